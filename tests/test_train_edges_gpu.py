"""GPU: the training operators at the ends of their ranges: tensors past 32-bit offsets, workspaces, sums in
parts, captured and concurrent calls, mixed lists."""

from __future__ import annotations

import numpy as np
import pytest

from oracle import train_oracle as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a16_group_quantized_amd import ops

    ops.load_library()
    return ops


def np64(t):
    return t.detach().double().cpu().numpy()


# ---- past 32 bits ---------------------------------------------------------------------
@pytest.mark.parametrize("stride,rows", [(2048, 1_100_000), (2051, 1_050_000)])
def test_rows_past_32_bit_offsets(ops, stride, rows):
    """A segment that begins more than 4 GB into the rows, aligned and not, against the same rows by themselves."""
    K, N, n = 2048, 72, 300
    g = torch.Generator(device="cuda").manual_seed(0)
    big = torch.empty(rows * stride, dtype=BF16, device="cuda")
    a = big.view(rows, stride)[:, :K]
    a[rows - n:] = torch.randn((n, K), generator=g, device="cuda").to(BF16)
    w = torch.randn((2, N, K), generator=g, device="cuda").to(BF16)
    off = torch.tensor([rows - n, rows - 100, rows], dtype=torch.int32, device="cuda")
    near = (off - (rows - n)).to(torch.int32)
    tail = a[rows - n:].contiguous()
    out = torch.empty((rows, N), dtype=BF16, device="cuda")
    ops.moe_grouped_gemm(a, w, off, out=out)
    want = np64(ops.moe_grouped_gemm(tail, w, near, dtype=F32))
    # one rounding to bf16 (2^-8), sums in another order: 2048 terms of about 1, 2^-23 each
    tol = 2.0 ** -8 * abs(want) + 2048 * 2.0 ** -23 * 2048
    assert (abs(np64(out[rows - n:]) - want) <= tol).all()
    grad = torch.randn((n, N), generator=g, device="cuda").to(BF16)
    out[rows - n:] = grad
    back = ops.moe_grouped_gemm_backward(out, w, off, out=a)
    want = np64(ops.moe_grouped_gemm_backward(grad, w, near, dtype=F32))
    assert (abs(np64(back[rows - n:]) - want) <= 2.0 ** -8 * abs(want) + 72 * 2.0 ** -23 * 72 * 16).all()
    a[rows - n:] = tail
    got = ops.moe_grouped_gemm_backward_weights(out, a, off, dtype=F32)
    want = ref.product_weights(np64(grad), np64(tail), near.cpu().numpy())
    size = ref.product_weights(abs(np64(grad)), abs(np64(tail)), near.cpu().numpy())
    assert (abs(np64(got) - want) <= 201 * 2.0 ** -23 * size).all()


def test_activation_past_32_bit_offsets(ops):
    rows, I = 1_400_000, 1608
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.empty((rows, 2 * I), dtype=BF16, device="cuda")
    h[-5:] = torch.randn((5, 2 * I), generator=g, device="cuda").to(BF16)
    off = torch.tensor([rows - 5, rows], dtype=torch.int32, device="cuda")
    act = ops.moe_silu_mul(h, off)
    assert torch.equal(act[-5:], ops.moe_silu_mul(h[-5:].clone()))
    grad = act
    grad[-5:] = torch.randn((5, I), generator=g, device="cuda").to(BF16)
    want = ops.moe_silu_mul_backward(grad[-5:].clone(), h[-5:].clone())
    ops.moe_silu_mul_backward(grad, h, off, out=h)
    assert torch.equal(h[-5:], want)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_32_bit_offsets(ops, bits):
    n, tail = (1 << 31) + (1 << 27) + 77, 1000
    g = torch.Generator(device="cuda").manual_seed(2)
    p, grad = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    p[-tail:] = torch.randn(tail, generator=g, device="cuda")
    grad[-tail:] = torch.randn(tail, generator=g, device="cuda")
    q, grad2 = p[-tail:].clone(), grad[-tail:].clone()
    m, v = ops.adamw_states(p, bits)
    m2, v2 = ops.adamw_states(q, bits)
    hyper = dict(lr=1e-2, step=1, seed=4, weight_decay=0.1)
    ops.moe_adamw([p], [grad], [m], [v], **hyper)
    ops.moe_adamw([q], [grad2], [m2], [v2], **hyper)
    assert torch.equal(p[-tail:], q) and p[: n - tail].eq(0).all()
    if bits == 32:
        assert torch.equal(m[-tail:], m2) and torch.equal(v[-tail:], v2)
    else:
        assert m[0][: n - tail].eq(0).all() and m[0][-tail:].ne(0).any()


# ---- sums in parts, workspaces, graphs ---------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_gradient_in_parts(ops, dtype):
    """A long sum that is shared out: uneven segments, one shorter than a part, one empty; added to a given tensor;
    in a captured graph with the caller's workspace."""
    counts, N, K, lead = [6000, 0, 5, 1800], 64, 136, 3
    E, R = len(counts), sum(counts) + lead
    need = ops.grouped_gemm_backward_weights_workspace_bytes(R, E, N, K)
    assert need > 0
    g = torch.Generator(device="cuda").manual_seed(3)
    grad = torch.randn((R, N), generator=g, device="cuda").to(BF16)
    a = torch.randn((R, K), generator=g, device="cuda").to(BF16)
    off = torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    want = ref.product_weights(np64(grad), np64(a), off.cpu().numpy())
    size = ref.product_weights(abs(np64(grad)), abs(np64(a)), off.cpu().numpy())
    eps = torch.finfo(dtype).eps / 2
    tol = 6001 * 2.0 ** -23 * size + eps * 1.01 * abs(want)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read unwritten
    first = ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=dtype, workspace=ws)
    assert (abs(np64(first) - want) <= tol).all() and first[1].eq(0).all()
    held = torch.ones_like(first)
    ops.moe_grouped_gemm_backward_weights(grad, a, off, out=held, accumulate=True, workspace=ws)
    assert (abs(np64(held) - want - 1) <= tol + eps * 1.01 * (abs(want) + 1) + 2.0 ** -22).all()
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe_grouped_gemm_backward_weights(grad, a, off, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(7)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    with pytest.raises(ops.MoEError):
        ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=dtype, workspace=ws[: need - 1])


def test_two_streams_at_once(ops):
    """Calls that overlap in time on two streams, each with its own outputs and workspace."""
    g = torch.Generator(device="cuda").manual_seed(4)
    cases = []
    for seed in range(2):
        a = torch.randn((5000, 256), generator=g, device="cuda").to(BF16)
        w = torch.randn((4, 512, 256), generator=g, device="cuda").to(BF16)
        grad = torch.randn((5000, 512), generator=g, device="cuda").to(BF16)
        off = torch.tensor([0, 2000 + seed, 2000 + seed, 4500, 5000], dtype=torch.int32, device="cuda")
        cases.append((a, w, grad, off))
    run = lambda a, w, grad, off: (ops.moe_grouped_gemm(a, w, off), ops.moe_grouped_gemm_backward(grad, w, off),  # noqa: E731
                                   ops.moe_grouped_gemm_backward_weights(grad[:, :64], a[:, :64], off, dtype=F32))
    want = [run(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(run(*c))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i]))


def test_column_ranges_of_one_buffer(ops):
    """Gate and up as column ranges: an operand and an output that interleave in one buffer."""
    g = torch.Generator(device="cuda").manual_seed(5)
    buf = torch.randn((100, 256), generator=g, device="cuda").to(BF16)
    a, out = buf[:, :128], buf[:, 128:192]
    w = torch.randn((1, 64, 128), generator=g, device="cuda").to(BF16)
    want = ops.moe_grouped_gemm(a.clone(), w)
    before = buf.clone()
    ops.moe_grouped_gemm(a, w, out=out)
    assert torch.equal(out, want) and torch.equal(buf[:, :128], before[:, :128])
    assert torch.equal(buf[:, 192:], before[:, 192:])


@pytest.mark.parametrize("size", ["256", "128", "64", "32"])
def test_every_shape_with_ragged_ends(ops, size):
    """Each tile shape with rows, columns and reduction that end inside a tile and a chunk, and rows that fill one."""
    counts, N, K = {"256": ([2049, 1, 700, 2048], 2552, 2552), "128": ([129, 0, 128, 255, 1, 130] * 8, 648, 648),
                    "64": ([65, 64, 1, 130], 1032, 1032), "32": ([33, 1, 0, 32], 72, 1352)}[size]
    g = torch.Generator(device="cuda").manual_seed(6)
    R, E = sum(counts), len(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    a = torch.randn((R, K), generator=g, device="cuda").to(F16)
    w = torch.randn((E, N, K), generator=g, device="cuda").to(F16)
    grad = torch.randn((R, N), generator=g, device="cuda").to(F16)
    seg = off.cpu().numpy()
    got = ops.moe_grouped_gemm(a, w, off, dtype=F32)
    back = ops.moe_grouped_gemm_backward(grad, w, off, dtype=F32)
    gw = ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=F32)
    for e in range(E):
        s = slice(int(seg[e]), int(seg[e + 1]))
        x, y, z = a[s].double(), w[e].double(), grad[s].double()
        for have, want, big, depth in (
                (got[s], x @ y.t(), x.abs() @ y.abs().t(), K), (back[s], z @ y, z.abs() @ y.abs(), N),
                (gw[e], z.t() @ x, z.abs().t() @ x.abs(), counts[e])):
            assert ((have.double() - want).abs() <= (depth + 1) * 2.0 ** -23 * big).all()


# ---- AdamW lists ------------------------------------------------------------------------
def test_adamw_mixed_lists(ops):
    """Types that differ from tensor to tensor, copies for some of them, shapes of any rank: as one call each."""
    g = torch.Generator(device="cuda").manual_seed(7)
    shapes, kinds = [(3, 50), (7,), (2, 3, 4), (5000,)], [F32, BF16, F16, F32]
    ps = [torch.randn(s, generator=g, device="cuda").to(k) for s, k in zip(shapes, kinds)]
    gs = [torch.randn(s, generator=g, device="cuda").to(k) for s, k in zip(shapes, [BF16, F32, F16, F32])]
    for bits in (32, 8):
        one, each = ([p.clone() for p in ps] for _ in range(2))
        copies = [torch.zeros(shapes[0], dtype=BF16, device="cuda"), None, None, torch.zeros(5000, dtype=F16, device="cuda")]
        st = [ops.adamw_states(p, bits) for p in ps]
        st2 = [ops.adamw_states(p, bits) for p in ps]
        kw = dict(lr=1e-2, step=3, seed=8)
        ops.moe_adamw(one, gs, [s[0] for s in st], [s[1] for s in st], copies=copies, **kw)
        for p, x, s in zip(each, gs, st2):
            ops.moe_adamw([p], [x], [s[0]], [s[1]], **kw)
        assert all(torch.equal(a, b) for a, b in zip(one, each))
        assert torch.equal(copies[0], one[0].to(BF16)) and torch.equal(copies[3], one[3].to(F16))
        flat = lambda s: [t for x in s for t in (x if isinstance(x, tuple) else (x,))]  # noqa: E731
        for a, b in zip(st, st2):
            assert all(torch.equal(x, y) for x, y in zip(flat(a), flat(b)))


def test_adamw_is_a_function_of_its_seed(ops):
    g = torch.Generator(device="cuda").manual_seed(9)
    grad = torch.randn(4096, generator=g, device="cuda")
    out = []
    for seed in (1, 1, 2):
        p = torch.zeros(4096, device="cuda")
        m, v = ops.adamw_states(p, 8)
        ops.moe_adamw([p], [grad], [m], [v], lr=1e-3, step=1, seed=seed)
        out.append((p, m[0], v[0]))
    assert all(torch.equal(a, b) for a, b in zip(out[0], out[1]))
    assert torch.equal(out[0][0], out[2][0])
    assert not torch.equal(out[0][1], out[2][1]) and not torch.equal(out[0][2], out[2][2])


def test_captured_adamw(ops):
    g = torch.Generator(device="cuda").manual_seed(10)
    make = lambda: [torch.full((n,), 0.5, device="cuda") for n in (100, 5000) * 30]  # noqa: E731
    grads = [torch.randn(p.numel(), generator=g, device="cuda") for p in make()]
    for bits in (32, 8):
        a, b = make(), make()
        sa, sb = [ops.adamw_states(p, bits) for p in a], [ops.adamw_states(p, bits) for p in b]
        step = lambda ps, st: ops.moe_adamw(ps, grads, [s[0] for s in st], [s[1] for s in st], lr=1e-2, step=2, seed=6)  # noqa: E731
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(a, sa)
        for _ in range(3):
            graph.replay()
            step(b, sb)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a, b))


# ---- narrow matrices -------------------------------------------------------------------
@pytest.mark.parametrize("counts,N,K", [([65], 8, 8), ([129, 65, 1, 193], 24, 16), ([70, 0, 130], 1024, 8),
                                        ([66] * 300, 8, 512)])
def test_weight_gradient_of_rows_shorter_than_a_tile(ops, counts, N, K):
    """The last segment ends with the tensors and with a few rows in its last chunk: what the rows before
    them read past their ends must stay inside.  Rows of other segments do not get in either."""
    g = torch.Generator(device="cuda").manual_seed(0)
    R = sum(counts)
    grad, a = (torch.randn((R, n), generator=g, device="cuda").to(BF16) for n in (N, K))
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    got = np64(ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=F32))
    seg, g_h, a_h = off.cpu().numpy(), np64(grad), np64(a)
    size = ref.product_weights(abs(g_h), abs(a_h), seg)
    assert (abs(got - ref.product_weights(g_h, a_h, seg)) <= (max(counts) + 1) * 2.0 ** -23 * size).all()


# ---- AdamW without eps --------------------------------------------------------------------
@pytest.mark.parametrize("eps", [0.0, 1e-21])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_subnormal_second_moments(ops, bits, eps):
    """Gradients of 1e-20 to 1e-16 square to fp32's subnormal numbers: the step is lr all the same."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n = 1000
    grad = 10.0 ** -(16 + 4 * torch.rand(n, generator=g, device="cuda")) * torch.randn(n, generator=g, device="cuda").sign()
    p = torch.ones(n, device="cuda")
    m, v = ops.adamw_states(p, bits)
    ops.moe_adamw([p], [grad], [m], [v], lr=1e-2, beta1=0.9, beta2=0.999, eps=eps, weight_decay=0.0, step=1)
    x = grad.cpu().numpy()
    m32, v32 = np.float32(1 - 0.9) * x, np.float32(1 - 0.999) * (x * x)  # in fp32, as the kernel's
    step = 1e-2 * (m32.astype(np.float64) / 0.1) / (np.sqrt(v32.astype(np.float64) / 0.001) + eps)
    assert (abs(np64(p) - (1 - step)) <= 2e-5 * abs(step) + 2.0 ** -23).all()


# ---- sizes off the 16-byte grid ---------------------------------------------------------
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("counts,N,K", [([9000], 63, 65), ([3000, 0, 5000], 33, 130), ([20000], 3, 7), ([6000], 1, 1),
                                        ([300, 2000], 257, 131)])
def test_weight_gradient_of_odd_sizes_and_long_sums(ops, counts, N, K, out_dtype):
    """Sums in parts and in one, plain and added to what is there, in a tensor with a value behind it."""
    g = torch.Generator(device="cuda").manual_seed(0)
    R, E = sum(counts), len(counts)
    grad, a = (torch.randn((R, n), generator=g, device="cuda").to(BF16) for n in (N, K))
    off = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    seg, g_h, a_h = off.cpu().numpy(), np64(grad), np64(a)
    want, size = ref.product_weights(g_h, a_h, seg), ref.product_weights(abs(g_h), abs(a_h), seg)
    half = torch.finfo(out_dtype).eps / 2
    for accumulate in (False, True):
        buf = torch.randn(E * N * K + 1, generator=g, device="cuda").to(out_dtype)
        before = np64(buf)
        held = before[:-1].reshape(E, N, K) * accumulate
        got = np64(ops.moe_grouped_gemm_backward_weights(grad, a, off, out=buf[:-1].view(E, N, K), accumulate=accumulate))
        tol = (max(counts) + 2) * 2.0 ** -23 * (size + abs(held)) + 1.01 * half * abs(want + held)
        assert (abs(got - (want + held)) <= tol).all()
        assert float(buf[-1]) == before[-1]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("E,R,N,K", [(3, 700, 521, 1031), (2, 2100, 1030, 513), (40, 3000, 259, 135)])
def test_products_of_odd_sizes_in_large_tiles(ops, E, R, N, K, dtype):
    """Rows behind and before the segments hold NaN, and the rows' ends another matrix's values."""
    g = torch.Generator(device="cuda").manual_seed(1)
    counts = np.bincount(np.random.default_rng(E).integers(0, E, R - 5), minlength=E)
    off = torch.tensor(3 + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    grad, a = (torch.randn((R, n + 3), generator=g, device="cuda").to(dtype)[:, 1:n + 1] for n in (N, K))
    w = (torch.randn((E, N, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    for t in (grad, a):
        t[:3], t[-2:] = float("nan"), float("nan")
    seg, g_h, a_h, w_h = off.cpu().numpy(), np64(grad), np64(a), np64(w)
    mine = slice(3, R - 2)
    for got, f, x, y, terms in ((ops.moe_grouped_gemm(a, w, off, dtype=F32), ref.product, a_h, w_h, K),
                                (ops.moe_grouped_gemm_backward(grad, w, off, dtype=F32), ref.product_rows, g_h, w_h, N)):
        size = f(abs(x), abs(y), seg)[mine]
        assert (abs(np64(got)[mine] - f(x, y, seg)[mine]) <= (terms + 1) * 2.0 ** -23 * size).all()
    got = np64(ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=F32))
    size = ref.product_weights(abs(g_h), abs(a_h), seg)
    assert (abs(got - ref.product_weights(g_h, a_h, seg)) <= (max(counts) + 1) * 2.0 ** -23 * size).all()


# ---- the most tokens --------------------------------------------------------------------
def test_route_backward_of_the_most_tokens(ops):
    """2^26 - 4 tokens of one choice: 2^32 - 256 threads."""
    T = (1 << 26) - 4
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) & 1).view(T, 1)
    w, grad = torch.full((T, 1), 0.5, device="cuda"), torch.arange(T, device="cuda").remainder(251).float().view(T, 1)
    out = ops.moe_route_backward(ids, w, grad, 2)
    want = torch.zeros(T, 2, device="cuda").scatter_(1, ids.long(), 0.25 * grad)  # w (g - w g): exact
    assert torch.equal(out, want)
    with pytest.raises(ops.MoEError):
        grow = lambda t: torch.cat([t, t[:1]])  # noqa: E731
        ops.moe_route_backward(grow(ids), grow(w), grow(grad), 2)
