"""GPU: grouped products with their gradients, the gated activation, the router's gradient and AdamW
against their oracle in 64 bits."""

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


def half_step(dtype):
    """Half a step of the type, relative to the value."""
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the smallest subnormal step: what a rounding near zero is off by."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rows_of(g, r, c, dtype, pad=0):
    """[r, c] with a row stride of c + pad."""
    return torch.randn((r, c + pad), generator=g, device="cuda").to(dtype)[:, :c]


def offsets_of(counts, lead=0):
    return torch.tensor(np.concatenate([[lead], lead + np.cumsum(counts)]), dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------------- #
# products
# --------------------------------------------------------------------------- #
def product_case(ops, counts, N, K, dtype, out_dtype, lead=0, tail=0, pad=0, seed=0, no_offsets=False):
    """All three products of one case, each against the oracle within the bound of an fp32 sum:
    (terms + 1) roundings of at most 2^-23 (the matrix instruction may cut instead of round) of the
    sum of magnitudes, and half a step of the output's type."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R, E = sum(counts) + lead + tail, len(counts)
    off = None if no_offsets else offsets_of(counts, lead)
    seg = None if no_offsets else off.cpu().numpy()
    a, grad = rows_of(g, R, K, dtype, pad), rows_of(g, R, N, dtype, pad)
    w = (torch.randn((E, N, K), generator=g, device="cuda") / K ** 0.5).to(dtype)
    # what no segment holds must not be read
    for t in (a, grad):
        t[:lead] = float("nan")
        t[R - tail:] = float("nan")
    a_h, g_h, w_h = np64(a), np64(grad), np64(w)

    def check(what, got, want, size, depth):
        got, held = np64(got), np.isfinite(want)
        tol = (depth + 1) * 2.0 ** -23 * size + half_step(out_dtype) * np.abs(want) * 1.01 + least(out_dtype)
        worst = (np.abs(got - want) / tol)[held]
        assert worst.size == 0 or worst.max() <= 1.0, f"{what}: {worst.max():.3g} of the bound"
        assert np.all(got[~held] == 7.0), f"{what}: a row outside the segments was written"

    def made(rows, cols):
        return torch.full((rows, cols + pad), 7.0, dtype=out_dtype, device="cuda")[:, :cols]

    with np.errstate(invalid="ignore"):
        out = ops.moe_grouped_gemm(a, w, off, out=made(R, N))
        check("out", out, ref.product(a_h, w_h, seg), np.nan_to_num(ref.product(abs(a_h), abs(w_h), seg)), K)
        ga = ops.moe_grouped_gemm_backward(grad, w, off, out=made(R, K))
        check("rows", ga, ref.product_rows(g_h, w_h, seg), np.nan_to_num(ref.product_rows(abs(g_h), abs(w_h), seg)), N)
    want = ref.product_weights(g_h, a_h, seg)
    size = ref.product_weights(abs(g_h), abs(a_h), seg)
    depth = max(counts) if counts else 0
    gw = ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=out_dtype)
    check("weights", gw, want, size, depth)
    held = torch.randn((E, N, K), generator=g, device="cuda").to(out_dtype)
    before = np64(held)
    got = ops.moe_grouped_gemm_backward_weights(grad, a, off, out=held, accumulate=True)
    check("added weights", got, want + before, size + abs(before), depth + 1)
    # a repeated call gives identical bits
    again = ops.moe_grouped_gemm(a, w, off, out=made(R, N))
    assert torch.equal(again.contiguous().view(torch.uint8), out.contiguous().view(torch.uint8))
    assert torch.equal(ops.moe_grouped_gemm_backward_weights(grad, a, off, dtype=out_dtype), gw)


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (BF16, F16)])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 8), ([5, 0, 3], 64, 96), ([0, 0, 40], 200, 136), ([33, 64, 65, 1], 264, 520),
    ([128, 127, 129], 512, 256), ([300, 0, 17], 1280, 640),
])
def test_products(ops, counts, N, K, dtype, out_dtype):
    product_case(ops, counts, N, K, dtype, out_dtype, lead=3, tail=5)


@pytest.mark.parametrize("counts,N,K,pad", [
    ([1], 1, 1, 0), ([2, 3], 1, 33, 0), ([7], 65, 3, 1), ([70, 0, 1], 63, 127, 0), ([40], 129, 64, 3),
    ([90, 20], 136, 72, 4), ([33], 72, 136, 8), ([64, 31], 96, 31, 0),
])
def test_products_any_size_and_stride(ops, counts, N, K, pad):
    product_case(ops, counts, N, K, BF16, F32, lead=1, tail=2, pad=pad)
    product_case(ops, counts, N, K, F16, F16, pad=pad, seed=1)


@pytest.mark.parametrize("rows", [1, 16, 17, 255, 256, 257, 1000])
def test_one_expert_without_offsets(ops, rows):
    product_case(ops, [rows], 264, 328, BF16, BF16, no_offsets=True)


@pytest.mark.parametrize("E,rows", [(64, 40), (130, 500), (512, 80), (600, 900), (4096, 300)])
def test_many_experts(ops, E, rows):
    counts = np.bincount(np.random.default_rng(E).integers(0, E, rows), minlength=E)
    product_case(ops, list(counts), 72, 64, BF16, F32, lead=2)


@pytest.mark.parametrize("counts,N,K", [
    ([700, 900], 1024, 768), ([2000], 520, 264), ([1500, 0, 300, 260], 256, 1024), ([513, 511, 1024], 776, 1288),
])
def test_products_of_large_tiles(ops, counts, N, K):
    product_case(ops, counts, N, K, BF16, BF16)
    product_case(ops, counts, N, K, F16, F32, lead=8, seed=2)


@pytest.mark.parametrize("rows,N,K", [(5000, 64, 64), (9000, 512, 264), (3001, 136, 128)])
def test_weight_gradient_of_many_rows_and_few_tiles(ops, rows, N, K):
    product_case(ops, [rows], N, K, BF16, F32)
    product_case(ops, [rows // 2, 7, rows // 3], N, K, F16, F16, tail=4, seed=3)


def test_unaligned_base(ops):
    """Rows that begin at an odd element."""
    g = torch.Generator(device="cuda").manual_seed(0)
    buf = torch.randn(40 * 64 + 1, generator=g, device="cuda").to(BF16)
    a, w = buf[1:].view(40, 64), torch.randn((1, 48, 64), generator=g, device="cuda").to(BF16)
    want = ops.moe_grouped_gemm(a.clone(), w, dtype=F32)
    got = ops.moe_grouped_gemm(a, w, dtype=F32)
    assert torch.allclose(got, want, rtol=0, atol=64 * 2.0 ** -22 * float((a.abs().float() @ w[0].abs().float().t()).max()))


def test_special_values(ops):
    """An infinity or NaN reaches its own row only, and zeros of an empty segment stay zeros."""
    g = torch.Generator(device="cuda").manual_seed(0)
    a = torch.randn((300, 128), generator=g, device="cuda").to(BF16)
    w = torch.randn((3, 136, 128), generator=g, device="cuda").to(BF16)
    off = offsets_of([100, 0, 200])
    clean = ops.moe_grouped_gemm(a, w, off)
    a[7, 3], a[150, 5] = float("nan"), float("inf")
    w[1] = float("nan")  # the expert without rows
    got = ops.moe_grouped_gemm(a, w, off)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[[7, 150]] = False
    assert torch.equal(got[keep], clean[keep])
    assert got[7].isnan().all() and not got[150].isfinite().any()
    grad = torch.randn((300, 136), generator=g, device="cuda").to(BF16)
    gw = ops.moe_grouped_gemm_backward_weights(grad, a, off)
    assert gw[1].eq(0).all()
    assert gw[0, :, 3].isnan().all() and gw[0, :, :3].isfinite().all() and gw[0, :, 4:].isfinite().all()
    assert not gw[2, :, 5].isfinite().any() and gw[2, :, :5].isfinite().all() and gw[2, :, 6:].isfinite().all()


def test_no_rows(ops):
    w = torch.ones((2, 16, 8), dtype=BF16, device="cuda")
    a, off = w.new_empty((0, 8)), offsets_of([0, 0])
    assert ops.moe_grouped_gemm(a, w, off).shape == (0, 16)
    assert ops.moe_grouped_gemm_backward(w.new_empty((0, 16)), w, off).shape == (0, 8)
    gw = torch.full((2, 16, 8), 3.0, device="cuda")
    ops.moe_grouped_gemm_backward_weights(w.new_empty((0, 16)), a, off, out=gw, accumulate=True)
    assert gw.eq(3).all()
    assert ops.moe_grouped_gemm_backward_weights(w.new_empty((0, 16)), a, off, out=gw).eq(0).all()


def test_offsets_outside_the_tensors(ops):
    """Entries outside [0, rows] do not lead out of the tensors."""
    a = torch.ones((20, 64), dtype=BF16, device="cuda")
    w = torch.ones((3, 64, 64), dtype=BF16, device="cuda")
    off = torch.tensor([-5, 10, 10, 999], dtype=torch.int32, device="cuda")
    out = torch.full((24, 64), 7.0, device="cuda")
    ops.moe_grouped_gemm(a, w, off, out=out[2:22])
    assert out[2:22].eq(64).all() and out[:2].eq(7).all() and out[22:].eq(7).all()
    gw = ops.moe_grouped_gemm_backward_weights(a, a, off, dtype=F32)
    assert gw[0].eq(10).all() and gw[1].eq(0).all() and gw[2].eq(10).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_products(ops, seed):
    rng = np.random.default_rng(seed)
    E = int(rng.choice([1, 3, 8, 37]))
    counts = rng.multinomial(int(np.exp(rng.uniform(0, 7))), rng.dirichlet(np.full(E, 0.5)))
    N, K = (8 * int(np.exp(rng.uniform(0, 5))) for _ in range(2))
    product_case(ops, [int(c) for c in counts], N, K, [BF16, F16][seed % 2], [BF16, F32, F16][seed % 3],
                 lead=int(rng.integers(0, 9)), tail=int(rng.integers(0, 9)), pad=int(rng.choice([0, 8])), seed=seed)


# --------------------------------------------------------------------------- #
# activation
# --------------------------------------------------------------------------- #
# fp32: an exponential of 2 units in the last place, a reciprocal of 1, and fewer than ten products and
# sums of one half each; 1 + gate (1 - s) has no cancellation beyond its own size of at least |gate (1 - s)|
FEW = 16 * 2.0 ** -23


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,I,pad", [(1, 1, 0), (3, 7, 0), (80, 640, 0), (257, 33, 5), (1000, 128, 8), (2, 8192, 0)])
def test_silu_mul(ops, rows, I, pad, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    h = rows_of(g, rows, 2 * I, dtype, pad) * 3
    grad = rows_of(g, rows, I, dtype, pad)
    want = ref.silu_mul(np64(h))
    got = np64(ops.moe_silu_mul(h))
    assert (abs(got - want) <= (FEW + half_step(dtype) * 1.01) * abs(want) + least(dtype) + 1e-37).all()
    want = ref.silu_mul_backward(np64(grad), np64(h))
    gate, up = np.split(np64(h), 2, axis=1)
    s = 1 / (1 + np.exp(-gate))
    size = np.concatenate([abs(np64(grad) * up) * s * (1 + abs(gate) * (1 - s)), abs(np64(grad) * gate) * s], axis=1)
    got = ops.moe_silu_mul_backward(grad, h)
    assert (abs(np64(got) - want) <= FEW * size + half_step(dtype) * 1.01 * abs(want) + least(dtype) + 1e-37).all()
    # in place
    inside = h.clone() if pad == 0 else h
    assert torch.equal(ops.moe_silu_mul_backward(grad, inside, out=inside), got)


def test_silu_mul_ends_of_the_range(ops):
    gate = torch.tensor([0.0, -0.0, 100.0, -100.0, 3e38, -3e38, float("inf"), float("nan"), -87.0, 88.0, 1e-40],
                        device="cuda")
    h = torch.cat([gate, torch.full_like(gate, 2.0)]).view(1, -1)
    got = ops.moe_silu_mul(h)[0]
    assert got[0] == 0 and got[1] == 0 and got[2] == 200 and abs(got[3]) < 1e-37 and got[4] == float("inf")
    assert got[5] == 0 and got[6] == float("inf") and got[7].isnan()
    back = ops.moe_silu_mul_backward(torch.ones_like(gate).view(1, -1), h)[0]
    n = gate.numel()
    assert back[0] == 1 and back[2] == 2 and abs(back[3]) < 1e-35 and back[4] == 2 and back[5] == 0
    assert back[n + 4] == 3e38 and back[n + 5] == 0 and back[7].isnan() and back[n + 7].isnan()


@pytest.mark.parametrize("counts,lead,tail", [([3, 0, 4], 2, 3), ([0, 0], 4, 1), ([9], 0, 0)])
def test_silu_mul_inside_segments(ops, counts, lead, tail):
    g = torch.Generator(device="cuda").manual_seed(0)
    R = sum(counts) + lead + tail
    h, grad, off = rows_of(g, R, 32, BF16), rows_of(g, R, 16, BF16), offsets_of(counts, lead)
    inside = slice(lead, R - tail)
    out = ops.moe_silu_mul(h, off, out=torch.full((R, 16), 7.0, dtype=BF16, device="cuda"))
    back = ops.moe_silu_mul_backward(grad, h, off, out=torch.full((R, 32), 7.0, dtype=BF16, device="cuda"))
    for got, want in ((out, ops.moe_silu_mul(h)), (back, ops.moe_silu_mul_backward(grad, h))):
        assert torch.equal(got[inside], want[inside])
        assert got[:lead].eq(7).all() and got[R - tail:].eq(7).all()


# --------------------------------------------------------------------------- #
# the router's gradient
# --------------------------------------------------------------------------- #
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (8, 512, 10), (257, 37, 5), (33, 4096, 64), (5, 64, 64), (100, 7, 3)])
def test_route_backward(ops, T, E, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(T)
    ids, w = ops.moe_route(torch.randn((T, E), generator=g, device="cuda"), k)
    grad = torch.randn((T, k), generator=g, device="cuda")
    got = np64(ops.moe_route_backward(ids, w, grad, E, dtype=dtype))
    want = ref.route_backward(ids.cpu().numpy(), np64(w), np64(grad), E)
    # a sum of k products (6 additions by halves for 64), one difference, one product
    size = (np64(w) * (abs(np64(grad)) + (np64(w) * abs(np64(grad))).sum(1, keepdims=True))).max()
    assert (abs(got - want) <= 10 * 2.0 ** -24 * size + half_step(dtype) * 1.01 * abs(want) + least(dtype)).all()
    assert (got != 0).sum() <= T * k


def test_route_backward_left_out_and_repeated(ops):
    ids = torch.tensor([[0, -1, 5], [2, 2, 9], [1 << 30, -7, 8]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25], [0.5, 0.25, 0.25], [0.5, 0.25, 0.25]], device="cuda")
    grad = torch.tensor([[1.0, 0.0, 2.0], [1.0, 3.0, -1.0], [1.0, 2.0, 4.0]], device="cuda")
    got = ops.moe_route_backward(ids, w, grad, 8)
    # token 0: sum 1; token 1: sum 1, both choices are expert 2
    want = torch.zeros((3, 8), device="cuda")
    want[0, 0], want[0, 5] = 0.0, 0.25
    want[1, 2] = 0.0 + 0.25 * 2.0
    assert torch.equal(got, want)


def test_route_backward_is_the_gradient(ops):
    """Against autograd through a softmax over the chosen logits, in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn((50, 64), generator=g, device="cuda")
    ids, w = ops.moe_route(logits, 6)
    grad = torch.randn((50, 6), generator=g, device="cuda")
    x = logits.double().cpu().requires_grad_()
    torch.softmax(x.gather(1, ids.long().cpu()), dim=1).backward(grad.double().cpu())
    got = ops.moe_route_backward(ids, w, grad, 64).double().cpu()
    # the weights themselves are off by a few units in the last place
    assert torch.allclose(got, x.grad, rtol=0, atol=32 * 2.0 ** -24 * float(grad.abs().max()) * 2)


# --------------------------------------------------------------------------- #
# AdamW
# --------------------------------------------------------------------------- #
HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)


def adamw_tensor(g, n, dtype, grad_dtype):
    p = torch.randn(n, generator=g, device="cuda").to(dtype)
    grad = (0.01 * torch.randn(n, generator=g, device="cuda")).to(grad_dtype)
    return p, grad


@pytest.mark.parametrize("dtype,grad_dtype,copy", [
    (F32, F32, None), (F32, BF16, BF16), (BF16, BF16, None), (F16, F32, F32), (F32, F16, F16)])
@pytest.mark.parametrize("sizes", [[1], [7, 2048, 2049, 0, 129], [100001], [640] * 95])
def test_adamw_fp32_states(ops, sizes, dtype, grad_dtype, copy):
    g = torch.Generator(device="cuda").manual_seed(len(sizes))
    pairs = [adamw_tensor(g, n, dtype, grad_dtype) for n in sizes]
    ps, gs = [p for p, _ in pairs], [x for _, x in pairs]
    ms = [0.01 * torch.randn(n, generator=g, device="cuda") for n in sizes]
    vs = [1e-4 * torch.rand(n, generator=g, device="cuda") for n in sizes]
    cs = None if copy is None else [torch.empty(n, dtype=copy, device="cuda") for n in sizes]
    before = [tuple(np64(t) for t in x) for x in zip(ps, gs, ms, vs)]
    ops.moe_adamw(ps, gs, ms, vs, step=7, copies=cs, **HYPER)
    f32 = lambda x: float(np.float32(x))  # noqa: E731  the scalars as the kernel holds them
    hyper = {**HYPER, "beta1": f32(0.9), "beta2": f32(0.999)}
    for i, (p, x, m, v) in enumerate(before):
        want_p, want_m, want_v = ref.adamw(p, x, m, v, step=7, **hyper)
        # two products and a sum in fp32, and 1 - beta rounded apart from beta
        assert (abs(np64(ms[i]) - want_m) <= 4 * 2.0 ** -24 * (abs(m) + abs(x))).all()
        # the rest 1 - beta2 = 1e-3 was rounded from the fp64 value: off from 1 - f32(beta2) by 2^-25
        assert (abs(np64(vs[i]) - want_v) <= 4 * 2.0 ** -24 * (v + x * x)).all()
        # the step: a root, a reciprocal and products, 2^-23 each at most; 1 - beta^7 of rounded betas
        step = HYPER["lr"] * (abs(want_p - p) / HYPER["lr"] + HYPER["weight_decay"] * abs(p))
        tol = 2e-5 * step + 2.0 ** -23 * abs(p)
        assert (abs(np64(ps[i]) - want_p) <= tol + half_step(dtype) * 1.01 * abs(want_p) + least(dtype)).all()
        if copy is not None:
            assert (abs(np64(cs[i]) - want_p) <= tol + half_step(copy) * 1.01 * abs(want_p) + least(copy)).all()


def code_bounds(x, scales, seed, signed):
    """Codes that the noise allows when the value's place is off by 8 roundings either way."""
    each = np.repeat(scales, ref.BLOCK)[: x.size]
    u = ref.noise(x.size, seed, 0 if signed else 1) / 2.0 ** 20
    low = ref.code_sizes(abs(x) * (1 - 2.0 ** -20), each, u, signed)
    high = ref.code_sizes(abs(x) * (1 + 2.0 ** -20), each, u + 2.0 ** -20, signed)
    return low, high


@pytest.mark.parametrize("dtype,copy", [(F32, BF16), (BF16, None)])
@pytest.mark.parametrize("sizes", [[1], [127, 128, 129, 0, 5000], [70001], [300] * 45])
def test_adamw_8bit_states(ops, sizes, dtype, copy):
    g = torch.Generator(device="cuda").manual_seed(len(sizes) + 5)
    pairs = [adamw_tensor(g, n, dtype, F32) for n in sizes]
    ps, gs = [p for p, _ in pairs], [x for _, x in pairs]
    states = [ops.adamw_states(p, 8) for p in ps]
    ms, vs = [s[0] for s in states], [s[1] for s in states]
    cs = None if copy is None else [torch.empty(n, dtype=copy, device="cuda") for n in sizes]
    for step in (1, 2, 3):
        before = [(np64(p), np64(x), np64(ops.adamw_state_values(m, True)), np64(ops.adamw_state_values(v, False)))
                  for p, x, m, v in zip(ps, gs, ms, vs)]
        ops.moe_adamw(ps, gs, ms, vs, step=step, seed=step * 1000 + 3, copies=cs, **HYPER)
        for i, (p, x, m, v) in enumerate(before):
            want_p, want_m, want_v = ref.adamw(p, x, m, v, step=step, **HYPER)
            move = abs(want_p - p) + HYPER["lr"] * HYPER["weight_decay"] * abs(p)
            # 1 - 0.999^step carries the rounding of beta2: 2^-24 / 1e-3 relative at step 1
            tol = 1e-4 * move + 2.0 ** -23 * abs(p)
            assert (abs(np64(ps[i]) - want_p) <= tol + half_step(dtype) * 1.01 * abs(want_p)).all()
            for state, want, signed in ((ms[i], want_m, True), (vs[i], want_v, False)):
                codes, scales = state[0].cpu().numpy().astype(int), np64(state[1])
                top = ref.block_scales(want)
                # beta's own rounding: 2^-25 of the state
                assert (abs(scales - top) <= 2.0 ** -21 * top).all()
                if signed:
                    nonzero = codes % 128 != 0
                    assert ((codes >= 128) == (want < 0))[nonzero].all()
                    codes = codes % 128
                low, high = code_bounds(want, scales, step * 1000 + 3, signed)
                assert ((low <= codes) & (codes <= high)).all(), (i, signed)
        # and each tensor gets other gradients next
        gs = [torch.randn(n, generator=g, device="cuda") * 0.01 for n in sizes]


def test_adamw_8bit_follows_fp32(ops):
    """The mean of the second moment after gradients that shrink: states rounded to nearest would stand still."""
    n, steps = 1 << 16, 60
    g = torch.Generator(device="cuda").manual_seed(0)
    p = torch.zeros(n, device="cuda")
    first = 0.01 * torch.randn(n, generator=g, device="cuda")
    m8, v8 = ops.adamw_states(p, 8)
    hyper = {**HYPER, "beta2": 0.99}
    ops.moe_adamw([p], [first], [m8], [v8], step=1, seed=1, **hyper)
    v0 = ops.adamw_state_values(v8, False).double()
    zero = torch.zeros_like(first)
    for step in range(2, steps + 2):
        ops.moe_adamw([p], [zero], [m8], [v8], step=step, seed=step, **hyper)
    v1 = ops.adamw_state_values(v8, False).double()
    # every rounding keeps the mean; a step's error is at most 2^-3 of the element, so after 60 steps the mean
    # over 65536 elements (weighted like v itself: kurtosis 3) is within 5 * 2^-3 sqrt(60 * 3 / 65536) / 2 = 1.6%
    assert abs(float(v1.sum() / v0.sum()) / 0.99 ** steps - 1) < 0.017


def test_adamw_special_values(ops):
    n = 512
    grad = torch.full((n,), 1e-3, device="cuda")
    grad[130] = float("nan")   # block 1
    grad[300] = 0.0            # block 2: a zero moment stays zero
    grad[384:] = 1e-25         # block 3: moments below the smallest scale
    p = torch.ones(n, device="cuda")
    m, v = ops.adamw_states(p, 8)
    ops.moe_adamw([p], [grad], [m], [v], step=1, seed=9, **HYPER)
    mv, vv = ops.adamw_state_values(m, True), ops.adamw_state_values(v, False)
    assert p[130].isnan() and p[:130].isfinite().all() and p[131:].isfinite().all()
    assert mv[:128].isfinite().all() and not mv[128:256].isfinite().any() and mv[256:].isfinite().all()
    assert vv[:128].isfinite().all() and not vv[128:256].isfinite().any()
    assert mv[300] == 0 and vv[300] == 0 and (vv[256:300] > 0).all()
    assert vv[384:].eq(0).all()


def test_adamw_second_moment_is_never_rounded_to_zero(ops):
    n = 1 << 14
    grad = torch.full((n,), 1e-7, device="cuda")
    grad[::128] = 1.0  # one large element a block: the others lie far below its smallest code
    p = torch.ones(n, device="cuda")
    m, v = ops.adamw_states(p, 8)
    for step in (1, 2, 3, 4):
        before = p.clone()
        ops.moe_adamw([p], [grad], [m], [v], step=step, seed=step, **{**HYPER, "weight_decay": 0.0})
        assert (v[0] > 0).all()
        # m may round up to 2^-17 of its scale (0.1 step / 1.875) while v is at least 2^-33 of its own
        # (1e-3 step / 1.875): |m / c1| / sqrt(v / c2) <= 2^-17 (1/1.875) / sqrt(2^-33 / 1.875) = 0.52,
        # doubled for beta's decay and v's own part of 1 - beta2
        assert ((p - before).abs() <= 2 * HYPER["lr"]).all()


def test_adamw_grad_scale(ops):
    g = torch.Generator(device="cuda").manual_seed(3)
    p, grad = adamw_tensor(g, 3000, F32, F32)
    m, v = ops.adamw_states(p)
    q, m2, v2 = p.clone(), m.clone(), v.clone()
    ops.moe_adamw([p], [grad * 0.25], [m], [v], step=1, **HYPER)
    ops.moe_adamw([q], [grad], [m2], [v2], step=1, grad_scale=torch.tensor([0.25], device="cuda"), **HYPER)
    assert torch.equal(p, q) and torch.equal(m, m2) and torch.equal(v, v2)


def test_adamw_views(ops):
    """Tensors at odd addresses inside larger ones; what lies beside them stays."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n = 1001
    def inside(dtype):
        buf = torch.full((n + 5,), 7, dtype=dtype, device="cuda")
        return buf, buf[3:3 + n]
    for bits in (32, 8):
        pb, p = inside(BF16)
        p.copy_(torch.randn(n, generator=g, device="cuda"))
        grad = torch.randn(n, generator=g, device="cuda")
        q = p.clone()
        if bits == 32:
            bufs, st = zip(*(inside(F32) for _ in range(2)))
            for s in st:
                s.zero_()
        else:
            bufs, st = [], []
            for _ in range(2):
                (cb, c), (sb, s) = inside(torch.uint8), (None, torch.zeros(8, device="cuda"))
                c.zero_()
                bufs.append(cb)
                st.append((c, s))
        plain = ops.adamw_states(q, bits)
        ops.moe_adamw([p], [grad], [st[0]], [st[1]], step=1, seed=2, **HYPER)
        ops.moe_adamw([q], [grad], [plain[0]], [plain[1]], step=1, seed=2, **HYPER)
        assert torch.equal(p, q)
        for b in (pb, *bufs):
            assert b[:3].eq(7).all() and b[3 + n:].eq(7).all()


# --------------------------------------------------------------------------- #
# together: a training step of the routed experts, streams, graphs
# --------------------------------------------------------------------------- #
class Step:
    """Routing, experts and weights' update of one layer as a training program calls them."""

    def __init__(self, ops, seed=0, T=96, E=8, k=2, H=64, I=48, bits=32):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.ops, self.T, self.E, self.k, self.H, self.I = ops, T, E, k, H, I
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x, self.target = r(T, H).to(BF16), r(T, H)
        self.master = [r(E, H) / 8, r(E, 2 * I, H) / 8, r(E, H, I) / 7]
        self.w = [m.to(BF16) for m in self.master]
        self.m, self.v = zip(*(ops.adamw_states(m, bits) for m in self.master))

    def gradients(self):
        ops, E, k = self.ops, self.E, self.k
        wg, w13, w2 = self.w
        logits = ops.moe_grouped_gemm(self.x, wg.view(1, E, self.H), dtype=F32)
        ids, weights = ops.moe_route(logits, k)
        perm = ops.moe_permute_masked(ids, E)
        off, slots = perm["expert_offsets"], perm["slot_rows"]
        rows = ops.moe_dispatch(self.x, slots, k)
        h = ops.moe_grouped_gemm(rows, w13, off)
        act = ops.moe_silu_mul(h, off)
        y = ops.moe_grouped_gemm(act, w2, off)
        out = ops.moe_combine_masked(y, weights, slots, dtype=F32)
        grad_out = ((out - self.target) / self.T).to(BF16)
        grad_y, grad_weights = ops.moe_combine_backward(grad_out, y, weights, slots)
        grad_act = ops.moe_grouped_gemm_backward(grad_y, w2, off)
        grad_w2 = ops.moe_grouped_gemm_backward_weights(grad_y, act, off, dtype=F32)
        grad_h = ops.moe_silu_mul_backward(grad_act, h, off)
        grad_w13 = ops.moe_grouped_gemm_backward_weights(grad_h, rows, off, dtype=F32)
        grad_x = ops.moe_dispatch_backward(ops.moe_grouped_gemm_backward(grad_h, w13, off), slots, k)
        grad_logits = ops.moe_route_backward(ids, weights, grad_weights, E, dtype=BF16)
        grad_wg = ops.moe_grouped_gemm_backward_weights(grad_logits, self.x, dtype=F32)[0]
        grad_x = grad_x + ops.moe_grouped_gemm_backward(grad_logits, wg.view(1, E, self.H))
        return out, grad_x, [grad_wg, grad_w13, grad_w2], ids

    def update(self, grads, step):
        self.ops.moe_adamw(self.master, grads, list(self.m), list(self.v), step=step, seed=step, copies=self.w,
                           **HYPER)

    def reference(self, ids):
        """Output and gradients by autograd in 64 bits, on the CPU, with the same choices."""
        x = self.x.double().cpu().requires_grad_()
        w = [t.double().cpu().requires_grad_() for t in self.w]
        ids = ids.long().cpu()
        weights = torch.softmax((x @ w[0].t()).gather(1, ids), dim=1)
        out = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            h = x[t] @ w[1][e].t()
            y = (torch.nn.functional.silu(h[:, :self.I]) * h[:, self.I:]) @ w[2][e].t()
            out = out.index_add(0, t, weights[t, j].unsqueeze(1) * y)
        (((out - self.target.double().cpu()) ** 2).sum() / (2 * self.T)).backward()
        return out.detach(), x.grad, [t.grad for t in w]


def close(got, want, steps):
    """Relative distance in norm: roundings to bf16 between the calls, each half a step (2^-8)."""
    got = got.double().cpu()
    return float((got - want).norm() / want.norm()) <= steps * 2.0 ** -8


def test_training_step_gradients(ops):
    s = Step(ops)
    out, grad_x, grads, ids = s.gradients()
    want_out, want_x, want = s.reference(ids)
    # rounded in between: h, act, y (out); grad_out, grad_y, grad_act, grad_h, rows (gradients) and the sums of both
    assert close(out, want_out, 4)
    for got, w in zip((grad_x, *grads), (want_x, *want)):
        assert close(got, w, 12)


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps_run(ops, bits):
    s = Step(ops, bits=bits)
    for step in (1, 2, 3):
        before = [m.clone() for m in s.master]
        s.update(s.gradients()[2], step)
        for m, b, w in zip(s.master, before, s.w):
            assert m.isfinite().all() and not torch.equal(m, b) and torch.equal(w, m.to(BF16))


def test_captured_training_step(ops):
    """Gradients and update captured once and replayed, with eager work in between: each replay as the eager call."""
    s, t = Step(ops, seed=1), Step(ops, seed=1)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        warm = Step(ops, seed=2)
        warm.update(warm.gradients()[2], 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grad_x, grads, _ = s.gradients()
        s.update(grads, 5)
    for _ in range(4):
        graph.replay()
        want = t.gradients()
        t.update(want[2], 5)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(grad_x, want[1])
        for a, b in zip((*grads, *s.master, *s.w, *s.m, *s.v), (*want[2], *t.master, *t.w, *t.m, *t.v)):
            assert torch.equal(a, b)


def test_behind_a_backlog_on_a_side_stream(ops):
    """The calls run on the current stream, behind what is queued there."""
    want = Step(ops, seed=3)
    want_grads = want.gradients()
    want.update(want_grads[2], 2)
    torch.cuda.synchronize()
    s = Step(ops, seed=3)
    x = s.x.clone()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.x.zero_()
        big = torch.randn((4096, 4096), device="cuda")
        for _ in range(20):
            big = big @ big * 1e-3
        s.x.copy_(x)
        got = s.gradients()
        s.update(got[2], 2)
    stream.synchronize()
    assert torch.equal(got[0], want_grads[0]) and torch.equal(got[1], want_grads[1])
    for a, b in zip((*got[2], *s.master), (*want_grads[2], *want.master)):
        assert torch.equal(a, b)
