"""GPU: the MXFP4 and row calls where ordinary inputs do not lead: sums near the ends
of fp32, rows without a token, scales at the ends of their range, empty batches, and
work that is still on its way on a side stream.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import mxfp4_oracle as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a16_group_quantized_amd import ops

    ops.load_library()
    return ops


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"\n[gpu-test] {request.node.nodeid}", flush=True)
    yield


def _gpu(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _host(t: torch.Tensor) -> np.ndarray:
    return (t.float() if t.is_floating_point() else t).cpu().numpy()


def _mx(values: np.ndarray, bytes_: np.ndarray):
    """Packed rows [..., K] of E2M1 values with the given scale bytes [..., K/32] (padding 255)."""
    K = values.shape[-1]
    flat = values.reshape(-1, K)
    code = np.abs(np.abs(flat)[..., None] - ref.E2M1).argmin(axis=-1) + 8 * np.signbit(flat)
    assert np.array_equal(ref.E2M1[code & 7], np.abs(flat))
    words, scales = ref.mx_pack(code.astype(np.uint8), bytes_.reshape(len(flat), -1).astype(np.uint8))
    scales[:, K // 32:] = 255
    return (words.reshape(*values.shape[:-1], -1), scales.reshape(*values.shape[:-1], -1))


# ---- SiLU over the whole of fp32 ------------------------------------------------------
# each gate is a 2^p + b 2^q, exact in fp32: about 17, 84, 88, 120, 1e30, 2.3e38, 2.4e38, 3.2e38
_GATES = [(1.0, 4, 1.0, 0), (1.5, 6, -1.5, 3), (1.0, 6, 1.5, 4), (1.0, 7, -1.0, 3), (1.5, 99, 0.0, 0),
          (1.5, 127, -1.0, 124), (1.5, 127, -1.0, 123), (1.5, 127, 1.5, 125)]


def _wide_gates(K: int):
    """(W13 [1, 2I, K] as MXFP4, gates [I], ups [I]) whose sums over a row with ones at columns 0 and
    32 are the gates of both signs, 32 columns each, and small ups."""
    I = 64 * len(_GATES)
    values, bytes_ = np.zeros((2 * I, K)), np.full((2 * I, K // 32), 127)
    ups = np.resize([0.5, 1.0, -1.5, 2.0, 3.0, -4.0], I)
    for i, (a, p, b, q) in enumerate(_GATES):
        for half, sign in enumerate((1.0, -1.0)):
            at = slice(64 * i + 32 * half, 64 * i + 32 * half + 32)
            values[at, 0], values[at, 32] = sign * a, sign * b
            bytes_[at, 0], bytes_[at, 1] = p + 127, q + 127
    values[I:, 0] = ups
    bytes_[I:, 0] = 127 - 20
    w = _mx(values[None], bytes_[None])
    h = ref.mx_values(*w)[0].sum(axis=1)
    return w, h[:I], h[I:]


def _silu_mul(gate: np.ndarray, up: np.ndarray):
    """SiLU(gate) * up in fp64, and what fp32 may be off by: a few roundings of the value (exponential,
    sum, quotient, two products), and a reciprocal below 2^-126 that counts as zero."""
    with np.errstate(over="ignore"):
        act = gate / (1.0 + np.exp(-gate)) * up
    return act, 8 * 2.0 ** -24 * np.abs(act) + 2.0 ** -126 * np.abs(gate * up)


@pytest.mark.parametrize("R,K", [(3, 64), (3, 1600), (900, 64)], ids=["stream", "stream-split", "tile"])
def test_gate_up_over_the_whole_range_of_gates(ops, R, K):
    w, gate, up = _wide_gates(K)
    ones = np.zeros((R, K))
    ones[:, [0, 32]] = 1.0
    a = _mx(ones, np.full((R, K // 32), 127))
    codes, scales = ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    I = len(gate)
    act, err = _silu_mul(gate, up)
    b = _host(scales)[:, : I // 32].astype(np.int64)
    top, off = np.abs(act).reshape(-1, 32), err.reshape(-1, 32)
    lo = ref.mx_exponent(np.maximum(top - off, 0).max(axis=1)) + 127
    hi = ref.mx_exponent((top + off).max(axis=1)) + 127
    assert ((lo <= b) & (b <= hi)).all(), (lo, hi, b[0])
    got = ref.mx_values(_host(codes), _host(scales))
    unit = np.repeat(np.exp2(b - 127.0), 32, axis=1)
    m = (np.abs(act) + err) / unit
    half = np.where(m <= 2, 0.25, np.where(m <= 4, 0.5, np.maximum(1.0, m - 6)))
    assert (np.abs(got - act) <= half * unit + err).all()


def test_gate_up_keeps_nan_and_infinite_gates(ops):
    """A NaN sum, and one past fp32: blocks of scale byte 255 and zero codes, in each kernel form."""
    for R in (3, 900):
        for value, byte in ((1.0, 255), (6.0, 254)):
            K, I = 64, 96
            v, s = np.zeros((1, 2 * I, K)), np.full((1, 2 * I, K // 32), 127)
            v[0, :, 0] = 1.0
            v[0, 40, 0], s[0, 40, 0] = value, byte  # gate 40, in the second block
            ones = np.zeros((R, K))
            ones[:, 0] = 1.0
            w, a = _mx(v, s), _mx(ones, np.full((R, K // 32), 127))
            codes, scales = ops.moe_mxfp4_gate_up(*(_gpu(t) for t in (*a, *w)))
            codes, scales = _host(codes), _host(scales)
            assert (scales[:, 1] == 255).all() and (codes[:, 4:8] == 0).all(), (R, byte)
            assert (scales[:, [0, 2]] != 255).all() and (codes[:, :4] != 0).all(), (R, byte)


@pytest.mark.parametrize("T", [1, 6, 7, 90])
def test_layer_over_the_whole_range_of_gates(ops, T):
    """The layer's gate/up, in its form for few tokens and in the calls' own: outputs of every gate
    apart (w2 picks one column of I each, its scale brings the product back to about 1)."""
    H = K = 64
    w13, gate, up = _wide_gates(K)
    I = len(gate)
    act, err = _silu_mul(gate, up)
    got_bytes = ref.mx_exponent(np.abs(act).reshape(-1, 32).max(axis=1))
    values, bytes_ = np.zeros((1, H, I)), np.full((1, H, I // 32), 127)
    picks = np.arange(H) * (I // H) + np.arange(H) % 7
    big = np.abs(act[picks]) > 2.0 ** -100
    for n, i in enumerate(picks):
        values[0, n, i] = 1.0
        bytes_[0, n, i // 32] = 127 - max(min(int(got_bytes[i // 32]), 127), -100)
    w2 = _mx(values, bytes_)
    x = torch.zeros(T, H, device="cuda")
    x[:, [0, 32]] = 1.0
    logits = torch.zeros(T, 1, device="cuda")
    w = {"w13_codes": _gpu(w13[0]), "w13_scales": _gpu(w13[1]), "w2_codes": _gpu(w2[0]), "w2_scales": _gpu(w2[1])}
    out = _host(ops.moe_mxfp4_layer_forward(logits, x, 1, w)).astype(np.float64)
    scale = ref.mx_values(*w2)[0][np.arange(H), picks]
    want = act[picks] * scale
    # an act is stored with half an E2M1 step of its block, at most 1 unit below 6 and 2 behind
    unit = np.exp2(got_bytes[picks // 32].astype(np.float64)) * scale
    assert np.isfinite(out).all()
    assert (np.abs(out - want)[:, big] <= (2.0 * unit + err[picks] * scale)[big]).all()
    assert (np.abs(out[:, big]) > 0).any(axis=0).sum() >= 24


# ---- rows without a token ---------------------------------------------------------------
ABSENT = [  # rows of A, top_k, E, N, K: streaming, K shared out, and tiles
    (23, 3, 5, 128, 416), (9, 2, 2, 128, 1600), (1500, 3, 40, 896, 640), (2150, 2, 2, 4160, 288), (300, 4, 64, 192, 1120),
]


@pytest.mark.parametrize("T,k,E,N,K", ABSENT)
def test_a_row_without_a_token_is_zero_whatever_the_weights_hold(ops, T, k, E, N, K):
    rng = np.random.default_rng(T)
    S = T * k
    words = lambda *s: rng.integers(0, 1 << 32, size=(*s, K // 8), dtype=np.uint32).view(np.int32)
    a = words(T), np.full((T, ref.mx_scale_bytes(K)), 125, np.uint8)
    w = words(E, N), np.full((E, N, ref.mx_scale_bytes(K)), 121, np.uint8)
    w[1][:, 17, 1] = 255  # column 17 of every expert
    slots = rng.permutation(S).astype(np.int32)
    gone = rng.random(S) < 0.2
    gone[[0, S - 1]] = True
    slots[gone] = rng.choice([-1, S, S + 5, -(1 << 31), (1 << 31) - 1], size=int(gone.sum()))
    off = np.sort(np.concatenate([[0, S], rng.integers(0, S + 1, E - 1)])).astype(np.int32)
    args = [_gpu(t) for t in (*a, *w, off)]
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((S, N), 7.0, device="cuda", dtype=dtype)
        got = _host(ops.moe_mxfp4_grouped_gemm(*args, row_slots=_gpu(slots), top_k=k, out=out))
        assert (got[gone] == 0).all()
        assert np.isnan(got[~gone][:, 17]).all() and np.isnan(got).sum() == (~gone).sum()
    codes, scales = ops.moe_mxfp4_gate_up(*args, row_slots=_gpu(slots), top_k=k)
    codes, scales = _host(codes), _host(scales)
    blocks = N // 64
    assert (codes[gone] == 0).all() and (scales[gone][:, :blocks] == 0).all()
    assert (scales[~gone][:, 0] == 255).all() and (codes[~gone][:, :4] == 0).all()
    assert (scales[:, 1:blocks] != 255).all()


# ---- an empty batch -----------------------------------------------------------------------
def test_permutation_of_no_tokens_into_given_buffers(ops):
    """A batch without tokens after one with some, both into the same buffers."""
    E, k = 6, 2
    out = ops.moe_permute_masked(torch.tensor([[1, 5], [1, 0]], dtype=torch.int32, device="cuda"), E)
    out["sorted_slots"], out["slot_rows"] = out["sorted_slots"][:0], out["slot_rows"][:0]
    ids = torch.empty(0, k, dtype=torch.int32, device="cuda")
    want = {n: torch.from_numpy(v) for n, v in ref.permute_masked(np.zeros((0, k), np.int32), E).items()}
    for got in (ops.moe_permute_masked(ids, E, out=out), ops.moe_permute_masked(ids, E)):
        for name, value in want.items():
            assert torch.equal(got[name].cpu(), value), name


# ---- scales at the ends of their range --------------------------------------------------
@pytest.mark.parametrize("E,R,N,K", [(1, 3, 48, 96), (1, 3, 48, 1600), (1, 900, 300, 288), (3, 800, 300, 1088)],
                         ids=["stream", "stream-split", "tile", "tile-long"])
@pytest.mark.parametrize("a_byte,w_byte", [(0, 254), (254, 0), (0, 127), (127, 0), (0, 140), (254, 100), (0, 0)])
def test_product_with_scale_bytes_0_and_254(ops, E, R, N, K, a_byte, w_byte):
    """Terms are multiples of 2^-2 of the scales' product, at most 36 of it.  Where that product is a
    normal number the bound is the usual one, K fp32 roundings; at byte 0 against 127 every sum is a
    multiple of 2^-129, which fp32 holds exactly up to 2^-105."""
    rng = np.random.default_rng(K + R)
    words = lambda *s: rng.integers(0, 1 << 32, size=(*s, K // 8), dtype=np.uint32).view(np.int32)
    a = words(R), np.full((R, ref.mx_scale_bytes(K)), a_byte, np.uint8)
    w = words(E, N), np.full((E, N, ref.mx_scale_bytes(K)), w_byte, np.uint8)
    off = np.linspace(0, R, E + 1).astype(np.int32)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off)
    got = _host(ops.moe_mxfp4_grouped_gemm(*(_gpu(t) for t in (*a, *w, off)))).astype(np.float64)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= K * 2.0 ** -24 * size * (a_byte + w_byte > 127 + 24) + 2.0 ** -150).all()


# ---- streams ------------------------------------------------------------------------------
def _stream_cases(ops):
    """name: (inputs that arrive late, call).  Zeros are valid in the place of every input."""
    rng = np.random.default_rng(31)
    T, k, E, H, I = 40, 4, 16, 256, 96
    S = T * k
    randn = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()
    ids = _gpu(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    perm = ops.moe_permute_masked(ids, E)
    xq = ops.moe_mxfp4_quantize(randn(S, H))
    w = {}
    for name, n, c in (("w13", 2 * I, H), ("w2", H, I)):
        codes, scales = ops.moe_mxfp4_quantize(randn(E * n, c) / c ** 0.5)
        w[name + "_codes"], w[name + "_scales"] = codes.view(E, n, -1), scales.view(E, n, -1)
    w13 = w["w13_codes"], w["w13_scales"]
    weights, rows = torch.rand(T, k, device="cuda"), perm["slot_rows"]
    return {
        "quantize": ([randn(S, H)], ops.moe_mxfp4_quantize),
        "dequantize": (list(xq), ops.moe_mxfp4_dequantize),
        "grouped_gemm": (list(xq), lambda c, s: ops.moe_mxfp4_grouped_gemm(c, s, *w13, perm["expert_offsets"])),
        "gate_up": (list(xq), lambda c, s: ops.moe_mxfp4_gate_up(c, s, *w13, perm["expert_offsets"])),
        "layer_few": ([randn(3, E), randn(3, H)], lambda g, x: ops.moe_mxfp4_layer_forward(g, x, k, w)),
        "layer": ([randn(T, E), randn(T, H)], lambda g, x: ops.moe_mxfp4_layer_forward(g, x, k, w)),
        "layer_many": ([randn(100, E), randn(100, H)], lambda g, x: ops.moe_mxfp4_layer_forward(g, x, k, w)),
        "permute_masked": ([ids], lambda i: tuple(ops.moe_permute_masked(i, E).values())),
        "dispatch": ([randn(T, H)], lambda x: ops.moe_dispatch(x, rows, k)),
        "dispatch_backward": ([randn(S, H)], lambda g: ops.moe_dispatch_backward(g, rows, k)),
        "combine_masked": ([randn(S, H)], lambda y: ops.moe_combine_masked(y, weights, rows)),
        "combine_backward": ([randn(T, H), randn(S, H)], lambda g, y: ops.moe_combine_backward(g, y, weights, rows)),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "grouped_gemm", "gate_up", "layer_few", "layer", "layer_many",
                                  "permute_masked", "dispatch", "dispatch_backward", "combine_masked", "combine_backward"])
def test_calls_wait_for_their_stream(ops, name):
    """Inputs that arrive on a side stream behind twenty large products: the call returns before
    they are there and computes from them, not from what the buffers held."""
    real, call = _stream_cases(ops)[name]
    as_tuple = lambda r: r if isinstance(r, tuple) else (r,)
    want = [t.clone() for t in as_tuple(call(*real))]
    late = [torch.zeros_like(t) for t in real]
    m = torch.randn(8192, 8192, device="cuda").to(torch.bfloat16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        product = torch.empty_like(m)
        torch.mm(m, m, out=product)
        call(*late)  # the side stream's buffers are there from here on
    torch.cuda.synchronize()
    arrived = torch.cuda.Event()
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.mm(m, m, out=product)
        for buffer, value in zip(late, real):
            buffer.copy_(value)
        arrived.record()
        got = as_tuple(call(*late))
        early = not arrived.query()
    s.synchronize()
    for g, v in zip(got, want):
        assert torch.equal(g, v)
    assert early
