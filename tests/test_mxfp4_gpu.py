"""GPU: the MXFP4 operators through the C ABI against the fp64 oracle.

Quantisation is compared bit for bit.  A product's bound counts fp32 roundings:
K of them at most along any path of a sum (2^-24 each, of the magnitudes summed)
and the half step of the result's type.  Buffers are filled with a pattern
before a call, so that a place that is not written, or written without reason,
shows.
"""

from __future__ import annotations

import numpy as np
import pytest

from oracle import mxfp4_oracle as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = [torch.float32, torch.float16, torch.bfloat16]
IDS = ["fp32", "fp16", "bf16"]


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


def _host(t: torch.Tensor) -> np.ndarray:
    return (t.float() if t.is_floating_point() else t).cpu().numpy()


def _random_mx(rng, *shape, low=120, high=130):
    *lead, K = shape
    words = rng.integers(0, 1 << 32, size=(*lead, K // 8), dtype=np.uint32).view(np.int32)
    scales = rng.integers(low, high + 1, size=(*lead, ref.mx_scale_bytes(K)), dtype=np.uint8)
    scales[..., K // 32:] = 255  # padding that would show as NaN
    return words, scales


def _gpu(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _close(got: torch.Tensor, want: np.ndarray, size: np.ndarray, K: int) -> None:
    """|got - want| within K fp32 roundings of the magnitudes and half a step of got's type."""
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * eps  # half a subnormal step
    off = np.abs(_host(got).astype(np.float64) - want)
    sums = K * 2.0 ** -24 * size
    bound = sums + eps * (np.abs(want) + sums) + tiny
    assert np.isfinite(_host(got)).all()
    assert (off <= bound).all(), f"worst {np.max(off - bound)} over its bound"


# ---- quantisation -----------------------------------------------------------------
def _special_rows(K: int) -> np.ndarray:
    """Rows that hold each border: ties, saturation, zeros of both signs, tiny and huge blocks."""
    rng = np.random.default_rng(7)
    rows = [np.zeros(K), -np.zeros(K), np.full(K, 7.99), np.full(K, -1.0)]
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0])
    for scale in (1.0, 2.0 ** -9, 2.0 ** 11):
        row = np.tile(np.concatenate([ties, -ties]), -(-K // 16))[:K] * scale
        rows += [row, np.nextafter(row.astype(np.float32), np.float32(np.inf)),
                 np.nextafter(row.astype(np.float32), np.float32(-np.inf))]
    rows += [rng.standard_normal(K) * 2.0 ** p for p in (-14, -24, 12)]
    return np.stack(rows).astype(np.float32)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("K", [32, 96, 128, 160, 2560])
def test_quantize_matches_the_oracle_bit_for_bit(ops, dtype, K):
    rows = np.concatenate([_special_rows(K), np.random.default_rng(K).standard_normal((37, K))
                           * np.exp(np.random.default_rng(1).standard_normal((37, 1)) * 4)])
    x = torch.from_numpy(rows.astype(np.float32)).to(dtype)
    want = ref.mx_pack(*ref.mx_quantize(x.float().numpy()))
    codes, scales = ops.moe_mxfp4_quantize(x.cuda())
    assert np.array_equal(_host(codes), want[0])
    assert np.array_equal(_host(scales), want[1])


def test_quantize_at_the_ends_of_fp32(ops):
    """Subnormal blocks, the largest finite values, infinities and NaN (blocks that read as NaN,
    their neighbours untouched)."""
    K = 128
    rng = np.random.default_rng(3)
    x = rng.standard_normal((12, K)).astype(np.float32)
    for i, p in enumerate((-149, -130, -127, -126, -125, -124, 126)):
        x[i] = np.ldexp(rng.uniform(1, 2, K), p).astype(np.float32)
    x[7] = np.float32(3.4028235e38)
    x[8, 5], x[8, 70] = np.inf, np.nan
    x[9, 33] = -np.inf
    want = ref.mx_pack(*ref.mx_quantize(x))
    codes, scales = ops.moe_mxfp4_quantize(_gpu(x))
    assert np.array_equal(_host(codes), want[0])
    assert np.array_equal(_host(scales), want[1])
    back = _host(ops.moe_mxfp4_dequantize(codes, scales, torch.float32))
    exact = ref.mx_values(*want)
    assert np.array_equal(np.isnan(back), np.isnan(exact))
    assert np.isnan(back[8, :32]).all() and not np.isnan(back[8, 32:64]).any()
    fine = ~np.isnan(exact)
    # values below 2^-149 round to a subnormal or zero, half a step off at most
    assert (np.abs(back[fine] - exact[fine]) <= 2.0 ** -150).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("K", [32, 96, 640])
def test_dequantize_rounds_once(ops, dtype, K):
    words, scales = _random_mx(np.random.default_rng(K), 33, K, low=113, high=140)
    scales[3, 0] = 255
    got = ops.moe_mxfp4_dequantize(_gpu(words), _gpu(scales), dtype)
    want = torch.from_numpy(ref.mx_values(words, scales)).to(dtype)
    assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(want))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_quantize_of_strided_unaligned_rows(ops, dtype):
    """Rows inside a wider buffer, at an address that is a multiple of the element only; the
    bytes around a dequantised slice stay."""
    R, K = 19, 160
    buf = torch.randn(R, K + 13, device="cuda").to(dtype)
    x = buf[:, 3:3 + K]
    codes, scales = ops.moe_mxfp4_quantize(x)
    want = ref.mx_pack(*ref.mx_quantize(_host(x)))
    assert np.array_equal(_host(codes), want[0]) and np.array_equal(_host(scales), want[1])
    back = torch.full_like(buf, 7.0)
    ops.moe_mxfp4_dequantize(codes, scales, dtype, out=back[:, 3:3 + K])
    assert np.array_equal(_host(back[:, 3:3 + K]), _host(ops.moe_mxfp4_dequantize(codes, scales, dtype)))
    assert (back[:, :3] == 7).all() and (back[:, 3 + K:] == 7).all()


@pytest.mark.parametrize("R", [1, 2, 127, 128, 129, 4097])
def test_quantize_row_counts(ops, R):
    x = torch.randn(R, 96, device="cuda", dtype=torch.bfloat16)
    want = ref.mx_pack(*ref.mx_quantize(_host(x)))
    codes, scales = ops.moe_mxfp4_quantize(x)
    assert np.array_equal(_host(codes), want[0]) and np.array_equal(_host(scales), want[1])


# ---- products ---------------------------------------------------------------------
def _offsets(rng, E, R, empty=0.3):
    """Segment borders with empty experts and one large one."""
    p = rng.random(E) * (rng.random(E) > empty) + 1e-9
    p[rng.integers(E)] += p.sum()
    counts = rng.multinomial(R, p / p.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


PRODUCTS = [  # E, rows, N, K
    (1, 1, 1, 32), (1, 1, 64, 128), (1, 17, 33, 160), (1, 300, 200, 512), (1, 129, 257, 1184),
    (3, 40, 96, 640), (8, 80, 80, 2560), (8, 1000, 130, 96), (37, 90, 48, 544), (512, 80, 64, 256),
    (64, 2500, 160, 256), (4096, 60, 32, 64), (2, 700, 320, 1024),
    (1, 1100, 300, 1440), (3, 2000, 520, 256), (16, 300, 260, 800), (16, 700, 136, 96),
    (1000, 12000, 64, 160), (600, 20000, 256, 96), (4096, 40000, 32, 64),
]


@pytest.mark.parametrize("E,R,N,K", PRODUCTS)
def test_grouped_gemm(ops, E, R, N, K):
    rng = np.random.default_rng(E * 1000 + R)
    a, w = _random_mx(rng, R, K), _random_mx(rng, E, N, K)
    off = _offsets(rng, E, R)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off)
    args = (_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off))
    for dtype in DTYPES:
        scale = 1.0
        out = torch.full((R, N), float("nan"), device="cuda", dtype=dtype)
        ops.moe_mxfp4_grouped_gemm(*args, out=out)
        _close(out, want * scale, size, K)
    again = ops.moe_mxfp4_grouped_gemm(*args, dtype=torch.bfloat16)
    assert torch.equal(again, out)


@pytest.mark.parametrize("E,R,N,K", [
    (1, 1, 1, 1568), (1, 37, 45, 2048), (5, 60, 200, 4000), (1, 16, 48, 16384), (1, 300, 130, 1600), (9, 50, 77, 1536),
    (200, 2000, 250, 2080), (500, 9000, 130, 96), (300, 9000, 200, 2080), (40, 4000, 900, 640),
    (70, 4900, 1000, 352), (3, 6000, 2100, 224), (1, 4001, 4200, 160), (2, 4300, 4100, 288),
])
def test_products_of_every_variant(ops, E, R, N, K):
    """Few columns over a K shared out to waves, then each of the tiles' shapes with odd ends; rows
    in order and mapped, bit for bit alike twice."""
    rng = np.random.default_rng(N)
    a, w = _random_mx(rng, R, K), _random_mx(rng, E, N, K)
    off = _offsets(rng, E, R, empty=0.0 if R < 100 else 0.2)
    values = ref.mx_values(*a), ref.mx_values(*w)
    args = (_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off))
    slots = rng.permutation(R).astype(np.int32)
    for rows, more in ((None, {}), (slots, {"row_slots": _gpu(slots)})):
        want, size = ref.mx_product(*values, off, rows)
        got = ops.moe_mxfp4_grouped_gemm(*args, **more)
        _close(got, want, size, K)
        assert torch.equal(got, ops.moe_mxfp4_grouped_gemm(*args, **more))


@pytest.mark.parametrize("R,N,K", [(1, 40, 96), (33, 128, 256), (515, 384, 544)])
def test_dense_product_without_offsets(ops, R, N, K):
    rng = np.random.default_rng(R)
    a, w = _random_mx(rng, R, K), _random_mx(rng, 1, N, K)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), [0, R])
    got = ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    _close(got, want, size, K)


@pytest.mark.parametrize("R,E", [(50, 4), (900, 3)])
def test_product_leaves_other_rows_and_columns_alone(ops, R, E):
    """Rows outside the segments, and the columns around a strided output, keep their values."""
    rng = np.random.default_rng(5)
    N, K = 70, 288
    a, w = _random_mx(rng, R, K), _random_mx(rng, E, N, K)
    off = _offsets(rng, E, R - 14) + np.int32(5)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off)
    for dtype in DTYPES:
        buf = torch.full((R, N + 9), 7.0, device="cuda", dtype=dtype)
        out = buf[:, 5:5 + N]
        ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off), out=out)
        lo, hi = int(off[0]), int(off[-1])
        _close(out[lo:hi], want[lo:hi], size[lo:hi], K)
        buf[lo:hi, 5:5 + N] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("seed", range(24))
def test_random_products(ops, seed):
    """Any sizes: dense and grouped, rows in order and mapped, strided outputs, gate/up."""
    rng = np.random.default_rng(1000 + seed)
    E = int(rng.choice([1, 2, 7, 64, 300, 700]))
    R = int(np.exp(rng.uniform(0, np.log(3000))))
    K = 32 * int(np.exp(rng.uniform(0, np.log(60))))
    N = int(np.exp(rng.uniform(0, np.log(900))))
    mapped = bool(rng.integers(2))
    k = int(rng.integers(1, 5)) if mapped else 1
    T = -(-R // k)
    a, w = _random_mx(rng, T if mapped else R, K), _random_mx(rng, E, N, K, low=118, high=124)
    slots = rng.integers(0, T * k, size=R).astype(np.int32)
    off = _offsets(rng, E, R)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off, slots // k if mapped else None)
    dtype = DTYPES[seed % 3]
    buf = torch.full((R, N + 3), 7.0, device="cuda", dtype=dtype)
    args = [_gpu(t) for t in (*a, *w, off)]
    more = {"row_slots": _gpu(slots), "top_k": k} if mapped else {}
    print(E, R, N, K, mapped, k, dtype, flush=True)
    out = ops.moe_mxfp4_grouped_gemm(*args, **more, out=buf[:, 2:2 + N])
    _close(out, want, size, K)
    assert (buf[:, :2] == 7).all() and (buf[:, 2 + N:] == 7).all()
    I = 32 * max(1, N // 64)
    w = _random_mx(rng, E, 2 * I, K, low=116, high=120)
    h, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off, slots // k if mapped else None)
    _check_act(*ops.moe_mxfp4_gate_up(args[0], args[1], _gpu(w[0]), _gpu(w[1]), args[4], **more), h, size, I, K)


def test_product_of_mapped_rows(ops):
    """row_slots: rows of tokens through the slots that hold them; a slot outside the tokens is a
    row of zeros."""
    rng = np.random.default_rng(11)
    T, k, E, N, K = 23, 3, 5, 96, 416
    S = T * k
    a, w = _random_mx(rng, T, K), _random_mx(rng, E, N, K)
    slots = rng.permutation(S).astype(np.int32)
    slots[[4, 40]] = [-1, S + 3]
    off = _offsets(rng, E, S)
    rows_of = np.where((slots >= 0) & (slots < S), slots // k, -1)
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off, rows_of)
    got = ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off),
                                     row_slots=_gpu(slots), top_k=k)
    _close(got, want, size, K)
    assert (got[4] == 0).all() and (got[40] == 0).all()


def test_product_past_32_bits(ops):
    """More than 2^32 bytes of output, and more than 2^31 of A's codes: rows near both ends."""
    rng = np.random.default_rng(6)
    R, N, K = 70000, 32768, 64
    a, w = _random_mx(rng, R, K), _random_mx(rng, 1, N, K)
    got = ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), dtype=torch.bfloat16)
    assert got.numel() * 2 > 1 << 32
    for rows in (slice(0, 3), slice(65534, 65538), slice(R - 3, R)):
        want, size = ref.mx_product(ref.mx_values(a[0][rows], a[1][rows]), ref.mx_values(*w), [0, rows.stop - rows.start])
        _close(got[rows], want, size, K)
    del got
    R, N, K = 140000, 32, 32768
    a_codes = torch.randint(-(1 << 31), 1 << 31, (R, K // 8), device="cuda", dtype=torch.int32)
    a_scales = torch.full((R, ref.mx_scale_bytes(K)), 126, device="cuda", dtype=torch.uint8)
    w = _random_mx(rng, 1, N, K)
    assert a_codes.numel() * 4 > 1 << 31
    got = ops.moe_mxfp4_grouped_gemm(a_codes, a_scales, _gpu(w[0]), _gpu(w[1]))
    slots = torch.arange(R, dtype=torch.int32, device="cuda")
    mapped = ops.moe_mxfp4_grouped_gemm(a_codes, a_scales, _gpu(w[0]), _gpu(w[1]), row_slots=slots)
    for rows in (slice(0, 3), slice(131070, 131075), slice(R - 3, R)):
        want, size = ref.mx_product(ref.mx_values(_host(a_codes[rows]), _host(a_scales[rows])), ref.mx_values(*w),
                                    [0, rows.stop - rows.start])
        _close(got[rows], want, size, K)
        _close(mapped[rows], want, size, K)


@pytest.mark.parametrize("R", [9, 700])
def test_nan_scales_reach_their_sums_only(ops, R):
    rng = np.random.default_rng(2)
    N, K = 96, 384
    a, w = _random_mx(rng, R, K), _random_mx(rng, 1, N, K)
    a[1][3, 5] = 255
    w[1][0, 17, 2] = 255
    want = np.isnan(ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), [0, R])[0])
    got = ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    assert np.array_equal(np.isnan(_host(got)), want)
    assert want[3].all() and want[:, 17].all() and want.sum() == R + N - 1


@pytest.mark.parametrize("R", [5, 400])
def test_product_at_the_ends_of_the_scales(ops, R):
    """Scale bytes 0 and 254, whose products with 2^0 stay in fp32's range."""
    rng = np.random.default_rng(4)
    K = 256
    a, w = _random_mx(rng, R, K, low=127, high=127), _random_mx(rng, 1, 64, K, low=127, high=127)
    w[1][0, :32, : K // 32] = 20
    w[1][0, 32:, : K // 32] = 240
    want, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), [0, R])
    got = ops.moe_mxfp4_grouped_gemm(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    _close(got, want, size, K)


# ---- gate/up ----------------------------------------------------------------------
def _check_act(codes, scales, h, size, I, K):
    """Stored MXFP4 against act = SiLU(gate) * up of exact sums h: the scale is that of a maximum
    within the sums' error, and each value within half an E2M1 step (or behind 6) of its act."""
    gate, up = h[:, :I], h[:, I:]
    act = gate / (1 + np.exp(-gate)) * up
    d = K * 2.0 ** -24 * size
    # |d act| <= |up| 1.1 d_gate + |SiLU(gate)| d_up + d_gate d_up, then a few fp32 roundings of
    # the value itself (exp, sum, quotient, product)
    err = 1.1 * np.abs(up) * d[:, :I] + np.abs(gate) * d[:, I:] + 1.1 * d[:, :I] * d[:, I:] + 8 * 2.0 ** -24 * np.abs(act)
    words, bytes_ = _host(codes), _host(scales)
    top = np.abs(act).reshape(len(act), -1, 32)
    e_err = err.reshape(top.shape)
    lo = ref.mx_exponent(np.maximum((top - e_err).max(axis=2), 0)) + 127
    hi = ref.mx_exponent((top + e_err).max(axis=2)) + 127
    b = bytes_[:, : I // 32].astype(np.int64)
    assert ((lo <= b) & (b <= hi)).all()
    assert (bytes_[:, I // 32:] == 127).all()
    unit = np.repeat(np.exp2(b - 127.0), 32, axis=1)
    m = (np.abs(act) + err) / unit
    half = np.where(m <= 2, 0.25, np.where(m <= 4, 0.5, np.where(m <= 6, 1.0, np.maximum(1.0, m - 6))))
    off = np.abs(ref.mx_values(words, bytes_) - act)
    assert (off <= half * unit + err).all()


@pytest.mark.parametrize("E,R,I,K", [(1, 1, 32, 32), (1, 20, 96, 160), (8, 80, 160, 2560),
                                     (5, 600, 64, 288), (512, 80, 32, 128), (2, 333, 640, 256),
                                     (16, 300, 160, 160), (16, 640, 96, 480), (1, 700, 96, 160), (2, 1500, 224, 416)])
def test_gate_up(ops, E, R, I, K):
    rng = np.random.default_rng(R + I)
    a = _random_mx(rng, R, K, low=124, high=126)
    w = _random_mx(rng, E, 2 * I, K, low=120, high=122)
    off = _offsets(rng, E, R)
    h, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off)
    out = (torch.full((R, I // 8), -1, dtype=torch.int32, device="cuda"),
           torch.full((R, ref.mx_scale_bytes(I)), 255, dtype=torch.uint8, device="cuda"))
    codes, scales = ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off),
                                          out=out)
    _check_act(codes, scales, h, size, I, K)


@pytest.mark.parametrize("E,R,I,K", [(1, 5, 64, 1568), (8, 40, 96, 2080), (3, 20, 32, 4096), (2, 1, 160, 8192)])
def test_gate_up_of_few_rows_with_long_sums(ops, E, R, I, K):
    rng = np.random.default_rng(K)
    a = _random_mx(rng, R, K, low=124, high=126)
    w = _random_mx(rng, E, 2 * I, K, low=120, high=122)
    off = _offsets(rng, E, R)
    h, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off)
    _check_act(*ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off)), h, size, I, K)


@pytest.mark.parametrize("E,R,I,K", [(300, 9000, 96, 2080), (40, 4000, 448, 640), (70, 4900, 512, 352),
                                     (500, 9000, 64, 96), (1, 3001, 2720, 160), (200, 2000, 160, 2080),
                                     (1, 200, 96, 1600), (2, 70, 64, 224)])
def test_gate_up_of_every_variant(ops, E, R, I, K):
    """Each of the tiles' shapes, and few tiles, with odd ends; rows mapped."""
    rng = np.random.default_rng(I)
    a = _random_mx(rng, R, K, low=124, high=126)
    w = _random_mx(rng, E, 2 * I, K, low=120, high=122)
    off = _offsets(rng, E, R)
    slots = rng.permutation(R).astype(np.int32)
    h, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off, slots)
    args = (_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off), _gpu(slots))
    got = ops.moe_mxfp4_gate_up(*args)
    _check_act(*got, h, size, I, K)
    for x, y in zip(got, ops.moe_mxfp4_gate_up(*args)):
        assert torch.equal(x, y)


def test_gate_up_of_mapped_rows_leaves_other_rows_alone(ops):
    rng = np.random.default_rng(12)
    T, k, E, I, K = 30, 4, 6, 96, 160
    S = T * k
    a, w = _random_mx(rng, T, K, low=124, high=126), _random_mx(rng, E, 2 * I, K, low=120, high=122)
    slots = rng.permutation(S).astype(np.int32)
    off = _offsets(rng, E, S - 10)
    h, size = ref.mx_product(ref.mx_values(*a), ref.mx_values(*w), off, slots // k)
    out = (torch.full((S, I // 8), -5, dtype=torch.int32, device="cuda"),
           torch.full((S, ref.mx_scale_bytes(I)), 99, dtype=torch.uint8, device="cuda"))
    codes, scales = ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]), _gpu(off),
                                          row_slots=_gpu(slots), top_k=k, out=out)
    n = int(off[-1])
    _check_act(codes[:n], scales[:n], h[:n], size[:n], I, K)
    assert (codes[n:] == -5).all() and (scales[n:] == 99).all()


@pytest.mark.parametrize("R", [4, 40, 300])
def test_gate_up_of_a_nan_row_is_a_nan_row(ops, R):
    """A NaN scale in a token's row: scale byte 255 and zero codes in all its blocks, the other
    rows as without it."""
    rng = np.random.default_rng(R)
    I, K = 96, 256
    a, w = _random_mx(rng, R, K, low=124, high=126), _random_mx(rng, 1, 2 * I, K, low=120, high=122)
    clean = ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    a[1][2, 3] = 255
    codes, scales = ops.moe_mxfp4_gate_up(_gpu(a[0]), _gpu(a[1]), _gpu(w[0]), _gpu(w[1]))
    assert (codes[2] == 0).all() and (scales[2, : I // 32] == 255).all()
    keep = [r for r in range(R) if r != 2]
    assert torch.equal(codes[keep], clean[0][keep]) and torch.equal(scales[keep], clean[1][keep])


# ---- the layer --------------------------------------------------------------------
def _layer_inputs(rng, T, E, H, I, dtype):
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).cuda().to(dtype)
    w13, w2 = _random_mx(rng, E, 2 * I, H, low=120, high=122), _random_mx(rng, E, H, I, low=121, high=123)
    w = {"w13_codes": _gpu(w13[0]), "w13_scales": _gpu(w13[1]), "w2_codes": _gpu(w2[0]),
         "w2_scales": _gpu(w2[1])}
    return logits, x, w, ref.mx_values(*w13), ref.mx_values(*w2)


def _layer_steps(ops, logits, x, k, w):
    """The layer as the separate calls, in its documented order."""
    E = logits.shape[1]
    ids, weights, perm = ops.moe_route_permute(logits, k)
    xq = ops.moe_mxfp4_quantize(x)
    act = ops.moe_mxfp4_gate_up(*xq, w["w13_codes"], w["w13_scales"], perm["expert_offsets"],
                                row_slots=perm["sorted_slots"], top_k=k)
    y = ops.moe_mxfp4_grouped_gemm(*act, w["w2_codes"], w["w2_scales"], perm["expert_offsets"])
    return ops.moe_combine_masked(y, weights, perm["slot_rows"], dtype=x.dtype)


LAYERS = [  # T, E, k, H, I
    (1, 8, 2, 256, 128), (4, 8, 2, 256, 128), (9, 37, 5, 96, 160), (63, 4, 4, 160, 96),
    (130, 16, 3, 288, 64), (700, 8, 2, 128, 96), (8, 512, 10, 256, 64),
    (2, 4, 4, 96, 32), (3, 100, 20, 544, 96), (4, 1000, 16, 1056, 224), (4, 200, 16, 64, 1088), (1, 64, 64, 128, 32),
    (5, 8, 3, 256, 96), (4, 8, 8, 2592, 64),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,E,k,H,I", LAYERS)
def test_layer_is_its_calls_and_near_the_oracle(ops, T, E, k, H, I, dtype):
    logits, x, w, w13, w2 = _layer_inputs(np.random.default_rng(T), T, E, H, I, dtype)
    ws = torch.full((ops.mxfp4_layer_workspace_bytes(T, k, E, H, I),), 255, dtype=torch.uint8, device="cuda")
    out = ops.moe_mxfp4_layer_forward(logits, x, k, w, workspace=ws)
    assert torch.equal(out, _layer_steps(ops, logits, x, k, w))
    assert torch.equal(out, ops.moe_mxfp4_layer_forward(logits, x, k, w))
    n = min(T, 40)
    want = ref.mx_layer(logits[:n].cpu().numpy(), _host(x[:n]), k, w13, w2)
    off = _host(out[:n]) - want
    # the layer's parity bar (relative RMS 1e-2): above bf16's rounding (2^-9 RMS) and the rare act
    # whose fp32 sum falls on the other side of a rounding border
    assert np.sqrt((off ** 2).sum() / (want ** 2).sum()) <= 1e-2


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,E,k,H,I", [
    (5, 512, 10, 256, 64), (6, 1000, 10, 96, 32), (6, 4, 4, 160, 1088), (6, 8, 2, 16384, 32), (5, 1024, 12, 64, 544),
    (4, 16, 16, 128, 1056), (6, 1, 1, 64, 2080), (2, 32, 32, 64, 96), (7, 64, 9, 128, 64), (6, 20, 11, 64, 64),
])
def test_layer_of_few_tokens_is_its_calls(ops, T, E, k, H, I, dtype):
    """Around the two-launch form's limits (6 tokens, 64 slots, 1024 experts, 16384 columns): many
    experts per wave, one or several windows of I, all slots on one expert, whole waves of slots."""
    logits, x, w, w13, w2 = _layer_inputs(np.random.default_rng(T * E), T, E, H, I, dtype)
    for same in (False, True):
        if same:  # every token the same experts
            logits[:] = logits[0].clone()
        out = ops.moe_mxfp4_layer_forward(logits, x, k, w)
        assert torch.equal(out, ops.moe_mxfp4_layer_forward(logits, x, k, w))
        want = ref.mx_layer(logits.cpu().numpy(), _host(x), k, w13, w2)
        for got in (out, _layer_steps(ops, logits, x, k, w)):
            assert np.sqrt(((_host(got) - want) ** 2).sum() / (want ** 2).sum()) <= 1e-2


def test_a_model_s_weights_through_the_layer(ops):
    """Float weights quantised at load time, expert by expert rows at once, then a decode and a
    prefill call on them."""
    rng = np.random.default_rng(17)
    E, k, H, I = 6, 2, 192, 96
    w13 = torch.from_numpy(rng.standard_normal((E, 2 * I, H)).astype(np.float32)).cuda() / H ** 0.5
    w2 = torch.from_numpy(rng.standard_normal((E, H, I)).astype(np.float32)).cuda() / I ** 0.5
    w, values = {}, {}
    for name, t in (("w13", w13), ("w2", w2)):
        codes, scales = ops.moe_mxfp4_quantize(t.flatten(0, 1))
        w[name + "_codes"], w[name + "_scales"] = (a.view(*t.shape[:2], -1) for a in (codes, scales))
        values[name] = ref.mx_values(_host(w[name + "_codes"]), _host(w[name + "_scales"]))
        assert np.array_equal(values[name], ref.mx_values(*ref.mx_pack(*ref.mx_quantize(_host(t.flatten(0, 1))))).reshape(t.shape))
    for T in (1, 30):
        logits = torch.randn(T, E, device="cuda")
        x = torch.randn(T, H, device="cuda", dtype=torch.float16)
        out = ops.moe_mxfp4_layer_forward(logits, x, k, w)
        want = ref.mx_layer(logits.cpu().numpy(), _host(x), k, values["w13"], values["w2"])
        assert np.sqrt(((_host(out) - want) ** 2).sum() / (want ** 2).sum()) <= 1e-2


@pytest.mark.parametrize("T,E,k", [(1, 512, 10), (3, 100, 7), (4, 37, 16), (1, 1000, 60), (9, 64, 5)])
def test_layer_with_tied_logits(ops, T, E, k):
    """Few distinct logits, all equal ones, and a list of choices longer than a wave's lanes hold:
    the lower expert comes first, as everywhere."""
    rng = np.random.default_rng(E)
    H, I = 128, 32
    logits, x, w, w13, w2 = _layer_inputs(rng, T, E, H, I, torch.float32)
    for step in (1.0, 100.0, 0.01):
        tied = torch.round(logits / step) * step
        out = ops.moe_mxfp4_layer_forward(tied, x, k, w)
        assert torch.equal(out, _layer_steps(ops, tied, x, k, w))
        want = ref.mx_layer(tied.cpu().numpy(), _host(x), k, w13, w2)
        assert np.sqrt(((_host(out) - want) ** 2).sum() / (want ** 2).sum()) <= 1e-2


def test_layer_in_a_graph_replayed(ops):
    """Replays with new inputs in the captured buffers, eager work between them."""
    rng = np.random.default_rng(8)
    T, E, k, H, I = 8, 64, 6, 256, 96
    logits, x, w, _, _ = _layer_inputs(rng, T, E, H, I, torch.bfloat16)
    ws = torch.empty(ops.mxfp4_layer_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    ops.moe_mxfp4_layer_forward(logits, x, k, w, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.moe_mxfp4_layer_forward(logits, x, k, w, workspace=ws, out=out)
    for i in range(4):
        new_logits, new_x, _, _, _ = _layer_inputs(rng, T, E, 256, 32, torch.bfloat16)
        logits.copy_(new_logits)
        x.copy_(new_x)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _layer_steps(ops, logits, x, k, w)), f"replay {i}"


@pytest.mark.parametrize("T", [1, 3, 100])
def test_two_layers_in_a_graph_share_buffers(ops, T):
    """Two layers in a row, the second reading the first's output, both with one workspace, replayed
    with new inputs: the calls of a captured model step."""
    rng = np.random.default_rng(T)
    E, k, H, I = 40, 4, 192, 96
    logits, x, w, _, _ = _layer_inputs(rng, T, E, H, I, torch.bfloat16)
    more, _, w2, _, _ = _layer_inputs(rng, T, E, H, I, torch.bfloat16)
    ws = torch.empty(ops.mxfp4_layer_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device="cuda")
    mid, out = torch.empty_like(x), torch.empty_like(x)

    def step(mid, out, ws):
        ops.moe_mxfp4_layer_forward(logits, x, k, w, workspace=ws, out=mid)
        ops.moe_mxfp4_layer_forward(more, mid, k, w2, workspace=ws, out=out)

    step(mid, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(mid, out, ws)
    for i in range(4):
        logits.copy_(torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
        x.copy_(torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)))
        want = torch.empty_like(out)
        step(torch.empty_like(mid), want, torch.empty_like(ws))
        out.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.isfinite(out).all(), f"replay {i}"
    # a layer's output may take the place of its input
    y = x.clone()
    ops.moe_mxfp4_layer_forward(logits, y, k, w, out=y)
    assert torch.equal(y, mid)


def test_calls_follow_the_current_stream(ops):
    """Work on a side stream: the call waits for its inputs there, not on the default stream."""
    s = torch.cuda.Stream()
    x = torch.randn(512, 2560, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            x = x * 1.0001
        codes, scales = ops.moe_mxfp4_quantize(x)
    s.synchronize()
    again = ops.moe_mxfp4_quantize(x)
    assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])


def test_empty_calls(ops):
    x = torch.empty(0, 64, device="cuda")
    codes, scales = ops.moe_mxfp4_quantize(x)
    assert codes.shape == (0, 8) and ops.moe_mxfp4_dequantize(codes, scales).shape == (0, 64)
    w = _random_mx(np.random.default_rng(0), 2, 32, 64)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert ops.moe_mxfp4_grouped_gemm(codes, scales, _gpu(w[0]), _gpu(w[1]), off).shape == (0, 32)
