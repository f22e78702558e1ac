"""CPU: refusals of the MXFP4 and dispatch entry points (nothing reaches a GPU),
and pins of their oracle."""

import os

import numpy as np
import pytest

from oracle import mxfp4_oracle as ref
from w4a16_group_quantized_amd import ops

torch = pytest.importorskip("torch")

FAKE = 0x1000  # aligned and never dereferenced: validation fails first
BAD, UNSUPPORTED, WORKSPACE = ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED, ops.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module", autouse=True)
def _built_library():
    if not os.path.exists(ops.LIB_PATH):
        from w4a16_group_quantized_amd import build_lib

        build_lib.build()


# ---- refusals through the C ABI ---------------------------------------------------
def _quantize(x=FAKE, dtype=1, rows=4, K=64, stride=64, codes=FAKE, scales=FAKE):
    return ops.load_library().moe_mxfp4_quantize(x, dtype, rows, K, stride, codes, scales, None)


@pytest.mark.parametrize("args,status", [
    ({"K": 48}, BAD), ({"K": 0}, BAD), ({"K": 65568, "stride": 65568}, UNSUPPORTED), ({"rows": -1}, BAD),
    ({"rows": 1 << 31}, UNSUPPORTED), ({"dtype": 3}, BAD), ({"dtype": -1}, BAD), ({"stride": 63}, BAD),
    ({"stride": (1 << 31) + 1}, UNSUPPORTED), ({"x": None}, BAD), ({"x": FAKE + 1}, BAD),
    ({"codes": FAKE + 8}, BAD), ({"scales": None}, BAD), ({"dtype": 0, "x": FAKE + 2}, BAD),
    ({"rows": 0, "x": None, "codes": None, "scales": None}, ops.MOE_OK),
])
def test_quantize_refusals(args, status):
    assert _quantize(**args) == status
    lib = ops.load_library()
    a = {"x": FAKE, "dtype": 1, "rows": 4, "K": 64, "stride": 64, "codes": FAKE, "scales": FAKE, **args}
    assert lib.moe_mxfp4_dequantize(a["codes"], a["scales"], a["rows"], a["K"], a["x"], a["dtype"],
                                    a["stride"], None) == status


def _gemm(a_codes=FAKE, a_rows=8, row_slots=None, top_k=1, rows=8, offsets=FAKE, E=2, w=FAKE, N=32, K=64,
          out=FAKE, dtype=0, stride=32):
    return ops.load_library().moe_mxfp4_grouped_gemm(a_codes, FAKE, a_rows, row_slots, top_k, rows, offsets,
                                                     E, w, FAKE, N, K, out, dtype, stride, None)


@pytest.mark.parametrize("args,status", [
    ({"K": 33}, BAD), ({"N": 0}, BAD), ({"E": 0}, BAD), ({"E": 4097}, UNSUPPORTED),
    ({"offsets": None}, BAD), ({"rows": 9}, BAD), ({"rows": -1}, BAD),
    ({"row_slots": FAKE, "top_k": 0}, BAD), ({"row_slots": FAKE + 4}, BAD), ({"stride": 31}, BAD),
    ({"dtype": 5}, BAD), ({"N": 65537, "stride": 65537}, UNSUPPORTED),
    ({"N": 65536, "K": 65536, "stride": 65536}, UNSUPPORTED),
    ({"rows": (1 << 27) + 1, "a_rows": 1 << 28}, UNSUPPORTED), ({"out": None}, BAD), ({"out": FAKE + 2}, BAD),
    ({"a_codes": None}, BAD), ({"w": FAKE + 4}, BAD),
    ({"rows": 0, "a_codes": None, "out": None, "w": None}, ops.MOE_OK),
])
def test_product_refusals(args, status):
    assert _gemm(**args) == status


def test_gate_up_refusals():
    lib = ops.load_library()

    def call(I=32, H=64, rows=8, act=FAKE, E=1):
        return lib.moe_mxfp4_gate_up(FAKE, FAKE, 8, None, 1, rows, FAKE, E, FAKE, FAKE, I, H, act, FAKE, None)

    assert call(I=16) == BAD and call(I=0) == BAD and call(I=32800) == UNSUPPORTED
    assert call(H=40) == BAD and call(act=None) == BAD and call(rows=9) == BAD
    assert call(rows=0, act=None) == ops.MOE_OK


def test_layer_refusals_and_workspace():
    lib = ops.load_library()

    def call(T=4, E=8, k=2, H=256, I=128, dtype=2, ws=1 << 40, x=FAKE):
        return lib.moe_mxfp4_layer_forward(FAKE, x, dtype, T, E, k, FAKE, FAKE, FAKE, FAKE, H, I, FAKE, FAKE,
                                           ws, None)

    assert call(k=9) == BAD and call(H=250) == BAD and call(I=100) == BAD and call(dtype=7) == BAD
    assert call(E=5000) == UNSUPPORTED and call(k=65, E=100) == UNSUPPORTED
    assert call(x=None) == BAD and call(T=-1) == BAD
    need = ops.mxfp4_layer_workspace_bytes(4, 2, 8, 256, 128)
    assert need > 8 * 256 * 4 and call(ws=need - 1) == WORKSPACE
    assert call(T=0, x=None) == ops.MOE_OK
    assert ops.mxfp4_layer_workspace_bytes(4, 9, 8, 256, 128) == 0


def test_permute_masked_refusals():
    lib = ops.load_library()

    def call(ids=FAKE, T=4, k=2, first=0, E=8, ws=None, ws_bytes=0):
        return lib.moe_permute_masked(ids, T, k, first, E, *[FAKE] * 5, ws, ws_bytes, None)

    assert call(ids=None) == BAD and call(T=-1) == BAD and call(k=0) == BAD and call(E=0) == BAD
    assert call(first=-1) == BAD and call(E=4097) == UNSUPPORTED and call(k=65) == UNSUPPORTED
    assert call(T=1 << 30, k=2) == UNSUPPORTED and call(first=(1 << 31) - 1) == UNSUPPORTED
    assert call(T=1000) == WORKSPACE
    need = ops.permute_masked_workspace_bytes(1000, 2, 8)
    assert call(T=1000, ws=None, ws_bytes=need) == BAD
    assert call(T=0, ids=None) == ops.MOE_OK
    assert ops.permute_masked_workspace_bytes(512, 2, 8) == 0
    assert ops.permute_masked_workspace_bytes(513, 2, 8) > 0


@pytest.mark.parametrize("args,status", [
    ({"T": -1}, BAD), ({"k": 0}, BAD), ({"k": 65}, UNSUPPORTED), ({"H": 0}, BAD), ({"H": 65537, "s": 65537}, UNSUPPORTED),
    ({"s": 4}, BAD), ({"dtype": 3}, BAD), ({"rows": -1}, BAD), ({"rows": 1 << 31}, UNSUPPORTED),
    ({"slots": None}, BAD), ({"x": None}, BAD), ({"x": FAKE + 1}, BAD), ({"T": 0, "x": None, "slots": None}, ops.MOE_OK),
])
def test_dispatch_and_combine_refusals(args, status):
    lib = ops.load_library()
    a = {"x": FAKE, "dtype": 1, "T": 3, "k": 2, "H": 5, "s": 5, "slots": FAKE, "rows": 6, **args}
    x, d, T, k, H, s, slots, rows = (a[n] for n in ("x", "dtype", "T", "k", "H", "s", "slots", "rows"))
    assert lib.moe_dispatch(x, d, T, k, H, s, slots, rows, FAKE, s, None) == status
    assert lib.moe_dispatch_backward(FAKE, d, T, k, H, s, slots, rows, x, s, None) == status
    assert lib.moe_combine_masked(x, d, T, k, H, s, FAKE, slots, rows, FAKE, d, s, None) == status
    assert lib.moe_combine_backward(x, d, s, FAKE, d, s, FAKE, slots, T, k, H, rows, FAKE, s, FAKE, None) == status


# ---- refusals in the binding --------------------------------------------------------
def test_tensors_off_the_gpu_are_refused():
    x = torch.zeros(4, 64)
    rows = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on a GPU"):
        ops.moe_mxfp4_quantize(x)
    with pytest.raises(ValueError, match="not on a GPU"):
        ops.moe_dispatch(x, rows, 2)
    with pytest.raises(ValueError, match="not on a GPU"):
        ops.moe_permute_masked(rows.view(4, 2), 8)
    with pytest.raises(ValueError, match="not on a GPU"):
        ops.moe_combine_backward(x, torch.zeros(8, 64), torch.zeros(4, 2), rows)


def test_shapes_types_and_layouts_are_refused():
    codes, scales = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 4, dtype=torch.uint8)
    w = torch.zeros(2, 32, 8, dtype=torch.int32), torch.zeros(2, 32, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="multiple of 32"):
        ops.moe_mxfp4_quantize(torch.zeros(4, 40))
    with pytest.raises(ValueError, match="float32"):
        ops.moe_mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous rows"):
        ops.moe_mxfp4_quantize(torch.zeros(64, 4).t())
    with pytest.raises(ValueError, match="overlap"):
        ops.moe_mxfp4_quantize(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError, match="scales"):
        ops.moe_mxfp4_dequantize(codes, scales[:, :2].contiguous())
    with pytest.raises(ValueError, match="columns"):
        ops.moe_mxfp4_grouped_gemm(codes[:, :4].contiguous(), scales, *w)
    with pytest.raises(ValueError, match="expert_offsets"):
        ops.moe_mxfp4_grouped_gemm(codes, scales, *w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="expert_offsets"):
        ops.moe_mxfp4_grouped_gemm(codes, scales, *w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="multiple of 64"):
        ops.moe_mxfp4_gate_up(codes, scales, *w, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="slot_rows"):
        ops.moe_dispatch(torch.zeros(4, 64), torch.zeros(9, dtype=torch.int32), 2)


def test_overlapping_outputs_are_refused():
    buf = torch.zeros(20, 16)
    ops._apart("out", buf[:8, :8], x=buf[:8, 8:])  # column ranges of one buffer
    ops._apart("out", buf[:8], x=buf[8:])
    ops._apart("out", buf[:0], x=buf)
    for a, b in ((buf[:8], buf[7:]), (buf[:8, :8], buf[:8, 7:15]), (buf[:, 4:12], buf[:, :5]), (buf, buf)):
        with pytest.raises(ValueError, match="overlaps"):
            ops._apart("out", a, x=b)


# ---- oracle pins --------------------------------------------------------------------
def test_oracle_codes_by_hand():
    x = np.zeros((1, 32))
    x[0, :12] = [4.0, -6.0, 0.25, 0.26, 0.75, 1.25, 2.5, 3.5, 5.0, 5.01, 7.9, -0.3]
    codes, scales = ref.mx_quantize(x)
    assert scales[0, 0] == 127  # max 7.9: floor(log2) = 2, exponent 0
    assert codes[0, :12].tolist() == [6, 15, 0, 1, 2, 2, 4, 6, 6, 7, 7, 9]
    codes, scales = ref.mx_quantize(x * 2.0 ** 5)
    assert scales[0, 0] == 132 and codes[0, :12].tolist() == [6, 15, 0, 1, 2, 2, 4, 6, 6, 7, 7, 9]
    assert ref.mx_quantize(np.full((1, 32), 8.0))[1][0, 0] == 128
    assert ref.mx_quantize(np.zeros((1, 32)))[1][0, 0] == 0


def test_oracle_packs_low_nibble_first_and_pads_scales():
    words, scales = ref.mx_pack(np.arange(64, dtype=np.uint8).reshape(1, 64) % 16, np.array([[5, 6]], np.uint8))
    assert words.view(np.uint32)[0, 0] == 0x76543210 and words.view(np.uint32)[0, 1] == 0xFEDCBA98
    assert scales.tolist() == [[5, 6, 127, 127]]
    v = ref.mx_values(words, scales)
    assert v[0, 7] == 6 * 2.0 ** -122 and v[0, 41] == -0.5 * 2.0 ** -121


def test_oracle_product_of_ones():
    one = ref.mx_pack(np.full((3, 64), 2, np.uint8), np.full((3, 2), 127, np.uint8))
    out, size = ref.mx_product(ref.mx_values(*one), ref.mx_values(one[0][None], one[1][None]), [0, 2])
    assert (out[:2] == 64).all() and (out[2] == 0).all() and (size[:2] == 64).all()


def test_oracle_permutation_by_hand():
    p = ref.permute_masked(np.array([[1, 5], [-1, 1], [0, 9]], np.int32), 2)
    assert p["expert_offsets"].tolist() == [0, 1, 3]
    assert p["sorted_slots"].tolist() == [4, 0, 3, -1, -1, -1]
    assert p["slot_rows"].tolist() == [1, -1, -1, 2, 0, -1]
    assert p["active_experts"].tolist() == [0, 1] and p["num_active"].tolist() == [2]


def test_oracle_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0], [5.0, 5.0]])
    out, size = ref.combine_masked(y, np.array([[0.5, 2.0], [3.0, -1.0]]), np.array([1, -1, 0, 7]))
    assert out.tolist() == [[5.0, 10.0], [3.0, 6.0]] and (size == out).all()
    gy, gw, _ = ref.combine_backward(np.array([[1.0, 1.0], [2.0, 0.0]]), y, np.array([[0.5, 2.0], [3.0, -1.0]]),
                                     np.array([1, -1, 0, 7]), np.full((3, 2), 9.0))
    assert gy.tolist() == [[6.0, 0.0], [0.5, 0.5], [9.0, 9.0]]
    assert gw.tolist() == [[30.0, 0.0], [2.0, 0.0]]
