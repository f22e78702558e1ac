"""CPU: what AdamW refuses before anything reaches a GPU."""

import ctypes
import os

import pytest

from w4a16_group_quantized_amd import ops

torch = pytest.importorskip("torch")

BAD = ops.MOE_ERR_INVALID_ARG
FP32, BF16 = 0, 2


@pytest.fixture(scope="module", autouse=True)
def _built_library():
    if not os.path.exists(ops.LIB_PATH):
        from w4a16_group_quantized_amd import build_lib

        build_lib.build()


# ---- buffers that share memory ------------------------------------------------------------
def _table(count, n, bits, copies=True):
    """`count` tensors of n elements in fp32, bf16 copies, all apart: addresses that are never used."""
    at = 0x100000

    def take(size):
        nonlocal at
        at += size + -size % 16
        return at - size - -size % 16

    rows, blocks = [], -(-n // ops.ADAMW_BLOCK) * 4
    for _ in range(count):
        rows.append({"n": n, "param": take(4 * n), "grad": take(4 * n), "m": take(n * bits // 8), "v": take(n * bits // 8),
                     "ms": take(blocks), "vs": take(blocks), "copy": take(2 * n) if copies else 0, "types": FP32,
                     "copy_type": BF16})
    return rows


def _step(rows, bits, scale=None):
    flat = [x for r in rows for x in r.values()]
    return ops.load_library().moe_adamw((ctypes.c_int64 * len(flat))(*flat), len(rows), bits, 1e-3, 0.9, 0.999, 1e-8,
                                        0.0, 1, 0, scale, None)


# (field of tensor i, bytes to move it by) takes the place of a field of tensor j
SHARED = [
    ("param", 0, "param", 1, 0), ("param", 0, "m", 0, 0), ("m", 0, "v", 0, 0), ("copy", 1, "copy", 0, 0),
    ("param", 0, "param", 1, 4), ("param", 0, "param", 1, 4 * 299), ("param", 1, "m", 0, -4), ("copy", 0, "v", 1, 596),
    ("grad", 0, "copy", 0, 0), ("grad", 0, "copy", 1, 1196), ("grad", 1, "param", 0, -4), ("m", 0, "grad", 0, 0),
]
SHARED_SCALES = [("ms", 0, "ms", 1, 0), ("ms", 0, "vs", 0, 0), ("vs", 1, "vs", 0, 8), ("m", 0, "vs", 0, 0),
                 ("ms", 0, "grad", 1, -4 * 299)]


@pytest.mark.parametrize("bits,place", [(b, p) for b in (32, 8) for p in SHARED] + [(8, p) for p in SHARED_SCALES])
def test_adamw_refuses_buffers_that_overlap(bits, place):
    field, i, other, j, move = place
    rows = _table(2, 300, bits)
    rows[j][other] = rows[i][field] + move
    assert _step(rows, bits) == BAD


def test_adamw_refuses_overlaps_among_many():
    for bits in (32, 8):
        rows = _table(300, 1000, bits)
        rows[290]["m"] = rows[3]["copy"] + 1996
        assert _step(rows, bits) == BAD


def test_adamw_refuses_a_gradients_scale_that_it_writes():
    rows = _table(2, 300, 32)
    for place in (rows[1]["v"] + 1196, rows[0]["param"]):
        assert _step(rows, 32, place) == BAD


def test_binding_names_tensors_that_overlap():
    flat = torch.zeros(64)
    p, q, g = flat[:32], flat[32:], torch.zeros(32)
    (m, v), (m2, v2) = ops.adamw_states(p), ops.adamw_states(p)
    (m8, v8), (m9, v9) = ops.adamw_states(p, 8), ops.adamw_states(p, 8)
    call = lambda *lists, **kw: ops.moe_adamw(*lists, lr=1e-3, step=1, seed=1, **kw)  # noqa: E731
    for args, kw, match in (
            (([p, flat[31:63]], [g, g], [m, m2], [v, v2]), {}, r"params\[1\] overlaps params\[0\]"),
            (([p, q], [g, g], [m8, (m9[0], m8[1])], [v8, v9]), {}, r"m scales\[1\] overlaps m scales\[0\]"),
            (([p], [g], [m8], [(v8[0], m8[1])]), {}, r"overlaps m scales\[0\]"),
            (([p], [q], [m], [v]), {"copies": [flat[33:].new_zeros(32)]}, "not on a GPU"),
            (([p], [g], [m], [v]), {"copies": [g]}, r"overlaps copies\[0\]"),
            (([p], [g], [m], [v]), {"grad_scale": v[3:4]}, r"grad_scale\[0\] overlaps v\[0\]"),
            # halves of one buffer, and one gradient for both, are no overlap
            (([p, q], [g, g], [m, m2], [v, v2]), {}, "not on a GPU")):
        with pytest.raises(ValueError, match=match):
            call(*args, **kw)
