"""CPU: what AdamW refuses before anything reaches a GPU, and how its 8-bit states have to be rounded."""

import ctypes
import os

import numpy as np
import pytest

from oracle import train_oracle as ref
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


# ---- why states are rounded by chance, and by another one at every step -------------------
def decays(signed, beta, steps, round_codes):
    """What is left of an 8-bit state's sum, over what should be, when one element per block keeps its block's
    scale and the others, between a quarter and the whole of a unit, get no gradients."""
    n = 1 << 13
    x = np.random.default_rng(0).uniform(0.25, 1.0, n)
    x[:: ref.BLOCK] = 3.0
    held = np.arange(n) % ref.BLOCK == 0
    scale = np.repeat(ref.block_scales(x), ref.BLOCK)
    values = ref.code_values(signed)
    x = values[round_codes(x, scale, 0, signed)] * scale
    first = x[~held].sum()
    for step in range(1, steps + 1):
        x = np.where(held, 3.0, beta * x)
        x = values[round_codes(x, scale, step, signed)] * scale
    return x[~held].sum() / first / beta ** steps


@pytest.mark.parametrize("signed,beta,steps", [(False, 0.999, 300), (True, 0.99, 60)])
def test_moments_follow_only_with_another_noise_each_step(signed, beta, steps):
    def by(noise):
        return lambda x, scale, step, signed: ref.code_sizes(x, scale, noise(x.size, step), signed)

    which = 0 if signed else 1
    each = decays(signed, beta, steps, by(lambda n, step: ref.noise(n, step, which) / 2.0 ** 20))
    once = decays(signed, beta, steps, by(lambda n, step: ref.noise(n, 0, which) / 2.0 ** 20))
    near = decays(signed, beta, steps, by(lambda n, step: np.full(n, 0.5)))
    # A code's step is at most an eighth of its value x, and a decay of (1 - beta) x is rounded to it or not: a
    # variance of (1 - beta) x^2 / 8 at most.  Over the steps and elements, x^2 in the mean 1.12 times the mean's
    # square, the sum's deviation is sqrt(steps (1 - beta) / 8 * 1.12 / n) of the first sum: five of them, over
    # what is left
    five = 5 * (steps * (1 - beta) / 8 * 1.12 / (1 << 13)) ** 0.5 / beta ** steps
    assert abs(each - 1) < five
    # the nearest code is the same one again where (1 - beta) is under half of a sixteenth: nothing decays
    assert near == pytest.approx(beta ** -steps)
    assert abs(once - 1) > 2 * five


# ---- scalars that fp32 does not hold -------------------------------------------------------
@pytest.mark.parametrize("lr,beta1,decay,step", [(1e39, 0.9, 0.0, 1), (1e38, 0.9, 0.0, 1), (1e30, 1 - 1e-9, 0.0, 1),
                                                 (1e20, 0.9, 1e19, 1000)])
def test_adamw_refuses_rates_past_fp32(lr, beta1, decay, step):
    """lr / (1 - beta1^step) or lr wd would be infinite, and NaN where it meets a zero."""
    rows = [x for r in _table(1, 300, 32) for x in r.values()]
    table = (ctypes.c_int64 * len(rows))(*rows)
    assert ops.load_library().moe_adamw(table, 1, 32, lr, beta1, 0.999, 1e-8, decay, step, 0, None, None) == BAD


@pytest.mark.parametrize("field,i,other,j", [("copy", 3, "m", 890), ("v", 899, "param", 0), ("grad", 899, "param", 0),
                                             ("grad", 0, "copy", 899), ("param", 898, "copy", 899)])
def test_adamw_refuses_overlaps_among_thousands_of_buffers(field, i, other, j):
    for bits in (32, 8):
        rows = _table(900, 1000, bits)
        rows[j][other] = rows[i][field] + 996
        assert _step(rows, bits) == BAD
