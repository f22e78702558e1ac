"""CPU: refusals of the training entry points (nothing reaches a GPU), and pins of their oracle."""

import ctypes
import os

import numpy as np
import pytest

from oracle import train_oracle as ref
from w4a16_group_quantized_amd import ops

torch = pytest.importorskip("torch")

FAKE = 0x1000  # aligned and never dereferenced: validation fails first
OK, BAD, UNSUPPORTED, WORKSPACE = (ops.MOE_OK, ops.MOE_ERR_INVALID_ARG, ops.MOE_ERR_UNSUPPORTED,
                                   ops.MOE_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def _built_library():
    if not os.path.exists(ops.LIB_PATH):
        from w4a16_group_quantized_amd import build_lib

        build_lib.build()


# ---- refusals through the C ABI ---------------------------------------------------
def _gemm(fn, **args):
    a = {"x": FAKE, "dtype": 2, "rows": 8, "x_ld": 64, "offsets": FAKE, "E": 2, "w": FAKE, "N": 64, "K": 64,
         "out": FAKE, "out_dtype": 2, "out_ld": 64, **args}
    return getattr(ops.load_library(), fn)(*(a[k] for k in ("x", "dtype", "rows", "x_ld", "offsets", "E", "w",
                                                            "N", "K", "out", "out_dtype", "out_ld")), None)


@pytest.mark.parametrize("fn", ["moe_grouped_gemm", "moe_grouped_gemm_backward"])
@pytest.mark.parametrize("args,status", [
    ({"dtype": 0}, UNSUPPORTED), ({"dtype": 3}, BAD), ({"out_dtype": -1}, BAD), ({"rows": -1}, BAD),
    ({"rows": (1 << 27) + 1}, UNSUPPORTED), ({"E": 0}, BAD), ({"E": 4097}, UNSUPPORTED), ({"offsets": None}, BAD),
    ({"offsets": FAKE + 4}, BAD), ({"N": 0}, BAD), ({"K": 0}, BAD), ({"x_ld": 63}, BAD), ({"out_ld": 63}, BAD),
    ({"x_ld": (1 << 31) + 1}, UNSUPPORTED), ({"N": 65537, "x_ld": 65537, "out_ld": 65537}, UNSUPPORTED),
    ({"N": 32768, "K": 32768, "x_ld": 32768, "out_ld": 32768}, UNSUPPORTED), ({"x": None}, BAD),
    ({"x": FAKE + 1}, BAD), ({"w": None}, BAD), ({"w": FAKE + 2}, BAD), ({"out": None}, BAD),
    ({"out": FAKE + 2, "out_dtype": 0}, BAD), ({"rows": 1 << 27, "N": 65536, "x_ld": 65536, "out_ld": 65536}, UNSUPPORTED),
    ({"rows": 0, "x": None, "w": None, "out": None}, OK),
])
def test_product_refusals(fn, args, status):
    assert _gemm(fn, **args) == status


@pytest.mark.parametrize("args,status", [
    ({"dtype": 0}, UNSUPPORTED), ({"out_dtype": 4}, BAD), ({"rows": -1}, BAD), ({"grad_ld": 63}, BAD),
    ({"a_ld": 31}, BAD), ({"offsets": None}, BAD), ({"accumulate": 2}, BAD), ({"out": None}, BAD),
    ({"out": FAKE + 8}, BAD), ({"grad": None}, BAD), ({"a": FAKE + 1}, BAD), ({"E": 0}, BAD),
    ({"N": 1 << 16, "K": 1 << 14, "grad_ld": 1 << 16, "a_ld": 1 << 14}, UNSUPPORTED),
])
def test_weight_gradient_refusals(args, status):
    a = {"grad": FAKE, "dtype": 1, "rows": 8, "grad_ld": 64, "a": FAKE, "a_ld": 32, "offsets": FAKE, "E": 2,
         "N": 64, "K": 32, "out": FAKE, "out_dtype": 0, "accumulate": 0, "ws": FAKE, "bytes": 1 << 40, **args}
    assert ops.load_library().moe_grouped_gemm_backward_weights(*a.values(), None) == status


def test_weight_gradient_workspace():
    lib = ops.load_library()
    sizes = [(r, E, N, K) for r in (1, 100, 5000, 100000) for E in (1, 8) for N, K in ((64, 64), (512, 2560))]
    for rows, E, N, K in sizes:
        need = ops.grouped_gemm_backward_weights_workspace_bytes(rows, E, N, K)
        if need:
            call = lambda ws, n: lib.moe_grouped_gemm_backward_weights(  # noqa: E731
                FAKE, 1, rows, N, FAKE, K, FAKE, E, N, K, FAKE, 0, 0, ws, n, None)
            assert call(FAKE, need - 1) == WORKSPACE and call(None, need) == BAD and call(FAKE + 8, need) == BAD
    assert ops.grouped_gemm_backward_weights_workspace_bytes(-1, 1, 8, 8) == 0


@pytest.mark.parametrize("args,status", [
    ({"dtype": 3}, BAD), ({"rows": -1}, BAD), ({"rows": 1 << 31}, UNSUPPORTED), ({"I": 0}, BAD),
    ({"I": 32769, "wide": 65538, "narrow": 32769}, UNSUPPORTED), ({"wide": 127}, BAD), ({"narrow": 63}, BAD),
    ({"offsets": FAKE, "E": 0}, BAD), ({"offsets": FAKE + 4, "E": 2}, BAD), ({"h": None}, BAD),
    ({"h": FAKE + 1}, BAD), ({"out": None}, BAD), ({"rows": 1 << 30, "I": 64}, UNSUPPORTED),
    ({"rows": 0, "h": None, "out": None, "grad": None}, OK),
])
def test_silu_mul_refusals(args, status):
    a = {"h": FAKE, "dtype": 2, "rows": 4, "I": 64, "wide": 128, "narrow": 64, "offsets": None, "E": 0,
         "out": FAKE, "grad": FAKE, **args}
    lib = ops.load_library()
    assert lib.moe_silu_mul(a["h"], a["dtype"], a["rows"], a["I"], a["wide"], a["offsets"], a["E"], a["out"],
                            a["narrow"], None) == status
    assert lib.moe_silu_mul_backward(a["grad"], a["narrow"], a["h"], a["wide"], a["dtype"], a["rows"], a["I"],
                                     a["offsets"], a["E"], a["out"], a["wide"], None) == status


@pytest.mark.parametrize("args,status", [
    ({"T": -1}, BAD), ({"E": 0}, BAD), ({"k": 0}, BAD), ({"k": 65}, UNSUPPORTED), ({"E": 4097}, UNSUPPORTED),
    ({"T": 1 << 40}, UNSUPPORTED), ({"T": 1 << 30, "k": 2}, UNSUPPORTED), ({"dtype": 3}, BAD), ({"ids": None}, BAD),
    ({"out": None}, BAD), ({"out": FAKE + 4}, BAD), ({"T": 0, "ids": None, "out": None}, OK),
])
def test_route_backward_refusals(args, status):
    a = {"ids": FAKE, "w": FAKE, "g": FAKE, "T": 4, "E": 8, "k": 2, "out": FAKE, "dtype": 0, **args}
    assert ops.load_library().moe_route_backward(*a.values(), None) == status


def _adamw(rows=((8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, 0),), count=None, bits=32, lr=1e-3, b1=0.9, b2=0.999,
           eps=1e-8, wd=0.0, step=1, scale=None):
    flat = [x for r in rows for x in r]
    table = (ctypes.c_int64 * max(1, len(flat)))(*flat)
    return ops.load_library().moe_adamw(table, len(rows) if count is None else count, bits, lr, b1, b2, eps, wd,
                                        step, 0, scale, None)


def _tensor(n=8, param=FAKE, grad=FAKE, m=FAKE, v=FAKE, ms=FAKE, vs=FAKE, copy=0, types=0, copy_type=0):
    return (n, param or 0, grad or 0, m or 0, v or 0, ms or 0, vs or 0, copy, types, copy_type)


@pytest.mark.parametrize("args,status", [
    ({"count": -1}, BAD), ({"bits": 16}, BAD), ({"lr": -1.0}, BAD), ({"lr": float("nan")}, BAD),
    ({"lr": float("inf")}, BAD), ({"b1": 1.0}, BAD), ({"b1": -0.1}, BAD), ({"b2": float("nan")}, BAD),
    ({"b2": 1.5}, BAD), ({"eps": -1e-9}, BAD), ({"wd": -0.1}, BAD), ({"step": 0}, BAD), ({"scale": FAKE + 2}, BAD),
    ({"rows": (_tensor(n=-1),)}, BAD), ({"rows": (_tensor(n=(1 << 33) + 1),)}, UNSUPPORTED),
    ({"rows": (_tensor(param=None),)}, BAD), ({"rows": (_tensor(grad=FAKE + 2),)}, BAD),
    ({"rows": (_tensor(m=None),)}, BAD), ({"rows": (_tensor(v=FAKE + 1),)}, BAD),
    ({"rows": (_tensor(types=3),)}, BAD), ({"rows": (_tensor(types=7 << 32),)}, BAD),
    ({"rows": (_tensor(copy=FAKE, copy_type=9),)}, BAD), ({"rows": (_tensor(copy=FAKE + 1, copy_type=2),)}, BAD),
    ({"rows": (_tensor(ms=None),), "bits": 8}, BAD), ({"rows": (_tensor(vs=FAKE + 2),), "bits": 8}, BAD),
    ({"rows": (_tensor(), _tensor(grad=None))}, BAD), ({"count": 0}, OK),
    ({"rows": (_tensor(n=0, param=None, grad=None, m=None),)}, OK),
])
def test_adamw_refusals(args, status):
    assert _adamw(**args) == status


# ---- refusals of the binding --------------------------------------------------------
def test_binding_refuses():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32)
    calls = [
        lambda: ops.moe_grouped_gemm(z(4, 8, d=torch.float32), z(2, 8, 8, d=torch.float32), off),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 8, d=torch.float16), off),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 16), off),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(8, 8), off),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 8), off.long()),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 8), off[:2]),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 8), off, out=z(4, 9)),
        lambda: ops.moe_grouped_gemm(z(4, 8), z(2, 8, 8), off, dtype=torch.int32),
        lambda: ops.moe_grouped_gemm(z(4, 16)[:, ::2], z(2, 8, 8), off),
        lambda: ops.moe_grouped_gemm_backward(z(4, 8), z(2, 4, 8), off),
        lambda: ops.moe_grouped_gemm_backward_weights(z(4, 8), z(5, 8), off),
        lambda: ops.moe_grouped_gemm_backward_weights(z(4, 8), z(4, 8), off, accumulate=True),
        lambda: ops.moe_grouped_gemm_backward_weights(z(4, 8), z(4, 8), off, out=z(2, 8, 9)),
        lambda: ops.moe_grouped_gemm_backward_weights(z(4, 8), z(4, 8), off, dtype=torch.int8),
        lambda: ops.moe_silu_mul(z(4, 7)),
        lambda: ops.moe_silu_mul(z(4, 8), off[:1]),
        lambda: ops.moe_silu_mul(z(4, 8), out=z(4, 4, d=torch.float16)),
        lambda: ops.moe_silu_mul_backward(z(4, 3), z(4, 8)),
        lambda: ops.moe_route_backward(off.view(1, 3).long(), z(1, 3, d=torch.float32), z(1, 3, d=torch.float32), 8),
        lambda: ops.moe_route_backward(off.view(1, 3), z(1, 3, d=torch.float32), z(1, 2, d=torch.float32), 8),
        lambda: ops.moe_adamw([z(4)], [], [z(4)], [z(4)], lr=1e-3, step=1),
        lambda: ops.moe_adamw([z(4)], [z(5)], [z(4, d=torch.float32)], [z(4, d=torch.float32)], lr=1e-3, step=1),
        lambda: ops.moe_adamw([z(4)], [z(4)], [z(4)], [z(4)], lr=1e-3, step=1),
        lambda: ops.moe_adamw([z(4)], [z(4)], [(z(4, d=torch.uint8), z(1, d=torch.float32))],
                              [z(4, d=torch.float32)], lr=1e-3, step=1),
        lambda: ops.moe_adamw([z(4)], [z(4)], [(z(4, d=torch.uint8), z(2, d=torch.float32))],
                              [(z(4, d=torch.uint8), z(1, d=torch.float32))], lr=1e-3, step=1),
        lambda: ops.adamw_states(z(4), 16),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_binding_refuses_shared_memory():
    """An output that shares memory with an input is refused before the device is looked at."""
    buf = torch.zeros(64, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    w = torch.zeros(1, 8, 8, dtype=torch.bfloat16)
    for call in (lambda: ops.moe_grouped_gemm(buf[:4, :8], w, off, out=buf[2:6, :8]),
                 lambda: ops.moe_grouped_gemm_backward(buf[:4, :8], w, off, out=buf[:4, 4:12]),
                 lambda: ops.moe_grouped_gemm_backward_weights(buf[:4, :8], w.view(8, 8)[:4], off, out=w),
                 lambda: ops.moe_silu_mul(buf[:4, :16], out=buf[:4, 8:16]),
                 lambda: ops.moe_silu_mul_backward(buf[:4, :8], buf[8:12, :16], out=buf[9:13, :16])):
        with pytest.raises(ValueError, match="overlaps"):
            call()


def test_states():
    p = torch.zeros(3, 50)
    m, v = ops.adamw_states(p)
    assert m.shape == p.shape and m.dtype == torch.float32
    (mc, ms), (vc, vs) = ops.adamw_states(p, 8)
    assert mc.shape == p.shape and mc.dtype == torch.uint8 and ms.shape == (2,) and vs.dtype == torch.float32
    codes = torch.arange(256, dtype=torch.uint8)
    scales = torch.tensor([0.5, 3.0])
    for signed in (True, False):
        got = ops.adamw_state_values((codes, scales), signed).double().numpy()
        assert np.array_equal(got, ref.decode(codes.numpy(), scales.numpy(), signed))


# ---- the oracle, by differences and by hand ----------------------------------------------
def _difference(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_oracle_gradients_by_differences():
    rng = np.random.default_rng(0)
    offsets = [0, 2, 2, 5]
    a, w, c = rng.normal(size=(5, 3)), rng.normal(size=(3, 4, 3)), rng.normal(size=(5, 4))
    loss = lambda a, w: (ref.product(a, w, offsets) * c).sum()  # noqa: E731
    assert np.allclose(ref.product_rows(c, w, offsets), _difference(lambda x: loss(x, w), a), atol=1e-7)
    assert np.allclose(ref.product_weights(c, a, offsets), _difference(lambda x: loss(a, x), w), atol=1e-7)
    h, c = rng.normal(size=(3, 8)) * 2, rng.normal(size=(3, 4))
    assert np.allclose(ref.silu_mul_backward(c, h), _difference(lambda x: (ref.silu_mul(x) * c).sum(), h), atol=1e-7)
    logits, ids, c = rng.normal(size=(3, 6)), np.array([[1, 4], [0, 2], [5, 3]]), rng.normal(size=(3, 2))
    want = _difference(lambda x: (ref.route_weights(x, ids) * c).sum(), logits)
    assert np.allclose(ref.route_backward(ids, ref.route_weights(logits, ids), c, 6), want, atol=1e-7)


def test_oracle_codes():
    for signed in (True, False):
        values = ref.code_values(signed)
        assert values[127 if signed else 255] == 1.875 and values[1] == 2.0 ** (-17 if signed else -33)
        # every code's value comes back as the code, whatever the noise
        x = values * 4.0
        for u in (0.0, 0.999999):
            c = ref.code_sizes(x, np.full(256, 4.0), np.full(256, u), signed)
            assert np.array_equal(c, np.arange(256) % 128 if signed else np.arange(256))
        # halfway between two codes: up for noise from 1/2 on
        mid = (values[1:127] + values[2:128]) / 2
        low = ref.code_sizes(mid, np.ones(126), np.full(126, 0.49), signed)
        high = ref.code_sizes(mid, np.ones(126), np.full(126, 0.51), signed)
        assert np.array_equal(low, np.arange(1, 127)) and np.array_equal(high, np.arange(2, 128))
    tiny = np.array([1e-30, 0.0])
    assert list(ref.code_sizes(tiny, np.ones(2), np.zeros(2), False)) == [1, 0]
    assert list(ref.code_sizes(tiny, np.ones(2), np.zeros(2), True)) == [0, 0]


def test_oracle_noise_is_even():
    u = ref.noise(1 << 16, 3, 0) / 2.0 ** 20
    # mean of 65536 even values: standard deviation 1 / sqrt(12 * 65536) = 0.0011
    assert abs(u.mean() - 0.5) < 5 * 0.0012 and u.max() < 1
    assert not np.array_equal(ref.noise(64, 3, 0), ref.noise(64, 4, 0))
    assert not np.array_equal(ref.noise(64, 3, 0), ref.noise(64, 3, 1))


def test_oracle_adamw_first_step():
    """From zero moments the first step moves by lr in the gradient's direction."""
    g = np.array([0.5, -2.0, 1e-3])
    p, m, v = ref.adamw(np.zeros(3), g, np.zeros(3), np.zeros(3), 0.1, 0.9, 0.999, 0.0, 0.0, 1)
    assert np.allclose(p, -0.1 * np.sign(g)) and np.allclose(m, 0.1 * g) and np.allclose(v, 1e-3 * g * g)


# ---- limits of a launch, and tensors given twice ------------------------------------------
@pytest.mark.parametrize("T", [1 << 26, (1 << 31) - 1])
def test_route_backward_of_more_tokens_than_a_launch_takes(T):
    assert ops.load_library().moe_route_backward(FAKE, FAKE, FAKE, T, 8, 1, FAKE, 0, None) == UNSUPPORTED


def test_binding_refuses_a_tensor_twice():
    p, q, g = (torch.zeros(8) for _ in range(3))
    (m, v), (m2, v2) = ops.adamw_states(p), ops.adamw_states(p)
    empty = torch.zeros(0)
    call = lambda *lists, copies=None: ops.moe_adamw(*lists, lr=1e-3, step=1, copies=copies)  # noqa: E731
    for args, copies in ((([p, p], [g, g], [m, m2], [v, v2]), None), (([p, q], [g, g], [m, m], [v, v2]), None),
                         (([p], [g], [m], [m]), None), (([p], [g], [m], [v]), [p]),
                         (([p, empty, empty, q], [g, empty, empty, g], [m, empty, empty, m], [v, empty, empty, v2]),
                          None)):
        with pytest.raises(ValueError, match="twice"):
            call(*args, copies=copies)


def test_binding_refuses_a_gradient_of_logits_over_its_inputs():
    ids, w, g = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8), torch.zeros(4, 8)
    for out in (w, g):
        with pytest.raises(ValueError, match="overlaps"):
            ops.moe_route_backward(ids, w, g, 8, out=out)
    with pytest.raises(ValueError):
        ops.moe_grouped_gemm_backward_weights(w.bfloat16(), w.bfloat16(), torch.zeros(0, dtype=torch.int32))


@pytest.mark.parametrize("T", [(1 << 26) - 3, (1 << 26) - 1])
def test_route_backward_of_the_last_tokens_that_make_a_launch_too_long(T):
    """Four tokens to a workgroup of 256 threads: one token behind 2^26 - 4 is the 2^24th workgroup."""
    assert ops.load_library().moe_route_backward(FAKE, FAKE, FAKE, T, 8, 1, FAKE, 0, None) == UNSUPPORTED
