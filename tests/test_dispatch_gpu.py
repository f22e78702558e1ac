"""GPU: the masked permutation, dispatch, combine and their gradients through the
C ABI against the fp64 oracle.

Moved rows and whole numbers are compared exactly.  A sum of n terms is off by
at most n fp32 roundings (2^-24 each) of the magnitudes summed (a product and
an addition are one rounding) and half a step of its type.
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


def _close(got: torch.Tensor, want, size, terms: int) -> None:
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * eps
    sums = (terms + 1) * 2.0 ** -24 * size
    off = np.abs(_host(got).astype(np.float64) - want)
    assert (off <= sums + eps * (np.abs(want) + sums) + tiny).all()


def _ids(rng, T, k, E, kind="some"):
    """kind: all kept, some tokens without experts, none, repeated ids, wild ids."""
    ids = np.stack([rng.permutation(max(E, k))[:k] % E for _ in range(T)]) if T else np.zeros((0, k))
    if kind == "some":
        ids[rng.random(T) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E + 3
    elif kind == "none":
        ids[:] = -1
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "wild":
        ids = rng.integers(-(1 << 31), 1 << 31, size=(T, k))
        ids[rng.random((T, k)) < 0.5] = E // 2
    return ids.astype(np.int32)


def _check_perm(got: dict, want: dict) -> None:
    for name, value in want.items():
        assert np.array_equal(_host(got[name]), value), name


SORTS = [  # T, k, E: one chunk of 1024 slots, a few, and more than 64 chunks
    (1, 1, 1), (1, 10, 512), (8, 10, 512), (64, 16, 37), (102, 10, 4096), (103, 10, 512),
    (205, 5, 1025), (1000, 8, 3), (6553, 10, 64), (6554, 10, 64), (9000, 9, 1500),
]


@pytest.mark.parametrize("kind", ["all", "some", "none", "one", "wild"])
@pytest.mark.parametrize("T,k,E", SORTS)
def test_permute_masked(ops, T, k, E, kind):
    ids = _ids(np.random.default_rng(T + k), T, k, E, kind)
    out = ops.moe_permute_masked(torch.from_numpy(ids).cuda(), E)
    _check_perm(out, ref.permute_masked(ids, E))


@pytest.mark.parametrize("T", [8, 300])
def test_permute_masked_equals_moe_permute_without_dropped_slots(ops, T):
    ids = torch.from_numpy(_ids(np.random.default_rng(T), T, 10, 512, "all")).cuda()
    a, b = ops.moe_permute_masked(ids, 512), ops.moe_permute(ids, 512)
    for name in b:
        assert torch.equal(a[name], b[name]), name


@pytest.mark.parametrize("T", [6, 400])
def test_permute_masked_of_a_range_of_experts(ops, T):
    """Two ranges of experts share out the slots of the whole."""
    ids = _ids(np.random.default_rng(1), T, 6, 96, "all")
    kept = 0
    for first, n in ((0, 40), (40, 56)):
        got = ops.moe_permute_masked(torch.from_numpy(ids).cuda(), n, first_expert=first)
        _check_perm(got, ref.permute_masked(ids, n, first))
        kept += int(got["expert_offsets"][-1])
    assert kept == T * 6


MOVES = [  # T, k, E, H
    (1, 1, 1, 1), (1, 10, 512, 2560), (5, 3, 4, 7), (33, 10, 37, 129), (130, 8, 16, 1000),
    (257, 17, 20, 64), (64, 64, 64, 37),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,k,E,H", MOVES)
def test_dispatch_and_its_gradient(ops, T, k, E, H, dtype):
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, k, E)
    perm = ref.permute_masked(ids, E)
    rows = torch.from_numpy(perm["slot_rows"]).cuda()
    x = torch.from_numpy(rng.standard_normal((T, H))).cuda().to(dtype)
    out = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    ops.moe_dispatch(x, rows, k, out=out)
    assert np.array_equal(_host(out), ref.dispatch(_host(x), perm["slot_rows"], k, np.full((T * k, H), 7.0, np.float32)))
    g = torch.from_numpy(rng.standard_normal((T * k, H))).cuda().to(dtype)
    g[int(perm["expert_offsets"][-1]):] = float("nan")  # rows without a slot are not read
    got = ops.moe_dispatch_backward(g, rows, k)
    want, size = ref.combine_masked(_host(g), np.ones((T, k)), perm["slot_rows"])
    _close(got, want, size, k)
    # the gradient is the transpose: <dispatch(x), g> = <x, gradient(g)>, in fp64
    kept = int(perm["expert_offsets"][-1])
    left = (_host(out)[:kept].astype(np.float64) * _host(g)[:kept]).sum()
    right = (_host(x).astype(np.float64) * want).sum()
    assert abs(left - right) <= 1e-9 * max(1.0, np.abs(_host(out)[:kept].astype(np.float64) * _host(g)[:kept]).sum())


@pytest.mark.parametrize("y_dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,k,E,H", MOVES)
def test_combine_and_its_gradients(ops, T, k, E, H, y_dtype):
    rng = np.random.default_rng(T + 1)
    ids = _ids(rng, T, k, E)
    perm = ref.permute_masked(ids, E)
    rows = torch.from_numpy(perm["slot_rows"]).cuda()
    R, kept = T * k, int(perm["expert_offsets"][-1])
    y = torch.from_numpy(rng.standard_normal((R, H))).cuda().to(y_dtype)
    y[kept:] = float("nan")
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    w[torch.from_numpy(perm["slot_rows"].reshape(T, k) < 0).cuda()] = float("inf")  # not used
    for dtype in DTYPES:
        got = ops.moe_combine_masked(y, w, rows, dtype=dtype)
        want, size = ref.combine_masked(_host(y), _host(w), perm["slot_rows"])
        _close(got, want, size, k)
        grad = torch.from_numpy(rng.standard_normal((T, H))).cuda().to(dtype)
        gy = torch.full((R, H), 7.0, dtype=y_dtype, device="cuda")
        gw = torch.full((T, k), float("nan"), device="cuda")
        ops.moe_combine_backward(grad, y, w, rows, out=gy, grad_weights=gw)
        want_y, want_w, size_w = ref.combine_backward(_host(grad), _host(y), _host(w),
                                                      perm["slot_rows"], np.full((R, H), 7.0))
        _close(gy, want_y, np.abs(want_y), 1)
        _close(gw, want_w, size_w, H)


@pytest.mark.parametrize("seed", range(16))
def test_random_moves(ops, seed):
    """Any sizes and kinds of ids through permutation, dispatch, combine and their gradients."""
    rng = np.random.default_rng(seed)
    T = int(np.exp(rng.uniform(0, np.log(1500))))
    k, E = int(rng.integers(1, 13)), int(rng.choice([1, 3, 50, 513, 4096]))
    H = int(np.exp(rng.uniform(0, np.log(400))))
    first = int(rng.integers(0, 3))
    ids = _ids(rng, T, k, E, ["all", "some", "one", "wild"][seed % 4])
    y_dtype, dtype = DTYPES[seed % 3], DTYPES[(seed // 3) % 3]
    print(T, k, E, H, first, y_dtype, dtype, flush=True)
    perm = ops.moe_permute_masked(torch.from_numpy(ids).cuda(), E, first_expert=first)
    want = ref.permute_masked(ids, E, first)
    _check_perm(perm, want)
    rows, R = perm["slot_rows"], T * k
    x = torch.randn(T, H, device="cuda").to(y_dtype)
    out = ops.moe_dispatch(x, rows, k)
    assert np.array_equal(_host(out), ref.dispatch(_host(x), want["slot_rows"], k, np.zeros((R, H), np.float32)))
    w = torch.randn(T, k, device="cuda")
    got = ops.moe_combine_masked(out, w, rows, dtype=dtype)
    value, size = ref.combine_masked(_host(out), _host(w), want["slot_rows"])
    _close(got, value, size, k)
    gy, gw = ops.moe_combine_backward(got, out, w, rows)
    value_y, value_w, size_w = ref.combine_backward(_host(got), _host(out), _host(w), want["slot_rows"], np.zeros((R, H)))
    _close(gy, value_y, np.abs(value_y), 1)
    _close(gw, value_w, size_w, H)
    value, size = ref.combine_masked(_host(gy), np.ones((T, k)), want["slot_rows"])
    _close(ops.moe_dispatch_backward(gy, rows, k), value, size, k)


def test_combine_gradients_against_differences(ops):
    """The outputs are linear in the rows and in the weights, so a difference of the fp64 oracle
    over a step of 1 is the directional derivative."""
    rng = np.random.default_rng(9)
    T, k, E, H = 12, 4, 6, 40
    perm = ref.permute_masked(_ids(rng, T, k, E), E)
    y, dy = rng.standard_normal((2, T * k, H)).astype(np.float32)
    w, dw = rng.standard_normal((2, T, k)).astype(np.float32)
    grad = rng.standard_normal((T, H)).astype(np.float32)
    gy, gw = ops.moe_combine_backward(*(torch.from_numpy(a).cuda() for a in (grad, y, w, perm["slot_rows"])))

    def loss(y, w):
        return (ref.combine_masked(y, w, perm["slot_rows"])[0] * grad).sum()

    base = loss(y.astype(np.float64), w.astype(np.float64))
    by_y = loss(y.astype(np.float64) + dy, w.astype(np.float64)) - base
    by_w = loss(y.astype(np.float64), w.astype(np.float64) + dw) - base
    got_y = (_host(gy).astype(np.float64) * dy)
    got_w = (_host(gw).astype(np.float64) * dw)
    assert abs(got_y.sum() - by_y) <= 2.0 ** -23 * np.abs(got_y).sum() + 1e-9
    size = np.abs(grad) @ np.abs(y).T  # at least any row's magnitude sum
    assert abs(got_w.sum() - by_w) <= H * 2.0 ** -24 * size.max() * np.abs(dw).sum() + 1e-9


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_strided_rows_and_short_buffers(ops, dtype):
    """Slices of wider buffers at odd addresses, and a row buffer shorter than the slots: rows
    behind it are skipped, the columns around a slice stay."""
    rng = np.random.default_rng(21)
    T, k, E, H = 40, 5, 8, 77
    perm = ref.permute_masked(_ids(rng, T, k, E), E)
    rows = torch.from_numpy(perm["slot_rows"]).cuda()
    R = 90
    xb = torch.from_numpy(rng.standard_normal((T, H + 10))).cuda().to(dtype)
    sb = torch.full((R, H + 6), 7.0, dtype=dtype, device="cuda")
    x, s = xb[:, 3:3 + H], sb[:, 1:1 + H]
    ops.moe_dispatch(x, rows, k, out=s)
    assert np.array_equal(_host(s), ref.dispatch(_host(x), perm["slot_rows"], k, np.full((R, H), 7.0, np.float32)))
    assert (sb[:, 0] == 7).all() and (sb[:, 1 + H:] == 7).all()
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    ob = torch.full((T, H + 4), 7.0, dtype=dtype, device="cuda")
    ops.moe_combine_masked(s, w, rows, out=ob[:, 2:2 + H])
    want, size = ref.combine_masked(_host(s), _host(w), perm["slot_rows"])
    _close(ob[:, 2:2 + H], want, size, k)
    assert (ob[:, :2] == 7).all() and (ob[:, 2 + H:] == 7).all()
    gb = torch.full((R, H + 3), 7.0, dtype=dtype, device="cuda")
    gy, gw = ops.moe_combine_backward(x, s, w, rows, out=gb[:, 2:2 + H])
    want_y, want_w, size_w = ref.combine_backward(_host(x), _host(s), _host(w), perm["slot_rows"],
                                                  np.full((R, H), 7.0))
    _close(gy, want_y, np.abs(want_y), 1)
    _close(gw, want_w, size_w, H)
    assert (gb[:, :2] == 7).all() and (gb[:, 2 + H:] == 7).all()


def test_dispatch_offsets_past_32_bits(ops):
    """A row buffer of more than 2^32 bytes: the last rows land where they should."""
    H, R = 65536, 33000
    out = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(2, H, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([R - 1, 0, 32769, -1], dtype=torch.int32, device="cuda")
    ops.moe_dispatch(x, rows, 2, out=out)
    assert torch.equal(out[R - 1], x[0]) and torch.equal(out[0], x[0]) and torch.equal(out[32769], x[1])
    assert int((out != 0).any(dim=1).sum()) == 3
    got = ops.moe_combine_masked(out, torch.ones(2, 2, device="cuda"), rows)
    assert torch.equal(got[1], x[1]) and torch.equal(got[0].float(), (2 * x[0].float()))


@pytest.mark.parametrize("T", [9, 600])
def test_a_run_of_them_in_a_graph(ops, T):
    """Permutation, dispatch, combine and the gradients captured once, replayed with new ids."""
    rng = np.random.default_rng(T)
    k, E, H = 6, 48, 200
    ids = torch.from_numpy(_ids(rng, T, k, E)).cuda()
    x = torch.randn(T, H, device="cuda", dtype=torch.bfloat16)
    w = torch.rand(T, k, device="cuda")
    S = T * k
    perm = ops.moe_permute_masked(ids, E)
    ws = torch.empty(max(1, ops.permute_masked_workspace_bytes(T, k, E)), dtype=torch.uint8, device="cuda")
    buf = {"x": torch.zeros(S, H, device="cuda", dtype=x.dtype), "out": torch.empty_like(x),
           "gy": torch.zeros(S, H, device="cuda", dtype=x.dtype), "gw": torch.empty(T, k, device="cuda"),
           "gx": torch.empty_like(x)}

    def step():
        ops.moe_permute_masked(ids, E, workspace=ws, out=perm)
        ops.moe_dispatch(x, perm["slot_rows"], k, out=buf["x"])
        ops.moe_combine_masked(buf["x"], w, perm["slot_rows"], out=buf["out"])
        ops.moe_combine_backward(buf["out"], buf["x"], w, perm["slot_rows"], out=buf["gy"],
                                 grad_weights=buf["gw"])
        ops.moe_dispatch_backward(buf["gy"], perm["slot_rows"], k, out=buf["gx"])

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        ids.copy_(torch.from_numpy(_ids(rng, T, k, E, ["some", "all", "none", "one"][i])).cuda())
        x.normal_()
        buf["x"].zero_()
        buf["gy"].zero_()
        g.replay()
        torch.cuda.synchronize()
        got = {**{n: t.clone() for n, t in buf.items()}, **{n: t.clone() for n, t in perm.items()}}
        buf["x"].zero_()
        buf["gy"].zero_()
        step()
        torch.cuda.synchronize()
        for n, t in {**buf, **perm}.items():
            assert torch.equal(t, got[n]), (i, n)
        _check_perm(got, ref.permute_masked(_host(ids), E))
