"""GPU: AdamW at the ends of its scalars' ranges, against the formula in 64 bits."""

from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from w4a16_group_quantized_amd import ops

    ops.load_library()
    return ops


def np64(t):
    return t.detach().double().cpu().numpy()


# ---- eps below fp32's normal numbers ------------------------------------------------------
@pytest.mark.parametrize("eps", [1e-37, 1e-38, 1e-40, 1e-45, 1e-50])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_subnormal_eps(ops, bits, eps):
    """Elements without moments (an expert that had no tokens) stay as they are; those whose second moment
    underflows are divided by eps, which fp32 holds as its smallest number at least; the others do not see it."""
    g = torch.Generator(device="cuda").manual_seed(0)
    n = 3000
    grad = torch.randn(n, generator=g, device="cuda")
    grad[::3] = 0.0
    grad[1::3] = 1e-24
    p = torch.randn(n, generator=g, device="cuda")
    before, x = np64(p), np64(grad)
    m, v = ops.adamw_states(p, bits)
    ops.moe_adamw([p], [grad], [m], [v], lr=1e-2, beta1=0.9, beta2=0.999, eps=eps, weight_decay=0.0, step=1, seed=1)
    got, held = np64(p), max(float(np.float32(eps)), 2.0 ** -149)
    assert np.array_equal(got[::3], before[::3])
    root = np.where(abs(x) > 1e-20, abs(x), 0.0)  # sqrt(v / (1 - beta2)); 0.001 * 1e-48 is 0 in fp32
    for part in (slice(1, None, 3), slice(2, None, 3)):
        step = 1e-2 * x[part] / (root[part] + held)
        # twelve roundings of 2^-24 at most (scalars, moments, root, reciprocal, products), and p's own
        want = before[part] - step
        assert (abs(got[part] - want) <= 12 * 2.0 ** -24 * abs(step) + 2.0 ** -24 * abs(want)).all()


# ---- weight decays next to fp32's steps ---------------------------------------------------
@pytest.mark.parametrize("lr,decay", [(1e-3, 0.01), (1e-5, 0.01), (1e-6, 0.031), (1e-6, 0.01), (0.5, 1.0), (1.0, 1.0)])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_a_small_weight_decay(ops, bits, lr, decay):
    """Without gradients a parameter becomes p (1 - lr wd), rounded once: decays of a few fp32 steps or less
    are not rounded to whole steps first."""
    g = torch.Generator(device="cuda").manual_seed(1)
    p = 4 * torch.randn(1 << 14, generator=g, device="cuda")
    before = np64(p)
    m, v = ops.adamw_states(p, bits)
    ops.moe_adamw([p], [torch.zeros_like(p)], [m], [v], lr=lr, weight_decay=decay, step=3, seed=1)
    move = lr * decay * before
    want = before - move
    # half of fp32's step there; the move's factor and product are rounded to 2^-24 each
    tol = np.spacing(abs(want).astype(np.float32)).astype(np.float64) / 2 + 3 * 2.0 ** -24 * abs(move)
    assert (abs(np64(p) - want) <= tol).all()


def test_adamw_of_infinite_parameters(ops):
    """An infinity stays one, with decay or without."""
    for decay in (0.0, 0.1):
        p = torch.tensor([float("inf"), -float("inf"), 1.0], device="cuda")
        m, v = ops.adamw_states(p)
        ops.moe_adamw([p], [torch.ones(3, device="cuda")], [m], [v], lr=1e-3, weight_decay=decay, step=1)
        assert p[0] == float("inf") and p[1] == -float("inf") and p[2].isfinite()


# ---- tensors side by side, and tensors that share memory ----------------------------------
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_views_side_by_side(ops, bits):
    """Neighbours in one buffer and one gradient for several tensors are taken, as if each were alone;
    a scales buffer that two tensors share, or a shifted view, is refused and nothing changes."""
    g = torch.Generator(device="cuda").manual_seed(2)
    sizes, count = [128, 256, 384], 3
    ends = np.cumsum(sizes)
    flat = torch.randn(int(ends[-1]), generator=g, device="cuda")
    whole_m, whole_v = ops.adamw_states(flat, bits)
    grad = torch.randn(384, generator=g, device="cuda")

    def part(state, i):
        cut = lambda t, unit: t[(ends[i] - sizes[i]) // unit: ends[i] // unit]  # noqa: E731
        return cut(state, 1) if bits == 32 else (cut(state[0], 1), cut(state[1], ops.ADAMW_BLOCK))

    ps = [flat[e - n: e] for e, n in zip(ends, sizes)]
    ms, vs = [part(whole_m, i) for i in range(count)], [part(whole_v, i) for i in range(count)]
    gs = [grad[:n] for n in sizes]
    alone = [p.clone() for p in ps]
    kw = dict(lr=1e-2, step=1, seed=3)
    for p, x in zip(alone, gs):
        m, v = ops.adamw_states(p, bits)
        ops.moe_adamw([p], [x], [m], [v], **kw)
    ops.moe_adamw(ps, gs, ms, vs, **kw)
    assert all(torch.equal(a, b) for a, b in zip(ps, alone))
    before = flat.clone()
    states = lambda: map(list, zip(*(ops.adamw_states(grad, bits) for _ in range(2))))  # noqa: E731
    with pytest.raises(ValueError, match="overlaps"):
        ops.moe_adamw([flat[:384], flat[383:767]], [grad, grad], *states(), **kw)
    with pytest.raises(ValueError, match="overlaps"):
        ops.moe_adamw([flat[:384]], [grad], [ms[2]], [vs[2]], grad_scale=flat[7:8], **kw)
    if bits == 8:
        m, v = states()
        m[1] = (m[1][0], m[0][1])
        with pytest.raises(ValueError, match="m scales"):
            ops.moe_adamw([flat[:384], flat[384:]], [grad, grad], m, v, **kw)
    assert torch.equal(flat, before)


# ---- what the rounding of 8-bit states goes by --------------------------------------------
def test_adamw_without_a_seed_rounds_by_the_step(ops):
    """The same states and gradients at two steps are rounded differently; the step's number is the seed."""
    g = torch.Generator(device="cuda").manual_seed(9)
    grad = torch.randn(4096, generator=g, device="cuda")
    out = []
    for kw in (dict(step=1), dict(step=2), dict(step=2, seed=2), dict(step=(1 << 32) + 2)):
        p = torch.zeros(4096, device="cuda")
        m, v = ops.adamw_states(p, 8)
        ops.moe_adamw([p], [grad], [m], [v], lr=1e-3, **kw)
        out.append((m[0], v[0]))
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))  # noqa: E731
    assert not torch.equal(out[0][0], out[1][0]) and not torch.equal(out[0][1], out[1][1])
    assert same(out[1], out[2]) and same(out[1], out[3])


@pytest.mark.parametrize("kind", ["seeds", "no seed"])
@pytest.mark.parametrize("which,beta,steps", [("v", 0.999, 300), ("m", 0.99, 60)])
def test_adamw_8bit_moments_decay_under_a_held_scale(ops, which, beta, steps, kind):
    """One element of each block has a gradient that keeps its moment, and with it the block's scale, where it is;
    the others had one gradient and decay to beta^steps.  Codes rounded to nearest, or by the same noise at
    every step, stand still."""
    n, signed = 1 << 16, which == "m"
    g = torch.Generator(device="cuda").manual_seed(3)
    first = 0.25 + 0.75 * torch.rand(n, generator=g, device="cuda")  # the moment, over 1 - beta
    held = torch.arange(n, device="cuda") % ops.ADAMW_BLOCK == 0
    first[held] = 3.0
    keep = torch.where(held, 3.0 * (1 - beta), 0.0)                  # beta M + (1 - beta) M = M = 3 (1 - beta)
    if which == "v":
        first, keep = first.sqrt(), keep.sqrt()
    p = torch.zeros(n, device="cuda")
    m, v = ops.adamw_states(p, 8)
    state = m if signed else v
    hyper = dict(lr=1e-3, weight_decay=0.0, beta1=beta if signed else 0.9, beta2=0.999 if signed else beta)
    seed = (lambda step: {"seed": 1000 - step}) if kind == "seeds" else (lambda step: {})
    ops.moe_adamw([p], [first], [m], [v], step=1, **seed(1), **hyper)
    before = ops.adamw_state_values(state, signed).double()
    for step in range(2, steps + 2):
        ops.moe_adamw([p], [keep], [m], [v], step=step, **seed(step), **hyper)
    after = ops.adamw_state_values(state, signed).double()
    # fp32 roundings of the held moment, 2^-22 a step at most
    assert torch.allclose(after[held], before[held], rtol=steps * 2.0 ** -22, atol=0)
    # a rounding's variance is (1 - beta) x^2 / 8 at most (a code's step is an eighth of x or less), and the mean of
    # x^2 1.12 times the mean's square: five deviations of the sum over steps and elements
    five = 5 * (steps * (1 - beta) / 8 * 1.12 / n) ** 0.5 / beta ** steps
    assert abs(float(after[~held].sum() / before[~held].sum()) / beta ** steps - 1) < five
