"""NumPy fp64 reference of the training operators: grouped products with their gradients, the
gated activation, the router's gradient, and AdamW with states in fp32 or in 8 bits.  Test
infrastructure only; shares no code with the GPU path."""

from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = 1.875  # value of an 8-bit state's largest code


# ---- products grouped by expert -----------------------------------------------------
def _segments(offsets, rows):
    if offsets is None:
        return [(0, 0, rows)]
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)]


def product(a, w, offsets):
    """out [R, N]; rows without an expert are NaN (left as they were)."""
    out = np.full((a.shape[0], w.shape[1]), np.nan)
    for e, r0, r1 in _segments(offsets, a.shape[0]):
        out[r0:r1] = a[r0:r1].astype(np.float64) @ w[e].astype(np.float64).T
    return out


def product_rows(grad, w, offsets):
    out = np.full((grad.shape[0], w.shape[2]), np.nan)
    for e, r0, r1 in _segments(offsets, grad.shape[0]):
        out[r0:r1] = grad[r0:r1].astype(np.float64) @ w[e].astype(np.float64)
    return out


def product_weights(grad, a, offsets):
    segs = _segments(offsets, grad.shape[0])
    out = np.zeros((len(segs), grad.shape[1], a.shape[1]))
    for e, r0, r1 in segs:
        out[e] = grad[r0:r1].astype(np.float64).T @ a[r0:r1].astype(np.float64)
    return out


# ---- the gated activation -------------------------------------------------------------
def _sigmoid(x):
    z = np.exp(-np.abs(x))
    return np.where(x >= 0, 1, z) / (1 + z)


def silu_mul(h):
    gate, up = np.split(h.astype(np.float64), 2, axis=1)
    return gate * _sigmoid(gate) * up


def silu_mul_backward(grad, h):
    gate, up = np.split(h.astype(np.float64), 2, axis=1)
    grad, s = grad.astype(np.float64), _sigmoid(gate)
    return np.concatenate([grad * up * s * (1 + gate * _sigmoid(-gate)), grad * gate * s], axis=1)


# ---- the router's gradient --------------------------------------------------------------
def route_weights(logits, ids):
    """Softmax over the chosen logits."""
    x = np.take_along_axis(logits.astype(np.float64), ids, axis=1)
    p = np.exp(x - x.max(axis=1, keepdims=True))
    return p / p.sum(axis=1, keepdims=True)


def route_backward(ids, weights, grad, E):
    w, g = weights.astype(np.float64), grad.astype(np.float64)
    each = w * (g - (w * g).sum(axis=1, keepdims=True))
    out = np.zeros((ids.shape[0], E))
    for t in range(ids.shape[0]):
        for j, e in enumerate(ids[t]):
            if 0 <= e < E:
                out[t, e] += each[t, j]
    return out


# ---- AdamW --------------------------------------------------------------------------------
def noise(n, seed, which):
    """20 bits per element: 0 for m, 1 for v."""
    i = np.arange(n, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    x = (i + (np.uint64(seed) + (i >> np.uint64(32))) * np.uint64(0x9E3779B9)) & low
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x6A09E667)) & low
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0xB7E15163)) & low
    x = x ^ (x >> np.uint64(16))
    if which:
        x = (x * np.uint64(0x9E3779B1)) & low
    return (x >> np.uint64(12)).astype(np.int64)


def code_values(signed):
    """The value of each code, 256 of them, by its fields."""
    bias = 15 if signed else 31
    out = np.zeros(256)
    for c in range(256):
        size = c % 128 if signed else c
        f, man = size // 8, size % 8 / 8
        v = (1 + man) * 2.0 ** (f - bias) if f else man * 2.0 ** (1 - bias)
        out[c] = -v if signed and c >= 128 else v
    return out


def decode(codes, scales, signed):
    n = codes.size
    return code_values(signed)[codes] * np.repeat(scales.astype(np.float64), BLOCK)[:n]


def block_scales(x):
    n = x.size
    top = np.abs(np.pad(x.astype(np.float64), (0, -n % BLOCK))).reshape(-1, BLOCK).max(axis=1)
    scale = top / TOP
    return np.where(scale < 2.0 ** -126, 0.0, scale)


def code_sizes(x, scale, u, signed):
    """Code without its sign of |x| / scale, rounded up where the part cut off plus u in [0, 1) carries."""
    bias = 15 if signed else 31
    t = np.divide(np.abs(x), scale, out=np.zeros_like(x), where=scale > 0)
    f = np.clip(np.floor(np.log2(np.maximum(t, 2.0 ** -200))), 1 - bias, None)
    f = np.where((2.0 ** f > t) & (f > 1 - bias), f - 1, f)
    step = 2.0 ** (f - 3)
    k = np.floor(t / step + u)              # in steps of this binade; 16 carries into the next
    c = np.where(t < 2.0 ** (1 - bias), k, (f + bias) * 8 + k - 8)
    c = np.minimum(c, 127 if signed else 255).astype(np.int64)
    return np.where(~np.asarray(signed) & (c == 0) & (x > 0), 1, c)


def encode(x, seed, signed):
    x = x.astype(np.float64)
    scale = block_scales(x)
    each = np.repeat(scale, BLOCK)[:x.size]
    c = code_sizes(x, each, noise(x.size, seed, 0 if signed else 1) / 2.0 ** 20, signed)
    if signed:
        c = c + 128 * np.signbit(x)
    return c.astype(np.uint8), scale


def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, grad_scale=1.0):
    """(p, m, v) after the step, from fp64 moments."""
    p, g = p.astype(np.float64), g.astype(np.float64) * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = m / (1 - beta1 ** step) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * update, m, v
