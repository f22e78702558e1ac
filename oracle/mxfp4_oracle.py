"""CPU oracle of the MXFP4 operators and of the masked, typed token permutation.

NumPy in fp64, from the definitions: E2M1 codes by distance to each of their
values, scales by comparison with powers of two, sums without regard to order.
"""

from __future__ import annotations

import numpy as np

from .moe_oracle import route, silu

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_scale_bytes(K: int) -> int:
    return 4 * -(-K // 128)


def mx_exponent(m: np.ndarray) -> np.ndarray:
    """clamp(floor(log2 m) - 2, -127, 127) of fp64 m >= 0 (m = 0: -127)."""
    e = np.full(m.shape, -127, dtype=np.int64)
    for p in range(-126, 128):
        e = np.where(m >= 2.0 ** (p + 2), p, e)
    return e


def mx_quantize(x: np.ndarray):
    """x [R, K] -> (codes uint8 [R, K], one per value, scale bytes uint8 [R, K/32])."""
    v = x.astype(np.float64).reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    e = mx_exponent(np.abs(v).max(axis=2))
    a = v / np.exp2(e.astype(np.float64))[..., None]
    m = np.abs(a)
    gap = np.abs(m[..., None] - E2M1)
    near = gap.min(axis=-1, keepdims=True)
    # of two equally near values the one with an even code
    code = np.argmin(np.where(gap == near, np.arange(8) % 2, 9), axis=-1)
    code = np.where(np.signbit(a), code + 8, code)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255, e + 127)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def mx_pack(codes: np.ndarray, bytes_: np.ndarray):
    """Codes one per value and bytes per block -> packed int32 words and padded scales (127)."""
    R, K = codes.shape
    words = np.zeros((R, K // 8), dtype=np.uint32)
    for j in range(8):
        words |= codes[:, j::8].astype(np.uint32) << np.uint32(4 * j)
    scales = np.full((R, mx_scale_bytes(K)), 127, dtype=np.uint8)
    scales[:, : K // 32] = bytes_
    return words.view(np.int32), scales


def mx_values(words: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 values of packed MXFP4 [..., K/8] and [..., B]; scale byte 255 is NaN."""
    w = words.view(np.uint32)
    code = np.stack([(w >> np.uint32(4 * j)) & np.uint32(15) for j in range(8)], axis=-1)
    code = code.reshape(*words.shape[:-1], -1)
    v = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])
    s = scales[..., : v.shape[-1] // 32].astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return v * np.repeat(s, 32, axis=-1)


def mx_product(a: np.ndarray, w: np.ndarray, offsets, rows_of=None):
    """(out, sum of the terms' magnitudes) of rows in expert order times w [E, N, K], both fp64;
    rows_of[r] is the row of a that r takes (-1: zeros).  Rows outside the segments stay zero."""
    R = len(a) if rows_of is None else len(rows_of)
    out = np.zeros((R, w.shape[1]))
    size = np.zeros_like(out)
    for e in range(w.shape[0]):
        for r in range(int(offsets[e]), int(offsets[e + 1])):
            src = r if rows_of is None else int(rows_of[r])
            if src < 0:
                continue
            with np.errstate(invalid="ignore"):
                out[r] = w[e] @ a[src]
                size[r] = np.abs(w[e]) @ np.abs(a[src])
    return out, size


def permute_masked(ids: np.ndarray, E: int, first: int = 0) -> dict:
    T, k = ids.shape
    S = T * k
    kept = [[] for _ in range(E)]
    for s in range(S):
        e = int(ids[s // k, s % k]) - first
        if 0 <= e < E:
            kept[e].append(s)
    offsets, order = [0], []
    for e in range(E):
        order += kept[e]
        offsets.append(len(order))
    slot_rows = np.full(S, -1, dtype=np.int32)
    for r, s in enumerate(order):
        slot_rows[s] = r
    active = [e for e in range(E) if kept[e]]
    return {"expert_offsets": np.array(offsets, dtype=np.int32),
            "sorted_slots": np.array(order + [-1] * (S - len(order)), dtype=np.int32),
            "slot_rows": slot_rows,
            "active_experts": np.array(active + [-1] * (E - len(active)), dtype=np.int32),
            "num_active": np.array([len(active)], dtype=np.int32)}


def dispatch(x: np.ndarray, slot_rows: np.ndarray, k: int, out: np.ndarray) -> np.ndarray:
    out = out.copy()
    for s, r in enumerate(slot_rows):
        if 0 <= r < len(out):
            out[r] = x[s // k]
    return out


def combine_masked(y: np.ndarray, weights: np.ndarray, slot_rows: np.ndarray):
    """(out [T, H] in fp64, sum of the terms' magnitudes)."""
    T, k = weights.shape
    out = np.zeros((T, y.shape[1]))
    size = np.zeros_like(out)
    for s, r in enumerate(slot_rows):
        if 0 <= r < len(y):
            term = float(weights[s // k, s % k]) * y[r].astype(np.float64)
            out[s // k] += term
            size[s // k] += np.abs(term)
    return out, size


def combine_backward(grad: np.ndarray, y: np.ndarray, weights: np.ndarray, slot_rows: np.ndarray,
                     grad_y: np.ndarray):
    """(grad_y, grad_weights, magnitudes of grad_weights' terms), from the formula, in fp64."""
    T, k = weights.shape
    grad_y = grad_y.astype(np.float64)
    gw = np.zeros((T, k))
    size = np.zeros((T, k))
    for s, r in enumerate(slot_rows):
        if 0 <= r < len(y):
            t, j = divmod(s, k)
            g = grad[t].astype(np.float64)
            grad_y[r] = float(weights[t, j]) * g
            gw[t, j] = g @ y[r].astype(np.float64)
            size[t, j] = np.abs(g) @ np.abs(y[r].astype(np.float64))
    return grad_y, gw, size


def mx_layer(logits: np.ndarray, x: np.ndarray, k: int, w13: np.ndarray, w2: np.ndarray):
    """The routed layer on MXFP4 experts (fp64 values w13 [E, 2I, H], w2 [E, H, I]): out [T, H]."""
    ids, weights = route(logits, k)
    I = w2.shape[2]
    xq = mx_values(*mx_pack(*mx_quantize(x)))
    out = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j in range(k):
            e = int(ids[t, j])
            h = w13[e] @ xq[t]
            act = (silu(h[:I]) * h[I:])[None]
            out[t] += weights[t, j] * (w2[e] @ mx_values(*mx_pack(*mx_quantize(act)))[0])
    return out
