"""What is measured of the MXFP4 experts and of the token permutation with its gradients.

Five operators around the routed-expert layer:

  quantize   rows of 32-wide microscaled 4-bit blocks (E2M1 codes, one E8M0 scale per block) and back
  product    grouped product of MXFP4 rows with MXFP4 expert weights (one expert: a plain product)
  dispatch   tokens sorted by expert, tokens or choices without an expert left out; and its gradient
  combine    expert rows weighted and added back into token order; and its gradients
  layer      the routed-expert layer on MXFP4 experts: routing, quantised dispatch, gate/up, SiLU, down, combine

A case's sizes: T tokens, E experts, k experts per token, H hidden size, I intermediate size, R rows, N output
columns, K reduction length.
"""

import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


# --------------------------------------------------------------------------- #
# cases
# --------------------------------------------------------------------------- #
def listed():
    return [
        # the activations of eight decoding sequences
        {"name": "quantize_fp16_r8_k2560", "op": "quantize", "R": 8, "K": 2560, "dtype": "fp16"},
        # one layer's share of gate/up weights, 64 experts of 1280 rows, turned to MXFP4 at load time
        {"name": "quantize_bf16_r81920_k2560", "op": "quantize", "R": 81920, "K": 2560, "dtype": "bf16"},
        # the gate/up product of eight decoding tokens, 512 experts and 10 per token
        {"name": "product_decode_e512_r80", "op": "product", "E": 512, "R": 80, "N": 1280, "K": 2560, "dtype": "fp32"},
        # the same product at a 4096-token prefill
        {"name": "product_prefill_e512_r40960", "op": "product", "E": 512, "R": 40960, "N": 1280, "K": 2560,
         "dtype": "fp16"},
        # a dense product of an odd number of rows, bound by the matrix cores
        {"name": "product_dense_r8191_n8192_k8192", "op": "product", "E": 1, "R": 8191, "N": 8192, "K": 8192,
         "dtype": "bf16"},
        # eight decoding tokens, one of them padding
        {"name": "dispatch_fp16_t8", "op": "dispatch", "T": 8, "E": 512, "k": 10, "H": 2560, "dtype": "fp16",
         "backward": False},
        # a 4096-token prefill or training step, some tokens padding
        {"name": "dispatch_bf16_t4096", "op": "dispatch", "T": 4096, "E": 512, "k": 10, "H": 2560, "dtype": "bf16",
         "backward": False},
        # its gradient in 32 bits, an odd number of tokens
        {"name": "dispatch_backward_fp32_t1021", "op": "dispatch", "T": 1021, "E": 512, "k": 10, "H": 2560,
         "dtype": "fp32", "backward": True},
        # back to token order after a decode step
        {"name": "combine_fp16_t8", "op": "combine", "T": 8, "E": 512, "k": 10, "H": 2560, "dtype": "fp16",
         "backward": False},
        # the gradients of a training step's combine: of the rows and of the router weights
        {"name": "combine_backward_bf16_t4096", "op": "combine", "T": 4096, "E": 512, "k": 10, "H": 2560,
         "dtype": "bf16", "backward": True},
        # the whole layer for one decoding token
        {"name": "layer_bf16_t1", "op": "layer", "T": 1, "E": 512, "k": 10, "H": 2560, "I": 640, "dtype": "bf16"},
        # the whole layer for a 1024-token prefill
        {"name": "layer_bf16_t1024", "op": "layer", "T": 1024, "E": 512, "k": 10, "H": 2560, "I": 640,
         "dtype": "bf16"},
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "dispatch", "combine", "layer"])
    kind = rng.choice(["fp32", "fp16", "bf16"])
    if op == "quantize":
        K = 32 * _log(rng, 1, 512)
        return {"op": op, "R": _log(rng, 1, min(200000, 81920 * 2560 // K)), "K": K, "dtype": kind}
    if op == "product":
        E = _log(rng, 1, 512)
        K = 32 * _log(rng, 2, 256)
        N = _log(rng, 16, 8192)
        if E * N * K > 512 * 1280 * 2560:
            N = max(16, 512 * 1280 * 2560 // (E * K))
        R = _log(rng, 1, min(40960, 8191 * 8192 * 8192 // (N * K)))
        return {"op": op, "E": E, "R": R, "N": N, "K": K, "dtype": kind}
    E = rng.choice([8, 37, 64, 128, 512])
    k = rng.randint(1, min(10, E))
    if op == "layer":
        H = 32 * _log(rng, 2, 80)
        I = 32 * _log(rng, 2, 20)
        return {"op": op, "T": _log(rng, 1, 1024), "E": E, "k": k, "H": H, "I": I,
                "dtype": rng.choice(["fp16", "bf16"])}
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": k, "H": _log(rng, 32, 2560), "dtype": kind,
            "backward": rng.random() < 0.5}


def _groups(K):
    """Bytes of one row's scales: one per 32 values, rows padded to whole 32-bit words."""
    return 4 * ((K + 127) // 128)


def _mx_bytes(rows, K):
    return rows * (K // 2 + K // 32)


def _active(E, R):
    """Expected number of experts that hold a row when R rows pick experts evenly."""
    return E * (1.0 - (1.0 - 1.0 / E) ** R) if E > 1 else 1


def work(case):
    op, c = case["op"], case
    if op == "quantize":
        n = c["R"] * c["K"]
        # values in, codes and scales out and in again, values out
        return {"bytes": 2 * n * SIZE[c["dtype"]] + 2 * _mx_bytes(c["R"], c["K"]), "flops": 0}
    if op == "product":
        experts = _active(c["E"], c["R"])
        return {"bytes": _mx_bytes(c["R"], c["K"]) + _mx_bytes(experts * c["N"], c["K"])
                + c["R"] * c["N"] * SIZE[c["dtype"]], "flops": 2 * c["R"] * c["N"] * c["K"]}
    S = c["T"] * c["k"]
    if op == "layer":
        H, I = c["H"], c["I"]
        experts = _active(c["E"], S)
        return {"bytes": experts * (_mx_bytes(2 * I, H) + _mx_bytes(H, I)) + 4 * c["T"] * c["E"] + 4 * c["T"] * H,
                "flops": 6 * S * H * I}
    size = SIZE[c["dtype"]]
    tokens, rows = c["T"] * c["H"] * size, S * c["H"] * size
    if op == "dispatch":
        routing = 4 * S if c["backward"] else 12 * S + 4 * c["E"]
        return {"bytes": tokens + rows + routing, "flops": S * c["H"] if c["backward"] else 0}
    if c["backward"]:
        return {"bytes": tokens + 2 * rows + 12 * S, "flops": 3 * S * c["H"]}
    return {"bytes": tokens + rows + 8 * S, "flops": 2 * S * c["H"]}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
def _codes(g, shape):
    return torch.randint(-(1 << 31), 1 << 31, shape, generator=g, device="cuda", dtype=torch.int32)


def _scales(g, shape, low, high):
    return torch.randint(low, high + 1, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)


def _weights(g, E, N, K):
    """Any codes, and scales that give rows of about unit norm."""
    middle = 127 + round(math.log2(1.0 / (2.93 * math.sqrt(K))))
    return _codes(g, (E, N, K // 8)), _scales(g, (E, N, _groups(K)), middle - 1, middle + 1)


def _activations(g, rows, cols, dtype):
    """Normal values with columns of unlike size, as hidden states have them."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    spread = torch.exp(torch.randn((cols,), generator=g, device="cuda"))
    return (x * spread).to(dtype)


def _padded_ids(g, T, E, k):
    """k distinct experts per token; every tenth token or so is padding and has none."""
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(dim=1)[:, :k].to(torch.int32)
    pad = torch.rand((T, 1), generator=g, device="cuda") < 0.1
    return torch.where(pad, torch.full_like(ids, -1), ids).contiguous()


def _sort_ids(ids, E):
    """(offsets [E + 1], sorted slots [S], rows of the slots [S]): slots by expert, in slot order; those without
    an expert come last and hold -1."""
    S = ids.numel()
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:E].cumsum(0)])
    at = torch.arange(S, device=ids.device)
    kept = at < offsets[E]
    rows = torch.empty_like(order)
    rows[order] = torch.where(kept, at, torch.full_like(at, -1))
    return (offsets.to(torch.int32), torch.where(kept, order, torch.full_like(order, -1)).to(torch.int32),
            rows.to(torch.int32))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    st = {"case": case}
    if op == "quantize":
        st["x"] = _activations(g, c["R"], c["K"], DTYPES[c["dtype"]])
    elif op == "product":
        st["a"] = (_codes(g, (c["R"], c["K"] // 8)), _scales(g, (c["R"], _groups(c["K"])), 125, 129))
        st["w"] = _weights(g, c["E"], c["N"], c["K"])
        counts = torch.bincount(torch.randint(0, c["E"], (c["R"],), generator=g, device="cuda"), minlength=c["E"])
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["most"] = int(counts.max())  # the plan of a program that pads: rows of the fullest expert
    elif op == "layer":
        st["logits"] = torch.randn((c["T"], c["E"]), generator=g, device="cuda")
        st["x"] = _activations(g, c["T"], c["H"], DTYPES[c["dtype"]])
        st["w13"] = _weights(g, c["E"], 2 * c["I"], c["H"])
        st["w2"] = _weights(g, c["E"], c["H"], c["I"])
        top = torch.topk(st["logits"], c["k"], dim=1)[1]
        st["most"] = int(torch.bincount(top.reshape(-1), minlength=c["E"]).max())
    else:
        T, k, H, dtype = c["T"], c["k"], c["H"], DTYPES[c["dtype"]]
        st["ids"] = _padded_ids(g, T, c["E"], k)
        if op == "dispatch" and not c["backward"]:
            st["x"] = _activations(g, T, H, dtype)
            st["sorted"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")
        else:
            st["rows"] = _sort_ids(st["ids"], c["E"])[2]
            if op == "dispatch":
                st["grad_sorted"] = _activations(g, T * k, H, dtype)
            else:
                st["weights"] = torch.rand((T, k), generator=g, device="cuda") + 0.05
                st["weights"] /= st["weights"].sum(1, keepdim=True)
                st["y"] = _activations(g, T * k, H, dtype)
                if c["backward"]:
                    st["grad"] = _activations(g, T, H, dtype)
                    st["grad_y"] = torch.zeros((T * k, H), dtype=dtype, device="cuda")
    return st


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantized(x):
    """The values that x [rows, K] stands for in MXFP4: per 32 values the scale 2^(floor(log2 max) - 2), then the
    nearest E2M1 value, ties to even, saturating at 6."""
    v = x.float().reshape(x.shape[0], -1, 32)
    exponent = (torch.frexp(v.abs().amax(2, keepdim=True))[1] - 3).clamp(-127, 127)
    a = torch.ldexp(v, -exponent)
    m = a.abs()
    q = (0.5 * (m > 0.25) + 0.5 * (m >= 0.75) + 0.5 * (m > 1.25) + 0.5 * (m >= 1.75) + 1.0 * (m > 2.5)
         + 1.0 * (m >= 3.5) + 2.0 * (m > 5.0))
    return torch.ldexp(torch.where(a < 0, -q, q), exponent).reshape(x.shape)


def _values(codes, scales):
    """fp32 values of MXFP4 codes [..., K/8] and scales [..., >= K/32]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=codes.device)
    shift = torch.arange(0, 32, 4, dtype=torch.int32, device=codes.device)
    v = table[((codes.unsqueeze(-1) >> shift) & 15)]
    v = v.reshape(*codes.shape[:-1], -1, 32)
    exponent = scales[..., : v.shape[-2]].to(torch.int32) - 127
    return torch.ldexp(v, exponent.unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _experts_product(a, w, offsets, most):
    """a [R, K] in expert order times each row's expert, w = (codes, scales) of [E, N, K]: fp32 [R, N].  Few rows
    take their expert's weights row by row; many are laid out in `most` places per expert."""
    E, N = w[0].shape[:2]
    R = a.shape[0]
    if E == 1:
        return a @ _values(w[0][0], w[1][0]).t()
    row = torch.arange(R, device=a.device)
    expert = torch.searchsorted(offsets[1:].contiguous(), row.to(torch.int32), right=True)
    if R <= E:
        return torch.bmm(_values(w[0][expert], w[1][expert]), a.unsqueeze(2)).squeeze(2)
    place = expert * most + row - offsets[expert].long()
    padded = torch.zeros((E * most, a.shape[1]), device=a.device)
    padded[place] = a
    y = torch.bmm(padded.view(E, most, -1), _values(*w).transpose(1, 2))
    return y.view(E * most, N)[place]


def _combined(y, weights, rows):
    """fp32 sum over a token's choices of weight times its row of y; choices without a row add nothing."""
    at = rows.view(weights.shape).long()
    picked = torch.where((at >= 0).unsqueeze(2), y[at.clamp(min=0)].float(), torch.zeros((), device=y.device))
    return (weights.unsqueeze(2) * picked).sum(1)


def _plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "quantize":
        return _quantized(st["x"]).to(st["x"].dtype)
    if op == "product":
        return _experts_product(_values(*st["a"]), st["w"], st["offsets"], st["most"]).to(DTYPES[c["dtype"]])
    if op == "layer":
        x, k = st["x"], c["k"]
        top, ids = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        weights = torch.softmax(top[:, :k], dim=1)
        offsets, slots, rows = _sort_ids(ids[:, :k].to(torch.int32), c["E"])
        h = _experts_product(_quantized(x)[slots.long() // k], st["w13"], offsets, st["most"])
        gate, up = h[:, :c["I"]], h[:, c["I"]:]
        y = _experts_product(_quantized(gate / (1.0 + torch.exp(-gate)) * up), st["w2"], offsets, st["most"])
        return _combined(y, weights, rows).to(x.dtype)
    if op == "dispatch" and not c["backward"]:
        offsets, slots, rows = _sort_ids(st["ids"], c["E"])
        kept = (slots >= 0).unsqueeze(1)
        st["sorted"] = torch.where(kept, st["x"][slots.clamp(min=0).long() // c["k"]], st["sorted"])
        return offsets, slots, rows, st["sorted"]
    if op == "dispatch":
        ones = torch.ones((c["T"], c["k"]), device="cuda")
        return _combined(st["grad_sorted"], ones, st["rows"]).to(st["grad_sorted"].dtype)
    if not c["backward"]:
        return _combined(st["y"], st["weights"], st["rows"]).to(st["y"].dtype)
    at = st["rows"].view(c["T"], c["k"]).long()
    kept = at >= 0
    grad = st["grad"].float().unsqueeze(1)
    picked = st["y"][at.clamp(min=0)].float()
    grad_weights = torch.where(kept, (grad * picked).sum(2), torch.zeros((), device="cuda"))
    st["grad_y"][at[kept]] = (st["weights"].unsqueeze(2) * grad)[kept].to(st["y"].dtype)
    return st["grad_y"], grad_weights


def _framework(st):
    from w4a16_group_quantized_amd import ops

    c, op = st["case"], st["case"]["op"]
    if op == "quantize":
        return ops.moe_mxfp4_dequantize(*ops.moe_mxfp4_quantize(st["x"]), st["x"].dtype)
    if op == "product":
        return ops.moe_mxfp4_grouped_gemm(*st["a"], *st["w"], st["offsets"], dtype=DTYPES[c["dtype"]])
    if op == "layer":
        w = {"w13_codes": st["w13"][0], "w13_scales": st["w13"][1], "w2_codes": st["w2"][0],
             "w2_scales": st["w2"][1]}
        return ops.moe_mxfp4_layer_forward(st["logits"], st["x"], c["k"], w)
    if op == "dispatch" and not c["backward"]:
        perm = ops.moe_permute_masked(st["ids"], c["E"])
        ops.moe_dispatch(st["x"], perm["slot_rows"], c["k"], out=st["sorted"])
        return perm["expert_offsets"], perm["sorted_slots"], perm["slot_rows"], st["sorted"]
    if op == "dispatch":
        return ops.moe_dispatch_backward(st["grad_sorted"], st["rows"], c["k"])
    if not c["backward"]:
        return ops.moe_combine_masked(st["y"], st["weights"], st["rows"])
    return ops.moe_combine_backward(st["grad"], st["y"], st["weights"], st["rows"], out=st["grad_y"])


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------- #
# from the definitions, in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    def _mx_decode(codes, scales):
        """MXFP4 as 64-bit values, from the bit fields: sign, two exponent bits with bias 1, one mantissa bit."""
        n = codes.shape[-1]
        parts = [((codes >> (4 * j)) & 15).to(torch.int64) for j in range(8)]
        code = torch.stack(parts, dim=-1).flatten(-2)
        sign = 1.0 - 2.0 * (code >> 3).double()
        field, mantissa = (code >> 1) & 3, (code & 1).double()
        size = torch.where(field == 0, 0.5 * mantissa, (1.0 + 0.5 * mantissa) * torch.exp2(field.double() - 1.0))
        scale = torch.exp2(scales[..., : n // 4].double() - 127.0)
        return sign * size * scale.repeat_interleave(32, dim=-1)

    def _mx_round(x):
        """The MXFP4 value of 64-bit x [rows, K], by distance to each E2M1 value (of two equally near, the even code)."""
        v = x.reshape(-1, 32)
        top = v.abs().max(dim=1).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        e = torch.where(torch.exp2(e) > top, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= top, e + 1, e) - 2
        e = torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(-127, 127)
        scale = torch.exp2(e).unsqueeze(1)
        m = (v / scale).abs()
        best, gap = torch.zeros_like(m), m.clone()
        for code in (2, 4, 6, 1, 3, 5, 7):  # even codes first: an odd one has to be strictly nearer
            near = (m - _E2M1[code]).abs()
            take = near < gap
            best, gap = torch.where(take, torch.full_like(m, _E2M1[code]), best), torch.where(take, near, gap)
        return (torch.sign(v) * best * scale).reshape(x.shape)

    def _by_expert(a, decoded, bounds, N):
        out = torch.zeros((a.shape[0], N), dtype=torch.float64, device=a.device)
        for e in range(len(bounds) - 1):
            lo, hi = bounds[e], bounds[e + 1]
            if hi > lo:
                out[lo:hi] = a[lo:hi] @ decoded(e).t()
        return out

    st, c, op = prepare(case, seed), case, case["op"]
    if op == "quantize":
        # in slices of rows: a 64-bit copy of the largest case does not pay
        step = max(1, (1 << 25) // c["K"])
        return torch.cat([_mx_round(st["x"][r:r + step].double()).to(torch.float32)
                          for r in range(0, c["R"], step)]).to(DTYPES[c["dtype"]])
    if op == "product":
        a, (codes, scales) = _mx_decode(*st["a"]), st["w"]
        return _by_expert(a, lambda e: _mx_decode(codes[e], scales[e]), st["offsets"].tolist(), c["N"])
    k = c["k"]
    if op == "layer":
        T, E, I = c["T"], c["E"], c["I"]
        logits = st["logits"].double()
        left, ids = logits.clone(), []
        for _ in range(k):
            ids.append(left.argmax(dim=1))
            left.scatter_(1, ids[-1].unsqueeze(1), -math.inf)
        ids = torch.stack(ids, dim=1)
        p = torch.exp(torch.gather(logits, 1, ids) - logits.max(dim=1, keepdim=True).values)
        p = p / p.sum(dim=1, keepdim=True)
        x = _mx_round(st["x"].double())
        out = torch.zeros((T, c["H"]), dtype=torch.float64, device="cuda")
        for e in range(E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if t.numel():
                h = x[t] @ _mx_decode(st["w13"][0][e], st["w13"][1][e]).t()
                act = _mx_round(torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:])
                out.index_add_(0, t, p[t, j].unsqueeze(1) * (act @ _mx_decode(st["w2"][0][e], st["w2"][1][e]).t()))
        return out
    T, S, H = c["T"], c["T"] * k, c["H"]
    if op == "dispatch" and not c["backward"]:
        flat = st["ids"].reshape(-1).long()
        keys = (flat * S + torch.arange(S, device="cuda"))[flat >= 0].sort().values
        moved = torch.zeros((S, H), dtype=torch.float64, device="cuda")
        moved[: keys.numel()] = st["x"][(keys % S) // k].double()
        return None, None, None, moved
    at = st["rows"].long()
    slots = torch.nonzero(at >= 0).squeeze(1)
    if op == "dispatch":
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        return out.index_add_(0, slots // k, st["grad_sorted"][at[slots]].double())
    w = st["weights"].double().reshape(-1)
    if not c["backward"]:
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        return out.index_add_(0, slots // k, w[slots].unsqueeze(1) * st["y"][at[slots]].double())
    grad_y = torch.zeros((S, H), dtype=torch.float64, device="cuda")
    grad = st["grad"].double()[slots // k]
    grad_y[at[slots]] = w[slots].unsqueeze(1) * grad
    grad_weights = torch.zeros(S, dtype=torch.float64, device="cuda")
    grad_weights[slots] = (grad * st["y"][at[slots]].double()).sum(dim=1)
    return grad_y, grad_weights.view(T, k)
