"""What is measured of the training side of the routed experts.

Four operators between dispatch and combine, and behind them:

  product  rows times their expert's weights, grouped by expert, in 16 bits: the product itself, and its gradients
           of the rows and of the weights
  act      SiLU(gate) * up between an expert's two products, and its gradient
  route    the gradient of the router's weights (softmax over the chosen experts) with respect to its logits
  adamw    one AdamW step over many tensors, the two states in fp32 or in 8 bits

A case's sizes: E experts, R rows in expert order, N output columns, K reduction length, I intermediate size, T
tokens, k experts per token; count tensors of about n elements.
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
        # gate/up of eight tokens on 512 experts, 10 per token: bound by reading the chosen experts' weights
        {"name": "product_bf16_e512_r80", "op": "product", "to": "out", "E": 512, "R": 80, "N": 1280, "K": 2560,
         "dtype": "bf16", "out": "bf16"},
        # gate/up of a 4096-token training step
        {"name": "product_bf16_e512_r40960", "op": "product", "to": "out", "E": 512, "R": 40960, "N": 1280,
         "K": 2560, "dtype": "bf16", "out": "bf16"},
        # few large experts, an odd number of rows: bound by the matrix cores
        {"name": "product_fp16_e8_r16381", "op": "product", "to": "out", "E": 8, "R": 16381, "N": 8192, "K": 4096,
         "dtype": "fp16", "out": "fp16"},
        # the gradient of the rows through the same experts
        {"name": "rows_bf16_e8_r16381", "op": "product", "to": "rows", "E": 8, "R": 16381, "N": 8192, "K": 4096,
         "dtype": "bf16", "out": "bf16"},
        # the gradient of the 512 experts' gate/up weights: bound by writing it
        {"name": "weights_bf16_e512_r40960", "op": "product", "to": "weights", "E": 512, "R": 40960, "N": 1280,
         "K": 2560, "dtype": "bf16", "out": "bf16"},
        # the gradient of few large experts' weights in fp32, as it is summed over micro-batches
        {"name": "weights_fp16_e8_r16381", "op": "product", "to": "weights", "E": 8, "R": 16381, "N": 8192,
         "K": 4096, "dtype": "fp16", "out": "fp32"},
        # the activation of eight tokens' rows
        {"name": "act_bf16_r80", "op": "act", "R": 80, "I": 640, "dtype": "bf16", "backward": False},
        # its gradient in a 4096-token training step
        {"name": "act_backward_bf16_r40960", "op": "act", "R": 40960, "I": 640, "dtype": "bf16", "backward": True},
        # the router's gradient for eight tokens, and for a training step
        {"name": "route_t8", "op": "route", "T": 8, "E": 512, "k": 10},
        {"name": "route_t4096", "op": "route", "T": 4096, "E": 512, "k": 10},
        # a block's small tensors (norms, a router): many of them, states in fp32, latency counts
        {"name": "adamw_fp32_30_small", "op": "adamw", "count": 30, "n": 2560, "bits": 32, "dtype": "fp32",
         "copy": False},
        # 32 experts' gate/up weights: fp32 parameters with a bf16 copy for the products, states in 8 bits
        {"name": "adamw_8bit_105m", "op": "adamw", "count": 1, "n": 32 * 1280 * 2560, "bits": 8, "dtype": "fp32",
         "copy": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "act", "route", "adamw", "adamw"])
    if op == "product":
        E = rng.choice([1, 8, 37, 64, 128, 512])
        K = 8 * _log(rng, 8, 512)
        N = 8 * _log(rng, 8, 1024)
        if E * N * K > 512 * 1280 * 2560:
            N = max(8, 512 * 1280 * 2560 // (E * K) // 8 * 8)
        R = _log(rng, 1, min(40960, 16381 * 8192 * 4096 // (N * K)))
        to = rng.choice(["out", "rows", "weights"])
        kind = rng.choice(["fp16", "bf16"])
        return {"op": op, "to": to, "E": E, "R": R, "N": N, "K": K, "dtype": kind,
                "out": rng.choice([kind, kind, "fp32"])}
    if op == "act":
        I = _log(rng, 16, 8192)
        return {"op": op, "R": _log(rng, 1, min(40960, 40960 * 640 // I)), "I": I,
                "dtype": rng.choice(["fp32", "fp16", "bf16"]), "backward": rng.random() < 0.5}
    if op == "route":
        E = rng.choice([8, 37, 64, 128, 512])
        return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(10, E))}
    count = _log(rng, 1, 60)
    return {"op": op, "count": count, "n": _log(rng, 1, 32 * 1280 * 2560 // count), "bits": rng.choice([8, 32]),
            "dtype": rng.choice(["fp32", "bf16", "fp16"]), "copy": rng.random() < 0.5}


def _sizes(c):
    """Elements of each tensor of an adamw case: odd ones and unequal ones among them."""
    return [max(1, c["n"] - (i * 37) % (c["n"] // 8 + 1)) for i in range(c["count"])]


def _active(E, R):
    """Expected number of experts that hold a row when R rows pick experts evenly."""
    return E * (1.0 - (1.0 - 1.0 / E) ** R) if E > 1 else 1


def work(case):
    c = case
    if c["op"] == "product":
        R, N, K, size, out = c["R"], c["N"], c["K"], SIZE[c["dtype"]], SIZE[c["out"]]
        weights = _active(c["E"], R) * N * K * size
        if c["to"] == "weights":
            return {"bytes": R * (N + K) * size + c["E"] * N * K * out, "flops": 2 * R * N * K}
        rows = R * (K * size + N * out) if c["to"] == "out" else R * (N * size + K * out)
        return {"bytes": weights + rows, "flops": 2 * R * N * K}
    if c["op"] == "act":
        return {"bytes": c["R"] * c["I"] * SIZE[c["dtype"]] * (5 if c["backward"] else 3),
                "flops": c["R"] * c["I"] * (12 if c["backward"] else 5)}
    if c["op"] == "route":
        return {"bytes": 12 * c["T"] * c["k"] + 4 * c["T"] * c["E"], "flops": 4 * c["T"] * c["k"]}
    size = SIZE[c["dtype"]]
    each = 2 * size + size + (2 if c["copy"] else 0) + (16 if c["bits"] == 32 else 4 + 16 / 128)
    return {"bytes": sum(_sizes(c)) * each, "flops": 14 * sum(_sizes(c))}


# --------------------------------------------------------------------------- #
# inputs
# --------------------------------------------------------------------------- #
LR, BETA1, BETA2, EPS, DECAY, STEP, SEED = 1e-4, 0.9, 0.999, 1e-8, 0.1, 1000, 77
BLOCK = 128


def _rows(g, rows, cols, dtype, scale=1.0):
    """Normal values with columns of unlike size, as hidden states and their gradients have them."""
    spread = scale * torch.exp(0.5 * torch.randn((cols,), generator=g, device="cuda"))
    return (torch.randn((rows, cols), generator=g, device="cuda") * spread).to(dtype)


def _states(g, n, bits):
    """The two moments of a tensor in mid-training: gradients of about 1e-3, a few elements far above the others."""
    size = 1e-3 * torch.exp(torch.randn((n,), generator=g, device="cuda"))
    m = 0.2 * size * torch.randn((n,), generator=g, device="cuda")
    v = size.square()
    if bits == 32:
        return m, v
    half = torch.full((n,), 1 << 19, dtype=torch.int64, device="cuda")
    return _encode(m, half, True), _encode(v, half, False)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    st = {"case": case}
    if op == "product":
        E, R, N, K, dtype = c["E"], c["R"], c["N"], c["K"], DTYPES[c["dtype"]]
        counts = torch.bincount(torch.randint(0, E, (R,), generator=g, device="cuda"), minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["most"] = int(counts.max())  # the plan of a program that pads: rows of the fullest expert
        if c["to"] != "rows":
            st["a"] = _rows(g, R, K, dtype)
        if c["to"] != "out":
            st["grad"] = _rows(g, R, N, dtype, 0.01)
        if c["to"] != "weights":
            st["w"] = torch.empty((E, N, K), dtype=dtype, device="cuda").normal_(0, 1 / math.sqrt(K), generator=g)
    elif op == "act":
        st["h"] = _rows(g, c["R"], 2 * c["I"], DTYPES[c["dtype"]])
        if c["backward"]:
            st["grad"] = _rows(g, c["R"], c["I"], DTYPES[c["dtype"]])
    elif op == "route":
        top, ids = torch.randn((c["T"], c["E"]), generator=g, device="cuda").topk(c["k"], dim=1)
        st["ids"], st["weights"] = ids.to(torch.int32), torch.softmax(top, dim=1)
        st["grad"] = torch.randn((c["T"], c["k"]), generator=g, device="cuda")
    else:
        dtype = DTYPES[c["dtype"]]
        st["params"], st["grads"], st["m"], st["v"] = [], [], [], []
        for n in _sizes(c):
            st["params"].append((0.05 * torch.randn((n,), generator=g, device="cuda")).to(dtype))
            m, v = _states(g, n, c["bits"])
            st["m"].append(m)
            st["v"].append(v)
            st["grads"].append((1e-3 * torch.randn((n,), generator=g, device="cuda")).to(dtype))
        st["copies"] = [torch.empty_like(p, dtype=torch.bfloat16) for p in st["params"]] if c["copy"] else None
    return st


# --------------------------------------------------------------------------- #
# plain forms
# --------------------------------------------------------------------------- #
def _padded(x, place, total):
    out = torch.zeros((total, x.shape[1]), device=x.device)
    out[place] = x.float()
    return out


def _product(st):
    """Few rows take their expert's weights row by row; many are laid out in `most` places per expert."""
    c, offsets, most = st["case"], st["offsets"], st["most"]
    E, R, N, K = c["E"], c["R"], c["N"], c["K"]
    row = torch.arange(R, device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), row.to(torch.int32), right=True)
    place = expert * most + row - offsets[expert].long()
    if c["to"] == "weights":
        grad = _padded(st["grad"], place, E * most).view(E, most, N)
        a = _padded(st["a"], place, E * most).view(E, most, K)
        return torch.bmm(grad.transpose(1, 2), a)
    if c["to"] == "out":
        if R <= E:
            return torch.bmm(st["w"][expert].float(), st["a"].float().unsqueeze(2)).squeeze(2)
        a = _padded(st["a"], place, E * most).view(E, most, K)
        return torch.bmm(a, st["w"].float().transpose(1, 2)).view(E * most, N)[place]
    if R <= E:
        return torch.bmm(st["grad"].float().unsqueeze(1), st["w"][expert].float()).squeeze(1)
    grad = _padded(st["grad"], place, E * most).view(E, most, N)
    return torch.bmm(grad, st["w"].float()).view(E * most, K)[place]


def _noise(index, seed, which):
    """20 bits per element, the same for everybody: a mix of the element's number and the seed in 32 bits."""
    low = 0xFFFFFFFF
    x = (index + seed * 0x9E3779B9) & low
    x = ((x ^ (x >> 16)) * 0x6A09E667) & low
    x = ((x ^ (x >> 15)) * 0xB7E15163) & low
    x = x ^ (x >> 16)
    return (x if which == 0 else (x * 0x9E3779B1) & low) >> 12


def _blocks(x):
    """x [n] as rows of 128, zeros behind the end."""
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _encode(x, noise, signed):
    """(codes uint8 [n], scales fp32 [blocks]): per block of 128 the scale max / 1.875 and floats of 3 mantissa bits,
    4 (signed) or 5 exponent bits, rounded up where the 20 bits behind them and the noise carry.  Positive values
    of an unsigned tensor do not become 0."""
    n = x.numel()
    b = _blocks(x)
    scale = b.abs().amax(1) / 1.875
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    inverse = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale)).unsqueeze(1)
    place = (b.abs() * inverse) * (2.0 ** -112 if signed else 2.0 ** -96)
    code = (place.view(torch.int32).long() + _blocks(noise)) >> 20
    code = code.clamp(max=127 if signed else 255)
    if signed:
        code = code + 128 * (b < 0)
    else:
        code = torch.where((code == 0) & (b > 0), torch.ones_like(code), code)
    return code.view(-1)[:n].to(torch.uint8), scale


def _decode(state, signed):
    codes, scales = state
    c = codes.to(torch.int32)
    value = ((c & 127 if signed else c) << 20).view(torch.float32) * (2.0 ** 112 if signed else 2.0 ** 96)
    value = (_blocks(value) * scales.unsqueeze(1)).view(-1)[: codes.numel()]
    return torch.where(c > 127, -value, value) if signed else value


def _adamw(st):
    """All tensors as one long one, each filled up to whole blocks of 128, and back."""
    c, sizes = st["case"], _sizes(st["case"])
    bits8 = c["bits"] == 8
    filled = [n + -n % BLOCK for n in sizes]
    flat = lambda parts: torch.cat([_blocks(x) for x in parts]).view(-1)  # noqa: E731
    p, g = flat(st["params"]).float(), flat(st["grads"]).float()
    if bits8:
        m, v = (_decode((flat([x[0] for x in st[k]]), torch.cat([x[1] for x in st[k]])), k == "m") for k in "mv")
    else:
        m, v = flat(st["m"]), flat(st["v"])
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    root = v.sqrt() * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS
    p = p * (1 - LR * DECAY) - (LR / (1 - BETA1 ** STEP)) * (m / root)
    changed = [(st["params"], p)] + ([(st["copies"], p)] if c["copy"] else [])
    if bits8:
        index = torch.cat([torch.arange(n, device="cuda") for n in filled])
        for k, x in (("m", m), ("v", v)):
            codes, scales = _encode(x, _noise(index, SEED, "mv".index(k)), k == "m")
            changed.append(([part[0] for part in st[k]], codes))
            for part, s in zip(st[k], scales.split([n // BLOCK for n in filled])):
                part[1].copy_(s)
    else:
        changed += [(st["m"], m), (st["v"], v)]
    for parts, x in changed:
        for part, new in zip(parts, x.split(filled)):
            part.copy_(new[: part.numel()])
    return _adamw_outputs(st)


def _adamw_outputs(st):
    """All that the step changed, one tensor of each kind; 8-bit states as the values they stand for (of 4
    significant bits, so 16-bit values hold them)."""
    whole = lambda parts: torch.cat(parts) if len(parts) > 1 else parts[0]  # noqa: E731
    if st["case"]["bits"] == 8:
        m = whole([_decode(x, True) for x in st["m"]]).to(torch.bfloat16)
        v = whole([_decode(x, False) for x in st["v"]]).to(torch.bfloat16)
    else:
        m, v = whole(st["m"]), whole(st["v"])
    return whole(st["params"]), m, v, whole(st["copies"]) if st["copies"] else None


def _plain(st):
    c, op = st["case"], st["case"]["op"]
    if op == "product":
        return _product(st).to(DTYPES[c["out"]])
    if op == "act":
        gate, up = st["h"][:, :c["I"]].float(), st["h"][:, c["I"]:].float()
        s = 1.0 / (1.0 + torch.exp(-gate))
        if not c["backward"]:
            return (gate * s * up).to(st["h"].dtype)
        grad = st["grad"].float()
        return torch.cat([grad * up * s * (1.0 + gate * (1.0 - s)), grad * gate * s], dim=1).to(st["h"].dtype)
    if op == "route":
        w, g = st["weights"], st["grad"]
        each = w * (g - (w * g).sum(1, keepdim=True))
        return torch.zeros((c["T"], c["E"]), device="cuda").scatter_(1, st["ids"].long(), each)
    return _adamw(st)


def _framework(st):
    from w4a16_group_quantized_amd import ops

    c, op = st["case"], st["case"]["op"]
    if op == "product":
        dtype = DTYPES[c["out"]]
        if c["to"] == "out":
            return ops.moe_grouped_gemm(st["a"], st["w"], st["offsets"], dtype=dtype)
        if c["to"] == "rows":
            return ops.moe_grouped_gemm_backward(st["grad"], st["w"], st["offsets"], dtype=dtype)
        return ops.moe_grouped_gemm_backward_weights(st["grad"], st["a"], st["offsets"], dtype=dtype)
    if op == "act":
        if c["backward"]:
            return ops.moe_silu_mul_backward(st["grad"], st["h"])
        return ops.moe_silu_mul(st["h"])
    if op == "route":
        return ops.moe_route_backward(st["ids"], st["weights"], st["grad"], c["E"])
    ops.moe_adamw(st["params"], st["grads"], st["m"], st["v"], lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS,
                  weight_decay=DECAY, step=STEP, seed=SEED, copies=st["copies"])
    return _adamw_outputs(st)


def run(state):
    return _framework(state) if own else _plain(state)


# --------------------------------------------------------------------------- #
# from the definitions, in 64 bits
# --------------------------------------------------------------------------- #
def exact(case, seed):
    c, op, st = case, case["op"], prepare(case, seed)
    if op == "product":
        bounds = st["offsets"].tolist()
        shape = {"out": (c["R"], c["N"]), "rows": (c["R"], c["K"]), "weights": (c["E"], c["N"], c["K"])}[c["to"]]
        # an expert at a time; kept in fp32 where the 64-bit whole would take tens of GB
        kept = torch.float32 if math.prod(shape) > 1 << 30 else torch.float64
        out = torch.zeros(shape, dtype=kept, device="cuda")
        for e in range(c["E"]):
            r = slice(bounds[e], bounds[e + 1])
            if r.start == r.stop:
                continue
            if c["to"] == "out":
                out[r] = st["a"][r].double() @ st["w"][e].double().t()
            elif c["to"] == "rows":
                out[r] = st["grad"][r].double() @ st["w"][e].double()
            else:
                out[e] = (st["grad"][r].double().t() @ st["a"][r].double()).to(kept)
        return out
    if op == "act":
        h = st["h"].double()
        gate, up = h[:, :c["I"]], h[:, c["I"]:]
        if not c["backward"]:
            return gate * torch.sigmoid(gate) * up
        grad, s, t = st["grad"].double(), torch.sigmoid(gate), torch.sigmoid(-gate)
        return torch.cat([grad * up * (s + gate * s * t), grad * gate * s], dim=1)
    if op == "route":
        w, g = st["weights"].double(), st["grad"].double()
        jacobian = torch.diag_embed(w) - w.unsqueeze(2) * w.unsqueeze(1)
        each = (jacobian * g.unsqueeze(1)).sum(2)
        out = torch.zeros((c["T"], c["E"]), dtype=torch.float64, device="cuda")
        out[torch.arange(c["T"], device="cuda").unsqueeze(1), st["ids"].long()] = each
        return out

    def mixed(n, which):
        x = (torch.arange(n, device="cuda") + SEED * 0x9E3779B9) % (1 << 32)
        for shift, factor in ((16, 0x6A09E667), (15, 0xB7E15163)):
            x = torch.bitwise_xor(x, x // (1 << shift)) * factor
            x = torch.bitwise_and(x, (1 << 32) - 1)
        x = torch.bitwise_xor(x, x // (1 << 16))
        if which:
            x = torch.bitwise_and(x * 0x9E3779B1, (1 << 32) - 1)
        return (x // 4096).double() / (1 << 20)

    def value(state, signed):
        """Codes by their fields: exponent f (bias 15 or 31, f = 0 subnormal) and three mantissa bits."""
        code = state[0].long()
        sign = 1.0 - 2.0 * (code // 128).double() if signed else 1.0
        code = code % 128 if signed else code
        f, man, bias = code // 8, (code % 8).double() / 8, 15 if signed else 31
        size = torch.where(f > 0, (1 + man) * torch.exp2((f - bias).double()), man * 2.0 ** (1 - bias))
        return sign * size * state[1].double().repeat_interleave(BLOCK)[: code.numel()]

    def rounded(x, u, signed):
        """Each value to the one of its two neighbours in the code that u picks."""
        n, bias = x.numel(), 15 if signed else 31
        top = torch.nn.functional.pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK).max(1).values
        scale = (top / 1.875).repeat_interleave(BLOCK)[:n]
        t = torch.where(scale > 0, x.abs() / scale, torch.zeros_like(x))
        f = torch.floor(torch.log2(torch.clamp(t, min=2.0 ** (1 - bias)))).clamp(min=1 - bias)
        f = torch.where(torch.exp2(f) > t, (f - 1).clamp(min=1 - bias), f)
        step = torch.exp2(f - 3)
        t = (torch.floor(t / step + u) * step).clamp(max=1.875)
        if not signed:
            t = torch.where((t == 0) & (x > 0), torch.full_like(t, 2.0 ** (-2 - bias)), t)
        return torch.sign(x) * t * scale

    outs = [[], [], [], []]
    for i, p in enumerate(st["params"]):
        g = st["grads"][i].double()
        m, v = st["m"][i], st["v"][i]
        m, v = (value(m, True), value(v, False)) if c["bits"] == 8 else (m.double(), v.double())
        m, v = m + (1 - BETA1) * (g - m), v + (1 - BETA2) * (g.square() - v)
        update = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)).sqrt() + EPS)
        p = p.double()
        p = p - LR * (update + DECAY * p)
        if c["bits"] == 8:
            m, v = rounded(m, mixed(p.numel(), 0), True), rounded(v, mixed(p.numel(), 1), False)
        for to, x in zip(outs, (p, m, v, p)):
            to.append(x)
    p, m, v, copy = (torch.cat(x) for x in outs)
    return p, m, v, copy if c["copy"] else None
