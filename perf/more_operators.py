"""The int4 layer with what surrounds it folded in: what is timed, and on what.

Five operators of a decoder block's linear and routed-expert layers (int4 codes q in
[-8, 7], eight offset-binary nibbles per 32-bit word along K, one fp16 scale per group
of 128 or 32 input features; fp16 activations and gradients):

  topk        the router's choice: each token's topk largest logits (ties: the lowest
              expert first), and their softmax over all experts or over the chosen ones
  topk_bwd    the gradient of the logits from the gradient of those weights
  moe         the whole routed feed-forward for a few tokens: sum over a token's experts
              of weight * down(SiLU(g) u), (g, u) = the expert's gate/up product
  linear      y = act(x . deq(W)^T + bias) + residual, for any number of rows; in training
              the fp16 pre-activations are kept for the backward pass
  linear_bwd  the gradient of the pre-activations, of the bias (their column sums) and of x

Where `own` is false, run() computes them in their plain form: elementary torch
operations in 32 bits, rounded once at the end.
"""

import math

import torch

own = False

# The dense feed-forward's hidden and intermediate widths; the routed experts' widths, number, and how many
# of them a token uses.
HIDDEN, INTER = 5120, 17408
EXPERT_HIDDEN, EXPERT_INTER, EXPERTS, TOPK = 2048, 512, 256, 8
FEW_TOKENS = 64
GELU_CUBIC = 0.044715


def _moe(name, tokens, **other):
    case = {"name": name, "op": "moe", "tokens": tokens, "experts": EXPERTS, "hidden": EXPERT_HIDDEN,
            "inter": EXPERT_INTER, "topk": TOPK, "group": 32, "spread": EXPERTS, "residual": True}
    case.update(other)
    return case


def listed():
    return [
        # the router of a single decoded token: launch latency counts
        {"name": "topk_1_256", "op": "topk", "tokens": 1, "experts": EXPERTS, "topk": TOPK, "half": False, "renormalize": True,
         "masked": False},
        # the router of a long prompt
        {"name": "topk_16384_256", "op": "topk", "tokens": 16384, "experts": EXPERTS, "topk": TOPK, "half": False,
         "renormalize": True, "masked": False},
        # a ragged training micro-batch, half-precision logits, some experts masked out, weights over all experts
        {"name": "topk_bwd_133_160", "op": "topk_bwd", "tokens": 133, "experts": 160, "topk": 6, "half": True,
         "renormalize": False, "masked": True},
        # a training batch
        {"name": "topk_bwd_8192_256", "op": "topk_bwd", "tokens": 8192, "experts": EXPERTS, "topk": TOPK, "half": False,
         "renormalize": True, "masked": False},
        # one decoded token through the routed experts: eight experts' weights, latency
        _moe("moe_1", 1),
        # an odd batch, routed to few experts of a bank with other widths and groups
        _moe("moe_13_skewed", 13, experts=60, hidden=1408, inter=384, topk=4, group=128, spread=9, residual=False),
        # a full decode batch: nearly every expert's weights once
        _moe("moe_64", FEW_TOKENS),
        # a decoded token's down projection, added to the residual stream
        {"name": "linear_1_down", "op": "linear", "m": 1, "n": HIDDEN, "k": INTER, "group": 128, "bias": False, "act": "none",
         "residual": True, "keep": False},
        # a ragged decode batch through a small odd layer with bias and GELU
        {"name": "linear_27_2003_2080", "op": "linear", "m": 27, "n": 2003, "k": 2080, "group": 32, "bias": True,
         "act": "gelu_tanh", "residual": False, "keep": False},
        # a training batch through the up projection, pre-activations kept
        {"name": "linear_4096_up", "op": "linear", "m": 4096, "n": INTER, "k": HIDDEN, "group": 128, "bias": True, "act": "gelu",
         "residual": False, "keep": True},
        # gradients of a few rows through an odd layer, and of a training batch
        {"name": "linear_bwd_19_1001_1120", "op": "linear_bwd", "m": 19, "n": 1001, "k": 1120, "group": 32, "bias": True,
         "act": "silu"},
        {"name": "linear_bwd_2048_up", "op": "linear_bwd", "m": 2048, "n": INTER, "k": HIDDEN, "group": 128, "bias": True,
         "act": "gelu"},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["topk", "topk_bwd", "moe", "moe", "linear", "linear", "linear_bwd"])
    if op in ("topk", "topk_bwd"):
        most = 16384 if op == "topk" else 8192
        experts = _log(rng, 4, 512)
        return {"op": op, "tokens": _log(rng, 1, min(most, most * EXPERTS // experts)), "experts": experts,
                "topk": rng.randint(1, min(10, experts)), "half": rng.random() < 0.5, "renormalize": rng.random() < 0.5,
                "masked": rng.random() < 0.3}
    group = rng.choice([32, 128])
    if op == "moe":
        hidden, inter = group * _log(rng, 1, 4096 // group), group * _log(rng, 1, 1024 // group)
        size = EXPERT_HIDDEN * EXPERT_INTER
        experts = _log(rng, 4, min(EXPERTS, EXPERTS * size // (hidden * inter)))
        topk = rng.randint(1, min(TOPK, experts))
        tokens = _log(rng, 1, max(1, min(FEW_TOKENS, FEW_TOKENS * TOPK * size // (topk * hidden * inter))))
        return {"op": op, "tokens": tokens, "experts": experts, "hidden": hidden, "inter": inter, "topk": topk, "group": group,
                "spread": rng.choice([experts, rng.randint(topk, experts)]), "residual": rng.random() < 0.5}
    case = {"op": op, "m": _log(rng, 1, 4096 if op == "linear" else 2048), "n": _log(rng, 9, INTER),
            "k": group * _log(rng, 1, HIDDEN // group), "group": group, "bias": rng.random() < 0.7,
            "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])}
    if rng.random() < 0.4:                          # the down projection's orientation
        case["n"], case["k"] = _log(rng, 9, HIDDEN), group * _log(rng, 1, INTER // group)
    if op == "linear":
        case["residual"] = rng.random() < 0.5
        case["keep"] = case["act"] != "none" and rng.random() < 0.5
    return case


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _half(gen, *shape, std=1.0):
    return (_randn(gen, *shape) * std).to(torch.float16)


def _weights(gen, rows, k, group):
    """Gaussian weights quantised symmetrically: (int32 words [rows, k/8], fp16 scales [rows, k/group])."""
    w = _randn(gen, rows, k // group, group) * 0.02
    s = (w.abs().amax(dim=2) / 7).to(torch.float16)
    q = (w / s.float().unsqueeze(2)).round().clamp(-8, 7).to(torch.int32).reshape(rows, k // 8, 8) + 8
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    return (q << shift).sum(dim=2, dtype=torch.int64).to(torch.int32), s


def _bank(gen, experts, rows, k, group):
    """An experts' bank: codes drawn evenly, scales of the size that such weights have."""
    words = torch.randint(-2 ** 31, 2 ** 31, (experts, rows, k // 8), generator=gen, device="cuda", dtype=torch.int64)
    s = torch.rand((experts, rows, k // group), generator=gen, device="cuda") * 1.5 + 1.5
    return words.to(torch.int32), (s * (0.02 / 7)).to(torch.float16)


def _logits(case, gen):
    """Router logits, some of them masked out; at most one in sixteen tokens is left fewer experts than it asks for."""
    x = _randn(gen, case["tokens"], case["experts"]) * 2
    if case["masked"]:
        drop = torch.rand(x.shape, generator=gen, device="cuda") < 0.2
        bare = torch.rand((x.shape[0], 1), generator=gen, device="cuda") < 1 / 16
        x = x.masked_fill(drop | (bare & (torch.rand(x.shape, generator=gen, device="cuda") < 0.97)), -math.inf)
    return x.to(torch.float16) if case["half"] else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] in ("topk", "topk_bwd"):
        st["logits"] = _logits(case, gen)
        if case["op"] == "topk_bwd":
            # what the forward pass left, and a gradient of the size a mean over the batch gives
            st["ids"], st["weights"] = _plain_topk(st["logits"], case["topk"], case["renormalize"])
            st["dweights"] = _randn(gen, case["tokens"], case["topk"]) * 0.05
        return st
    if case["op"] == "moe":
        t, e, h, i, group = case["tokens"], case["experts"], case["hidden"], case["inter"], case["group"]
        st["gate_up"], st["gate_up_scales"] = _bank(gen, e, 2 * i, h, group)
        st["down"], st["down_scales"] = _bank(gen, e, h, i, group)
        st["x"] = _half(gen, t, h)
        used = torch.randperm(e, generator=gen, device="cuda")[:case["spread"]]
        top, at = torch.topk(_randn(gen, t, case["spread"]) * 2, case["topk"], dim=1)
        st["ids"], st["weights"] = used[at].to(torch.int32), torch.softmax(top, dim=1)
        st["residual"] = _half(gen, t, h) if case["residual"] else None
        st["out"] = torch.empty((t, h), dtype=torch.float16, device="cuda")
        return st
    m, n, k = case["m"], case["n"], case["k"]
    st["packed"], st["scales"] = _weights(gen, n, k, case["group"])
    half = dict(dtype=torch.float16, device="cuda")
    if case["op"] == "linear":
        st["x"] = _half(gen, m, k)
        st["bias"] = _half(gen, n, std=0.5) if case["bias"] else None
        st["residual"] = _half(gen, m, n) if case["residual"] else None
        st["pre"] = torch.empty((m, n), **half) if case["keep"] else None
        st["out"] = torch.empty((m, n), **half)
    else:
        # pre-activations of the size N(0, 1) inputs give, and loss-scaled gradients
        st["dy"] = _half(gen, m, n, std=0.05)
        st["pre"] = _half(gen, m, n, std=0.02 * k ** 0.5) if case["act"] != "none" else None
        st["dpre"] = torch.empty((m, n), **half) if case["act"] != "none" else None
        st["dbias"] = torch.empty(n, dtype=torch.float32, device="cuda") if case["bias"] else None
        st["out"] = torch.empty((m, k), **half)
    return st


def _dequantised(packed, scales, group):
    """[..., k/8] words and [..., k/group] scales -> fp32 [..., k]."""
    shift = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    codes = ((packed.unsqueeze(-1) >> shift) & 15).sub(8).to(torch.float32).flatten(-2)
    return codes * scales.to(torch.float32).repeat_interleave(group, dim=-1)


def _act(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + GELU_CUBIC * z * z * z)))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if name == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    sig = 1 / (1 + torch.exp(-c * (z + GELU_CUBIC * z * z * z)))
    return sig + z * sig * (1 - sig) * c * (1 + 3 * GELU_CUBIC * z * z)


def _plain_topk(logits, topk, renormalize):
    x = logits.to(torch.float32)
    order = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = order.values[:, :topk], order.indices[:, :topk]
    chosen = top > -math.inf                        # an expert that is masked out is not chosen
    peak = torch.where(top[:, :1] > -math.inf, top[:, :1], torch.zeros_like(top[:, :1]))
    e = torch.exp(top - peak)
    total = e.sum(dim=1, keepdim=True) if renormalize else torch.exp(x - peak).sum(dim=1, keepdim=True)
    weights = torch.where(chosen, e / total, torch.zeros_like(e))
    return torch.where(chosen, ids, torch.full_like(ids, -1)).to(torch.int32), weights


def _plain_topk_backward(st, renormalize):
    ids, weights, dw = st["ids"].to(torch.int64), st["weights"], st["dweights"]
    chosen = ids >= 0
    mean = torch.where(chosen, weights * dw, torch.zeros_like(dw)).sum(dim=1, keepdim=True)
    x = st["logits"].to(torch.float32)
    if renormalize:
        dlogits = torch.zeros_like(x)
    else:
        peak = x.amax(dim=1, keepdim=True)
        e = torch.exp(x - torch.where(peak > -math.inf, peak, torch.zeros_like(peak)))
        total = e.sum(dim=1, keepdim=True)
        dlogits = -mean * e / torch.where(total > 0, total, torch.ones_like(total))
    part = torch.where(chosen, weights * (dw - mean if renormalize else dw), torch.zeros_like(dw))
    return dlogits.scatter_add(1, ids.clamp(min=0), part).to(st["logits"].dtype)


def _plain_moe(st, group):
    rows = []
    for t in range(st["x"].shape[0]):
        ids = st["ids"][t].to(torch.int64)
        x = st["x"][t].to(torch.float32)
        z = _dequantised(st["gate_up"][ids], st["gate_up_scales"][ids], group) @ x
        g, u = z[:, 0::2], z[:, 1::2]
        h = g / (1 + torch.exp(-g)) * u * st["weights"][t].unsqueeze(1)
        w = _dequantised(st["down"][ids], st["down_scales"][ids], group)
        y = torch.matmul(w, h.unsqueeze(2)).squeeze(2).sum(dim=0)
        rows.append(y if st["residual"] is None else y + st["residual"][t].to(torch.float32))
    return torch.stack(rows).to(torch.float16)


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "topk":
        return _plain_topk(st["logits"], case["topk"], case["renormalize"])
    if op == "topk_bwd":
        return (_plain_topk_backward(st, case["renormalize"]),)
    if op == "moe":
        return (_plain_moe(st, case["group"]),)
    w = _dequantised(st["packed"], st["scales"], case["group"])
    if op == "linear":
        z = st["x"].to(torch.float32) @ w.t()
        if st["bias"] is not None:
            z = z + st["bias"].to(torch.float32)
        y = _act(case["act"], z)
        if st["residual"] is not None:
            y = y + st["residual"].to(torch.float32)
        return (y.to(torch.float16),) if st["pre"] is None else (y.to(torch.float16), z.to(torch.float16))
    dz = st["dy"].to(torch.float32)
    if st["pre"] is not None:
        dz = dz * _act_slope(case["act"], st["pre"].to(torch.float32))
    # the pre-activations' gradient is an fp16 output of its own, and the product's input
    outs = ((dz.to(torch.float16).to(torch.float32) @ w).to(torch.float16),)
    if st["pre"] is not None:
        outs += (dz.to(torch.float16),)
    return outs + (dz.sum(dim=0),) if st["dbias"] is not None else outs


def run(st):
    if not own:
        return _plain(st)
    import w4a16_int4_weight_linear_amd as w4
    case, op = st["case"], st["case"]["op"]
    if op == "topk":
        return w4.moe_topk(st["logits"], case["topk"], renormalize=case["renormalize"])
    if op == "topk_bwd":
        return (w4.moe_topk_backward(st["dweights"], st["logits"], st["ids"], st["weights"], renormalize=case["renormalize"]),)
    if op == "moe":
        return (w4.moe_ffn(st["x"], st["ids"], st["weights"], st["gate_up"], st["gate_up_scales"], st["down"], st["down_scales"],
                           case["group"], residual=st["residual"], out=st["out"]),)
    if op == "linear":
        y = w4.linear(st["x"], st["packed"], st["scales"], case["group"], bias=st["bias"], activation=case["act"],
                      residual=st["residual"], pre=st["pre"], out=st["out"])
        return (y,) if st["pre"] is None else (y, st["pre"])
    dx, dpre, dbias = w4.linear_backward(st["dy"], st["packed"], st["scales"], case["group"], pre=st["pre"],
                                         activation=case["act"], out=st["out"], dpre=st["dpre"], dbias=st["dbias"])
    return tuple(t for t in (dx, dpre, dbias) if t is not None)


def work(case):
    op = case["op"]
    if op in ("topk", "topk_bwd"):
        t, e, k, size = case["tokens"], case["experts"], case["topk"], 2 if case["half"] else 4
        if op == "topk":
            return {"bytes": t * e * size + t * k * 8, "flops": 4 * t * e}
        reads = 0 if case["renormalize"] else t * e * size
        return {"bytes": reads + t * e * size + t * k * 12, "flops": 4 * t * e}
    group = case["group"]
    if op == "moe":
        t, h, i, k, spread = case["tokens"], case["hidden"], case["inter"], case["topk"], case["spread"]
        experts = spread * (1 - (1 - k / spread) ** t)          # that receive a token, on average
        bank = 3 * i * h // 2 + 2 * (2 * i * (h // group) + h * (i // group))
        return {"bytes": int(experts * bank) + t * (2 * h * (3 if case["residual"] else 2) + 8 * k), "flops": 6 * t * k * i * h}
    m, n, k = case["m"], case["n"], case["k"]
    words, scales = n * k // 2, n * (k // group) * 2
    if op == "linear":
        planes = 1 + case["residual"] + case["keep"]
        return {"bytes": words + scales + 2 * m * k + 2 * m * n * planes + 2 * n * case["bias"], "flops": 2 * m * n * k}
    planes = 1 if case["act"] == "none" else 3
    return {"bytes": words + scales + 2 * m * k + 2 * m * n * planes + 4 * n * case["bias"], "flops": 2 * m * n * k}


def _exact_weights(packed, scales, group):
    """The definition: code (u - 8) of nibble i of word j is weight k = 8 j + i, times its group's scale."""
    words = packed.to(torch.int64) & 0xFFFFFFFF
    code = torch.stack([(words // 16 ** i) % 16 for i in range(8)], dim=-1).flatten(-2).double() - 8.0
    shape = code.shape
    return (code.view(*shape[:-1], shape[-1] // group, group) * scales.double().unsqueeze(-1)).view(shape)


def _exact_choice(logits, topk):
    """Rank of each expert among its token's (more, or as many and before it); ids and whether they count."""
    t, e = logits.shape
    ids = torch.empty((t, topk), dtype=torch.int64, device=logits.device)
    before = torch.ones((e, e), dtype=torch.bool, device=logits.device).tril(-1)      # [e, j]: j < e
    for t0 in range(0, t, 512):
        x = logits[t0:t0 + 512]
        more = (x[:, None, :] > x[:, :, None]) | ((x[:, None, :] == x[:, :, None]) & before)
        rank = more.sum(dim=2)
        slots = torch.arange(topk, device=logits.device)
        ids[t0:t0 + 512] = (rank[:, None, :] == slots[None, :, None]).int().argmax(dim=2)
    return ids, torch.gather(logits, 1, ids) != -math.inf


def _exact_slope(name, z):
    if name == "relu":
        return torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
    if name == "silu":
        s = torch.sigmoid(z)
        return s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    u = math.sqrt(2 / math.pi) * (z + GELU_CUBIC * z.pow(3))
    return (1 + torch.tanh(u)) / 2 + z * (1 - torch.tanh(u).square()) / 2 * math.sqrt(2 / math.pi) * (1 + 3 * GELU_CUBIC * z.square())


def _exact_act(name, z):
    if name == "relu":
        return z.clamp(min=0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + GELU_CUBIC * z.pow(3)))) / 2
    return z


def exact(case, seed):
    """The definitions in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "topk":
        x = st["logits"].double()
        ids, counts = _exact_choice(x, case["topk"])
        over = torch.where(counts, torch.gather(x, 1, ids), -math.inf) if case["renormalize"] else x
        norm = torch.logsumexp(over, dim=1, keepdim=True)
        w = torch.exp(torch.gather(x, 1, ids) - norm)
        return ids.masked_fill(~counts, -1).to(torch.int32), w.masked_fill(~counts, 0.0)
    if op == "topk_bwd":
        x, dw = st["logits"].double(), st["dweights"].double()
        ids, w = st["ids"].long(), st["weights"].double()
        of = torch.zeros((x.shape[0], x.shape[1] + 1), dtype=torch.float64, device=x.device)   # last column: no expert
        of.scatter_(1, torch.where(ids < 0, x.shape[1], ids), dw)
        of = of[:, :-1]
        share = torch.zeros_like(of).scatter_(1, ids.clamp(min=0), torch.zeros_like(dw))
        for s in range(ids.shape[1]):
            hit = ids[:, s] >= 0
            share[hit, ids[hit, s]] = w[hit, s]
        mean = (share * of).sum(dim=1, keepdim=True)
        if case["renormalize"]:
            return (share * (of - mean),)
        p = torch.nan_to_num(torch.softmax(x, dim=1), nan=0.0)
        return (share * of - p * mean,)
    if op == "moe":
        y = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
        for e in torch.unique(st["ids"]).tolist():
            t, s = torch.nonzero(st["ids"] == e, as_tuple=True)
            w = _exact_weights(st["gate_up"][e], st["gate_up_scales"][e], case["group"])
            z = torch.mm(st["x"][t].double(), w.t().contiguous()).view(t.shape[0], -1, 2)
            h = torch.sigmoid(z[..., 0]) * z[..., 0] * z[..., 1]
            w = _exact_weights(st["down"][e], st["down_scales"][e], case["group"])
            y.index_add_(0, t, torch.mm(h, w.t().contiguous()) * st["weights"][t, s].double().unsqueeze(1))
        return (y if st["residual"] is None else y + st["residual"].double(),)
    w = _exact_weights(st["packed"], st["scales"], case["group"])
    if op == "linear":
        z = torch.mm(st["x"].double(), w.t().contiguous())
        if case["bias"]:
            z += st["bias"].double()
        y = _exact_act(case["act"], z)
        if case["residual"]:
            y = y + st["residual"].double()
        return (y, z) if case["keep"] else (y,)
    dz = st["dy"].double()
    if case["act"] != "none":
        dz = dz * _exact_slope(case["act"], st["pre"].double())
    outs = (torch.mm(dz.half().double(), w),)
    if case["act"] != "none":
        outs += (dz,)
    return outs + (dz.sum(dim=0),) if case["bias"] else outs
