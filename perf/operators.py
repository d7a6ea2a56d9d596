"""The feed-forward block's training operators on int4 weights: what is timed, and on what.

Four operators of the W4A16 layer (int4 codes q in [-8, 7], eight offset-binary
nibbles per 32-bit word along K, one fp16 scale per group of 128 or 32 input
features; fp16 activations and gradients):

  swiglu      h = SiLU(g) * u with (g, u) = x . deq(W)^T interleaved, for any number of rows;
              in training the fp16 (g, u) pairs are kept for the backward pass
  swiglu_bwd  (dg, du) from dh and the kept pairs, then dx = (dg, du) . deq(W)
  t           y = d . deq(W): the product with the weights' other side (the input
              gradient of every linear layer), from one row to a whole prompt
  dscales     ds[n, group] = sum over the group of q * (d^T . x): the gradient of the scales

Where `own` is false, run() computes them in their plain form: elementary torch
operations in 32 bits, rounded once at the end.
"""

import torch

own = False

# The dense feed-forward's hidden and intermediate widths, and the MoE expert's.
HIDDEN, INTER = 5120, 17408
EXPERT_HIDDEN, EXPERT_INTER = 2048, 512


def listed():
    return [
        # a few tokens through one expert-sized block: launch latency counts
        {"name": "swiglu_17_512_2048", "op": "swiglu", "m": 17, "n": EXPERT_INTER, "k": EXPERT_HIDDEN, "group": 32, "keep": True},
        # one training micro-batch through the dense gate/up pair, keeping (g, u)
        {"name": "swiglu_512_dense", "op": "swiglu", "m": 512, "n": INTER, "k": HIDDEN, "group": 128, "keep": True},
        # prefill of a long prompt: nothing kept
        {"name": "swiglu_4096_dense", "op": "swiglu", "m": 4096, "n": INTER, "k": HIDDEN, "group": 128, "keep": False},
        # input gradient of a single token (a sensitivity, the last token of a prefix), small and full size
        {"name": "t_1_1024_1024", "op": "t", "m": 1, "n": 1024, "k": 1024, "group": 128},
        {"name": "t_1_up", "op": "t", "m": 1, "n": INTER, "k": HIDDEN, "group": 128},
        # a handful of rows through the down projection
        {"name": "t_16_down", "op": "t", "m": 16, "n": HIDDEN, "k": INTER, "group": 128},
        # ragged batch, odd number of weight rows, small groups
        {"name": "t_300_2003_2080", "op": "t", "m": 300, "n": 2003, "k": 2080, "group": 32},
        # input gradient of a whole training batch
        {"name": "t_4096_up", "op": "t", "m": 4096, "n": INTER, "k": HIDDEN, "group": 128},
        # the block's backward: a few rows, and a training batch
        {"name": "swiglu_bwd_19_512_2048", "op": "swiglu_bwd", "m": 19, "n": EXPERT_INTER, "k": EXPERT_HIDDEN, "group": 32},
        {"name": "swiglu_bwd_2048_dense", "op": "swiglu_bwd", "m": 2048, "n": INTER, "k": HIDDEN, "group": 128},
        # learned scales: a ragged small layer, and the dense up projection
        {"name": "dscales_133_1001_1120", "op": "dscales", "m": 133, "n": 1001, "k": 1120, "group": 32},
        {"name": "dscales_2048_up", "op": "dscales", "m": 2048, "n": INTER, "k": HIDDEN, "group": 128},
    ]


def _log(rng, lo, hi):
    """An integer spread evenly over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["swiglu", "swiglu_bwd", "t", "t", "dscales"])
    group = rng.choice([32, 128])
    top = {"swiglu": 4096, "swiglu_bwd": 2048, "t": 4096, "dscales": 2048}[op]
    case = {"op": op, "m": _log(rng, 1, top), "n": _log(rng, 9, INTER), "k": group * _log(rng, 1, HIDDEN // group), "group": group}
    if op == "t" and rng.random() < 0.5:            # the down projection's orientation
        case["n"], case["k"] = _log(rng, 9, HIDDEN), group * _log(rng, 1, INTER // group)
    if op == "swiglu":
        case["keep"] = rng.random() < 0.5
    return case


def _rows(case):
    """Weight rows: the gate/up pair has two per output."""
    return case["n"] * (2 if case["op"].startswith("swiglu") else 1)


def _normal(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(torch.float16)


def _weights(gen, rows, k, group):
    """Gaussian weights quantised symmetrically: (int32 words [rows, k/8], fp16 scales [rows, k/group])."""
    w = (torch.randn((rows, k // group, group), generator=gen, device="cuda") * 0.02)
    s = (w.abs().amax(dim=2) / 7).to(torch.float16)
    q = (w / s.float().unsqueeze(2)).round().clamp(-8, 7).to(torch.int32).reshape(rows, k // 8, 8) + 8
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    return (q << shift).sum(dim=2, dtype=torch.int64).to(torch.int32), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    m, n, k, group, op = case["m"], case["n"], case["k"], case["group"], case["op"]
    packed, scales = _weights(gen, _rows(case), k, group)
    st = {"op": op, "group": group, "packed": packed, "scales": scales}
    half = dict(dtype=torch.float16, device="cuda")
    if op == "swiglu":
        st["x"] = _normal(gen, m, k)
        st["out"] = torch.empty((m, n), **half)
        st["gate_up"] = torch.empty((m, 2 * n), **half) if case["keep"] else None
    elif op == "swiglu_bwd":
        # preactivations of the size N(0, 1) inputs give, and loss-scaled gradients
        st["gate_up"] = _normal(gen, m, 2 * n, std=0.02 * k ** 0.5)
        st["dy"] = _normal(gen, m, n, std=0.05)
        st["out"], st["dgate_up"] = torch.empty((m, k), **half), torch.empty((m, 2 * n), **half)
    elif op == "t":
        st["dy"] = _normal(gen, m, n, std=0.05)
        st["out"] = torch.empty((m, k), **half)
    else:
        st["dy"] = _normal(gen, m, n, std=0.05)
        st["x"] = _normal(gen, m, k)
        st["out"] = torch.empty((n, k // group), dtype=torch.float32, device="cuda")
    return st


def _codes(packed):
    """int32 words [n, k/8] -> codes [n, k] as fp32."""
    shift = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    return ((packed.unsqueeze(2) >> shift) & 15).sub(8).to(torch.float32).reshape(packed.shape[0], -1)


def _dequantised(st):
    return _codes(st["packed"]) * st["scales"].to(torch.float32).repeat_interleave(st["group"], dim=1)


def _plain(st):
    op = st["op"]
    if op == "swiglu":
        z = st["x"].to(torch.float32) @ _dequantised(st).t()
        g, u = z[:, 0::2], z[:, 1::2]
        h = (g / (1 + torch.exp(-g)) * u).to(torch.float16)
        return (h,) if st["gate_up"] is None else (h, z.to(torch.float16))
    if op == "swiglu_bwd":
        z, dh = st["gate_up"].to(torch.float32), st["dy"].to(torch.float32)
        g, u = z[:, 0::2], z[:, 1::2]
        sig = 1 / (1 + torch.exp(-g))
        dz = torch.stack((dh * u * sig * (1 + g * (1 - sig)), dh * g * sig), dim=2).reshape(z.shape).to(torch.float16)
        # the pairs' gradient is an fp16 output of its own, and the product's input
        return (dz.to(torch.float32) @ _dequantised(st)).to(torch.float16), dz
    if op == "t":
        return ((st["dy"].to(torch.float32) @ _dequantised(st)).to(torch.float16),)
    dw = st["dy"].to(torch.float32).t() @ st["x"].to(torch.float32)
    return ((dw * _codes(st["packed"])).reshape(dw.shape[0], -1, st["group"]).sum(dim=2),)


def run(st):
    if not own:
        return _plain(st)
    import w4a16_int4_weight_linear_amd as w4
    op = st["op"]
    if op == "swiglu":
        h = w4.gemm_swiglu(st["x"], st["packed"], st["scales"], st["group"], gate_up=st["gate_up"], out=st["out"])
        return (h,) if st["gate_up"] is None else (h, st["gate_up"])
    if op == "swiglu_bwd":
        return w4.gemm_swiglu_backward(st["dy"], st["gate_up"], st["packed"], st["scales"], st["group"], out=st["out"],
                                       dgate_up=st["dgate_up"])
    if op == "t":
        return (w4.gemm_t(st["dy"], st["packed"], st["scales"], st["group"], out=st["out"]),)
    return (w4.gemm_dscales(st["dy"], st["x"], st["packed"], st["group"], out=st["out"]),)


def work(case):
    m, n, k, rows = case["m"], case["n"], case["k"], _rows(case)
    words, scales, product = rows * k // 2, rows * (k // case["group"]) * 2, 2 * m * rows * k
    if case["op"] == "swiglu":
        return {"bytes": words + scales + 2 * m * k + 2 * m * n * (3 if case["keep"] else 1), "flops": product}
    if case["op"] == "swiglu_bwd":
        return {"bytes": words + scales + 2 * m * k + 2 * m * n * 5, "flops": product}
    if case["op"] == "t":
        return {"bytes": words + scales + 2 * m * n + 2 * m * k, "flops": product}
    return {"bytes": words + 2 * scales + 2 * m * n + 2 * m * k, "flops": product}


def exact(case, seed):
    """The definitions in fp64: code (u - 8) of nibble i of word j is weight k = 8 j + i."""
    st = prepare(case, seed)
    words = st["packed"].to(torch.int64) & 0xFFFFFFFF
    code = torch.stack([(words // 16 ** i) % 16 for i in range(8)], dim=2).flatten(1).double() - 8.0
    n, k = code.shape
    group, op = st["group"], st["op"]
    if op == "dscales":
        grad = torch.mm(st["dy"].double().t().contiguous(), st["x"].double())
        return (torch.mul(code, grad).view(n, k // group, group).sum(2),)
    w = (code.view(n, k // group, group) * st["scales"].double()[:, :, None]).view(n, k)
    del code, words
    if op == "swiglu":
        z = torch.mm(st["x"].double(), w.t().contiguous())
        pair = z.view(z.shape[0], -1, 2)
        h = torch.sigmoid(pair[..., 0]) * pair[..., 0] * pair[..., 1]
        return (h,) if not case["keep"] else (h, z)
    if op == "swiglu_bwd":
        pair = st["gate_up"].double().view(st["gate_up"].shape[0], -1, 2)
        g, u, dh = pair[..., 0], pair[..., 1], st["dy"].double()
        s = torch.sigmoid(g)
        dz = torch.empty_like(pair)
        dz[..., 0] = dh * u * (s + g * s * torch.sigmoid(-g))
        dz[..., 1] = dh * s * g
        dz = dz.flatten(1)
        return torch.mm(dz.half().double(), w), dz
    return (torch.mm(st["dy"].double(), w),)
