"""The routed experts' feed-forward for a few tokens against the fp64 formula.

Bar (fixed before the first run), per output: 2^-11 |y| (the one rounding) + the fp32 parts: gate and up sums are
off by at most e = (hidden + 64) 2^-24 sum |x w|; h = SiLU(g) u by 1.1 |u| e_g + |SiLU(g)| e_u + 2^-18 (|h| +
|g u| 2^-6) (exponential, 22 bits between the kernels) + 2^-27; the down sums by (inter + 64) 2^-24 sum |w2 h|, and
each of these is weighted as the output is: sum_s w sum_i |w2| (...).  The slots' sum adds (topk + 2) 2^-23 sum |w y_s|.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


class Layer:
    def __init__(self, w4, experts, hidden, inter, group, seed):
        rng = self.rng = np.random.default_rng(seed)
        self.w4, self.group, self.hidden, self.inter, self.experts = w4, group, hidden, inter, experts
        self.gu = synth.code_bank(rng, experts, 2 * inter, hidden), synth.scale_bank(rng, experts, 2 * inter, hidden // group)
        self.dn = synth.code_bank(rng, experts, hidden, inter), synth.scale_bank(rng, experts, hidden, inter // group)
        pack = lambda b: dev(np.stack([w4.pack(q) for q in b[0]]))  # noqa: E731
        self.args = pack(self.gu), dev(self.gu[1]), pack(self.dn), dev(self.dn[1])

    def __call__(self, x, ids, w, **kw):
        return self.w4.moe_ffn(x, ids, w, *self.args, self.group, **kw)

    def formula(self, x, ids, w, residual=None):
        """(y, bar) in fp64."""
        t, topk = ids.shape
        y = np.zeros((t, self.hidden)) if residual is None else residual.astype(np.float64)
        extra = np.zeros((t, self.hidden))
        part = np.abs(y)
        for e in np.unique(ids):
            if not 0 <= e < self.experts:
                continue
            w1, w2 = (oracle.dequantize(b[0][e], b[1][e], self.group) for b in (self.gu, self.dn))
            at, slot = np.nonzero(ids == e)
            for a, s in zip(at, slot):
                xa = x[a].astype(np.float64)
                z, ez = w1 @ xa, (self.hidden + 64) * 2.0 ** -24 * (np.abs(w1) @ np.abs(xa))
                g, u, eg, eu = z[0::2], z[1::2], ez[0::2], ez[1::2]
                act = g / (1 + np.exp(-g))
                h = act * u
                eh = 1.1 * np.abs(u) * eg + np.abs(act) * eu + 2.0 ** -18 * (np.abs(h) + np.abs(g * u) * 2.0 ** -6) + 2.0 ** -27
                ws = float(w[a, s])
                ys = w2 @ h
                y[a] += ws * ys
                part[a] += np.abs(ws * ys)
                extra[a] += abs(ws) * (np.abs(w2) @ eh + (self.inter + 64) * 2.0 ** -24 * (np.abs(w2) @ np.abs(h)))
        return y, 2.0 ** -11 * np.abs(y) + extra + (topk + 2) * 2.0 ** -23 * part + 2.0 ** -25


def routed(rng, tokens, topk, experts, spread=None):
    used = rng.permutation(experts)[:spread or experts]
    ids = np.stack([rng.choice(used, topk, replace=False) for _ in range(tokens)]).astype(np.int32)
    w = rng.random((tokens, topk)).astype(np.float32)
    return ids, w / w.sum(axis=1, keepdims=True)


def check(layer, tokens, topk, ids=None, w=None, spread=None, residual=False):
    rng = layer.rng
    if ids is None:
        ids, w = routed(rng, tokens, topk, layer.experts, spread)
    x = synth.activations(rng, tokens, layer.hidden)
    r = synth.activations(rng, tokens, layer.hidden) if residual else None
    y = host(layer(dev(x), dev(ids), dev(w), residual=dev(r) if residual else None)).astype(np.float64)
    want, bar = layer.formula(x, ids, w, r)
    bad = np.argwhere(~(np.abs(y - want) <= bar))
    assert bad.size == 0, f"{len(bad)} of {y.size} wrong, first {tuple(bad[0])}: {y[tuple(bad[0])]} want {want[tuple(bad[0])]}"


# (tokens, topk, experts, hidden, inter, group, spread): one token; widths below, at and past a step; odd numbers of
# steps; one expert for all tokens (many passes over its rows); every pair in use
SIZES = [(1, 1, 1, 32, 32, 32, 1), (1, 8, 16, 512, 128, 32, 16), (2, 2, 4, 544, 96, 32, 4), (3, 4, 9, 128, 128, 128, 9),
         (5, 3, 7, 2080, 544, 32, 5), (7, 8, 20, 1408, 384, 128, 9), (13, 4, 60, 640, 1152, 128, 12), (33, 2, 5, 288, 64, 32, 2),
         (64, 8, 24, 256, 160, 32, 24), (64, 1, 3, 96, 608, 32, 1), (10, 8, 8, 4224, 128, 128, 8), (64, 8, 256, 64, 32, 32, 256),
         (8, 64, 70, 96, 64, 32, 70), (31, 5, 40, 1000 // 32 * 32, 96, 32, 30)]


@pytest.mark.parametrize("tokens,topk,experts,hidden,inter,group,spread", SIZES)
def test_sizes(w4, tokens, topk, experts, hidden, inter, group, spread):
    layer = Layer(w4, experts, hidden, inter, group, 91000 + tokens + hidden + inter)
    check(layer, tokens, topk, spread=spread, residual=tokens % 2 == 1)


def test_ids_that_name_no_expert(w4):
    """Slots without an expert contribute nothing, whatever their weight; a token may have none at all."""
    layer = Layer(w4, 6, 256, 64, 32, 92000)
    ids, w = routed(layer.rng, 9, 4, 6)
    ids[0] = -1
    ids[1, 2], ids[2, 0], ids[3, 3] = -1, 6, 2 ** 31 - 1
    w[0], w[1, 2] = np.nan, np.inf
    x = synth.activations(layer.rng, 9, 256)
    y = host(layer(dev(x), dev(ids), dev(w))).astype(np.float64)
    want, bar = layer.formula(x, ids, w)
    assert np.all(np.abs(y - want) <= bar) and np.all(y[0] == 0)
    r = synth.activations(layer.rng, 9, 256)
    y = host(layer(dev(x), dev(np.full((9, 4), -1, np.int32)), dev(w), residual=dev(r)))
    assert np.array_equal(y, r)


def test_an_expert_named_twice(w4):
    layer = Layer(w4, 5, 160, 96, 32, 93000)
    ids, w = routed(layer.rng, 6, 4, 5)
    ids[0] = 3
    ids[2, :2] = ids[2, 2]
    check(layer, 6, 4, ids, w, residual=True)


def test_residual_in_place(w4):
    layer = Layer(w4, 12, 512, 128, 128, 94000)
    ids, w = routed(layer.rng, 20, 4, 12)
    x, r = dev(synth.activations(layer.rng, 20, 512)), dev(synth.activations(layer.rng, 20, 512))
    want = layer(x, dev(ids), dev(w), residual=r).clone()
    got = layer(x, dev(ids), dev(w), residual=r, out=r)
    assert got.data_ptr() == r.data_ptr() and np.array_equal(host(got).view(np.uint16), host(want).view(np.uint16))


def test_rows_do_not_see_their_neighbours(w4):
    """A token that is not finite leaves the others' bits as they are, and a token's result does not depend on its batch."""
    layer = Layer(w4, 4, 576, 160, 32, 95000)
    ids, w = routed(layer.rng, 11, 3, 4)
    x = synth.activations(layer.rng, 11, 576)
    y = host(layer(dev(x), dev(ids), dev(w)))
    bad = x.copy()
    bad[4, 100], bad[7, :] = np.inf, np.nan
    yb = host(layer(dev(bad), dev(ids), dev(w)))
    rest = [t for t in range(11) if t not in (4, 7)]
    assert np.array_equal(yb[rest].view(np.uint16), y[rest].view(np.uint16))
    assert not np.any(np.isfinite(yb[7])) and not np.all(np.isfinite(yb[4]))
    for t in range(11):
        one = host(layer(dev(x[t:t + 1]), dev(ids[t:t + 1]), dev(w[t:t + 1])))
        assert np.array_equal(one[0].view(np.uint16), y[t].view(np.uint16)), t


def test_large_gate_products(w4):
    """SiLU(g) u past fp16's range is kept between the kernels (here up to about 10^6)."""
    layer = Layer(w4, 2, 128, 64, 32, 96000)
    ids, w = routed(layer.rng, 5, 2, 2)
    x = (synth.activations(layer.rng, 5, 128) * np.float16(3000)).astype(np.float16)
    y = host(layer(dev(x), dev(ids), dev(w))).astype(np.float64)
    want, bar = layer.formula(x, ids, w)
    inside = np.abs(want) < 60000
    assert inside.sum() > 100 and np.all(np.abs(y - want)[inside] <= bar[inside])


def test_rows_behind_the_last_token_stay(w4):
    torch = torch_mod()
    layer = Layer(w4, 8, 544, 64, 32, 97000)
    ids, w = routed(layer.rng, 7, 4, 8)
    out = torch.full((16, 544), 7.0, dtype=torch.float16, device="cuda")
    layer(dev(synth.activations(layer.rng, 7, 544)), dev(ids), dev(w), out=out[4:11])
    assert bool((out[:4] == 7).all()) and bool((out[11:] == 7).all()) and not bool((out[4:11] == 7).all())


def test_a_bank_past_two_gigabytes(w4):
    """Experts behind 2^31 bytes of packed weights (and 2^32: 5 GB)."""
    torch = torch_mod()
    experts, hidden, inter, group = 1200, 2048, 2048, 128       # 4.2 MB an expert's gate/up, 2.1 its down
    gu = torch.randint(-2 ** 31, 2 ** 31, (experts, 2 * inter, hidden // 8), dtype=torch.int32, device="cuda")
    dn = torch.randint(-2 ** 31, 2 ** 31, (experts, hidden, inter // 8), dtype=torch.int32, device="cuda")
    gs = torch.full((experts, 2 * inter, hidden // group), 0.002, dtype=torch.float16, device="cuda")
    ds = torch.full((experts, hidden, inter // group), 0.002, dtype=torch.float16, device="cuda")
    x = torch.randn(2, hidden, device="cuda").to(torch.float16)
    ids = torch.tensor([[3, 700], [1100, 1199]], dtype=torch.int32, device="cuda")
    w = torch.full((2, 2), 0.5, device="cuda")
    y = w4.moe_ffn(x, ids, w, gu, gs, dn, ds, group)
    used = ids.flatten().long()
    small = w4.moe_ffn(x, torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda"), w, gu[used].contiguous(),
                       gs[used].contiguous(), dn[used].contiguous(), ds[used].contiguous(), group)
    assert torch.equal(y.view(torch.int16), small.view(torch.int16)) and bool(y.isfinite().all())
