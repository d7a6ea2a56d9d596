"""The routed experts' feed-forward past 64 (token, slot) pairs, where workgroups sort the pairs into blocks of one
expert: how the ids fall (runs, repeats, one expert, collisions of the table's places, no expert at all), against the
fp64 formula with the bars of the other tests of this call."""

import numpy as np
import pytest

import synth
from gpu_util import dev, host, torch_mod
from test_moe_ffn_gpu import Layer, check, routed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def ids_like(kind, rng, tokens, topk, experts):
    pairs = tokens * topk
    if kind == "one":
        flat = np.full(pairs, experts - 1)
    elif kind == "alternate":
        flat = np.arange(pairs) % 2 * (experts - 1)
    elif kind == "runs":                                    # five of each: blocks of four and of one, across waves
        flat = np.arange(pairs) // 5 % experts
    elif kind == "repeats":                                 # tokens that name an expert several times
        flat = np.repeat(rng.integers(0, experts, pairs // 2 + 1), 2)[:pairs]
    elif kind == "stride":                                  # an expert's pairs 64 apart: one per wave
        flat = np.arange(pairs) % 64 % experts
    else:                                                   # some ids name no expert
        flat = rng.integers(0, experts, pairs)
        flat[rng.random(pairs) < 0.4] = -1
        flat[:2 * topk] = -1                                # two tokens have none
        flat[-1], flat[-2], flat[-3] = experts, 2 ** 31 - 1, -2 ** 31
    return flat.astype(np.int32).reshape(tokens, topk)


@pytest.mark.parametrize("kind", ["one", "alternate", "runs", "repeats", "stride", "missing"])
@pytest.mark.parametrize("tokens,topk", [(13, 5), (64, 8), (9, 40), (47, 3)])
def test_how_ids_fall(w4, tokens, topk, kind):
    layer = Layer(w4, 70, 96, 64, 32, 99000 + tokens)
    ids = ids_like(kind, layer.rng, tokens, topk, 70)
    w = layer.rng.random((tokens, topk)).astype(np.float32)
    if kind == "missing":
        w[0], w[-1, -1] = np.nan, np.inf                    # of slots that name no expert
    check(layer, tokens, topk, ids, w, residual=True)


def test_all_ids_missing(w4):
    layer = Layer(w4, 6, 256, 64, 32, 99100)
    r = synth.activations(layer.rng, 30, 256)
    y = host(layer(dev(synth.activations(layer.rng, 30, 256)), dev(np.full((30, 4), -1, np.int32)),
                   dev(np.full((30, 4), np.nan, np.float32)), residual=dev(r)))
    assert np.array_equal(y, r)


def test_colliding_places(w4):
    """512 different experts, most of which fall on a few places of the table (the upper ten bits of a product)."""
    experts = 40000
    all_ids = np.arange(experts, dtype=np.uint64)
    place = ((all_ids * 0x9E3779B1) & 0xFFFFFFFF) >> 22
    near = all_ids[np.isin(place, np.concatenate([np.arange(1016, 1024), np.arange(0, 4)]))][:440]     # round the end too
    rng = np.random.default_rng(99200)
    rest = rng.choice(np.setdiff1d(all_ids, near), 512 - len(near), replace=False)
    assert len(near) > 300
    ids = rng.permutation(np.concatenate([near, rest]).astype(np.int64)).reshape(64, 8).astype(np.int32)
    layer = Layer(w4, 64, 32, 32, 32, 99201)                # the bank: 64 experts over and over
    torch = torch_mod()
    times = experts // 64
    bank = [t.repeat((times,) + (1,) * (t.dim() - 1)) for t in layer.args]
    x, w = dev(synth.activations(layer.rng, 64, 32)), dev(layer.rng.random((64, 8)).astype(np.float32))
    got = w4.moe_ffn(x, dev(ids), w, *bank, 32)
    want, bar = layer.formula(host(x), ids % 64, host(w))
    assert np.all(np.abs(host(got) - want) <= bar)
    # the lists are in the pairs' order whatever order the places were taken in
    for _ in range(3):
        assert torch.equal(w4.moe_ffn(x, dev(ids), w, *bank, 32), got)


def test_rows_do_not_see_their_neighbours_in_blocks(w4):
    layer = Layer(w4, 4, 576, 160, 32, 99300)
    ids, w = routed(layer.rng, 30, 3, 4)
    x = synth.activations(layer.rng, 30, 576)
    y = host(layer(dev(x), dev(ids), dev(w)))
    bad = x.copy()
    bad[4, 100], bad[17, :] = np.inf, np.nan
    yb = host(layer(dev(bad), dev(ids), dev(w)))
    rest = [t for t in range(30) if t not in (4, 17)]
    assert np.array_equal(yb[rest].view(np.uint16), y[rest].view(np.uint16))
    assert not np.any(np.isfinite(yb[17])) and not np.all(np.isfinite(yb[4]))
    # the same tokens in another batch and order, as many pairs that they are sorted too
    order = layer.rng.permutation(30)[:23]
    again = host(layer(dev(x[order]), dev(ids[order]), dev(w[order])))
    assert np.array_equal(again.view(np.uint16), y[order].view(np.uint16))


# more than one step of h (512) and piece of x (2048), ragged ones; columns that end inside a band; few and many experts
@pytest.mark.parametrize("tokens,topk,experts,hidden,inter,group,spread",
                         [(24, 4, 30, 160, 544, 32, 30), (20, 4, 11, 2176, 1152, 128, 11), (33, 2, 40, 4128, 1600, 32, 40),
                          (64, 8, 9, 32, 2080, 32, 9), (64, 2, 128, 1056, 512, 32, 100), (22, 3, 3, 2048, 1024, 128, 3)])
def test_long_rows_in_blocks(w4, tokens, topk, experts, hidden, inter, group, spread):
    layer = Layer(w4, experts, hidden, inter, group, 99400 + tokens + inter)
    check(layer, tokens, topk, spread=spread, residual=tokens % 2 == 0)
