"""The router's choice and its gradient against plain fp64 code.

Bars (fixed before the first run).  ids: equal to a stable sort's (largest first, equal ones by expert), -1 where
only masked experts are left.  weights: fp32 with l - max rounded once (2^-24 |l - max|), an exponential within
four half steps, sums of up to E terms: relative error <= (E + 16) 2^-24 + 2^-23 |l - max|.  dlogits: a few fp32
operations on w, dw, p and a sum of topk products, |err| <= eps |v| + (E + topk + 32) 2^-23 (w |dw| + p sum |w dw|
(1 + |l - max|)) + tiny, with eps 2^-11 (fp16) or 2^-23 (fp32) for the one rounding and tiny half the smallest subnormal.
"""

import numpy as np
import pytest

from gpu_util import dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def choice(x, topk):
    """ids [t, topk] (-1: none left) of logits without NaN."""
    ids = np.argsort(-x.astype(np.float64), axis=1, kind="stable")[:, :topk]
    return np.where(np.isneginf(np.take_along_axis(x, ids, 1)), -1, ids)


def softmax_weights(x, ids, renormalize):
    """(weights, |l - max| of the chosen) in fp64."""
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        peak = np.where(np.isneginf(x.max(axis=1)), 0, x.max(axis=1))[:, None]
        e = np.exp(x - peak)
    top = np.where(ids >= 0, np.take_along_axis(e, np.maximum(ids, 0), 1), 0)
    total = (top if renormalize else e).sum(axis=1, keepdims=True)
    far = np.where(ids >= 0, peak - np.take_along_axis(x, np.maximum(ids, 0), 1), 0)
    return top / np.where(total > 0, total, 1), far


def check_choice(w4, x, topk, renormalize):
    ids, w = (host(t) for t in w4.moe_topk(dev(x), topk, renormalize=renormalize))
    want = choice(x, topk)
    assert np.array_equal(ids, want), f"first at {np.argwhere(ids != want)[0]}"
    ww, far = softmax_weights(x, want, renormalize)
    assert w.dtype == np.float32 and np.all(w[want < 0] == 0)
    assert np.all(np.abs(w - ww) <= ((x.shape[1] + 16) * 2.0 ** -24 + 2.0 ** -23 * far) * ww + 2.0 ** -149)
    return ids, w


# (tokens, experts, topk): one token, single experts, rows of every alignment, every number of lanes and values
SIZES = [(1, 1, 1), (1, 256, 8), (5, 3, 3), (17, 64, 6), (33, 65, 16), (100, 127, 1), (9, 160, 10), (1000, 256, 8), (3, 255, 17),
         (70, 256, 64), (12, 257, 8), (4, 512, 2), (130, 511, 33), (2, 1024, 64), (21, 1001, 5), (4099, 4, 2)]


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("tokens,experts,topk", SIZES)
def test_choice(w4, tokens, experts, topk, dtype, renormalize):
    rng = np.random.default_rng(81000 + tokens + experts)
    check_choice(w4, (rng.standard_normal((tokens, experts)) * 3).astype(dtype), topk, renormalize)


@pytest.mark.parametrize("experts,topk", [(8, 4), (200, 10), (256, 40), (1000, 20)])
def test_ties_go_to_the_lowest_expert(w4, experts, topk):
    rng = np.random.default_rng(82000 + experts)
    x = rng.integers(-2, 3, (60, experts)).astype(np.float32)
    x[0] = 0
    x[1] = np.where(np.arange(experts) % 2, 0.0, -0.0)        # the two zeros are equal
    x[2] = -1e30
    check_choice(w4, x, topk, True)
    check_choice(w4, x.astype(np.float16).clip(-60000, 60000), topk, False)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("experts,topk", [(6, 6), (100, 8), (256, 8), (700, 30)])
def test_masked_experts(w4, experts, topk, renormalize):
    """-inf is never chosen: fewer experts than slots, one, none at all; and the lowest finite values are."""
    rng = np.random.default_rng(83000 + experts)
    x = (rng.standard_normal((64, experts)) * 2).astype(np.float32)
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[3] = -np.inf
    x[4] = -np.inf
    x[4, experts - 1] = -5
    x[5] = -np.inf
    x[5, ::2] = np.finfo(np.float32).min
    x[6] = np.finfo(np.float32).min
    ids, w = check_choice(w4, x, topk, renormalize)
    assert np.all(ids[3] == -1) and np.all(w[3] == 0)
    assert ids[4, 0] == experts - 1 and w[4, 0] == 1 and np.all(ids[4, 1:] == -1)


def test_not_finite_logits(w4):
    x = np.zeros((4, 32), np.float32)
    x[0, 7], x[0, 3] = np.nan, 5
    x[1, 9] = np.inf
    x[2, 1] = 2
    for renormalize in (True, False):
        ids, w = (host(t) for t in w4.moe_topk(dev(x), 4, renormalize=renormalize))
        assert list(ids[0][:2]) == [7, 3] and ids[1][0] == 9 and ids[2][0] == 1
        assert np.all(np.isnan(w[:2])) and np.all(np.isfinite(w[2:]))


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("tokens,experts,topk", [s for s in SIZES if s[0] < 1000])
def test_backward(w4, tokens, experts, topk, dtype, renormalize):
    rng = np.random.default_rng(84000 + tokens + experts)
    x = (rng.standard_normal((tokens, experts)) * 2).astype(dtype)
    if experts > 2:
        x[rng.random(x.shape) < 0.2] = -np.inf
        x[0] = -np.inf
    dw = rng.standard_normal((tokens, topk)).astype(np.float32)
    xd = dev(x)
    ids, w = w4.moe_topk(xd, topk, renormalize=renormalize)
    got = w4.moe_topk_backward(dev(dw), xd, ids, w, renormalize=renormalize)
    assert got.dtype == xd.dtype
    got, ids, w = host(got).astype(np.float64), host(ids), host(w).astype(np.float64)
    want, size = np.zeros((tokens, experts)), np.zeros((tokens, experts))
    for t in range(tokens):
        ok = ids[t] >= 0
        mean, total = np.sum(w[t, ok] * dw[t, ok]), np.sum(np.abs(w[t, ok] * dw[t, ok]))
        if not renormalize and ok.any():
            l = x[t].astype(np.float64)
            p = np.exp(l - l.max())
            p /= p.sum()
            far = np.where(np.isneginf(l), 0, l.max() - l)
            want[t], size[t] = -p * mean, p * total * (1 + far)
        for e, ws, d in zip(ids[t][ok], w[t][ok], dw[t][ok]):
            want[t, e] += ws * (d - mean) if renormalize else ws * d
            size[t, e] += ws * (abs(d) + total)
    eps, tiny = (2.0 ** -11, 2.0 ** -25) if dtype == np.float16 else (2.0 ** -23, 2.0 ** -140)
    assert np.all(np.abs(got - want) <= eps * np.abs(want) + (experts + topk + 32) * 2.0 ** -23 * size + tiny)
    assert np.all(got[np.isneginf(x)] == 0)


def test_backward_against_differences(w4):
    """Central differences of sum(weights dw) in fp64, the choice held."""
    rng = np.random.default_rng(85000)
    t, e, k = 6, 40, 5
    x = rng.standard_normal((t, e)).astype(np.float32)
    dw = rng.standard_normal((t, k)).astype(np.float32)
    for renormalize in (True, False):
        ids, w = w4.moe_topk(dev(x), k, renormalize=renormalize)
        got = host(w4.moe_topk_backward(dev(dw), dev(x), ids, w, renormalize=renormalize))
        at, step = host(ids), 1e-5
        for j in range(e):
            d = np.zeros(e); d[j] = step
            up = softmax_weights(x.astype(np.float64) + d, at, renormalize)[0]
            dn = softmax_weights(x.astype(np.float64) - d, at, renormalize)[0]
            diff = np.sum((up - dn) * dw, axis=1) / (2 * step)
            assert np.all(np.abs(got[:, j] - diff) <= 1e-5)   # step^2 and 2^-23 (E + 32) of sums of at most 5 |dw|


def test_ids_that_name_no_expert(w4):
    """Given ids outside the experts count for nothing and nothing is written for them."""
    x = dev(np.zeros((3, 20), np.float32))
    ids = dev(np.array([[-1, 4], [20, 2 ** 31 - 1], [-2 ** 31, 19]], np.int32))
    w, dw = dev(np.full((3, 2), 0.5, np.float32)), dev(np.array([[9, 1], [1, 2], [3, 1]], np.float32))
    got = host(w4.moe_topk_backward(dw, x, ids, w))
    want = np.zeros((3, 20), np.float32)
    want[0, 4] = want[2, 19] = 0.25
    assert np.array_equal(got, want)


def test_rows_behind_the_last_token_stay(w4):
    torch = torch_mod()
    x = torch.randn(37, 96, device="cuda")
    ids = torch.full((40, 4), 77, dtype=torch.int32, device="cuda")
    w = torch.full((40, 4), 7.0, device="cuda")
    out = torch.full((40, 96), 7.0, device="cuda")
    w4.moe_topk(x, 4, ids=ids[:37], weights=w[:37])
    w4.moe_topk_backward(torch.randn(37, 4, device="cuda"), x, ids[:37], w[:37], renormalize=False, out=out[:37])
    assert bool((ids[37:] == 77).all()) and bool((w[37:] == 7).all()) and bool((out[37:] == 7).all())
