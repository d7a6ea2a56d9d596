"""The router's choice and its gradient over many tokens (sixteen lanes of a wave per token), with the bars of few
tokens' tests: every number of values per lane, odd rows, ties, masks, and more slots than such a kernel takes."""

import numpy as np
import pytest

from gpu_util import dev, host, torch_mod
from test_moe_topk_gpu import check_choice

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


# (tokens, experts, topk): either side of the number of tokens where the kernel changes; one, two and four runs of four
# experts per lane, whole and ragged; 17 slots stay on whole waves
SIZES = [(2047, 256, 8), (2048, 256, 8), (2049, 256, 8), (2050, 64, 4), (2051, 37, 16), (2052, 128, 1), (2053, 101, 6),
         (2054, 200, 10), (2055, 255, 16), (2056, 256, 17), (2060, 300, 8), (5000, 1, 1), (2100, 129, 3)]


def logits(tokens, experts, dtype):
    rng = np.random.default_rng(86000 + tokens + experts)
    x = (rng.standard_normal((tokens, experts)) * 2).astype(dtype)
    if experts > 2:
        x[rng.random(x.shape) < 0.2] = -np.inf
        x[0] = -np.inf                                  # nothing left
        x[-1] = -np.inf
        x[-1, experts // 2] = np.finfo(dtype).min       # the lowest finite value alone
        x[1] = rng.integers(-1, 2, experts)             # ties
    return rng, x


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("tokens,experts,topk", SIZES)
def test_choice_of_many_tokens(w4, tokens, experts, topk, dtype, renormalize):
    _, x = logits(tokens, experts, dtype)
    check_choice(w4, x, topk, renormalize)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("tokens,experts,topk", SIZES)
def test_gradient_of_many_tokens(w4, tokens, experts, topk, dtype, renormalize):
    rng, x = logits(tokens, experts, dtype)
    dw = rng.standard_normal((tokens, topk)).astype(np.float32)
    xd = dev(x)
    ids, w = w4.moe_topk(xd, topk, renormalize=renormalize)
    got = host(w4.moe_topk_backward(dev(dw), xd, ids, w, renormalize=renormalize)).astype(np.float64)
    ids, w = host(ids), host(w).astype(np.float64)
    chosen, at = ids >= 0, (np.arange(tokens)[:, None], np.maximum(ids, 0))
    wd = np.where(chosen, w * dw, 0)
    mean, total = wd.sum(axis=1, keepdims=True), np.abs(wd).sum(axis=1, keepdims=True)
    want, size = np.zeros((tokens, experts)), np.zeros((tokens, experts))
    if not renormalize:
        l = x.astype(np.float64)
        peak = np.where(np.isneginf(l.max(axis=1)), 0, l.max(axis=1))[:, None]
        p = np.exp(l - peak)
        p /= np.maximum(p.sum(axis=1, keepdims=True), 1e-300)
        want, size = -p * mean, p * total * (1 + np.where(np.isneginf(l), 0, peak - l))
    # (a token's experts differ: no two slots add to one place; slots without an expert add zeros)
    np.add.at(want, at, np.where(chosen, w * (dw - mean) if renormalize else wd, 0))
    np.add.at(size, at, np.where(chosen, w * (np.abs(dw) + total), 0))
    eps, tiny = (2.0 ** -11, 2.0 ** -25) if dtype == np.float16 else (2.0 ** -23, 2.0 ** -140)
    assert np.all(np.abs(got - want) <= eps * np.abs(want) + (experts + topk + 32) * 2.0 ** -23 * size + tiny)
    assert np.all(got[np.isneginf(x)] == 0)


def test_many_tokens_leave_what_is_behind_them(w4):
    torch = torch_mod()
    t, e, k = 2051, 130, 5
    x = torch.randn(t, e, device="cuda")
    ids = torch.full((t + 40, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((t + 40, k), 7.0, device="cuda")
    out = torch.full((t + 40, e), 7.0, device="cuda")
    w4.moe_topk(x, k, ids=ids[:t], weights=w[:t])
    w4.moe_topk_backward(torch.randn(t, k, device="cuda"), x, ids[:t], w[:t], renormalize=False, out=out[:t])
    assert bool((ids[t:] == 77).all()) and bool((w[t:] == 7).all()) and bool((out[t:] == 7).all())
    # ids are exact whichever kernel chose them
    assert torch.equal(w4.moe_topk(x[:100].contiguous(), k)[0], ids[:100])
