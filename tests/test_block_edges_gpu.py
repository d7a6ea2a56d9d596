"""The edges of the linear layer's, the router's and the few-token experts' calls, on the device."""

import numpy as np
import pytest

from gpu_util import dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def test_the_most_tokens_of_a_router(w4):
    """2^26 - 1 tokens with a wave each (17 slots): past 2^32 threads, so two rows of workgroups.  Choice and gradient of every token of
    a repeating batch; a permutation of all experts each, so their sum says that every row was written."""
    torch = torch_mod()
    tokens, experts, few = (1 << 26) - 1, 17, 8191
    rng = np.random.default_rng(87000)
    some = torch.from_numpy(rng.standard_normal((few, experts)).astype(np.float16)).cuda()
    logits = torch.empty((tokens, experts), dtype=torch.float16, device="cuda")
    for a in range(0, tokens, few * 1024):
        b = min(a + few * 1024, tokens)
        logits[a:b] = some.repeat(1024, 1)[:b - a]
    ids = torch.full((tokens, experts), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((tokens, experts), -7.0, device="cuda")
    want_ids, want_w = w4.moe_topk(some, experts)
    w4.moe_topk(logits, experts, ids=ids, weights=weights)
    dw = torch.from_numpy(rng.standard_normal((few, experts)).astype(np.float32)).cuda()
    want_d = w4.moe_topk_backward(dw, some, want_ids, want_w)
    for a in range(0, tokens, few * 1024):
        b = min(a + few * 1024, tokens)
        assert torch.equal(ids[a:b], want_ids.repeat(1024, 1)[:b - a]), a
        assert torch.equal(weights[a:b], want_w.repeat(1024, 1)[:b - a]), a
    dws = torch.empty_like(weights)
    for a in range(0, tokens, few * 1024):
        b = min(a + few * 1024, tokens)
        dws[a:b] = dw.repeat(1024, 1)[:b - a]
    w4.moe_topk_backward(dws, logits, ids, weights, out=logits.fill_(7))
    for a in range(0, tokens, few * 1024):
        b = min(a + few * 1024, tokens)
        assert torch.equal(logits[a:b], want_d.repeat(1024, 1)[:b - a]), a


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens", [500, 4096])
def test_equal_logits_have_equal_weights(w4, tokens, renormalize):
    """A token's slots are divided by one total, whichever lane holds them (six equal logits lie in lanes of different fours)."""
    rng = np.random.default_rng(87100)
    x = np.repeat(rng.standard_normal((tokens, 20)).astype(np.float32), 6, axis=1)
    ids, w = (host(t) for t in w4.moe_topk(dev(x), 16, renormalize=renormalize))
    picked = np.take_along_axis(x, ids, 1)
    same = picked[:, 1:] == picked[:, :-1]
    assert same.sum() >= 13 * tokens and np.array_equal(w[:, 1:][same], w[:, :-1][same])


def graph_nodes(w4, graph):
    """How many nodes a captured graph has."""
    import ctypes
    get, count = w4.lib.hipGraphGetNodes, ctypes.c_size_t(0)       # (of the runtime that the library is linked with)
    get.restype, get.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
    assert get(graph.raw_cuda_graph(), None, ctypes.byref(count)) == 0
    return count.value


@pytest.mark.parametrize("call,kernels", [("experts of one token", 2), ("experts of 40 tokens", 3), ("split tiles", 2)])
def test_a_captured_call_is_its_kernels(w4, call, kernels):
    """No fill of counters that a call does not use in front of it; replays give the eager result."""
    torch = torch_mod()
    from test_moe_ffn_gpu import Layer
    rng = np.random.default_rng(87200)
    if call == "split tiles":
        p = torch.randint(-2 ** 31, 2 ** 31 - 1, (520, 256), dtype=torch.int32, device="cuda")
        s, x = torch.rand(520, 16, device="cuda").half() * 0.01, torch.randn(300, 2048, device="cuda").half()
        assert w4.ffn_workspace("linear", 300, 520, 2048, 128) is not None
        step = lambda: w4.linear(x, p, s, 128, activation="silu")  # noqa: E731
    else:
        tokens = 1 if "one" in call else 40
        layer = Layer(w4, 9, 256, 128, 32, 87201)
        x, ids = dev(rng.standard_normal((tokens, 256)).astype(np.float16)), dev(rng.integers(0, 9, (tokens, 3)).astype(np.int32))
        w = dev(rng.random((tokens, 3)).astype(np.float32))
        step = lambda: layer(x, ids, w)  # noqa: E731
    want = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        out = step()
    assert graph_nodes(w4, graph) == kernels
    graph.instantiate()
    for _ in range(3):
        out.fill_(float("nan"))
        torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k,group", [(1, 40, 64, 32), (21, 131, 64, 32), (30, 3001, 2560, 32), (70, 264, 128, 128), (70, 33, 64, 32)])
def test_gradient_of_pre_activations_past_fp16(w4, m, n, k, group, act):
    """A pre-activation past 65504 is kept as infinity: y is finite (0 at that end), or infinite as fp16 has it, and the
    gradient is dy times 0 or 1, not NaN; in the product, in front of it, on odd rows and tiles."""
    torch = torch_mod()
    from test_linear_gpu import weights
    rng = np.random.default_rng(87300 + m + n)
    q, s = weights(rng, n, k, group)
    # through the call itself: codes of 7, scales of 16 and x of +-1000 give z = +-7 16 1000 k
    x = np.full((m, k), 1000, np.float16)
    x[::2] = -1000
    pre = torch.empty((m, n), dtype=torch.float16, device="cuda")
    big = dev(w4.pack(np.full((n, k), 7, np.int8))), dev(np.full((n, k // group), 16, np.float16))
    y = host(w4.linear(dev(x), *big, group, activation=act, pre=pre))
    z = host(pre)
    assert np.all(np.isneginf(z[::2])) and np.all(np.isposinf(z[1::2])) and np.all(np.abs(y[::2]) == 0) and np.all(np.isposinf(y[1::2]))
    z[:, ::3] = rng.standard_normal(z[:, ::3].shape)
    z[m - 1, n - 1] = np.nan
    dy = rng.standard_normal((m, n)).astype(np.float16)
    dx, dpre, dbias = (host(t) for t in w4.linear_backward(dev(dy), dev(w4.pack(q)), dev(s), group, pre=dev(z), activation=act, dbias=True))
    assert np.array_equal(dpre[np.isneginf(z)], 0 * dy[np.isneginf(z)]) and np.array_equal(dpre[np.isposinf(z)], dy[np.isposinf(z)])
    rest = ~np.isnan(z)
    assert np.all(np.isfinite(dpre[rest])) and np.isnan(dpre[m - 1, n - 1])
    assert np.all(np.isfinite(dx[:m - 1])) and np.all(np.isfinite(dbias[:n - 1])) and np.isnan(dbias[n - 1])


# decode kernels, weight-streaming kernel (scales that come in one load and that do not), tiles where weights are exact
@pytest.mark.parametrize("m,k,group", [(1, 416, 32), (1, 640, 128), (3, 416, 32), (4, 512, 128), (5, 416, 32), (9, 512, 32), (16, 640, 128),
                                       (16, 512, 128), (17, 416, 32), (32, 512, 32), (32, 640, 128), (40, 512, 128), (70, 640, 128)])
def test_linear_has_exact_weights(w4, m, k, group):
    """Each output is the difference of two weights that nearly cancel, 2048 (s1 q1 - s2 q2): exact in fp32, and far off if a
    weight was rounded to fp16."""
    torch = torch_mod()
    rng = np.random.default_rng(87400 + m + k)
    n = 131
    q = rng.integers(5, 8, (n, 1)).astype(np.int8) * np.ones((1, k), np.int8) * rng.choice([-1, 1], (n, 1)).astype(np.int8)
    # scales in 1..2 (ulp 2^-10), neighbours up to three ulps apart
    s = (1 + (rng.integers(0, 1000, (n, 1)) + rng.integers(0, 4, (n, k // group))) / 1024).astype(np.float16)
    x = np.zeros((m, k), np.float16)
    for r in range(m):
        a, b = rng.choice(k // group, 2, replace=False) * group + rng.integers(0, group, 2)
        x[r, a], x[r, b] = 2048, -2048
    pre = torch.empty((m, n), dtype=torch.float16, device="cuda")
    y = host(w4.linear(dev(x), dev(w4.pack(q)), dev(s), group, pre=pre))
    want = x.astype(np.float64) @ (q * np.repeat(s.astype(np.float64), group, axis=1)).T
    assert np.array_equal(y, want.astype(np.float16)) and np.array_equal(host(pre), want.astype(np.float16))


# More tiles (128 x 256; up to 64 rows: 64 x 256) than workgroups, so that one takes a second whole tile while its first one's
# outputs are on their way: rows that are whole 16-byte pieces and odd ones; leftover tiles whole (short k) and split
@pytest.mark.parametrize("m,n,k,group,split", [(2177, 4104, 256, 32, False), (2177, 4099, 256, 128, False), (2177, 4104, 2560, 128, True),
                                               (2177, 4099, 2560, 32, True), (2177, 4104, 2208, 32, True), (50, 66000, 256, 32, False),
                                               (61, 66001, 256, 128, False), (4400, 8197, 96, 32, False)])
@pytest.mark.parametrize("act,residual,keep", [("relu", "in place", True), ("none", "apart", False), ("silu", "in place", True)])
def test_linear_of_many_tiles(w4, m, n, k, group, split, act, residual, keep):
    """Integers, so z is exact (relu, none: y too) and any element that went astray shows."""
    torch = torch_mod()
    tiles = -(-m // (64 if m <= 64 else 128)) * -(-n // 256)
    assert tiles > torch.cuda.get_device_properties(0).multi_processor_count
    assert (w4.lib.w4a16_linear_workspace_bytes(m, n, k, group) > 0) == split
    gen = torch.Generator(device="cuda").manual_seed(87500 + m + n + k)
    ints = lambda lo, hi, *shape: torch.randint(lo, hi + 1, shape, generator=gen, device="cuda")  # noqa: E731
    codes = ints(-8, 7, n, k // 8, 8)
    packed = ((codes + 8) << torch.arange(0, 32, 4, device="cuda")).sum(dim=2).to(torch.int32)
    scales = torch.ones((n, k // group), dtype=torch.float16, device="cuda")
    scales[:, ::2] = 0.5
    x, bias, res = ints(-2, 2, m, k).half(), ints(-8, 8, n).half(), ints(-64, 64, m, n).half()
    w = codes.view(n, k).float() * scales.float().repeat_interleave(group, dim=1)
    z = x.float() @ w.t() + bias.float()
    want = {"relu": z.clamp(min=0), "none": z, "silu": z.double() * torch.sigmoid(z.double())}[act] + res.double()
    pre = torch.full((m, n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    y = w4.linear(x, packed, scales, group, bias=bias, activation=act, residual=res, pre=pre, out=res if residual == "in place" else None)
    if act == "silu":         # y's one rounding, and the exponential's and reciprocal's (some fp32 units in the last place)
        assert bool(((y.double() - want).abs() <= 2.0 ** -11 * want.abs() + 2.0 ** -20 * (z.abs() + 1)).all())
    else:
        assert torch.equal(y, want.half())
    if keep:
        assert torch.equal(pre, z.half())


@pytest.mark.parametrize("tokens,topk", [(2, 3), (7, 9), (40, 4)])
@pytest.mark.parametrize("size", [2.0 ** -3, 2.0 ** -8, 2.0 ** -13, 2.0 ** -18])
def test_small_products_between_the_experts_kernels(w4, tokens, topk, size):
    """h = SiLU(g) u about `size` and down scales about 1: y is as far off as an h within 2^-23 of its size or 2^-28 makes it.
    Bar: gate/up weights are sums of one term each and h's own arithmetic is fp32 (g u sigmoid: 2^-20 |h|, as the
    exponential and reciprocal are within some units in the last place); then |w2| times that, fp32 sums, one rounding."""
    torch = torch_mod()
    from test_moe_ffn_gpu import Layer
    experts, hidden, inter, group = 5, 64, 96, 32
    layer = Layer(w4, experts, hidden, inter, group, 87600 + tokens)
    rng = layer.rng
    # g near 1 (gate rows: code 4, scale 1/4, at x[0] = 1), u near size (up rows: at x[1] = size)
    gu, gs = np.zeros((experts, 2 * inter, hidden), np.int8), np.full((experts, 2 * inter, hidden // group), 0.25, np.float16)
    gu[:, 0::2, 0], gu[:, 1::2, 1] = 4, rng.integers(2, 8, (experts, inter))
    ds = (0.5 + rng.random((experts, hidden, inter // group))).astype(np.float16)
    x = np.zeros((tokens, hidden), np.float16)
    x[:, 0], x[:, 1] = 0.5 + rng.random(tokens), size * (0.5 + rng.random(tokens))
    ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    w = rng.random((tokens, topk)).astype(np.float32)
    pack = lambda b: dev(np.stack([w4.pack(c) for c in b]))  # noqa: E731
    y = host(w4.moe_ffn(dev(x), dev(ids), dev(w), pack(gu), dev(gs), pack(layer.dn[0]), dev(ds), group)).astype(np.float64)
    want, bar = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for t in range(tokens):
        for e, ws in zip(ids[t], w[t].astype(np.float64)):
            w2 = layer.dn[0][e] * np.repeat(ds[e].astype(np.float64), group, axis=1)
            g = float(x[t, 0])
            u = gu[e, 1::2, 1] * 0.25 * float(x[t, 1])
            h = g / (1 + np.exp(-g)) * u
            want[t] += ws * (w2 @ h)
            bar[t] += ws * (np.abs(w2) @ (2.0 ** -20 * np.abs(h) + np.maximum(2.0 ** -23 * np.abs(h), 2.0 ** -28)
                                          + (inter + topk + 8) * 2.0 ** -24 * np.abs(h)))
    assert np.all(np.abs(y - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + bar)


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("tokens", [5, 60, 300])
def test_masked_router_into_the_experts(w4, tokens, renormalize):
    """Tokens that the router leaves with fewer experts than slots, or none, go through the four calls, and (few tokens)
    through moe_ffn, as through the formula with the slots left out."""
    torch = torch_mod()
    from gpu_util import assert_close
    from test_moe_ffn_gpu import Layer
    experts, topk, hidden = 12, 4, 256
    layer = Layer(w4, experts, hidden, 128, 32, 87700 + tokens)
    rng = layer.rng
    logits = rng.standard_normal((tokens, experts)).astype(np.float32)
    logits[rng.random(logits.shape) < 0.7] = -np.inf
    logits[1] = -np.inf
    x = dev(rng.standard_normal((tokens, hidden)).astype(np.float16))
    ids, w = w4.moe_topk(dev(logits), topk, renormalize=renormalize)
    assert bool((ids == -1).any(dim=1).any()) and bool((ids[1] == -1).all())
    want, bar = layer.formula(host(x), host(ids), host(w))
    gu, gs, dn, ds = layer.args
    offs, tok, row = w4.moe_route(ids, experts)
    h = w4.grouped_gemm_swiglu(x, gu, gs, offs, 32, pair_token=tok)
    y = host(w4.moe_combine(w4.grouped_gemm(h, dn, ds, offs, 32), row, w))
    assert np.all(y[1] == 0)
    some = np.abs(want).sum(axis=1) > 0
    assert_close(y[some], want[some], "four calls")
    if tokens <= 64:
        y = host(layer(x, ids, w)).astype(np.float64)
        assert np.all(np.abs(y - want) <= bar) and np.all(y[1] == 0)
