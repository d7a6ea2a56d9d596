"""The block's calls one after another as a model makes them: a decoded token's step (output projection with the
residual, router, routed experts), a training step's forward and backward, both captured and replayed, on
other streams, from two host threads and with given workspaces.

Each stage is checked against fp64 from the device's own result of the stage before, with the bars of the calls'
own tests; the runs among each other bit by bit (the kernels' results do not depend on timing).
"""

import threading

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_close, dev, host, torch_mod
from test_linear_gpu import act64, slope64, weights
from test_moe_ffn_gpu import Layer
from test_moe_topk_gpu import choice, softmax_weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


class Block:
    """Output projection [hidden, width], router [experts, hidden] (a plain fp32 product), routed experts."""

    def __init__(self, w4, hidden, width, experts, inter, topk, group, seed):
        self.w4, self.group, self.topk = w4, group, topk
        self.experts = Layer(w4, experts, hidden, inter, group, seed)
        rng = self.rng = self.experts.rng
        self.proj = weights(rng, hidden, width, group)
        self.packed, self.scales = dev(w4.pack(self.proj[0])), dev(self.proj[1])
        self.router = dev((rng.standard_normal((experts, hidden)) / np.sqrt(hidden)).astype(np.float32))

    def inputs(self, tokens):
        return (dev(synth.activations(self.rng, tokens, self.packed.shape[1] * 8)),
                dev(synth.activations(self.rng, tokens, self.packed.shape[0])))

    def step(self, attended, stream_in, **kw):
        h = self.w4.linear(attended, self.packed, self.scales, self.group, residual=stream_in, **kw)
        logits = (h.float()[:, None, :] * self.router).sum(dim=2)
        ids, w = self.w4.moe_topk(logits, self.topk, **kw)
        return h, logits, ids, w, self.experts(h, ids, w, residual=h, **kw)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("tokens", [1, 4, 11, 40, 64])
def test_decode_step(w4, tokens, group):
    b = Block(w4, 384, 640, 12, 256, 3, group, 91000 + tokens + group)
    attended, stream_in = b.inputs(tokens)
    h, logits, ids, w, y = b.step(attended, stream_in)
    want = host(attended).astype(np.float64) @ oracle.dequantize(*b.proj, group).T + host(stream_in).astype(np.float64)
    size = np.abs(host(attended).astype(np.float64)) @ np.abs(oracle.dequantize(*b.proj, group)).T
    assert np.all(np.abs(host(h) - want) <= 2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 704 * 2.0 ** -24) * size
                  + 2.0 ** -18 * (2 * np.abs(want) + 1))
    l = host(logits)
    assert np.array_equal(host(ids), choice(l, 3))
    ww, far = softmax_weights(l, host(ids), True)
    assert np.all(np.abs(host(w) - ww) <= (28 * 2.0 ** -24 + 2.0 ** -23 * far) * ww)
    want, bar = b.experts.formula(host(h), host(ids), host(w), host(h))
    assert np.all(np.abs(host(y) - want) <= bar)


# fewer rows than the weight-streaming kernel takes, where the epilogue's gradient is made in it, in front of it (longer
# ranges per wave), odd rows of both kinds, and tiles
TRAIN = [(6, 264, 384, 128), (19, 515, 640, 32), (32, 7000, 5120, 128), (5, 6203, 5120, 128), (30, 3001, 2560, 32),
         (70, 330, 256, 128)]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "none"])
@pytest.mark.parametrize("m,n,k,group", TRAIN)
def test_training_step(w4, m, n, k, group, act):
    """linear with kept pre-activations, linear_backward from them, gemm_dscales from its dpre."""
    torch = torch_mod()
    rng = np.random.default_rng(92000 + m + n)
    q, s = weights(rng, n, k, group)
    x, dy = synth.activations(rng, m, k), synth.activations(rng, m, n)
    b = synth.activations(rng, 1, n)[0]
    p, sd, has = dev(w4.pack(q)), dev(s), act != "none"
    z = torch.empty((m, n), dtype=torch.float16, device="cuda") if has else None
    y = w4.linear(dev(x), p, sd, group, bias=dev(b), activation=act, pre=z)
    dx, dz, dbias = w4.linear_backward(dev(dy), p, sd, group, pre=z, activation=act, dbias=True)
    ds = w4.gemm_dscales(dz if has else dev(dy), dev(x), p, group)
    w, x64, dy64 = oracle.dequantize(q, s, group), x.astype(np.float64), dy.astype(np.float64)
    pre = x64 @ w.T + b.astype(np.float64)
    size = (2.0 ** -11 + (k + 64) * 2.0 ** -24) * (np.abs(x64) @ np.abs(w).T) + 2.0 ** -25
    want = act64(act, pre)
    assert np.all(np.abs(host(y) - want) <= 2.0 ** -11 * np.abs(want) + 1.13 * size
                  + 2.0 ** -18 * (np.abs(pre) + np.abs(want) + 1))
    got = dy64
    if has:
        assert np.all(np.abs(host(z) - pre) <= 2.0 ** -11 * np.abs(pre) + size)
        z64 = host(z).astype(np.float64)
        v, slack = dy64 * slope64(act, z64), 2.0 ** -18 * np.abs(dy64) * (1 + np.minimum(np.abs(z64), 100))
        got = host(dz).astype(np.float64)
        assert np.all(np.abs(got - v) <= 2.0 ** -11 * np.abs(v) + slack + 2.0 ** -25)
    else:
        v, slack = dy64, 0 * dy64
    assert np.all(np.abs(host(dbias) - v.sum(axis=0)) <= (m + 32) * 2.0 ** -23 * np.abs(v).sum(axis=0) + slack.sum(axis=0))
    assert_close(host(dx), got @ w, "dx")
    # the scales' gradient: sum over a group's k of (dz^T x) q, fp32 sums of exact products
    per = (got.T @ x64) * q
    bound = (np.abs(got).T @ np.abs(x64)) * np.abs(q)
    per, bound = (t.reshape(n, k // group, group).sum(axis=2) for t in (per, bound))
    assert np.all(np.abs(host(ds) - per) <= (m + group + 64) * 2.0 ** -23 * bound)


def same(a, b):
    return all(x is y or bool((x.view(-1) == y.view(-1)).all()) for x, y in zip(a, b))


@pytest.mark.parametrize("tokens", [1, 24])
def test_captured_decode_steps(w4, tokens):
    """Two graphs of two blocks that live at once and are replayed in turn, on two streams, with eager steps between;
    the topk gradient is part of them."""
    torch = torch_mod()
    blocks = [Block(w4, 256, 384, 9, 128, 2, 32, 93000 + i) for i in range(2)]
    ins = [b.inputs(tokens) for b in blocks]

    def step(i):
        b, (attended, stream_in) = blocks[i], ins[i]
        h, logits, ids, w, y = b.step(attended, stream_in)
        return h, logits, ids, w, y, w4.moe_topk_backward(w * 2, logits, ids, w)

    for i in range(2):
        step(i)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i))
        graphs.append(g)
    sides = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(4):
        for attended, stream_in in ins:
            attended.copy_(torch.randn_like(attended))
            stream_in.copy_(torch.randn_like(stream_in))
        want = [[t.clone() for t in step(i)] for i in range(2)]
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for g, side in zip(graphs, sides):             # both in flight at once
            with torch.cuda.stream(side):
                g.replay()
        step(0)
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1]), f"replay {rep}"


@pytest.mark.parametrize("m,n,k,group", [(3, 264, 640, 128), (21, 515, 640, 32), (70, 330, 1024, 128), (140, 2003, 1024, 128)])
def test_captured_training_step(w4, m, n, k, group):
    """Forward and backward in one graph, while eager steps of the same leaves run before, between and after."""
    torch = torch_mod()
    rng = np.random.default_rng(94000 + m)
    q, s = weights(rng, n, k, group)
    p, sd, b = dev(w4.pack(q)), dev(s), dev(synth.activations(rng, 1, n)[0])
    x, dy = dev(synth.activations(rng, m, k)), dev(synth.activations(rng, m, n))

    def step():
        z = torch.empty((m, n), dtype=torch.float16, device="cuda")
        y = w4.linear(x, p, sd, group, bias=b, activation="gelu", residual=dy, pre=z)
        return (z, y) + w4.linear_backward(y, p, sd, group, pre=z, activation="gelu", dbias=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for rep in range(4):
        x.copy_(torch.randn_like(x))
        want = step()
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want), f"replay {rep}"


def test_on_a_stream_given(w4):
    """Every call on a stream given by argument, behind its own work, operands dropped at once."""
    torch = torch_mod()
    b = Block(w4, 256, 384, 9, 128, 2, 32, 95000)
    attended, stream_in = b.inputs(30)
    side = torch.cuda.Stream()
    h, _, ids, w, y = b.step(attended, stream_in)
    logits = torch.randn(30, 9, device="cuda")
    pre, dy = torch.randn_like(h), torch.randn_like(h)
    want = [h, y, *w4.moe_topk(logits, 2), *w4.linear_backward(dy, b.packed, b.scales, 32, pre=pre, activation="silu", dbias=True)]
    want.append(w4.moe_topk_backward(want[3], logits, want[2], want[3]))
    work = torch.zeros((8192, 8192), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            for _ in range(8):
                work = work @ work
        copies = [t.clone() for t in (attended, stream_in, logits, pre, dy, h, ids, w)]
        side.wait_stream(torch.cuda.current_stream())
        a2, s2, l2, p2, d2, h2, i2, w2 = copies
        got = [w4.linear(a2, b.packed, b.scales, 32, residual=s2, stream=side),
               b.experts(h2, i2, w2, residual=h2, stream=side)]
        got.extend(w4.moe_topk(l2, 2, stream=side))
        got.extend(w4.linear_backward(d2, b.packed, b.scales, 32, pre=p2, activation="silu", dbias=True, stream=side))
        got.append(w4.moe_topk_backward(got[3], l2, got[2], got[3], stream=side))
        sizes = [(t.numel(), t.dtype) for t in copies]
        del copies, a2, s2, l2, p2, d2, h2, i2, w2
        again = [torch.full((count,), -1, dtype=dtype, device="cuda") for count, dtype in sizes]
        torch.cuda.synchronize()
        assert same(got, want) and all(bool((t == -1).all()) for t in again)


def test_two_threads_at_once(w4):
    """Two host threads on two streams, each with its own block and the same workspaces' sizes."""
    torch = torch_mod()
    blocks = [Block(w4, 256, 384, 9, 128, 2, 128, 96000 + i) for i in range(2)]
    ins = [b.inputs(50) for b in blocks]
    f16 = dict(dtype=torch.float16, device="cuda")
    big = dict(group=128, packed=torch.randint(-2 ** 31, 2 ** 31 - 1, (520, 128), dtype=torch.int32, device="cuda"),
               scales=torch.rand(520, 8, **f16) * 0.01)
    xs, dys = [torch.randn(140, 1024, **f16) for _ in range(2)], [torch.randn(140, 520, **f16) for _ in range(2)]

    def run(i):
        return list(blocks[i].step(*ins[i])) + [w4.linear(xs[i], **big, activation="gelu")] + \
            list(w4.linear_backward(dys[i], **big, pre=dys[i], activation="silu", dbias=True))

    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    bad = []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(25):
                    got = run(i)
                torch.cuda.current_stream().synchronize()
                if not same(got, want[i]):
                    bad.append(i)
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("m,n,k,group", [(1, 1024, 1024, 128), (19, 1001, 1120, 32), (70, 330, 1024, 128), (140, 2003, 1024, 128)])
def test_given_workspace(w4, m, n, k, group):
    """A workspace of the size asked for serves call after call: nothing is written behind it and its counters end at zero."""
    torch = torch_mod()
    rng = np.random.default_rng(97000 + m)
    q, s = weights(rng, n, k, group)
    p, sd = dev(w4.pack(q)), dev(s)
    x, dy, z = (dev(synth.activations(rng, m, c)) for c in (k, n, n))
    runs = {"linear": lambda **kw: (w4.linear(x, p, sd, group, activation="silu", **kw),),
            "linear_backward": lambda **kw: w4.linear_backward(dy, p, sd, group, pre=z, activation="silu", dbias=True, **kw)}
    for call, run in runs.items():
        made = w4.ffn_workspace(call, m, n, k, group)
        words = 0 if made is None else made.numel()
        buf = torch.full((words + 65536,), 77, dtype=torch.int32, device="cuda")
        ws = buf[:words]
        ws[:4096] = 0
        want = run()
        for _ in range(3):
            assert same(run(workspace=ws if words else None), want)
        assert bool((buf[words:] == 77).all())
        assert int(ws[:4096].abs().sum()) == 0


@pytest.mark.parametrize("tokens", [3, 20])
def test_given_workspace_of_the_experts(w4, tokens):
    torch = torch_mod()
    layer = Layer(w4, 10, 256, 384, 128, 98000 + tokens)
    x = dev(synth.activations(layer.rng, tokens, 256))
    ids = dev(layer.rng.integers(0, 10, (tokens, 4)).astype(np.int32))
    w = dev(layer.rng.random((tokens, 4)).astype(np.float32))
    words = -(-w4.lib.w4a16_moe_ffn_workspace_bytes(tokens, 4, 256, 384, 128) // 4)
    buf = torch.full((words + 65536,), 77, dtype=torch.int32, device="cuda")
    buf[:4096] = 0
    want = layer(x, ids, w)
    for _ in range(3):
        assert torch.equal(layer(x, ids, w, workspace=buf[:words]), want)
    assert bool((buf[words:] == 77).all())
    with pytest.raises(w4.W4A16Error, match="WORKSPACE"):
        layer(x, ids, w, workspace=buf[:words - 4])
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [2, 40])
def test_workspace_made_for_the_experts(w4, tokens):
    """moe_ffn_workspace's tensor serves calls on another stream, and within a capture that makes it."""
    torch = torch_mod()
    layer = Layer(w4, 7, 256, 128, 32, 99500 + tokens)
    x = dev(synth.activations(layer.rng, tokens, 256))
    ids = dev(layer.rng.integers(0, 7, (tokens, 3)).astype(np.int32))
    w = dev(layer.rng.random((tokens, 3)).astype(np.float32))
    want = layer(x, ids, w)
    ws = w4.moe_ffn_workspace(tokens, 3, 256, 128, 32)
    assert ws.numel() * 4 >= w4.lib.w4a16_moe_ffn_workspace_bytes(tokens, 3, 256, 128, 32) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [layer(x, ids, w, workspace=ws, stream=side) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert w4.moe_ffn_workspace(65, 3, 256, 128, 32) is None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, ids, w, workspace=w4.moe_ffn_workspace(tokens, 3, 256, 128, 32))
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
