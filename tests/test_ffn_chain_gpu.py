"""The feed-forward block's calls together, as a training step makes them: forward, input
gradients and scale gradients against the fp64 formulas; captured, replayed and on several
streams at once; with shared workspaces, neighbouring memory, infinities and large offsets.

Bars (fixed before the first run): the oracle's per element and per row (each stage is
compared with the fp64 formula on the fp16 inputs that the stage itself was given, so the
derivations of the single calls' tests hold); scale gradients (rows + group) 2^-22 of the
sum of magnitudes.  Repeated, replayed and concurrent calls must agree bit for bit: every
sum has a fixed order.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_close, dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


class Block:
    """A small feed-forward block with its inputs on the device (gate/up [2 n, k], down [k, n])."""

    def __init__(self, w4, m, n, k, group, seed):
        rng = np.random.default_rng(seed)
        self.w4, self.m, self.n, self.k, self.group = w4, m, n, k, group
        self.gu = synth.code_bank(rng, 1, 2 * n, k)[0], synth.scale_bank(rng, 1, 2 * n, k // group)[0]
        self.dn = synth.code_bank(rng, 1, k, n)[0], synth.scale_bank(rng, 1, k, n // group)[0]
        self.x, self.dy = synth.activations(rng, m, k), (synth.activations(rng, m, k) * np.float16(0.1)).astype(np.float16)
        self.gu_d = dev(w4.pack(self.gu[0])), dev(self.gu[1])
        self.dn_d = dev(w4.pack(self.dn[0])), dev(self.dn[1])
        self.x_d, self.dy_d = dev(self.x), dev(self.dy)
        self.gemm_ws = w4.gemm_workspace(m, k, n, group)     # the down projection's own: gemm keeps state in it

    def step(self, stream=None):
        """One training step's calls: outputs by name."""
        torch, w4, g = torch_mod(), self.w4, self.group
        z = torch.empty((self.m, 2 * self.n), dtype=torch.float16, device="cuda")
        h = w4.gemm_swiglu(self.x_d, *self.gu_d, g, gate_up=z, stream=stream)
        y = w4.gemm(h, *self.dn_d, g, workspace=self.gemm_ws, stream=stream)
        dh = w4.gemm_t(self.dy_d, *self.dn_d, g, stream=stream)
        ds_dn = w4.gemm_dscales(self.dy_d, h, self.dn_d[0], g, stream=stream)
        dx, dz = w4.gemm_swiglu_backward(dh, z, *self.gu_d, g, stream=stream)
        ds_gu = w4.gemm_dscales(dz, self.x_d, self.gu_d[0], g, stream=stream)
        return dict(z=z, h=h, y=y, dh=dh, ds_dn=ds_dn, dx=dx, dz=dz, ds_gu=ds_gu)


def assert_scale_gradient(ds, d, x, q, group, what):
    n, k = q.shape
    d, x, q = (a.astype(np.float64) for a in (d, x, q))
    grouped = lambda a: a.reshape(n, k // group, group).sum(axis=2)  # noqa: E731
    want, size = grouped(q * (d.T @ x)), grouped(np.abs(q) * (np.abs(d).T @ np.abs(x)))
    assert np.all(np.abs(ds - want) <= (d.shape[0] + group) * 2.0 ** -22 * size), what


# (m, n, k, group): one token, a few, a ragged batch, a batch past a tile
@pytest.mark.parametrize("m,n,k,group", [(1, 256, 384, 128), (20, 544, 288, 32), (77, 1056, 416, 32), (300, 512, 640, 128)])
def test_training_step(w4, m, n, k, group):
    b = Block(w4, m, n, k, group, 51000 + m)
    o = {a: host(t) for a, t in b.step().items()}
    gu, dn = oracle.dequantize(*b.gu, group), oracle.dequantize(*b.dn, group)
    f64 = {a: t.astype(np.float64) for a, t in o.items()}
    assert_close(o["z"], b.x.astype(np.float64) @ gu.T, "kept products")
    assert_close(o["h"], oracle.swiglu_linear(b.x, oracle.pack(b.gu[0]), b.gu[1], group), "h")
    assert_close(o["y"], f64["h"] @ dn.T, "y")
    assert_close(o["dh"], b.dy.astype(np.float64) @ dn, "dh")
    z, dh = f64["z"], f64["dh"]
    sig = 1 / (1 + np.exp(-z[:, 0::2]))
    dz = np.empty_like(z)
    dz[:, 0::2] = dh * z[:, 1::2] * sig * (1 + z[:, 0::2] * (1 - sig))
    dz[:, 1::2] = dh * z[:, 0::2] * sig
    assert_close(o["dz"], dz, "dz")
    assert_close(o["dx"], f64["dz"] @ gu, "dx")
    assert_scale_gradient(o["ds_gu"], o["dz"], b.x, b.gu[0], group, "gate/up scales")
    assert_scale_gradient(o["ds_dn"], b.dy, o["h"], b.dn[0], group, "down scales")


def same(a, b):
    return all(np.array_equal(host(a[n]).view(np.uint8), host(b[n]).view(np.uint8)) for n in b)


@pytest.mark.parametrize("m,n,k,group", [(5, 256, 384, 128), (150, 1056, 416, 32)])
def test_graph_replays_match_eager(w4, m, n, k, group):
    """The step captured, replayed with new inputs, other eager work and other streams' calls between."""
    torch = torch_mod()
    b, other = Block(w4, m, n, k, group, 52000 + m), Block(w4, m + 9, n, k, group, 52500 + m)
    want_other = {a: t.clone() for a, t in other.step().items()}
    b.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.step()
    for rep in range(4):
        b.x_d.copy_(torch.randn_like(b.x_d))
        b.dy_d.copy_(torch.randn_like(b.dy_d) * 0.1)
        want = {a: t.clone() for a, t in b.step().items()}
        for t in out.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert same(out, want), f"replay {rep}"
        assert same(other.step(), want_other), f"eager work after replay {rep}"


def test_two_graphs_on_two_streams(w4):
    """Two captured steps replayed at once: they share no workspace."""
    torch = torch_mod()
    blocks = [Block(w4, 40, 512, 384, 128, 53000), Block(w4, 140, 512, 384, 128, 53001)]
    wants = [{a: t.clone() for a, t in b.step().items()} for b in blocks]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b in blocks:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.step())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for t in (t for o in outs for t in o.values()):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip(outs, wants))


def test_calls_on_several_streams_at_once(w4):
    """Steps of two sizes interleaved on three streams, the streams given by argument."""
    torch = torch_mod()
    blocks = [Block(w4, 24, 512, 640, 128, 54000), Block(w4, 200, 512, 640, 128, 54001), Block(w4, 1, 512, 640, 128, 54002)]
    wants = [{a: t.clone() for a, t in b.step().items()} for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(6):
        outs = [b.step(stream=s) for b, s in zip(blocks, streams)]
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip(outs, wants))


def test_one_workspace_for_every_call(w4):
    """A caller's own workspace, sized for the largest call, used by all of them in turn; its counters stay 0."""
    torch = torch_mod()
    b = Block(w4, 70, 544, 416, 32, 55000)
    n, k, g = 544, 416, 32
    sizes = [w4.ffn_workspace(c, m, nn, k, g) for c, m, nn in (("gemm_swiglu", 70, n), ("gemm_swiglu_backward", 70, n),
                                                              ("gemm_t", 1, 2 * n), ("gemm_dscales", 70, 2 * n))]
    ws = max((t for t in sizes if t is not None), key=torch.numel)
    ws[4096:].fill_(-1)                                    # only the counters have to be clear
    want = b.step()
    z, dz = want["z"], want["dz"]
    for _ in range(3):
        z2 = torch.empty_like(z)
        h = w4.gemm_swiglu(b.x_d, *b.gu_d, g, gate_up=z2, workspace=ws)
        dx, dz2 = w4.gemm_swiglu_backward(want["dh"], z2, *b.gu_d, g, workspace=ws)
        y1 = w4.gemm_t(dz[:1].contiguous(), *b.gu_d, g, workspace=ws)
        ds = w4.gemm_dscales(dz, b.x_d, b.gu_d[0], g, workspace=ws)
        y2 = w4.gemm_t(dz[:1].contiguous(), *b.gu_d, g)
        got = dict(z=z2, h=h, dx=dx, dz=dz2, ds_gu=ds)
        assert same(got, {a: want[a] for a in got}) and torch.equal(y1, y2)
        assert int(ws[:4096].abs().sum()) == 0
    # 1024 rows need one (the work is split along them): too small a one is refused
    rows = torch.zeros((1024, 2 * n), dtype=torch.float16, device="cuda"), torch.zeros((1024, k), dtype=torch.float16, device="cuda")
    assert w4.ffn_workspace("gemm_dscales", 1024, 2 * n, k, g) is not None
    with pytest.raises(w4.W4A16Error, match="WORKSPACE"):
        w4.gemm_dscales(*rows, b.gu_d[0], g, workspace=ws[:4096].contiguous())


@pytest.mark.parametrize("m", [1, 17, 50, 300])
def test_nothing_else_is_written(w4, m):
    """Outputs in the middle of larger buffers (16-byte aligned): the neighbours keep their values."""
    torch = torch_mod()
    n, k, g = 1003, 416, 32
    rng = np.random.default_rng(56000 + m)
    q, s = synth.code_bank(rng, 1, 2 * n, k)[0], synth.scale_bank(rng, 1, 2 * n, k // g)[0]
    p, s = dev(w4.pack(q)), dev(s)
    x, dy = dev(synth.activations(rng, m, k)), dev(synth.activations(rng, m, n))

    def framed(rows, cols, dtype=torch.float16):
        buf = torch.full((rows * cols + 128,), 777.0, dtype=dtype, device="cuda")
        return buf, buf[64:64 + rows * cols].view(rows, cols)

    frames = {a: framed(*shape) for a, shape in dict(h=(m, n), z=(m, 2 * n), dz=(m, 2 * n), dx=(m, k), t=(m, k)).items()}
    frames["ds"] = framed(2 * n, k // g, torch.float32)
    w4.gemm_swiglu(x, p, s, g, gate_up=frames["z"][1], out=frames["h"][1])
    w4.gemm_swiglu_backward(dy, frames["z"][1], p, s, g, out=frames["dx"][1], dgate_up=frames["dz"][1])
    w4.gemm_t(frames["dz"][1], p, s, g, out=frames["t"][1])
    w4.gemm_dscales(frames["dz"][1], x, p, g, out=frames["ds"][1])
    torch.cuda.synchronize()
    for name, (buf, view) in frames.items():
        assert bool((buf[:64] == 777).all()) and bool((buf[-64:] == 777).all()), name
        assert torch.isfinite(view).all(), name
    assert torch.equal(frames["t"][1], frames["dx"][1])


@pytest.mark.parametrize("m,n", [(2, 40), (2, 43), (20, 1001), (70, 40), (70, 43), (300, 1001)])
def test_infinities_and_nans_stay_in_their_row(w4, m, n):
    """Row 1 of d (x) all infinity and NaN: every other row's result is untouched, row 1's is not finite."""
    torch = torch_mod()
    k, g = 416, 32
    rng = np.random.default_rng(57000 + m + n)
    p, s = dev(w4.pack(synth.code_bank(rng, 1, 2 * n, k)[0])), dev(synth.scale_bank(rng, 1, 2 * n, k // g)[0])
    d = dev(synth.activations(rng, m, 2 * n))
    x = dev(synth.activations(rng, m, k))
    bad_d, bad_x = d.clone(), x.clone()
    for t in (bad_d, bad_x):
        t[1, 0::2], t[1, 1::2] = float("inf"), float("nan")
    keep = torch.arange(m, device="cuda") != 1
    for good, bad in ((w4.gemm_t(d, p, s, g), w4.gemm_t(bad_d, p, s, g)),
                      (w4.gemm_swiglu(x, p, s, g), w4.gemm_swiglu(bad_x, p, s, g))):
        assert torch.equal(good[keep], bad[keep]) and not torch.isfinite(bad[1]).any()
    # an infinity meets the formula's: every product with a code other than 0 is infinite
    one = torch.zeros_like(d)
    one[0, 3] = float("inf")
    q = torch.from_numpy(w4.unpack(host(p).view(np.uint32), k)).cuda()[3].float()
    y = w4.gemm_t(one, p, s, g)[0].float()
    assert torch.equal(torch.isnan(y), q == 0) and torch.equal(torch.sign(y[q != 0]), torch.sign(q[q != 0]))
    # a column of d in the scale gradient: only its row of the result
    bad_d = d.clone()
    bad_d[0, 5] = float("nan")
    a, b = w4.gemm_dscales(d, x, p, g), w4.gemm_dscales(bad_d, x, p, g)
    keep = torch.arange(2 * n, device="cuda") != 5
    assert torch.equal(a[keep], b[keep]) and torch.isnan(b[5]).all()


def test_empty_sizes(w4):
    torch = torch_mod()
    f16 = dict(dtype=torch.float16, device="cuda")
    p0, s0 = torch.zeros((0, 16), dtype=torch.int32, device="cuda"), torch.zeros((0, 1), **f16)
    assert torch.equal(w4.gemm_t(torch.zeros((3, 0), **f16), p0, s0, 128), torch.zeros((3, 128), **f16))
    dx, dz = w4.gemm_swiglu_backward(torch.zeros((3, 0), **f16), torch.zeros((3, 0), **f16), p0, s0, 128)
    assert torch.equal(dx, torch.zeros((3, 128), **f16)) and dz.shape == (3, 0)
    p, s = torch.zeros((6, 16), dtype=torch.int32, device="cuda"), torch.ones((6, 1), **f16)
    assert w4.gemm_t(torch.zeros((0, 6), **f16), p, s, 128).shape == (0, 128)
    assert w4.gemm_swiglu(torch.zeros((0, 128), **f16), p, s, 128).shape == (0, 3)
    ds = w4.gemm_dscales(torch.zeros((0, 6), **f16), torch.zeros((0, 128), **f16), p, 128)
    assert torch.equal(ds, torch.zeros((6, 1), dtype=torch.float32, device="cuda"))


def test_large_offsets(w4):
    """Buffers near their limit of 2 GiB: 36 rows of d with 2^24 + 40 columns (1.2 GB), k = 32."""
    torch = torch_mod()
    m, n, k, g = 36, (1 << 24) + 40, 32, 32
    gen = torch.Generator(device="cuda").manual_seed(58000)
    p = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, k // 8), dtype=torch.int32, device="cuda", generator=gen)
    s = torch.full((n, 1), 2.0 ** -10, dtype=torch.float16, device="cuda")
    d = torch.zeros((m, n), dtype=torch.float16, device="cuda")
    at = torch.randint(0, n, (m, 64), device="cuda", generator=gen)
    at[:, 0], at[:, 1] = n - 1, 0
    d.scatter_(1, at, 1.0)
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)

    def codes(rows):
        return (((p[rows].unsqueeze(2) >> shift) & 15) - 8).reshape(len(rows), k).double()

    want = torch.stack([codes(torch.unique(at[r])).sum(dim=0) for r in range(m)]) * 2.0 ** -10
    assert torch.equal(w4.gemm_t(d, p, s, g).double(), want)                 # exact: at most 64 codes of 10 bits
    for rows in (1, 32):                                                     # the weight-streaming kernels
        assert torch.equal(w4.gemm_t(d[:rows].contiguous(), p, s, g).double(), want[:rows])
    x = torch.ones((m, k), dtype=torch.float16, device="cuda")
    ds = w4.gemm_dscales(d, x, p, g)
    rows = torch.unique(at)
    assert torch.equal(ds[rows, 0].double(), codes(rows).sum(dim=1) * d[:, rows].double().sum(dim=0))
    assert int((ds != 0).sum()) <= len(rows)


def test_threads_on_one_stream(w4):
    """Two host threads call at once on the same stream: their calls' kernels interleave there."""
    import threading
    torch = torch_mod()
    blocks = [Block(w4, 70, 512, 640, 128, 57000), Block(w4, 300, 512, 640, 128, 57001)]
    wants = [{a: t.clone() for a, t in b.step().items()} for b in blocks]
    torch.cuda.synchronize()
    start, results = threading.Barrier(2), [None, None]

    def work(i):
        start.wait()
        results[i] = [blocks[i].step() for _ in range(20)]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for r, want in zip(results, wants):
        assert r is not None and all(same(o, want) for o in r)


def test_pairs_gradient_is_not_written_over_the_pairs(w4):
    b = Block(w4, 3, 64, 128, 32, 57100)
    z = torch_mod().zeros((3, 128), dtype=torch_mod().float16, device="cuda")
    dh = torch_mod().zeros((3, 64), dtype=torch_mod().float16, device="cuda")
    with pytest.raises(ValueError, match="must not be gate_up"):
        w4.gemm_swiglu_backward(dh, z, *b.gu_d, 32, dgate_up=z)
