"""The feed-forward block's calls and the memory they are given: operands that share some, and
workspaces used on other streams than the one they were made on."""

import numpy as np
import pytest

import synth
from gpu_util import dev, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def pair_weights(w4, rng, n, k, group):
    """Packed words and scales of 2 n weight rows on the device."""
    return dev(w4.pack(synth.code_bank(rng, 1, 2 * n, k)[0])), dev(synth.scale_bank(rng, 1, 2 * n, k // group)[0])


@pytest.mark.parametrize("m", [2, 40])
def test_shared_memory_is_refused(w4, m):
    """Views of one buffer that overlap by 16 bytes or more: refused, and nothing is written; just apart: accepted."""
    torch = torch_mod()
    n, k, g = 64, 128, 32
    rng = np.random.default_rng(61000 + m)
    p, s = pair_weights(w4, rng, n, k, g)
    buf = dev(synth.activations(rng, 1, 4 * m * 2 * n))[0]
    before = buf.clone()

    def view(at, rows, cols):
        return buf[at:at + rows * cols].view(rows, cols)

    size = m * 2 * n
    z, dh, x = view(0, m, 2 * n), dev(synth.activations(rng, m, n)), view(0, m, k)
    refused = [lambda: w4.gemm_swiglu_backward(dh, z, p, s, g, dgate_up=view(size - 8, m, 2 * n)),
               lambda: w4.gemm_swiglu_backward(dh, z, p, s, g, out=view(size - 8, m, k)),
               lambda: w4.gemm_swiglu_backward(dh, z, p, s, g, dgate_up=view(size, m, 2 * n), out=view(2 * size - 8, m, k)),
               lambda: w4.gemm_swiglu_backward(view(size, m, n), z, p, s, g, out=view(size, m, k)),      # over dy
               lambda: w4.gemm_swiglu(x, p, s, g, out=view(size - 8, m, n)),
               lambda: w4.gemm_swiglu(x, p, s, g, gate_up=view(size - 8, m, 2 * n)),
               lambda: w4.gemm_t(z, p, s, g, out=z),                                                      # 2 n == k
               lambda: w4.gemm_dscales(z, x, p, g, out=buf[:2 * 2 * n * (k // g)].view(torch.float32).view(2 * n, k // g))]
    for i, call in enumerate(refused):
        with pytest.raises(w4.W4A16Error, match="OVERLAP") as e:
            call()
        assert e.value.status == w4.ERR_OVERLAP, i
    torch.cuda.synchronize()
    assert torch.equal(buf, before)
    want = w4.gemm_swiglu_backward(dh, z.clone(), p, s, g)
    got = w4.gemm_swiglu_backward(dh, z, p, s, g, dgate_up=view(size, m, 2 * n), out=view(2 * size, m, k))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def busy(torch, work, times=12):
    """Some milliseconds of work on the current stream."""
    for _ in range(times):
        work[0] = work[0] @ work[1]


@pytest.mark.parametrize("drop", [False, True])
def test_workspace_used_on_another_stream_at_once(w4, drop):
    """Made behind other work on one stream, in memory that held other values, and used at once on a second
    stream by a call whose workgroups count their arrivals in it; then dropped while that call still waits,
    with its memory asked for again on the first stream."""
    torch = torch_mod()
    m, n, k, g = 1, 1024, 1024, 128
    rng = np.random.default_rng(62000)
    p, s = dev(w4.pack(synth.code_bank(rng, 1, n, k)[0])), dev(synth.scale_bank(rng, 1, n, k // g)[0])
    d = dev(synth.activations(rng, m, n))
    want = w4.gemm_t(d, p, s, g)
    first, second = torch.cuda.Stream(), torch.cuda.Stream()
    work = [torch.zeros((8192, 8192), dtype=torch.float16, device="cuda") for _ in range(4)]
    words = w4.ffn_workspace("gemm_t", m, n, k, g).numel()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(first):
            used = torch.full((words,), -1, dtype=torch.int32, device="cuda")
            busy(torch, work[:2])
            del used                                   # its memory goes to the next request on this stream
        ws = w4.ffn_workspace("gemm_t", m, n, k, g, stream=first)
        with torch.cuda.stream(second):
            busy(torch, work[2:])
        out = torch.full_like(want, float("nan"))
        second.wait_stream(torch.cuda.current_stream())
        w4.gemm_t(d, p, s, g, out=out, workspace=ws, stream=second)
        if drop:
            del ws
            with torch.cuda.stream(first):
                taken = torch.full((words,), -1, dtype=torch.int32, device="cuda")
        else:
            w4.gemm_t(d, p, s, g, workspace=ws, stream=second)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        if drop:
            assert bool((taken == -1).all())
        else:
            assert int(ws[:4096].abs().sum()) == 0


def test_workspace_stream_and_device_agree(w4):
    torch = torch_mod()
    side = torch.cuda.Stream()
    ws = w4.ffn_workspace("gemm_t", 1, 1024, 1024, 128, device=side.device, stream=side)
    assert ws.device == side.device and int(ws[:4096].abs().sum()) == 0
    assert w4.ffn_workspace("gemm_t", 1, 1024, 1024, 128, device="cuda").device == side.device
    g = torch.cuda.CUDAGraph()
    d = torch.ones((1, 1024), dtype=torch.float16, device="cuda")
    p, s = torch.zeros((1024, 128), dtype=torch.int32, device="cuda"), torch.ones((1024, 8), dtype=torch.float16, device="cuda")
    want = w4.gemm_t(d, p, s, 128)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):                          # made and used within one capture
        out = w4.gemm_t(d, p, s, 128, workspace=w4.ffn_workspace("gemm_t", 1, 1024, 1024, 128))
    for _ in range(3):
        out.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and float(out[0, 0]) == -8 * 1024


@pytest.mark.parametrize("m", [2, 40])
def test_operands_dropped_before_their_call_has_run(w4, m):
    """Calls queued on a busy stream given by argument, every operand dropped at once and its memory filled
    again on the stream it came from."""
    torch = torch_mod()
    n, k, g = 512, 1024, 128
    rng = np.random.default_rng(63000 + m)
    p, s = pair_weights(w4, rng, n, k, g)
    x, dh = dev(synth.activations(rng, m, k)), dev(synth.activations(rng, m, n))
    z = torch.empty((m, 2 * n), dtype=torch.float16, device="cuda")
    h = w4.gemm_swiglu(x, p, s, g, gate_up=z)
    dx, dz = w4.gemm_swiglu_backward(dh, z, p, s, g)
    want = [h, dx, dz, w4.gemm_t(z, p, s, g), w4.gemm_dscales(z, x, p, g)]
    side = torch.cuda.Stream()
    work = [torch.zeros((8192, 8192), dtype=torch.float16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            busy(torch, work)
        got = []
        copies = [t.clone() for t in (x, p, s, dh, z)]
        side.wait_stream(torch.cuda.current_stream())
        x2, p2, s2, dh2, z2 = copies
        got.append(w4.gemm_swiglu(x2, p2, s2, g, gate_up=torch.empty_like(z), stream=side))
        got.extend(w4.gemm_swiglu_backward(dh2, z2, p2, s2, g, stream=side))
        got.append(w4.gemm_t(z2, p2, s2, g, stream=side))
        got.append(w4.gemm_dscales(z2, x2, p2, g, stream=side))
        sizes = [(t.numel(), t.dtype) for t in copies]
        del copies, x2, p2, s2, dh2, z2
        again = [torch.full((count,), -1, dtype=dtype, device="cuda") for count, dtype in sizes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool((t == -1).all()) for t in again)


# split tiles on few workgroups: (call, m, n, k, group), n as ffn_workspace takes it, and the plan's sizes: tiles of
# the product, steps per tile, fewest steps of a part, fp32 values of a partial tile
SPLIT = [("gemm_t", 64, 768, 1024, 128, 4, 12, 4, 256 * 256), ("gemm_t", 300, 2003, 2080, 32, 18, 32, 4, 256 * 256),
         ("gemm_swiglu", 64, 256, 1024, 128, 2, 8, 3, 64 * 256), ("gemm_swiglu_backward", 70, 300, 544, 32, 3, 10, 4, 256 * 256),
         ("gemm_dscales", 512, 1024, 1024, 128, 16, 16, 4, 256 * 2)]


@pytest.mark.parametrize("call,m,n,k,g,tiles,steps,least,tile", SPLIT)
def test_workspace_is_as_large_as_its_split(w4, call, m, n, k, g, tiles, steps, least, tile):
    """No larger than the partial tiles of the workgroups that split tiles, and nothing behind it is written."""
    torch = torch_mod()
    rng = np.random.default_rng(64000 + m + n)
    rows = 2 * n if "swiglu" in call else n
    p, s = dev(w4.pack(synth.code_bank(rng, 1, rows, k)[0])), dev(synth.scale_bank(rng, 1, rows, k // g)[0])
    x, d, dh = (dev(synth.activations(rng, m, c)) for c in (k, rows, n))
    run = {"gemm_t": lambda **kw: w4.gemm_t(d, p, s, g, **kw), "gemm_swiglu": lambda **kw: w4.gemm_swiglu(x, p, s, g, **kw),
           "gemm_swiglu_backward": lambda **kw: w4.gemm_swiglu_backward(dh, d, p, s, g, **kw)[0],
           "gemm_dscales": lambda **kw: w4.gemm_dscales(d, x, p, g, **kw)}[call]
    words = w4.ffn_workspace(call, m, n, k, g).numel()
    buf = torch.full((words + 65536,), 77, dtype=torch.int32, device="cuda")
    ws = buf[:words]
    ws[:4096] = 0
    want = run()
    assert torch.equal(run(workspace=ws), want) and bool((buf[words:] == 77).all())
    # two places for each workgroup that may split: of the 8 dies, each with its share of the tiles, one per `least` steps;
    # behind them a left side with padded rows
    per_die = min(32, -(-tiles // 8) * steps // least)
    assert words <= 4096 + 16 * per_die * tile + m * (rows + 8) // 2 + 64


def test_kept_workspaces_are_bounded_and_released(w4):
    torch = torch_mod()
    d = torch.ones((1, 1024), dtype=torch.float16, device="cuda")
    p, s = torch.zeros((1024, 128), dtype=torch.int32, device="cuda"), torch.ones((1024, 8), dtype=torch.float16, device="cuda")
    want = w4.gemm_t(d, p, s, 128)
    torch.cuda.synchronize()
    # more handles than torch's pool of streams has, as a program with streams of its own may use
    kept = w4._FFN_WORKSPACES.of
    for i in range(100):
        kept[(0, -1 - i)] = kept[(0, torch.cuda.current_stream().cuda_stream)]
    side = torch.cuda.Stream()
    assert torch.equal(w4.gemm_t(d, p, s, 128, stream=side), want)
    assert len(kept) <= 32 and (0, side.cuda_stream) in kept
    side.synchronize()
    w4.ffn_release_workspaces()
    assert not kept
    assert torch.equal(w4.gemm_t(d, p, s, 128), want)


@pytest.mark.parametrize("m", [1, 20, 70])
def test_no_input_features(w4, m):
    """k == 0: empty sums, zeros; the pairs' gradient does not depend on k."""
    torch = torch_mod()
    n, g = 24, 32
    f16 = dict(dtype=torch.float16, device="cuda")
    p0, s0, x0 = torch.zeros((2 * n, 0), dtype=torch.int32, device="cuda"), torch.zeros((2 * n, 0), **f16), torch.zeros((m, 0), **f16)
    z = torch.full((m, 2 * n), float("nan"), **f16)
    h = w4.gemm_swiglu(x0, p0, s0, g, gate_up=z)
    assert torch.equal(h, torch.zeros((m, n), **f16)) and torch.equal(z, torch.zeros((m, 2 * n), **f16))
    rng = np.random.default_rng(65000 + m)
    p, s = pair_weights(w4, rng, n, 32, g)
    z, dh = dev(synth.activations(rng, m, 2 * n)), dev(synth.activations(rng, m, n))
    want = w4.gemm_swiglu_backward(dh, z, p, s, g)[1]
    dx, dz = w4.gemm_swiglu_backward(dh, z, p0, s0, g)
    assert dx.shape == (m, 0) and torch.equal(dz, want)
    assert w4.gemm_t(z, p0, s0, g).shape == (m, 0) and w4.gemm_dscales(z, x0, p0, g).shape == (2 * n, 0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("m", [2, 150])
def test_captured_on_a_forked_stream(w4, m):
    """A capture that forks: one branch's calls on a stream given by argument, their inputs made (and dropped)
    on the capturing stream, one of them with a workspace of its own."""
    torch = torch_mod()
    n, k, g = 512, 1024, 128
    rng = np.random.default_rng(66000 + m)
    p, s = pair_weights(w4, rng, n, k, g)
    x, dh = dev(synth.activations(rng, m, k)), dev(synth.activations(rng, m, n))
    side = torch.cuda.Stream()

    def step(fork):
        z = torch.empty((m, 2 * n), dtype=torch.float16, device="cuda")
        h = w4.gemm_swiglu(x, p, s, g, gate_up=z)
        twice = dh * 2
        if fork:
            side.wait_stream(torch.cuda.current_stream())
            dx, dz = w4.gemm_swiglu_backward(twice, z, p, s, g, stream=side)
            del twice
            ws = w4.ffn_workspace("gemm_t", m, 2 * n, k, g)
            t = w4.gemm_t(z, p, s, g, workspace=ws)
            torch.cuda.current_stream().wait_stream(side)
        else:
            dx, dz = w4.gemm_swiglu_backward(twice, z, p, s, g)
            t = w4.gemm_t(z, p, s, g)
        return h, dx, dz, t

    want = [t.clone() for t in step(False)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(True)
    for rep in range(4):
        x.copy_(torch.randn_like(x))
        want = step(False)
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), f"replay {rep}"
