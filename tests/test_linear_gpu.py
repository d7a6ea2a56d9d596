"""The linear layer with bias, activation and residual, and its backward pass, against the fp64 formulas.

Bars (fixed before the first run).  y: with size = sum |x w| and slope <= 1.13 (the largest slope of
any of the activations), |err| <= 2^-11 |y| (the one rounding) + 1.13 (2^-11 + (k + 64) 2^-24) size (weights
at worst fp16(s q), half a step each; fp32 additions) + 2^-18 (|z| + |y| + 1) (exponentials and the formula's
terms at fp32, with room) + 2^-25 (half the smallest subnormal).  z: the same without the activation's terms.
Integer inputs with act none or relu: every partial sum is exact, so y and z are the rounded exact values.  dpre:
|err| <= 2^-11 |v| + 2^-18 |dy| (1 + |z|) + 2^-25.  dbias: fp32 sums of the unrounded values, |err| <=
(rows + 32) 2^-23 sum |v| + 2^-18 sum |dy| (1 + |z|).  dx: the oracle's bars on the fp16 dpre the call returned.
"""

import math

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_close, dev, host, torch_mod

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def erf(z):
    return np.vectorize(math.erf, otypes=[np.float64])(z)


def act64(name, z):
    if name == "relu":
        return np.maximum(z, 0)
    if name == "silu":
        return z / (1 + np.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def slope64(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return np.ones_like(z)


def weights(rng, n, k, group):
    return synth.code_bank(rng, 1, n, k)[0], synth.scale_bank(rng, 1, n, k // group)[0]


def aligned_away(w4, scales, shift):
    """The scales on the device, `shift` elements past a 16-byte boundary."""
    torch = torch_mod()
    buf = torch.empty(scales.size + 16, dtype=torch.float16, device="cuda")
    view = buf[shift:shift + scales.size].view(scales.shape)
    view.copy_(dev(scales))
    return view


def check_linear(w4, m, n, k, group, act, bias, residual, keep, seed, shift=0):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    q, s = weights(rng, n, k, group)
    x = synth.activations(rng, m, k)
    b = (synth.activations(rng, 1, n)[0] * np.float16(0.5)).astype(np.float16) if bias else None
    r = synth.activations(rng, m, n) if residual else None
    sd = aligned_away(w4, s, shift) if shift else dev(s)
    pre = torch.full((m, n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    y = w4.linear(dev(x), dev(w4.pack(q)), sd, group, bias=dev(b) if bias else None, activation=act,
                  residual=dev(r) if residual else None, pre=pre)
    torch.cuda.synchronize()
    w = oracle.dequantize(q, s, group)
    x64 = x.astype(np.float64)
    z = x64 @ w.T
    size = np.abs(x64) @ np.abs(w).T
    if bias:
        z = z + b.astype(np.float64)
    want = act64(act, z)
    if residual:
        want = want + r.astype(np.float64)
    sums = (2.0 ** -11 + (k + 64) * 2.0 ** -24) * size + 2.0 ** -25
    got = host(y).astype(np.float64)
    bar = 2.0 ** -11 * np.abs(want) + 1.13 * sums + 2.0 ** -18 * (np.abs(z) + np.abs(want) + 1)
    bad = np.argwhere(~(np.abs(got - want) <= bar))
    assert bad.size == 0, f"{len(bad)} of {got.size} outputs wrong, first {tuple(bad[0])}: {got[tuple(bad[0])]} want {want[tuple(bad[0])]}"
    if keep:
        zg = host(pre).astype(np.float64)
        bad = np.argwhere(~(np.abs(zg - z) <= 2.0 ** -11 * np.abs(z) + sums))
        assert bad.size == 0, f"{len(bad)} of {zg.size} pre-activations wrong, first {tuple(bad[0])}"


# (m, n, k, group): each kernel's sizes (one row; 2-4; weight-streaming up to 16 and 32; tiles of 64 and of 128
# rows), single outputs, odd n, K tails, split tiles, many tiles
SIZES = [(1, 1, 32, 32), (1, 1003, 1056, 32), (1, 520, 2176, 128), (2, 9, 96, 32), (3, 1001, 640, 128), (4, 2000, 1024, 32),
         (5, 17, 32, 32), (16, 999, 2080, 32), (17, 2003, 512, 128), (32, 64, 4128, 32), (33, 130, 416, 32),
         (64, 515, 2048, 128), (65, 257, 256, 128), (130, 1000, 1120, 32), (300, 520, 2048, 128), (257, 33, 160, 32)]


@pytest.mark.parametrize("m,n,k,group", SIZES)
def test_linear_sizes(w4, m, n, k, group):
    act = ACTS[(m + n) % 5]
    check_linear(w4, m, n, k, group, act, bias=True, residual=m % 2 == 1, keep=m % 3 != 0, seed=61000 + m + n + k)


@pytest.mark.parametrize("m", [1, 3, 20, 40, 200])
@pytest.mark.parametrize("act", ACTS)
def test_linear_activations(w4, m, act):
    """Each activation on each kernel, with and without each of the other operands."""
    i = ACTS.index(act)
    check_linear(w4, m, 264, 256, 128, act, bias=i % 2 == 0, residual=i % 3 == 0, keep=i % 2 == 1, seed=62000 + 7 * m + i)
    check_linear(w4, m, 131, 288, 32, act, bias=i % 3 != 0, residual=True, keep=True, seed=62500 + 7 * m + i)


@pytest.mark.parametrize("m", [1, 2, 9, 50, 140])
def test_linear_unaligned_scales(w4, m):
    for group, k in ((32, 1024), (128, 640)):
        check_linear(w4, m, 300, k, group, "silu", True, True, False, 63000 + m, shift=1)


# one row past the on-chip row buffers, and two: the weight-streaming kernel takes over
@pytest.mark.parametrize("m,k", [(1, 40960), (4, 24576)])
def test_linear_long_rows(w4, m, k):
    check_linear(w4, m, 40, k, 128, "none", True, True, False, 64000 + m)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("m,n,k,group", [(1, 77, 256, 32), (4, 300, 128, 128), (13, 64, 544, 32), (29, 131, 256, 128),
                                         (50, 263, 1056, 32), (260, 520, 896, 128)])
def test_linear_is_exact_on_integers(w4, m, n, k, group, act):
    torch = torch_mod()
    rng = np.random.default_rng(65000 + m)
    q = synth.integer_codes(rng, n, k)
    s = np.ones((n, k // group), np.float16)
    x = synth.integer_activations(rng, m, k)
    b = rng.integers(-8, 9, n).astype(np.float16)
    r = rng.integers(-64, 65, (m, n)).astype(np.float16)
    pre = torch.empty((m, n), dtype=torch.float16, device="cuda")
    y = host(w4.linear(dev(x), dev(w4.pack(q)), dev(s), group, bias=dev(b), activation=act, residual=dev(r), pre=pre))
    z = x.astype(np.int64) @ q.astype(np.int64).T + b.astype(np.int64)
    want = (np.maximum(z, 0) if act == "relu" else z) + r.astype(np.int64)
    assert np.array_equal(host(pre), z.astype(np.float16))
    assert np.array_equal(y, want.astype(np.float16))


@pytest.mark.parametrize("m", [1, 4, 16, 31, 64, 190])
def test_linear_into_the_residual(w4, m):
    """residual and out are one tensor: the residual stream is updated in place, as the separate call computes it."""
    rng = np.random.default_rng(66000 + m)
    n, k, group = 333, 1280, 128
    q, s = weights(rng, n, k, group)
    x, r = dev(synth.activations(rng, m, k)), dev(synth.activations(rng, m, n))
    p, sd = dev(w4.pack(q)), dev(s)
    want = w4.linear(x, p, sd, group, activation="gelu", residual=r).clone()
    got = w4.linear(x, p, sd, group, activation="gelu", residual=r, out=r)
    assert got.data_ptr() == r.data_ptr() and np.array_equal(host(got).view(np.uint16), host(want).view(np.uint16))


@pytest.mark.parametrize("m", [1, 3, 12, 60, 129])
def test_linear_without_epilogue_is_the_product(w4, m):
    """No bias, activation or residual: within a rounding of the plain product's bars."""
    rng = np.random.default_rng(67000 + m)
    q, s = weights(rng, 200, 512, 128)
    x = synth.activations(rng, m, 512)
    assert_close(host(w4.linear(dev(x), dev(w4.pack(q)), dev(s), 128)), x.astype(np.float64) @ oracle.dequantize(q, s, 128).T)


@pytest.mark.parametrize("m", [1, 4, 30, 70])
def test_linear_special_values(w4, m):
    """An infinite activation, bias or residual reaches its own row or column alone; relu keeps NaN."""
    torch = torch_mod()
    rng = np.random.default_rng(68000 + m)
    n, k, group = 96, 256, 128
    q, s = weights(rng, n, k, group)
    x = synth.activations(rng, m, k)
    b, r = np.zeros(n, np.float16), synth.activations(rng, m, n)
    b[5], r[m - 1, 7], r[0, 9] = np.inf, -np.inf, np.nan
    y = host(w4.linear(dev(x), dev(w4.pack(q)), dev(s), group, bias=dev(b), activation="relu", residual=dev(r)))
    assert np.all(np.isposinf(y[:, 5])) and np.isneginf(y[m - 1, 7]) and np.isnan(y[0, 9])
    ok = np.ones_like(y, bool)
    ok[:, 5], ok[m - 1, 7], ok[0, 9] = False, False, False
    assert np.all(np.isfinite(y[ok]))
    x[0, 3] = np.nan
    y = host(w4.linear(dev(x), dev(w4.pack(q)), dev(s), group, activation="relu"))
    assert np.all(np.isnan(y[0])) and np.all(np.isfinite(y[1:]))
    # far tails of every activation: 0 or the value itself
    z = np.array([-60000, -200, -30, 30, 200, 60000], np.float16)
    w1, s1 = np.zeros((6, 128), np.int8), np.ones((6, 1), np.float16)
    xm = np.zeros((m, 128), np.float16)
    for act in ACTS[2:]:
        y = host(w4.linear(dev(xm), dev(w4.pack(w1)), dev(s1), 128, bias=dev(z), activation=act)).astype(np.float64)
        assert np.all(np.abs(y[:, :3]) <= 1e-9) and np.array_equal(y[:, 3:], np.tile(z[3:].astype(np.float64), (m, 1))), act
    torch.cuda.synchronize()


def test_linear_leaves_its_neighbours(w4):
    """Nothing is written outside y and pre: guard rows before and behind keep their values."""
    torch = torch_mod()
    rng = np.random.default_rng(69000)
    for m, n, k, group in ((1, 40, 96, 32), (3, 9, 128, 128), (18, 50, 64, 32), (45, 70, 256, 128), (140, 264, 288, 32)):
        q, s = weights(rng, n, k, group)
        x = synth.activations(rng, m, k)
        bufs = [torch.full(((m * n + 7) // 8 * 8 + 1024,), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
        views = [t[512:512 + m * n].view(m, n) for t in bufs]
        w4.linear(dev(x), dev(w4.pack(q)), dev(s), group, activation="silu", out=views[0], pre=views[1])
        for t in bufs:
            assert bool((t[:512] == 7).all()) and bool((t[512 + m * n:] == 7).all())


# ---- backward ----
BACK = [(1, 1, 32, 32), (1, 500, 1024, 128), (3, 77, 416, 32), (19, 1001, 1120, 32), (40, 1003, 640, 128), (129, 136, 256, 32),
        (300, 300, 256, 128), (700, 129, 96, 32)]


@pytest.mark.parametrize("m,n,k,group", BACK)
@pytest.mark.parametrize("act", ACTS)
def test_linear_backward(w4, m, n, k, group, act):
    rng = np.random.default_rng(71000 + m + n + k)
    q, s = weights(rng, n, k, group)
    z = (synth.activations(rng, m, n) * np.float16(1.5)).astype(np.float16)
    z[0, 0], z[-1, -1] = -30, 25
    if n > 4:
        z[0, 1], z[0, 2], z[0, 3] = 0, 60000, -60000
    dy = (synth.activations(rng, m, n) * np.float16(0.25)).astype(np.float16)
    has = act != "none"
    dx, dpre, dbias = w4.linear_backward(dev(dy), dev(w4.pack(q)), dev(s), group, pre=dev(z) if has else None, activation=act,
                                         dbias=True)
    torch_mod().cuda.synchronize()
    dy64, z64 = dy.astype(np.float64), z.astype(np.float64)
    v = dy64 * slope64(act, z64)
    slack = 2.0 ** -18 * np.abs(dy64) * (1 + np.minimum(np.abs(z64), 100)) if has else 0 * v
    if has:
        got = host(dpre).astype(np.float64)
        assert np.all(np.abs(got - v) <= 2.0 ** -11 * np.abs(v) + slack + 2.0 ** -25)
    else:
        assert dpre is None
        got = dy64
    assert np.all(np.abs(host(dbias) - v.sum(axis=0)) <= (m + 32) * 2.0 ** -23 * np.abs(v).sum(axis=0) + slack.sum(axis=0) + 1e-30)
    assert_close(host(dx), got @ oracle.dequantize(q, s, group), "dx")
    # without the bias's gradient: the same bits
    dx2, dpre2, none = w4.linear_backward(dev(dy), dev(w4.pack(q)), dev(s), group, pre=dev(z) if has else None, activation=act)
    assert none is None and np.array_equal(host(dx2).view(np.uint16), host(dx).view(np.uint16))
    if has:
        assert np.array_equal(host(dpre2).view(np.uint16), host(dpre).view(np.uint16))


@pytest.mark.parametrize("act", ACTS[1:])
def test_linear_gradient_against_differences(w4, act):
    """Central differences of sum(y dy) in x and in the bias, in fp64 by the definition, against the library's chain."""
    torch = torch_mod()
    rng = np.random.default_rng(72000)
    m, n, k, group = 21, 40, 64, 32
    q, s = weights(rng, n, k, group)
    s = (s * np.float16(4)).astype(np.float16)
    x, dy = synth.activations(rng, m, k), synth.activations(rng, m, n)
    b = (synth.activations(rng, 1, n)[0] * np.float16(0.5)).astype(np.float16)
    pre = torch.empty((m, n), dtype=torch.float16, device="cuda")
    p, sd = dev(w4.pack(q)), dev(s)
    w4.linear(dev(x), p, sd, group, bias=dev(b), activation=act, pre=pre)
    dx, _, dbias = w4.linear_backward(dev(dy), p, sd, group, pre=pre, activation=act, dbias=True)
    w = oracle.dequantize(q, s, group)
    dy64 = dy.astype(np.float64)
    rows = lambda xv, bv: np.sum(act64(act, xv @ w.T + bv) * dy64, axis=1)  # noqa: E731
    x64, b64, step = x.astype(np.float64), b.astype(np.float64), 1e-5
    diff = np.empty_like(x64)
    for j in range(k):
        e = np.zeros(k); e[j] = step
        diff[:, j] = (rows(x64 + e, b64) - rows(x64 - e, b64)) / (2 * step)
    # pre, dpre and dx are rounded to fp16 and the weights once: 4 half steps per row (the second derivative
    # is at most 1.2); relu's slope jumps where a pre-activation lies within its own rounding of 0
    err = np.linalg.norm(host(dx) - diff, axis=1) / np.linalg.norm(diff, axis=1)
    assert err.max() <= 4 * 2.0 ** -11
    db = np.empty(n)
    for j in range(n):
        e = np.zeros(n); e[j] = step
        db[j] = np.sum(rows(x64, b64 + e) - rows(x64, b64 - e)) / (2 * step)
    z = x64 @ w.T + b64
    # pre's rounding seen through the second derivative, per row: 1.2 2^-11 |z| |dy|, doubled
    bar = 2.4 * 2.0 ** -11 * np.sum(np.abs(z * dy64), axis=0) + 1e-6 * np.sum(np.abs(dy64), axis=0)
    assert np.all(np.abs(host(dbias) - db) <= bar)
