"""The gate/up SwiGLU product for any number of rows, and its kept products, against the fp64 oracle.

Bars (fixed before the first run): the oracle's (per element 4e-3 of the largest,
per row 1e-3 in relative L2).  Three roundings of half a step 2^-11 enter a row:
each weight q s (fp16 operand), seen once through u and once through g with
|g SiLU'(g)| of the size of |SiLU(g)|, and the output; independent, they add to at
most sqrt(3) 2^-11 / sqrt(3) = 4.9e-4 of the row's norm.  Integer inputs with
power-of-two scales have no rounding before the output: the kept products must be
bit-exact there.
"""

import numpy as np
import pytest

import oracle
import synth
from gpu_util import assert_bit_exact, assert_close, dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    torch_mod()
    import w4a16_int4_weight_linear_amd as w4
    return w4


def codes_and_scales(rng, rows, k, group):
    return synth.code_bank(rng, 1, rows, k)[0], synth.scale_bank(rng, 1, rows, k // group)[0]


# (m, n outputs, k, group): decode, weight-streaming and tiled sizes, ragged n, a K
# tail inside a step, scale rows that are not 16-byte aligned, fewer and more tiles
# than workgroups.
CASES = [(1, 300, 2080, 32), (4, 129, 640, 128), (9, 33, 384, 128), (16, 777, 1536, 32), (17, 512, 2048, 32),
         (32, 65, 416, 32), (33, 1000, 1280, 128), (130, 77, 2080, 32), (300, 1003, 640, 128), (1000, 2176, 1024, 128)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,group", CASES)
def test_swiglu_any_rows(w4, m, n, k, group, keep):
    torch = torch_mod()
    rng = np.random.default_rng(21000 + m + n + k)
    q, s = codes_and_scales(rng, 2 * n, k, group)
    x = synth.activations(rng, m, k)
    p = w4.pack(q)
    z = torch.full((m, 2 * n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    y = w4.gemm_swiglu(dev(x), dev(p), dev(s), group, gate_up=z)
    torch.cuda.synchronize()
    what = f"m={m} n={n} k={k} g={group}"
    assert_close(host(y), oracle.swiglu_linear(x, oracle.pack(q), s, group), what)
    if keep:
        assert_close(host(z), oracle.linear(x, oracle.pack(q), s, group), what + " kept products")


@pytest.mark.parametrize("m,n,k,group", [(13, 40, 256, 128), (77, 150, 1056, 32), (513, 600, 768, 128)])
def test_kept_products_are_bit_exact_on_integers(w4, m, n, k, group):
    torch = torch_mod()
    rng = np.random.default_rng(22000 + m)
    q = synth.integer_codes(rng, 2 * n, k)
    s = synth.power_of_two_scales(rng, 2 * n, k // group, lo=-6, hi=-3)
    x = synth.integer_activations(rng, m, k)
    z = torch.empty((m, 2 * n), dtype=torch.float16, device="cuda")
    y1 = host(w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s), group, gate_up=z))
    assert_bit_exact(host(z), oracle.linear(x, oracle.pack(q), s, group), f"m={m}")
    # again, without keeping: the same bits
    y2 = host(w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s), group))
    if m > 16:      # up to 16 rows the call without kept products may run another kernel
        assert np.array_equal(y1.view(np.uint16), y2.view(np.uint16))
    s0 = s.copy(); s0[1::2] = 0
    assert np.all(host(w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s0), group)).astype(np.float64) == 0)


def test_large_negative_and_infinite_gates(w4):
    """SiLU at the ends: g far below zero gives (minus) zero, an infinite product is carried, no NaN appears of itself."""
    torch = torch_mod()
    n, k, group, m = 64, 128, 128, 40
    q = np.zeros((2 * n, k), np.int8); q[:, 0] = 1
    s = np.ones((2 * n, 1), np.float16)
    x = np.zeros((m, k), np.float16)
    x[:, 0] = np.linspace(-60000, 60000, m).astype(np.float16)
    y = host(w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s), group)).astype(np.float64)
    with np.errstate(over="ignore"):
        want = oracle.swiglu_linear(x, oracle.pack(q), s, group).astype(np.float16).astype(np.float64)
    neg = x[:, 0] < -200
    assert np.all(y[neg] == 0) and np.array_equal(np.isinf(y), np.isinf(want)) and not np.isnan(y).any()
    torch.cuda.synchronize()


# tiles of 64 rows: full and ragged, split and whole, and few rows of weights too large for two passes
TILES_64 = [(33, 600, 2080, 32), (63, 2176, 1024, 128), (64, 1003, 1280, 128), (64, 8192, 1056, 32), (20, 8200, 4096, 128)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,group", TILES_64)
def test_swiglu_tiles_of_64_rows(w4, m, n, k, group, keep):
    test_swiglu_any_rows(w4, m, n, k, group, keep)


# tiles of one to three steps (not split), the last with more tiles than workgroups and a partial last round
FEW_STEPS = [(40, 5, 32, 32), (33, 1, 128, 128), (70, 300, 96, 32), (200, 9, 384, 128), (2000, 2500, 256, 128)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k,group", FEW_STEPS)
def test_swiglu_few_steps(w4, m, n, k, group, keep):
    """Sums so short that roundings do not average out and rows so short that one cancelled product is a
    row: the bar is the arithmetic itself.  Weights enter as fp16(q s), each off by at most 2^-11 of
    itself, so a product z = sum x w is off by dz <= 2^-11 sum |x w| (and fp32 sums of up to 384 terms by
    2^-15 of that, within the factor 1 + 2^-4).  |SiLU'| <= 1.1, so h = SiLU(g) u is off by at most
    1.1 dg (|u| + du) + |SiLU(g)| du, and its rounding adds 2^-11 |h| (fp32 SiLU: within 2^-4 of that);
    results below 2^-14 round by 2^-25."""
    torch = torch_mod()
    rng = np.random.default_rng(21000 + m + n + k)
    q, s = codes_and_scales(rng, 2 * n, k, group)
    x = synth.activations(rng, m, k)
    z = torch.full((m, 2 * n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    h = host(w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s), group, gate_up=z)).astype(np.float64)
    w, x64 = oracle.dequantize(q, s, group).astype(np.float64), x.astype(np.float64)
    z64, half = x64 @ w.T, 2.0 ** -11 * (1 + 2.0 ** -4)
    dz = half * (np.abs(x64) @ np.abs(w).T)
    g, u, dg, du = z64[:, 0::2], z64[:, 1::2], dz[:, 0::2], dz[:, 1::2]
    silu = g / (1 + np.exp(-g))
    want = silu * u
    assert np.all(np.abs(h - want) <= 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + half * np.abs(want) + 2.0 ** -24)
    if keep:
        assert np.all(np.abs(host(z).astype(np.float64) - z64) <= dz + half * np.abs(z64) + 2.0 ** -24)
