"""The product with the weights' other side (y = d . deq(W)) against the fp64 definition.

Bars (fixed before the first run): the oracle's (per element 4e-3 of the largest, per
row 1e-3 in relative L2).  Two roundings of half a step 2^-11 enter, the fp16 operand
s q and the output, together at most sqrt(2) 2^-11 / sqrt(3) = 4e-4 of a row's norm.
Integers with power-of-two scales are exact until the output and must match bit for bit.
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


def reference(d, q, s, group):
    return d.astype(np.float64) @ oracle.dequantize(q, s, group)


# (m, n, k, group): single rows to several tiles, n of one, odd and no multiple of 8 or of
# a step, k below, at and past a tile, one step and many.
CASES = [(1, 1, 32, 32), (1, 1000, 1024, 128), (2, 63, 384, 128), (5, 300, 96, 32), (16, 129, 1056, 32),
         (17, 2048, 256, 128), (33, 513, 2080, 32), (64, 72, 4096, 128), (65, 1001, 640, 128), (130, 64, 160, 32),
         (257, 2003, 2080, 32), (300, 1016, 768, 128), (1000, 4104, 512, 128), (2050, 200, 8448, 128), (3, 17408, 5120, 128), (31, 5120, 1760, 32), (50, 2500, 8192, 32),
         (8, 40, 70016, 128)]


@pytest.mark.parametrize("m,n,k,group", CASES)
def test_exact_on_integers(w4, m, n, k, group):
    rng = np.random.default_rng(31000 + m + n + k)
    q = synth.integer_codes(rng, n, k)
    s = synth.power_of_two_scales(rng, n, k // group, lo=-5, hi=-3)
    d = synth.integer_activations(rng, m, n)
    y = w4.gemm_t(dev(d), dev(w4.pack(q)), dev(s), group)
    torch_mod().cuda.synchronize()
    assert_bit_exact(host(y), reference(d, q, s, group), f"m={m} n={n} k={k} g={group}")


@pytest.mark.parametrize("m,n,k,group", CASES[1:])
def test_gaussian(w4, m, n, k, group):
    rng = np.random.default_rng(32000 + m + n + k)
    q, s = synth.code_bank(rng, 1, n, k)[0], synth.scale_bank(rng, 1, n, k // group)[0]
    d = synth.activations(rng, m, n)
    y = w4.gemm_t(dev(d), dev(w4.pack(q)), dev(s), group)
    torch_mod().cuda.synchronize()
    assert_close(host(y), reference(d, q, s, group), f"m={m} n={n} k={k} g={group}")


@pytest.mark.parametrize("m,n", [(5, 63), (17, 37), (3, 257), (40, 63), (9, 62)])
def test_rows_do_not_see_their_neighbours(w4, m, n):
    """Rows that start inside a dword or a chunk: infinities and NaN of one row stay in it."""
    rng = np.random.default_rng(34000 + m + n)
    k, group = 96, 32
    q, s = synth.code_bank(rng, 1, n, k)[0], synth.scale_bank(rng, 1, n, k // group)[0]
    d = synth.activations(rng, m, n)
    p, s_d = dev(w4.pack(q)), dev(s)
    want = host(w4.gemm_t(dev(d), p, s_d, group))
    for row in (1, m // 2, m - 1):
        bad = d.copy()
        bad[row, :] = np.inf
        bad[row, -1] = np.nan
        got = host(w4.gemm_t(dev(bad), p, s_d, group))
        others = np.arange(m) != row
        assert np.array_equal(got[others].view(np.uint16), want[others].view(np.uint16))
        assert np.isnan(got[row]).all()


# tiles of one or two steps (not split), more of them than workgroups, a partial last round
@pytest.mark.parametrize("m,n,k,group", [(33, 1, 32, 32), (4100, 72, 4992, 32), (4100, 33, 4992, 128)])
def test_exact_on_integers_few_steps(w4, m, n, k, group):
    test_exact_on_integers(w4, m, n, k, group)
