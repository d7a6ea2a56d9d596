"""The gate/up SwiGLU product: kernel instances that the ragged cases of its other tests miss (group 32
with whole steps of 128, scale rows on 16-byte boundaries and off them, tiles of 64 and 128 rows, split
and whole), and the precision with which weights enter where the library promises exact ones.

Bars (fixed before the first run).  Values: the oracle's, as derived for the product's other tests.
Exact weights: the share of kept products that are not the fp16 value nearest to the exact one, at
most 4%.  With exact weights a kept product z of standard deviation t differs from the exact one by
fp32 sums alone: with an addition for every four of 2048 products, each off by at most a step 2^-23 of a
partial sum (of size t / sqrt(2) on average), independently, e = sqrt(512) 2^-23 t / sqrt(2) / sqrt(3) =
2^-20 t.  A value moves to another neighbour with probability at most 2 e / (its fp16 step), and
the step is at least 2^-11 |z|: over a Gaussian z that is 2 pdf(0) t (c + c ln(1 / c)) with c = 2 e 2^11 / t
= 2^-8, i.e. 2.1%; twice that for the tails of the assumptions.  Weights rounded to fp16(q s), each off
by 2^-12 of itself on average, give c = 0.7 and a share near 40%.

Up to 16 rows at group 128 with scale rows on their boundary, codes enter the sums on top of a bias 2^10
times their unit, taken off group by group, so the sums are not those of products of z's size and the
derivation above does not hold: a group's sums are of size sqrt(64) 2^-10 = 2^-7 (x of size 1; the bias of
every second k), its 32 additions off by sqrt(32) 2^-23 2^-7 / sqrt(6) = 2^-28.8, in units of the codes'
2^-20 by 2^-8.8, over 16 groups by 2^-6.8, against z of size 4.3 sqrt(2048) = 2^7.6: e = 2^-14.4 t =
0.5e-4 t.  There the bar is the relative error over all values.  Rounding z to fp16 alone gives
sqrt(E[v^-2] / 12) 2^-10 = 2.1e-4 (v: the mantissa, log-uniform; 2.3e-4 for the unluckiest place of t in
its octave), with e 2.35e-4; weights rounded to fp16(q s), exact for the codes 1, 2 and 4 only, add 1.9e-4,
together 2.8e-4.  The bar is 2.4e-4.
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


def inputs(m, n, k, group, seed):
    rng = np.random.default_rng(seed)
    q, s = synth.code_bank(rng, 1, 2 * n, k)[0], synth.scale_bank(rng, 1, 2 * n, k // group)[0]
    return q, s, synth.activations(rng, m, k)


def unaligned(s):
    """The scales two bytes past a 16-byte boundary."""
    torch = torch_mod()
    buf = torch.empty(s.size + 8, dtype=torch.float16, device="cuda")
    view = buf[1:1 + s.size].view(*s.shape)
    view.copy_(dev(s))
    return view


# (m, n outputs, k): 64-row tiles split and whole, 128-row tiles split and whole; k / 32 a multiple of 8 (2048, 256) or not
# (384, 640); n no multiple of 8 or of a tile
G32_TILES = [(40, 300, 2048), (64, 8300, 384), (33, 129, 640), (70, 515, 2048), (130, 77, 384), (1500, 600, 256), (300, 1003, 640)]


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("m,n,k", G32_TILES)
def test_group_32_in_whole_steps(w4, m, n, k, off, keep):
    torch = torch_mod()
    q, s, x = inputs(m, n, k, 32, 71000 + m + n + k)
    z = torch.full((m, 2 * n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    y = w4.gemm_swiglu(dev(x), dev(w4.pack(q)), unaligned(s) if off else dev(s), 32, gate_up=z)
    what = f"m={m} n={n} k={k} off={off}"
    assert_close(host(y), oracle.swiglu_linear(x, oracle.pack(q), s, 32), what)
    if keep:
        assert_close(host(z), oracle.linear(x, oracle.pack(q), s, 32), what + " kept products")


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("m,n,k", [(40, 300, 1024), (130, 77, 640), (20, 129, 384), (9, 300, 640)])
def test_group_128_with_scales_off_their_boundary(w4, m, n, k, keep):
    torch = torch_mod()
    q, s, x = inputs(m, n, k, 128, 72000 + m + n + k)
    z = torch.full((m, 2 * n), float("nan"), dtype=torch.float16, device="cuda") if keep else None
    y = w4.gemm_swiglu(dev(x), dev(w4.pack(q)), unaligned(s), 128, gate_up=z)
    assert_close(host(y), oracle.swiglu_linear(x, oracle.pack(q), s, 128), f"m={m} n={n} k={k}")
    if keep:
        assert_close(host(z), oracle.linear(x, oracle.pack(q), s, 128), f"m={m} n={n} k={k} kept products")


# group 128: the tiles of 64 and 128 rows and the weight-streaming kernel; group 32: the weight-streaming kernel
@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("m,n,k,group", [(40, 512, 2048, 128), (300, 512, 1024, 128), (16, 512, 2048, 128), (17, 512, 2048, 32),
                                         (5, 512, 1056, 32)])
def test_kept_products_have_exact_weights(w4, m, n, k, group, off):
    torch = torch_mod()
    q, s, x = inputs(m, n, k, group, 73000 + m + n + k)
    z = torch.empty((m, 2 * n), dtype=torch.float16, device="cuda")
    w4.gemm_swiglu(dev(x), dev(w4.pack(q)), unaligned(s) if off else dev(s), group, gate_up=z)
    exact = x.astype(np.float64) @ oracle.dequantize(q, s, group).astype(np.float64).T
    if group == 128 and m <= 16 and not off:
        error = np.linalg.norm(host(z).astype(np.float64) - exact) / np.linalg.norm(exact)
        assert error <= 2.4e-4, f"relative error {error:.2e}"
        return
    want = exact.astype(np.float16)
    share = np.mean(host(z) != want)
    assert share <= 0.04, f"{100 * share:.2f}% of the kept products are not the nearest fp16"
