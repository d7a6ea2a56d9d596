"""The SwiGLU block's backward pass and the scales' gradient against the fp64 formulas and against differences.

Bars (fixed before the first run).  dgate_up: one fp32 formula of about ten operations
rounded to fp16, so within one unit of 2^-10 of the formula's terms: |err| <= 2^-10
|value| + 2^-17 |dy| (|u| + 1)(1 + |g|) + 2^-25 (the terms that cancel in 1 + g (1 - sig), at
fp32 precision with room, and half the smallest subnormal).  dx: as the transposed
product (the oracle's bars) on the fp16 dgate_up the call returned.  dscales: fp32
sums of exact products, |err| <= (m + group) 2^-22 sum |q d x| (m + group additions
of half a step 2^-24 each, a factor 4 for the matrix cores' inner sums).
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


def pair_gradient(dy, z):
    dy, z = dy.astype(np.float64), z.astype(np.float64)
    g, u = z[:, 0::2], z[:, 1::2]
    sig = 1 / (1 + np.exp(-g))
    out = np.empty_like(z)
    out[:, 0::2] = dy * u * sig * (1 + g * (1 - sig))
    out[:, 1::2] = dy * g * sig
    return out


# (m, n outputs, k, group): single rows, odd n (rows of 2 n that are no multiple of 8), K tails
CASES = [(1, 1, 32, 32), (1, 500, 1024, 128), (3, 77, 416, 32), (19, 512, 2048, 32), (40, 1003, 640, 128),
         (130, 64, 1056, 32), (300, 300, 256, 128)]


@pytest.mark.parametrize("m,n,k,group", CASES)
def test_block_backward(w4, m, n, k, group):
    rng = np.random.default_rng(41000 + m + n + k)
    q, s = synth.code_bank(rng, 1, 2 * n, k)[0], synth.scale_bank(rng, 1, 2 * n, k // group)[0]
    z = (synth.activations(rng, m, 2 * n) * np.float16(1.5)).astype(np.float16)
    z[0, :2] = (-30, 3)
    z[-1, -2:] = (25, -0.5)
    dy = (synth.activations(rng, m, n) * np.float16(0.25)).astype(np.float16)
    dx, dz = w4.gemm_swiglu_backward(dev(dy), dev(z), dev(w4.pack(q)), dev(s), group)
    torch_mod().cuda.synchronize()
    dx, dz = host(dx), host(dz)
    want = pair_gradient(dy, z)
    z64 = z.astype(np.float64)
    size = np.repeat(np.abs(dy.astype(np.float64)) * (np.abs(z64[:, 1::2]) + 1) * (1 + np.abs(z64[:, 0::2])), 2, axis=1)
    assert np.all(np.abs(dz - want) <= 2.0 ** -10 * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -25)
    assert_close(dx, dz.astype(np.float64) @ oracle.dequantize(q, s, group), f"m={m} n={n} k={k} dx")


# up to 32 rows: pairs' gradient within the product (n a multiple of 4, short ranges per wave: one to
# four units of 32 rows of W) and in front of it (the last: ranges of more units)
FEW_ROWS = [(1, 4, 32, 32), (16, 36, 544, 32), (32, 1028, 1056, 32), (17, 4100, 256, 128), (5, 16300, 512, 128),
            (2, 2100, 16384, 128)]


@pytest.mark.parametrize("m,n,k,group", FEW_ROWS)
def test_block_backward_few_rows(w4, m, n, k, group):
    test_block_backward(w4, m, n, k, group)


def test_block_gradient_against_differences(w4):
    """Central differences of sum(h * dy) in x, in fp64 by the definition, against the library's whole chain."""
    torch = torch_mod()
    rng = np.random.default_rng(42000)
    m, n, k, group = 33, 24, 128, 128
    q, s = synth.code_bank(rng, 1, 2 * n, k)[0], synth.scale_bank(rng, 1, 2 * n, 1)[0]
    x = synth.activations(rng, m, k)
    dy = synth.activations(rng, m, n)
    z = torch.empty((m, 2 * n), dtype=torch.float16, device="cuda")
    w4.gemm_swiglu(dev(x), dev(w4.pack(q)), dev(s), group, gate_up=z)
    dx, _ = w4.gemm_swiglu_backward(dev(dy), z, dev(w4.pack(q)), dev(s), group)
    dx = host(dx).astype(np.float64)
    w = oracle.dequantize(q, s, group)

    def value(xv):
        zz = xv @ w.T
        return np.sum(oracle.silu(zz[:, 0::2]) * zz[:, 1::2] * dy, axis=1)

    x64, step = x.astype(np.float64), 1e-4
    diff = np.empty_like(x64)
    for j in range(k):
        e = np.zeros(k); e[j] = step
        diff[:, j] = (value(x64 + e) - value(x64 - e)) / (2 * step)
    # the kept products and their gradient are rounded to fp16 on the way (2^-11 each, seen
    # through SiLU'' of at most one half), the weights and dx once: 4 half steps per row
    err = np.linalg.norm(dx - diff, axis=1) / np.linalg.norm(diff, axis=1)
    assert err.max() <= 4 * 2.0 ** -11


# (m, n, k, group): one row, rows below / at / past a step, odd n, partial tiles, many tiles
SCALE_CASES = [(1, 1, 32, 32), (1, 300, 384, 128), (31, 257, 1056, 32), (32, 256, 256, 128), (133, 1001, 1120, 32),
               (500, 64, 2176, 128), (1000, 8200, 2304, 128), (2048, 520, 512, 32)]


@pytest.mark.parametrize("m,n,k,group", SCALE_CASES)
def test_scale_gradient(w4, m, n, k, group):
    rng = np.random.default_rng(43000 + m + n + k)
    q = synth.integer_codes(rng, n, k)
    d, x = synth.activations(rng, m, n), synth.activations(rng, m, k)
    ds = host(w4.gemm_dscales(dev(d), dev(x), dev(w4.pack(q)), group))
    torch_mod().cuda.synchronize()
    d64, x64, q64 = d.astype(np.float64), x.astype(np.float64), q.astype(np.float64)
    grouped = lambda a: a.reshape(n, k // group, group).sum(axis=2)  # noqa: E731
    want = grouped(q64 * (d64.T @ x64))
    size = grouped(np.abs(q64) * (np.abs(d64).T @ np.abs(x64)))
    assert ds.shape == want.shape and ds.dtype == np.float32
    bad = np.argwhere(~(np.abs(ds - want) <= (m + group) * 2.0 ** -22 * size))
    assert bad.size == 0, f"{len(bad)} of {ds.size} wrong, first {tuple(bad[0])}: {ds[tuple(bad[0])]} want {want[tuple(bad[0])]}"


@pytest.mark.parametrize("m,n,k,group", [(7, 9, 64, 32), (100, 300, 640, 128), (600, 700, 416, 32)])
def test_scale_gradient_is_exact_on_integers(w4, m, n, k, group):
    rng = np.random.default_rng(44000 + m)
    q = synth.integer_codes(rng, n, k)
    d, x = synth.integer_activations(rng, m, n), synth.integer_activations(rng, m, k)
    ds = host(w4.gemm_dscales(dev(d), dev(x), dev(w4.pack(q)), group))
    want = (q.astype(np.int64) * (d.astype(np.int64).T @ x.astype(np.int64))).reshape(n, k // group, group).sum(axis=2)
    assert np.array_equal(ds.astype(np.int64), want) and np.array_equal(ds, ds.astype(np.int64))


# tiles of one or two steps (not split), more of them than workgroups, a partial last round
@pytest.mark.parametrize("m,n,k,group", [(33, 1, 32, 32), (40, 4500, 4992, 32), (17, 4501, 4992, 128)])
def test_scale_gradient_few_steps(w4, m, n, k, group):
    test_scale_gradient(w4, m, n, k, group)
