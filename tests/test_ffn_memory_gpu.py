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
