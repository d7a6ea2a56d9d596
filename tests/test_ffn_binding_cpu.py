"""The binding's refusals for the feed-forward block's calls: dtype, contiguity, shape and
device of every argument, before anything reaches the C ABI (CPU tensors only)."""

import pytest
import torch

import w4a16_int4_weight_linear_amd as w4

F16, F32, I32 = torch.float16, torch.float32, torch.int32


def operands(m=3, n=64, k=256, group=128):
    """Every tensor of the four calls, n outputs of the gated pair (2 n weight rows)."""
    z = lambda *shape, dtype=F16: torch.zeros(shape, dtype=dtype)  # noqa: E731
    return dict(x=z(m, k), packed=z(2 * n, k // 8, dtype=I32), scales=z(2 * n, k // group), gate_up=z(m, 2 * n),
                dy=z(m, n), d=z(m, 2 * n))


def call(name, o, **changed):
    o = {**o, **{a: t for a, t in changed.items() if a in o}}
    extra = {a: t for a, t in changed.items() if a not in o}
    args = {"gemm_swiglu": ("x", "packed", "scales"), "gemm_t": ("d", "packed", "scales"),
            "gemm_swiglu_backward": ("dy", "gate_up", "packed", "scales"), "gemm_dscales": ("d", "x", "packed")}[name]
    group = extra.pop("group", 128)
    return getattr(w4, name)(*(o[a] for a in args), group, **extra)


CALLS = {"gemm_swiglu": ("x", "packed", "scales"), "gemm_t": ("d", "packed", "scales"),
         "gemm_swiglu_backward": ("dy", "gate_up", "packed", "scales"), "gemm_dscales": ("d", "x", "packed")}


@pytest.mark.parametrize("name,arg", [(c, a) for c, args in CALLS.items() for a in args])
def test_each_argument_is_checked(name, arg):
    o = operands()
    t = o[arg]
    with pytest.raises(TypeError, match=arg):
        call(name, o, **{arg: t.numpy()})
    with pytest.raises(ValueError, match="dtype"):
        call(name, o, **{arg: t.to(torch.float64)})
    with pytest.raises(ValueError, match="2-D"):
        call(name, o, **{arg: t[0]})
    with pytest.raises(ValueError):                       # a row less than the others say
        call(name, o, **{arg: t[1:].contiguous()})
    with pytest.raises(ValueError, match="contiguous"):
        call(name, o, **{arg: t.t().contiguous().t()})


@pytest.mark.parametrize("name", CALLS)
def test_group_and_device(name):
    o = operands()
    with pytest.raises(ValueError, match="group"):
        call(name, o, group=64)
    with pytest.raises(ValueError):
        call(name, operands(k=96, group=32), group=128)   # k is no multiple of the group
    with pytest.raises(ValueError, match="HIP device"):
        call(name, o)                                     # everything right, but host memory
    with pytest.raises(ValueError, match="dtype"):
        call(name, o, workspace=torch.zeros(16, dtype=F32))


def test_outputs_are_checked():
    o = operands()
    z = torch.zeros
    for name, good in (("gemm_swiglu", (3, 64)), ("gemm_t", (3, 256)), ("gemm_swiglu_backward", (3, 256))):
        with pytest.raises(ValueError, match="out has shape"):
            call(name, o, out=z((good[0], good[1] + 1), dtype=F16))
        with pytest.raises(ValueError, match="out has dtype"):
            call(name, o, out=z(good, dtype=F32))
    with pytest.raises(ValueError, match="out has dtype"):
        call("gemm_dscales", o, out=z((128, 2), dtype=F16))
    with pytest.raises(ValueError, match="gate_up has shape"):
        call("gemm_swiglu", {k: v for k, v in o.items() if k != "gate_up"}, gate_up=z((3, 64), dtype=F16))
    with pytest.raises(ValueError, match="dgate_up has shape"):
        call("gemm_swiglu_backward", o, dgate_up=z((3, 64), dtype=F16))
    with pytest.raises(ValueError, match="multiple of 2 rows"):
        call("gemm_swiglu", {**o, "packed": o["packed"][1:].contiguous(), "scales": o["scales"][1:].contiguous()})
    with pytest.raises(ValueError, match="even"):
        call("gemm_swiglu_backward", {**o, "gate_up": z((3, 127), dtype=F16)})
    with pytest.raises(ValueError, match="no workspace"):
        w4.ffn_workspace("gemm", 1, 1, 32, 32, device="cpu")
