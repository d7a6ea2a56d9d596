"""Refusals of the linear layer's, the router's and the few-token feed-forward's calls: the binding's (dtype,
contiguity, shape and device of every argument, CPU tensors only) and the C ABI's (no GPU)."""

import ctypes

import pytest
import torch

import w4a16_int4_weight_linear_amd as w4

F16, F32, I32 = torch.float16, torch.float32, torch.int32


def z(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def linear_operands(m=3, n=64, k=256, group=128):
    return dict(x=z(m, k), packed=z(n, k // 8, dtype=I32), scales=z(n, k // group), dy=z(m, n), bias=z(n), residual=z(m, n),
                pre=z(m, n), out=z(m, n), dpre=z(m, n), dbias=z(n, dtype=F32))


def call_linear(**changed):
    o = {**linear_operands(), **changed}
    return w4.linear(o["x"], o["packed"], o["scales"], o.get("group", 128), bias=o["bias"], activation=o.get("activation", "silu"),
                     residual=o["residual"], pre=o["pre"], out=o["out"], workspace=o.get("workspace"))


def call_backward(**changed):
    o = {**linear_operands(), **changed}
    return w4.linear_backward(o["dy"], o["packed"], o["scales"], o.get("group", 128), pre=o["pre"],
                              activation=o.get("activation", "silu"), dpre=o["dpre"], dbias=o["dbias"], workspace=o.get("workspace"))


@pytest.mark.parametrize("call,args", [(call_linear, ("x", "packed", "scales", "bias", "residual", "pre", "out")),
                                       (call_backward, ("dy", "packed", "scales", "pre", "dpre", "dbias"))])
def test_linear_arguments(call, args):
    o = linear_operands()
    for a in args:
        t = o[a]
        with pytest.raises(TypeError, match=a):
            call(**{a: t.numpy()})
        with pytest.raises(ValueError, match="dtype"):
            call(**{a: t.to(torch.float64)})
        with pytest.raises(ValueError):
            call(**{a: t[1:].contiguous()})
        if t.dim() == 2:
            with pytest.raises(ValueError, match="contiguous"):
                call(**{a: t.t().contiguous().t()})
    with pytest.raises(ValueError, match="HIP device"):
        call()
    with pytest.raises(ValueError, match="group"):
        call(group=64)
    with pytest.raises(ValueError, match="activation"):
        call(activation="tanh")
    with pytest.raises(ValueError, match="dtype"):
        call(workspace=z(16, dtype=F32))


def test_linear_backward_needs_its_pre_activations():
    with pytest.raises(ValueError, match="missing"):
        call_backward(pre=None)
    with pytest.raises(ValueError, match="with an activation"):
        call_backward(activation="none")
    with pytest.raises(ValueError, match="dpre"):
        call_backward(activation="none", pre=None)


def test_topk_arguments():
    logits = z(5, 20, dtype=F32)
    ids, w = z(5, 4, dtype=I32), z(5, 4, dtype=F32)
    with pytest.raises(TypeError, match="logits"):
        w4.moe_topk(logits.numpy(), 4)
    with pytest.raises(ValueError, match="dtype"):
        w4.moe_topk(logits.to(torch.bfloat16), 4)
    with pytest.raises(ValueError, match="tokens, experts"):
        w4.moe_topk(logits[0], 4)
    with pytest.raises(ValueError, match="contiguous"):
        w4.moe_topk(z(20, 5, dtype=F32).t(), 4)
    for topk in (0, -1, 21):
        with pytest.raises(ValueError, match="topk"):
            w4.moe_topk(logits, topk)
    with pytest.raises(ValueError, match="topk"):
        w4.moe_topk(z(2, 100, dtype=F32), 65)
    with pytest.raises(ValueError, match="experts"):
        w4.moe_topk(z(2, 1025, dtype=F32), 4)
    with pytest.raises(ValueError, match="ids has shape"):
        w4.moe_topk(logits, 3, ids=ids)
    with pytest.raises(ValueError, match="weights has dtype"):
        w4.moe_topk(logits, 4, weights=z(5, 4))
    with pytest.raises(ValueError, match="HIP device"):
        w4.moe_topk(logits, 4)
    with pytest.raises(ValueError, match="ids"):
        w4.moe_topk_backward(w, logits, ids[0], w)
    with pytest.raises(ValueError, match="dweights has shape"):
        w4.moe_topk_backward(w[:4], logits, ids, w)
    with pytest.raises(ValueError, match="out has dtype"):
        w4.moe_topk_backward(w, logits, ids, w, out=z(5, 20))
    with pytest.raises(ValueError, match="HIP device"):
        w4.moe_topk_backward(w, logits, ids, w)


def ffn_operands(t=3, e=4, h=256, i=128, k=2, g=128):
    return dict(x=z(t, h), ids=z(t, k, dtype=I32), weights=z(t, k, dtype=F32), gate_up=z(e, 2 * i, h // 8, dtype=I32),
                gate_up_scales=z(e, 2 * i, h // g), down=z(e, h, i // 8, dtype=I32), down_scales=z(e, h, i // g))


def call_ffn(group=128, **changed):
    o = ffn_operands()
    extra = {a: t for a, t in changed.items() if a not in o}
    o.update({a: t for a, t in changed.items() if a in o})
    return w4.moe_ffn(*o.values(), group, **extra)


def test_ffn_arguments():
    for a, t in ffn_operands().items():
        with pytest.raises(TypeError, match=a):
            call_ffn(**{a: t.numpy()})
        with pytest.raises(ValueError, match="dtype"):
            call_ffn(**{a: t.to(torch.float64)})
        with pytest.raises(ValueError):
            call_ffn(**{a: t[1:].contiguous()})
        with pytest.raises(ValueError):
            call_ffn(**{a: t[..., :-1].contiguous()})
        with pytest.raises(ValueError):
            call_ffn(**{a: t[0]})
    with pytest.raises(ValueError, match="group"):
        call_ffn(group=64)
    with pytest.raises(ValueError, match="out has shape"):
        call_ffn(out=z(3, 255))
    with pytest.raises(ValueError, match="residual has dtype"):
        call_ffn(residual=z(3, 256, dtype=F32))
    with pytest.raises(ValueError, match="HIP device"):
        call_ffn()


# ---- the C ABI: pointers are never followed before the checks ----
P = ctypes.c_void_p
A = [P((i + 1) << 24) for i in range(10)]      # aligned places 16 MB apart


def linear(x=A[0], p=A[1], s=A[2], bias=A[3], res=A[4], y=A[5], pre=A[6], m=4, n=64, k=128, group=128, act=1, ws=A[7], nb=1 << 20):
    return w4.lib.w4a16_linear(x, p, s, bias, res, y, pre, m, n, k, group, act, ws, nb, None)


def backward(dy=A[0], pre=A[1], p=A[2], s=A[3], dpre=A[4], db=A[5], dx=A[6], m=4, n=64, k=128, group=128, act=1, ws=A[7], nb=1 << 20):
    return w4.lib.w4a16_linear_backward(dy, pre, p, s, dpre, db, dx, m, n, k, group, act, ws, nb, None)


NULL, ODD = P(0), P((1 << 24) + 8)


def test_linear_abi_refusals():
    for f in (linear, backward):
        assert f(act=5) == w4.ERR_RANGE and f(act=-1) == w4.ERR_RANGE
        assert f(group=64) == w4.ERR_GROUP
        assert f(m=-1) == f(n=-1) == f(k=-128) == f(k=96) == f(m=1 << 31) == f(n=1 << 31) == w4.ERR_SHAPE
        assert f(n=1 << 26, k=128) == f(m=1 << 25, n=64) == w4.ERR_SHAPE     # 4 GB of weights, of outputs
        assert f(ws=ODD) == w4.ERR_ALIGN
    assert linear(k=0) == w4.ERR_SHAPE
    for a in ("x", "p", "s", "y"):
        assert linear(**{a: NULL}) == w4.ERR_NULL
    for a in ("x", "p", "bias", "res", "y", "pre"):
        assert linear(**{a: ODD}) == w4.ERR_ALIGN
    assert linear(m=0) == linear(n=0) == w4.OK
    for a in ("dy", "pre", "p", "s", "dpre", "dx"):
        assert backward(**{a: NULL}) == w4.ERR_NULL
    for a in ("dy", "pre", "p", "dpre", "db", "dx"):
        assert backward(**{a: ODD}) == w4.ERR_ALIGN
    assert backward(act=0) == w4.ERR_SHAPE                                   # pre and dpre without an activation
    assert backward(act=0, dpre=NULL) == w4.ERR_SHAPE
    assert backward(m=0, db=NULL) == w4.OK and backward(n=0, k=0) == w4.OK


def topk(x=A[0], dtype=0, ids=A[1], w=A[2], t=4, e=32, k=4):
    return w4.lib.w4a16_moe_topk(x, dtype, ids, w, t, e, k, 1, None)


def topk_back(dw=A[0], x=A[1], dtype=0, ids=A[2], w=A[3], out=A[4], t=4, e=32, k=4, norm=0):
    return w4.lib.w4a16_moe_topk_backward(dw, x, dtype, ids, w, out, t, e, k, norm, None)


def test_topk_abi_refusals():
    for f in (topk, topk_back):
        assert f(dtype=2) == f(dtype=-1) == w4.ERR_RANGE
        assert f(t=-1) == f(k=0) == f(k=33) == f(e=1025, k=4) == f(e=200, k=65) == f(e=0, k=1) == f(t=1 << 31) == w4.ERR_SHAPE
        assert f(t=0) == w4.OK
        assert f(x=NULL) == f(ids=NULL) == f(w=NULL) == w4.ERR_NULL
        assert f(x=ODD) == f(ids=P(0x1000002)) == f(w=P(0x1000002)) == w4.ERR_ALIGN
    assert topk(ids=A[2]) == topk(ids=A[0]) == topk(w=P(A[0].value + 16)) == w4.ERR_OVERLAP
    assert topk_back(out=NULL) == topk_back(dw=NULL) == w4.ERR_NULL
    assert topk_back(out=A[1]) == topk_back(out=A[0]) == topk_back(out=A[2], norm=1) == w4.ERR_OVERLAP


def ffn(x=A[0], ids=A[1], w=A[2], gu=A[3], gs=A[4], dn=A[5], ds=A[6], res=A[7], y=A[8], t=4, k=2, e=3, h=128, i=64, group=32, ws=A[9],
        nb=1 << 22):
    return w4.lib.w4a16_moe_ffn(x, ids, w, gu, gs, dn, ds, res, y, t, k, e, h, i, group, ws, nb, None)


def test_ffn_abi_refusals():
    assert ffn(group=64) == w4.ERR_GROUP
    assert ffn(t=-1) == ffn(t=65) == ffn(k=0) == ffn(t=64, k=9) == ffn(k=513) == ffn(k=2 ** 31 - 1) == w4.ERR_SHAPE
    assert ffn(e=0) == ffn(e=-1) == ffn(h=-32) == ffn(h=100) == ffn(i=0) == ffn(i=48) == ffn(i=-32) == w4.ERR_SHAPE
    assert ffn(h=1 << 20, i=1 << 11) == w4.ERR_SHAPE                         # 2 GiB of an expert's weights
    assert ffn(t=0) == ffn(h=0) == w4.OK
    for a in ("x", "ids", "w", "gu", "gs", "dn", "ds", "y"):
        assert ffn(**{a: NULL}) == w4.ERR_NULL, a
    for a in ("x", "gu", "dn", "res", "y", "ws"):
        assert ffn(**{a: ODD}) == w4.ERR_ALIGN, a
    assert ffn(ids=P(0x1000002)) == ffn(w=P(0x1000002)) == ffn(gs=P(0x1000001)) == w4.ERR_ALIGN
    need = w4.lib.w4a16_moe_ffn_workspace_bytes(4, 2, 128, 64, 32)
    assert need > 0 and ffn(nb=need - 1) == w4.ERR_WORKSPACE and ffn(ws=NULL) == w4.ERR_WORKSPACE
    for a in ("x", "ids", "w", "gu", "gs", "dn", "ds"):
        assert ffn(**{a: A[8]}) == w4.ERR_OVERLAP, a                         # y over an input
        assert ffn(**{a: A[9]}) == w4.ERR_OVERLAP, a                         # the workspace over an input
    assert ffn(res=P(A[8].value + 16)) == w4.ERR_OVERLAP                     # the residual over part of y
    for sizes in ((0, 2, 128, 64, 32), (65, 2, 128, 64, 32), (4, 2, 128, 64, 48), (4, 2, 100, 64, 32)):
        assert w4.lib.w4a16_moe_ffn_workspace_bytes(*sizes) == 0


def test_the_experts_workspace_is_device_memory():
    with pytest.raises(ValueError, match="HIP device"):
        w4.moe_ffn_workspace(4, 2, 256, 128, 32, device="cpu")
