"""Calls whose gradient torch would have to record are refused, not answered without one."""

import pytest
import torch

from rank_structured_matmul_b200 import layers


def _fake(cls, **attrs):
    """A layer without a handle, its device the CPU: the binding's checks run
    before any call of the library."""
    x = cls.__new__(cls)
    x._setup("bf16")
    x.device, x.index = torch.device("cpu"), -1
    for k, v in attrs.items():
        setattr(x, k, v)
    return x


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


class Reached(Exception):
    pass


def reached(stream):
    raise Reached()


def check(layer, call, args):
    """Refused with each floating-point argument requiring a gradient; past the checks
    without one, under no_grad and in inference mode."""
    layer._on = reached
    for name, t in args.items():
        if not t.is_floating_point():
            continue
        kw = dict(args, **{name: t.clone().requires_grad_()})
        with pytest.raises(ValueError, match="gradient"):
            call(**kw)
        with torch.no_grad(), pytest.raises(Reached):
            call(**kw)
        with torch.inference_mode(), pytest.raises(Reached):
            call(**kw)
        # a result of a recorded operation, not a leaf
        with pytest.raises(ValueError, match="gradient"):
            call(**dict(kw, **{name: kw[name] * 1}))
    with pytest.raises(Reached):
        call(**args)


def test_dense():
    layer = _fake(layers.DenseLinear, d_in=8, d_out=24)
    check(layer, layer.forward, dict(X=z(4, 8), W=z(24, 8), bias=z(24), residual=z(4, 24),
                                     Y=z(4, 24)))
    check(layer, lambda **kw: layer.backward(act="gelu", **kw),
          dict(dY=z(4, 24), X=z(4, 8), W=z(24, 8), Z=z(4, 24)))


def test_experts():
    layer = _fake(layers.MoeLayer, d_model=8, d_ff=24, experts_n=5, top_k=2)
    experts = dict(X=z(4, 8), Wgu=z(5, 48, 8), Wd=z(5, 8, 24), residual=z(4, 8), Y=z(4, 8))
    check(layer, layer.route, dict(X=z(4, 8), Wr=z(5, 8)))
    check(layer, layer.forward, dict(experts, Wr=z(5, 8)))
    check(layer, layer.experts, dict(experts, ids=z(4, 2, dtype=torch.int32),
                                     weights=z(4, 2, dtype=torch.float32)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameters_under_no_grad(dtype):
    """A training step on leaves that require gradients, the way the message says."""
    layer = layers.DenseLinear(64, 128, "bf16" if dtype == torch.bfloat16 else "f32")
    g = torch.Generator(device="cuda").manual_seed(0)
    X, W, b, dY = (torch.randn(*s, generator=g, device="cuda").to(dtype)
                   for s in ((33, 64), (128, 64), (128,), (33, 128)))
    W, b = W.requires_grad_(), b.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        layer.forward(X, W, bias=b)
    with torch.no_grad():
        Y, Z = layer.forward(X, W, bias=b, act="silu", save_z=True)
        grads = layer.backward(dY, X, W, Z=Z, act="silu")
    W, b = W.detach(), b.detach()
    Y2, Z2 = layer.forward(X, W, bias=b, act="silu", save_z=True)
    for a, c in zip((Y, Z, *grads), (Y2, Z2, *layer.backward(dY, X, W, Z=Z2, act="silu"))):
        assert torch.equal(a, c) and not a.requires_grad
    layer.close()
