"""The exact layers' ABI and binding without a GPU: refusals of arguments."""

import ctypes

import pytest
import torch

from rank_structured_matmul_b200 import dyra, layers

INV, ALIGN = dyra.DYRA_ERR_INVALID_ARG, dyra.DYRA_ERR_ALIGNMENT
F32, BF16 = dyra.DYRA_F32, dyra.DYRA_BF16


@pytest.mark.parametrize("args,code", [
    ((0, 64, F32), INV),      # d_in < 1
    ((64, 0, F32), INV),      # d_out < 1
    ((64, -8, BF16), INV),
    ((64, 64, 2), INV),       # unknown type
    ((60, 64, BF16), ALIGN),  # d_in % 8
    ((64, 60, BF16), ALIGN),  # d_out % 8
    ((2 ** 31 - 504, 64, BF16), INV),  # beyond 2^31 - 512
    ((64, 2 ** 31 - 511, F32), INV),
])
def test_dense_create_rejects(args, code):
    h = ctypes.c_void_p()
    assert dyra.lib().dyra_dense_create(ctypes.byref(h), *args) == code
    assert h.value is None


@pytest.mark.parametrize("args,code", [
    ((0, 64, 8, 2, 4, 1, F32), INV),     # d_model < 1
    ((64, 0, 8, 2, 4, 1, F32), INV),     # d_ff < 1
    ((2 ** 20 + 8, 64, 8, 2, 4, 1, F32), INV),  # d_model > 2^20
    ((64, 2 ** 20 + 8, 8, 2, 4, 1, BF16), INV),
    ((64, 64, 0, 1, 4, 1, F32), INV),    # experts < 1
    ((64, 64, 513, 2, 4, 1, F32), INV),  # experts > 512
    ((64, 64, 8, 0, 4, 1, F32), INV),    # top_k < 1
    ((64, 64, 8, 9, 4, 1, F32), INV),    # top_k > experts
    ((64, 64, 64, 17, 4, 1, F32), INV),  # top_k > 16
    ((64, 64, 8, 2, 5, 1, F32), INV),    # unknown activation
    ((64, 64, 8, 2, -1, 1, F32), INV),
    ((64, 64, 8, 2, 4, 2, F32), INV),    # renorm neither 0 nor 1
    ((64, 64, 8, 2, 4, 1, 9), INV),      # unknown type
    ((60, 64, 8, 2, 4, 1, BF16), ALIGN),
    ((64, 60, 8, 2, 4, 1, BF16), ALIGN),
])
def test_moe_create_rejects(args, code):
    h = ctypes.c_void_p()
    assert dyra.lib().dyra_moe_create(ctypes.byref(h), *args) == code
    assert h.value is None


def test_null_handles_and_outputs():
    lib = dyra.lib()
    n = None
    assert lib.dyra_dense_create(n, 64, 64, F32) == INV
    assert lib.dyra_moe_create(n, 64, 64, 8, 2, 4, 1, F32) == INV
    assert lib.dyra_dense_forward(n, n, n, n, n, 0, n, n, 1, n) == INV
    assert lib.dyra_dense_backward(n, n, n, n, n, 0, n, n, n, n, 1, n) == INV
    assert lib.dyra_moe_route(n, n, n, n, n, 1, n) == INV
    assert lib.dyra_moe_experts(n, n, n, n, n, n, n, n, 1, n) == INV
    assert lib.dyra_moe_forward(n, n, n, n, n, n, n, n, n, 1, n) == INV
    assert lib.dyra_dense_status(n) == INV and lib.dyra_moe_status(n) == INV
    assert lib.dyra_dense_device_bytes(n) == 0 and lib.dyra_moe_device_bytes(n) == 0
    assert lib.dyra_dense_destroy(n) == 0 and lib.dyra_moe_destroy(n) == 0


def test_constants_match_the_header():
    import os
    import re
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                        "dyra_layers.h")
    text = open(path).read()
    for name in ("DYRA_ACT_NONE", "DYRA_ACT_RELU", "DYRA_ACT_GELU", "DYRA_ACT_GELU_TANH",
                 "DYRA_ACT_SILU"):
        assert int(re.search(name + r" = (\d+)", text).group(1)) == getattr(layers, name)
    for name in ("DYRA_MOE_MAX_TOP_K", "DYRA_MOE_MAX_EXPERTS"):
        assert int(re.search("#define " + name + r" (\d+)", text).group(1)) == getattr(layers, name)


def test_without_a_gpu_creation_fails_cleanly():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(dyra.DyraError):
        layers.dyra_dense_create(64, 64, BF16)
    with pytest.raises(dyra.DyraError):
        layers.dyra_moe_create(64, 64, 8, 2, 4, 1, BF16)


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


@pytest.mark.parametrize("kw", [
    dict(X=z(4, 16)),                                    # wrong width
    dict(X=z(4)),                                        # not a matrix
    dict(X=z(4, 8, dtype=torch.float32)),                # wrong type
    dict(X=z(8, 4).t()),                                 # not contiguous
    dict(W=z(8, 24)),                                    # transposed weight
    dict(W=None),
    dict(bias=z(8)),                                     # wrong length
    dict(residual=z(3, 24)),                             # wrong rows
    dict(Y=z(4, 8)),
    dict(act="swish"),                                   # unknown activation
])
def test_dense_forward_refuses(kw):
    layer = _fake(layers.DenseLinear, d_in=8, d_out=24)
    args = dict(X=z(4, 8), W=z(24, 8))
    args.update(kw)
    with pytest.raises(ValueError):
        layer.forward(**args)


@pytest.mark.parametrize("kw", [
    dict(dY=z(4, 8)), dict(X=z(3, 8)), dict(X=None), dict(W=None), dict(Z=None),
    dict(Z=z(4, 24, dtype=torch.float32)), dict(act="swish"),
])
def test_dense_backward_refuses(kw):
    layer = _fake(layers.DenseLinear, d_in=8, d_out=24)
    args = dict(dY=z(4, 24), X=z(4, 8), W=z(24, 8), Z=z(4, 24), act="gelu")
    args.update(kw)
    with pytest.raises(ValueError):
        layer.backward(**args)


@pytest.mark.parametrize("kw", [
    dict(ids=z(4, 2, dtype=torch.int64)), dict(ids=z(4, 3, dtype=torch.int32)),
    dict(weights=z(4, 2)), dict(Wgu=z(5, 24, 8)), dict(Wd=z(5, 24, 8)), dict(X=z(4, 16)),
    dict(residual=z(4, 16)), dict(Y=z(5, 8)),
])
def test_moe_experts_refuses(kw):
    layer = _fake(layers.MoeLayer, d_model=8, d_ff=24, experts_n=5, top_k=2)
    args = dict(X=z(4, 8), ids=z(4, 2, dtype=torch.int32), weights=z(4, 2, dtype=torch.float32),
                Wgu=z(5, 48, 8), Wd=z(5, 8, 24))
    args.update(kw)
    with pytest.raises(ValueError):
        layer.experts(**args)


def test_layer_type_refused():
    with pytest.raises(ValueError):
        layers.DenseLinear(8, 8, "f16")
    with pytest.raises(ValueError):
        layers.MoeLayer(8, 8, 4, 2, act="swish")
