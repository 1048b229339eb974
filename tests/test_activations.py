"""The layers' activations and their slopes by themselves: weights of zero (or one
product with 1), the argument through the bias, every bf16 value of 2^-10 to 14 and
both signs, against 64 bits.

Bounds, derived from how the functions are evaluated. An output is rounded once, off
by at most u = 2^-8 (bf16) or 2^-24 (f32) of itself.
  bf16  GELU: Phi(-|z|) = 2^P(|z|) within 2^-12 of itself, and z Phi adds a few fp32
        roundings: 2^-11 of |z| Phi(-|z|) on the negative side, less on the positive.
        The others are logistic functions of v = z or v = 1.6 z (1 + 0.045 z^2): the
        exponent's rounding is 2^-23 |v| of the result, the hardware's 2^x and
        reciprocal 2^-21 together; |v| <= 126 before it underflows, so 2^-15 in all.
        2^x flushes results below 2^-126 to zero: times |z| <= 14 and a slope's
        |v'| <= 26, 2^-117.
  f32   erfc, exp and the division are within 2^-20 of themselves for exact arguments.
        An argument's rounding (three operations) moves erfc(z / sqrt 2) by z^2 2^-22
        and exp(v) by |v| 2^-22 of itself.
A slope is a sum of two terms and is off by its terms' errors.
"""

import math

import pytest
import torch

from rank_structured_matmul_b200 import layers

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
C = math.sqrt(2 / math.pi)


def arguments():
    bits = torch.arange(0x3A80, 0x4161, 1, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = torch.cat([z, -z, torch.zeros(6, dtype=torch.bfloat16)]).cuda()
    assert z.numel() % 8 == 0
    return z


def parts64(z, act):
    """(value, slope, its terms' magnitudes, argument) in 64 bits."""
    z = z.double()
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        t = z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return z * p, p + t, p + t.abs(), z * z
    v, dv = z, torch.ones_like(z)
    if act == "gelu_tanh":
        v, dv = 2 * C * (z + 0.044715 * z ** 3), 2 * C * (1 + 3 * 0.044715 * z * z)
    p, n = torch.special.expit(v), torch.special.expit(-v)
    t = z * p * n * dv
    return z * p, p + t, p + t.abs(), v.abs()


def rel(act, arg, dtype):
    if dtype == "bf16":
        return torch.full_like(arg, 2.0 ** -11 if act == "gelu" else 2.0 ** -15)
    return 2.0 ** -20 + arg * 2.0 ** -22


def check(got, want, size, r, dtype, what):
    tol = U[dtype] * (want.abs() + r * size) + r * size + 2.0 ** -117
    err = (got.double() - want).abs()
    worst = (err / tol).max().item()
    assert worst <= 1.0, "%s: error is %.2f of its bound" % (what, worst)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype,N", [("bf16", 1), ("bf16", 6500), ("f32", 1), ("simt", 1)])
def test_values(dtype, N, act, monkeypatch):
    """One row (clusters) and many (pairs: alone, with Z, with a residual of zeros)."""
    if dtype == "simt":
        monkeypatch.setenv("DYRA_KERNELS", "simt")
        dtype = "bf16"
    z = arguments().to(DT[dtype])
    n = z.numel()
    layer = layers.DenseLinear(8, n, dtype)
    X = torch.zeros(N, 8, device="cuda", dtype=DT[dtype])
    W = torch.zeros(n, 8, device="cuda", dtype=DT[dtype])
    y, _, _, arg = parts64(z, act)
    outs = [layer.forward(X, W, bias=z, act=act),
            layer.forward(X, W, bias=z, act=act, residual=torch.zeros_like(X).new_zeros(N, n)),
            layer.forward(X, W, bias=z, act=act, save_z=True)[0]]
    for Y in outs:
        assert bool((Y == Y[:1]).all())
        check(Y[0], y, y.abs(), rel(act, arg, dtype), dtype, act)
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slopes(dtype, act):
    z = arguments().to(DT[dtype])
    n = z.numel()
    layer = layers.DenseLinear(8, n, dtype)
    one = torch.ones(1, n, device="cuda", dtype=DT[dtype])
    _, _, got = layer.backward(one, None, None, Z=z.view(1, n), act=act, need_dX=False,
                               need_dW=False)
    _, slope, size, arg = parts64(z, act)
    check(got, slope, size, rel(act, arg, dtype), dtype, act)
    layer.close()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates(dtype, act):
    """An expert whose gate rows give z, its up rows 1, its down product the identity:
    the hidden values, rounded once, come out as they are."""
    z = arguments()[::5][:704].to(DT[dtype])
    f = z.numel()
    assert f % 8 == 0
    layer = layers.MoeLayer(f, f, 1, 1, dtype, act=act)
    X = torch.zeros(2, f, device="cuda", dtype=DT[dtype])
    X[:, :2] = 1
    Wgu = torch.zeros(1, 2 * f, f, device="cuda", dtype=DT[dtype])
    Wgu[0, :f, 0], Wgu[0, f:, 1] = z, 1
    Wd = torch.eye(f, device="cuda", dtype=DT[dtype])[None]
    ids = torch.zeros(2, 1, device="cuda", dtype=torch.int32)
    Y = layer.experts(X, ids, torch.ones(2, 1, device="cuda"), Wgu, Wd)
    y, _, _, arg = parts64(z, act)
    assert torch.equal(Y[0], Y[1])
    check(Y[0], y, y.abs(), rel(act, arg, dtype), dtype, act)
    assert layer.status() == 0
    layer.close()
