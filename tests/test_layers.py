"""The dense and expert layers on the GPU against plain 64-bit arithmetic.

Tolerances are bounds, derived here once. u = 2^-8 (bf16) or 2^-24 (f32) is
half a step of the stored type. A sum of K products in fp32 is off by at most
(K + 8) 2^-23 of the sum of the products' magnitudes (a unit in the last place
per addition covers accumulators that truncate; 8 more for the epilogue's
few operations). The activations have slopes of at most 1.2 and are themselves
within 2^-20 of |z|. An output is rounded once, u |y|. Gradients add the one
rounding of dZ to the stored type, u |dZ| per element.
"""

import math

import pytest
import torch

from rank_structured_matmul_b200 import dyra, layers

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def rand(g, *shape, dtype="bf16", scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(DT[dtype])


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def assert_within(got, want, tol, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), what
    worst = (err / tol).max().item() if err.numel() else 0.0
    assert worst <= 1.0, "%s: error is %.2f of its bound" % (what, worst)


def dense_case(N, d_in, d_out, dtype, seed=0):
    g = gen(seed + 7 * N + d_in + d_out)
    X = rand(g, N, d_in, dtype=dtype)
    W = rand(g, d_out, d_in, dtype=dtype, scale=d_in ** -0.5)
    b = rand(g, d_out, dtype=dtype, scale=0.5)
    R = rand(g, N, d_out, dtype=dtype)
    return X, W, b, R


def check_forward(layer, X, W, b, R, act, dtype):
    Y, Z = layer.forward(X, W, bias=b, residual=R, act=act, save_z=True)
    z = X.double() @ W.double().t()
    mag = X.double().abs() @ W.double().abs().t()
    if b is not None:
        z, mag = z + b.double(), mag + b.double().abs()
    u, k = U[dtype], (X.shape[1] + 8) * 2.0 ** -23
    y = act64(z, act)
    tol_y = u * y.abs() + 1.2 * k * mag + 2.0 ** -20 * z.abs() + 1e-30
    if R is not None:
        y = y + R.double()
        tol_y = tol_y + u * y.abs() + 2.0 ** -23 * (y.abs() + R.double().abs())
    assert_within(Z, z, u * z.abs() + k * mag + 1e-30, "Z")
    assert_within(Y, y, tol_y, "Y")
    assert layer.status() == 0
    return Y, Z


# rows from one token to several tiles and odd counts between; widths below,
# at and beyond the tiles' and the k steps' sizes
SIZES_BF16 = [(1, 8, 8), (1, 64, 128), (2, 72, 136), (5, 4096, 264), (16, 256, 1000),
              (17, 1000, 512), (33, 128, 2048), (64, 512, 128), (65, 640, 384), (127, 64, 64),
              (128, 200, 248), (129, 1024, 1024), (200, 8, 520), (257, 136, 8), (300, 2048, 392),
              (511, 264, 640), (777, 512, 1032), (1500, 320, 256), (2049, 192, 1288)]
SIZES_F32 = [(1, 1, 1), (1, 250, 190), (3, 17, 33), (16, 1024, 512), (64, 256, 256), (65, 63, 65),
             (77, 250, 190), (128, 128, 128), (129, 127, 131), (300, 511, 64), (1000, 100, 1001)]


@pytest.mark.parametrize("N,d_in,d_out", SIZES_BF16)
def test_forward_bf16(N, d_in, d_out):
    layer = layers.DenseLinear(d_in, d_out, "bf16")
    X, W, b, R = dense_case(N, d_in, d_out, "bf16")
    check_forward(layer, X, W, b, R, ACTS[(N + d_in) % 5], "bf16")
    check_forward(layer, X, W, None, None, "none", "bf16")
    layer.close()


@pytest.mark.parametrize("N,d_in,d_out", SIZES_F32)
def test_forward_f32(N, d_in, d_out):
    layer = layers.DenseLinear(d_in, d_out, "f32")
    X, W, b, R = dense_case(N, d_in, d_out, "f32")
    check_forward(layer, X, W, b, R, ACTS[(N + d_in) % 5], "f32")
    check_forward(layer, X, W, None, R, "none", "f32")
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [3, 70, 600])
def test_forward_activations(N, act, dtype):
    layer = layers.DenseLinear(96, 160, dtype)
    X, W, b, R = dense_case(N, 96, 160, dtype, seed=3)
    X = X * 4  # pre-activations well into both tails
    for bias, res in ((b, R), (b, None), (None, R)):
        check_forward(layer, X, W, bias, res, act, dtype)
    layer.close()


def grads64(dY, X, W, Z, act):
    z = Z.double().requires_grad_(True)
    dZ, = torch.autograd.grad(act64(z, act), z, dY.double())
    return dZ, dZ @ W.double(), dZ.t() @ X.double(), dZ.sum(0)


def check_backward(layer, X, W, Z, dY, act, dtype):
    dX, dW, db = layer.backward(dY, X, W, Z=Z, act=act)
    dZ64, dX64, dW64, db64 = grads64(dY, X, W, Z, act)
    u = U[dtype]
    N, d_out = dY.shape
    # dZ: its slope within 2^-20 of (1 + |z|), then rounded for the products
    slope = 2.0 ** -20 * (1 + Z.double().abs()) * dY.double().abs()
    a = dZ64.abs()
    per = slope + (u * a if act != "none" else 0)

    def tol(mag, off, k, y):
        return off + (k + 8) * 2.0 ** -23 * mag + u * y.abs() + 1e-30

    Wa, Xa = W.double().abs(), X.double().abs()
    assert_within(dX, dX64, tol(a @ Wa, per @ Wa, d_out, dX64), "dX")
    assert_within(dW, dW64, tol(a.t() @ Xa, per.t() @ Xa, N, dW64), "dW")
    assert_within(db, db64, tol(a.sum(0), slope.sum(0), N, db64), "dbias")
    # the bound above is a worst case; roundings being independent, the whole
    # gradient is off by at most sqrt(2) u / sqrt(3) of its norm, and the sums'
    # share. The norm needs many elements to be told apart from its parts.
    if dtype == "bf16" and dX64.numel() > 1000 and N > 8:
        for got, want in ((dX, dX64), (dW, dW64)):
            rel = ((got.double() - want).norm() / want.norm()).item()
            assert rel <= math.sqrt(2.0 / 3.0) * u + 1e-4, rel
    assert layer.status() == 0
    return dX, dW, db


@pytest.mark.parametrize("N,d_in,d_out", SIZES_BF16)
def test_backward_bf16(N, d_in, d_out):
    layer = layers.DenseLinear(d_in, d_out, "bf16")
    X, W, b, R = dense_case(N, d_in, d_out, "bf16")
    act = ACTS[(N + d_out) % 5]
    _, Z = layer.forward(X, W, bias=b, act=act, save_z=True)
    check_backward(layer, X, W, Z, R, act, "bf16")
    check_backward(layer, X, W, Z, R, "none", "bf16")
    layer.close()


@pytest.mark.parametrize("N,d_in,d_out", SIZES_F32)
def test_backward_f32(N, d_in, d_out):
    layer = layers.DenseLinear(d_in, d_out, "f32")
    X, W, b, R = dense_case(N, d_in, d_out, "f32")
    act = ACTS[(N + d_out) % 5]
    _, Z = layer.forward(X, W, bias=b, act=act, save_z=True)
    check_backward(layer, X, W, Z, R, act, "f32")
    layer.close()


@pytest.mark.parametrize("N,d_in,d_out", [(9700, 1024, 512), (6500, 264, 4096), (2600, 520, 1544)])
def test_forward_many_tiles(N, d_in, d_out):
    """More 256 x 256 tiles than pairs of SMs, with a last round of few tiles
    (76 of 74), of most, and ragged in both directions: every form of the
    epilogue."""
    layer = layers.DenseLinear(d_in, d_out, "bf16")
    X, W, b, R = dense_case(N, d_in, d_out, "bf16")
    z = X.double() @ W.double().t()
    mag = X.double().abs() @ W.double().abs().t() + b.double().abs()
    k, u = (d_in + 8) * 2.0 ** -23, U["bf16"]
    for act, bias, res, save in (("gelu", b, R, False), ("silu", b, R, True), ("none", None, R, False),
                                 ("gelu_tanh", b, None, True), ("relu", b, None, False),
                                 ("none", None, None, False)):
        zb = z if bias is None else z + b.double()
        y = act64(zb, act)
        tol = u * y.abs() + 1.2 * k * mag + 2.0 ** -20 * zb.abs()
        if res is not None:
            y = y + R.double()
            tol = tol + u * y.abs() + 2.0 ** -23 * (y.abs() + R.double().abs())
        out = layer.forward(X, W, bias=bias, residual=res, act=act, save_z=save)
        Y, Z = out if save else (out, None)
        assert_within(Y, y, tol, "Y %s" % act)
        if save:
            assert_within(Z, zb, u * zb.abs() + k * mag, "Z")
        again = layer.forward(X, W, bias=bias, residual=res, act=act)
        assert torch.equal(again, Y)
    got = R.clone()
    layer.forward(X, W, bias=b, residual=got, act="gelu", Y=got)
    assert torch.equal(got, layer.forward(X, W, bias=b, residual=R, act="gelu"))
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("N,d_in,d_out", [(9700, 512, 4096), (6000, 1280, 5120), (12345, 264, 136)])
def test_backward_many_rows(N, d_in, d_out):
    """Long sums and last rounds of few tiles (dX of 76 tiles, dW of 100)."""
    layer = layers.DenseLinear(d_in, d_out, "bf16")
    X, W, b, R = dense_case(N, d_in, d_out, "bf16")
    _, Z = layer.forward(X, W, bias=b, act="gelu", save_z=True)
    first = check_backward(layer, X, W, Z, R, "gelu", "bf16")
    for a, c in zip(first, layer.backward(R, X, W, Z=Z, act="gelu")):
        assert torch.equal(a, c)
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(act, dtype):
    layer = layers.DenseLinear(96, 160, dtype)
    X, W, b, R = dense_case(130, 96, 160, dtype, seed=3)
    _, Z = layer.forward(X * 4, W, bias=b, act=act, save_z=True)
    check_backward(layer, X, W, Z, R, act, dtype)
    layer.close()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences(act):
    """Directional derivatives of sum(dY * Y) from the gradients, against
    central differences of the 64-bit forward. With h = 1e-4 a central
    difference is off by about h^2 = 1e-8 of the derivatives' size; the f32
    gradients by (K + 8) 2^-23 of the summed magnitudes."""
    N, d_in, d_out = 33, 40, 56
    layer = layers.DenseLinear(d_in, d_out, "f32")
    X, W, b, dY = dense_case(N, d_in, d_out, "f32", seed=11)
    _, Z = layer.forward(X, W, bias=b, act=act, save_z=True)
    dX, dW, db = layer.backward(dY, X, W, Z=Z, act=act)

    def loss(x, w, c):
        return (dY.double() * act64(x @ w.t() + c, act)).sum()

    g = gen(5)
    h = 1e-4
    base = (X.double(), W.double(), b.double())
    for i, grad in enumerate((dX, dW, db)):
        v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * v, base[i] - h * v
        want = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.double() * v).sum()
        size = (grad.double() * v).abs().sum()
        assert abs(got - want) <= 2e-5 * size, (i, got.item(), want.item())
    layer.close()


def test_backward_parts_and_bits():
    """Each gradient alone equals the same gradient of the whole call, and two
    equal calls give equal bits."""
    layer = layers.DenseLinear(264, 392, "bf16")
    X, W, b, dY = dense_case(333, 264, 392, "bf16")
    _, Z = layer.forward(X, W, bias=b, act="gelu", save_z=True)
    whole = layer.backward(dY, X, W, Z=Z, act="gelu")
    again = layer.backward(dY, X, W, Z=Z, act="gelu")
    only_x = layer.backward(dY, None, W, Z=Z, act="gelu", need_dW=False, need_dbias=False)
    only_w = layer.backward(dY, X, None, Z=Z, act="gelu", need_dX=False, need_dbias=False)
    only_b = layer.backward(dY, None, None, Z=Z, act="gelu", need_dX=False, need_dW=False)
    for a, c in zip(whole, again):
        assert torch.equal(a, c)
    assert torch.equal(only_x[0], whole[0]) and only_x[1] is None and only_x[2] is None
    assert torch.equal(only_w[1], whole[1]) and torch.equal(only_b[2], whole[2])
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dtype):
    """Y over the residual; dZ over Z and over dY (through the C ABI)."""
    for N in (7, 150, 1100):
        layer = layers.DenseLinear(128, 264, dtype)
        X, W, b, R = dense_case(N, 128, 264, dtype)
        want, Z = layer.forward(X, W, bias=b, residual=R, act="silu", save_z=True)
        got = R.clone()
        layer.forward(X, W, bias=b, residual=got, act="silu", Y=got)
        assert torch.equal(got, want)
        dX, dW, db = layer.backward(R, X, W, Z=Z, act="silu")
        s = torch.cuda.current_stream().cuda_stream
        for over in ("Z", "dY"):
            z2, dy2 = Z.clone(), R.clone()
            x2, w2, b2 = torch.empty_like(dX), torch.empty_like(dW), torch.empty_like(db)
            layers.dyra_dense_backward(layer.handle, dy2, X, W, z2, layers.DYRA_ACT_SILU,
                                       z2 if over == "Z" else dy2, x2, w2, b2, N, s)
            assert torch.equal(x2, dX) and torch.equal(w2, dW) and torch.equal(b2, db)
        assert layer.status() == 0
        layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(dtype):
    layer = layers.DenseLinear(64, 128, dtype)
    e = lambda w: torch.empty(0, w, device="cuda", dtype=DT[dtype])  # noqa: E731
    W = torch.ones(128, 64, device="cuda", dtype=DT[dtype])
    assert layer.forward(e(64), W).shape == (0, 128)
    dX, dW, db = layer.backward(e(128), e(64), W, Z=e(128), act="gelu")
    assert dX.shape == (0, 64) and not dW.any() and not db.any()
    layer.close()


@pytest.mark.parametrize("N", [1, 40, 200, 1000])
def test_rows_behind_the_last_are_left_alone(N):
    """Rows behind the last, NaN in the inputs, neither read into the results
    nor written."""
    d_in, d_out, pad = 136, 264, 300
    layer = layers.DenseLinear(d_in, d_out, "bf16")
    X, W, b, R = dense_case(N + pad, d_in, d_out, "bf16")
    want, wz = layer.forward(X[:N].clone(), W, bias=b, residual=R[:N].clone(), act="gelu",
                             save_z=True)
    gw = layer.backward(R[:N].clone(), X[:N].clone(), W, Z=wz, act="gelu")
    Xp, Rp = X.clone(), R.clone()
    Xp[N:], Rp[N:] = float("nan"), float("nan")
    Y = torch.full((N + pad, d_out), 7.0, device="cuda", dtype=torch.bfloat16)
    layer.forward(Xp[:N], W, bias=b, residual=Rp[:N], act="gelu", Y=Y[:N])
    assert torch.equal(Y[:N], want) and bool((Y[N:] == 7.0).all())
    Zp = torch.full_like(Rp, float("nan"))
    Zp[:N] = wz
    for a, c in zip(layer.backward(Rp[:N], Xp[:N], W, Z=Zp[:N], act="gelu"), gw):
        assert torch.equal(a, c)
    assert layer.status() == 0
    layer.close()


def test_nan_stays_in_its_row():
    layer = layers.DenseLinear(128, 256, "bf16")
    for N in (5, 90, 700):
        X, W, b, R = dense_case(N, 128, 256, "bf16")
        want = layer.forward(X, W, bias=b, act="relu")
        X2 = X.clone()
        X2[N // 2, 3] = float("nan")
        got = layer.forward(X2, W, bias=b, act="relu")
        rows = torch.ones(N, dtype=torch.bool, device="cuda")
        rows[N // 2] = False
        assert torch.equal(got[rows], want[rows]) and torch.isnan(got[N // 2]).all()
    layer.close()


def test_refusals_on_the_device():
    layer = layers.DenseLinear(64, 64, "bf16")
    X, W, b, R = dense_case(4, 64, 64, "bf16")
    s = torch.cuda.current_stream().cuda_stream
    Y = torch.full((4, 64), 7.0, device="cuda", dtype=torch.bfloat16)

    def refused(code, call, *a):
        with pytest.raises(dyra.DyraError) as e:
            call(layer.handle, *a)
        assert e.value.code == code

    fwd, bwd = layers.dyra_dense_forward, layers.dyra_dense_backward
    inv, al = dyra.DYRA_ERR_INVALID_ARG, dyra.DYRA_ERR_ALIGNMENT
    refused(inv, fwd, None, W, None, None, 0, Y, None, 4, s)
    refused(inv, fwd, X, None, None, None, 0, Y, None, 4, s)
    refused(inv, fwd, X, W, None, None, 0, None, None, 4, s)
    refused(inv, fwd, X, W, None, None, 5, Y, None, 4, s)
    refused(inv, fwd, X, W, None, None, 0, Y, None, -1, s)
    refused(inv, fwd, X, W, None, None, 0, Y, None, 2 ** 31, s)
    refused(al, fwd, X.data_ptr() + 2, W, None, None, 0, Y, None, 3, s)
    refused(al, fwd, X, W, b.data_ptr() + 8, None, 0, Y, None, 4, s)
    refused(al, fwd, X, W, None, None, 0, Y.data_ptr() + 4, None, 3, s)
    refused(inv, bwd, None, X, W, None, 0, None, Y, None, None, 4, s)
    refused(inv, bwd, R, None, W, None, 0, None, None, Y, None, 4, s)   # dW without X
    refused(inv, bwd, R, X, None, None, 0, None, Y, None, None, 4, s)   # dX without W
    refused(inv, bwd, R, X, W, None, 2, Y, Y, None, None, 4, s)         # act without Z
    refused(inv, bwd, R, X, W, R, 2, None, Y, None, None, 4, s)         # act without dZ
    torch.cuda.synchronize()
    assert bool((Y == 7.0).all()) and layer.status() == 0
    layer.close()


def test_streams_and_graphs():
    """A call on another stream than the current one, two handles at once on
    two streams, and captured calls replayed on new inputs."""
    d = 264
    a, c = layers.DenseLinear(d, d, "bf16"), layers.DenseLinear(d, d, "bf16")
    cases = [dense_case(n, d, d, "bf16", seed=n) for n in (3, 600)]
    want = [a.forward(X, W, bias=b, residual=R, act="gelu") for X, W, b, R in cases]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        (X, W, b, R), (X2, W2, b2, R2) = cases
        got.append((a.forward(X, W, bias=b, residual=R, act="gelu", stream=s1),
                    c.forward(X2, W2, bias=b2, residual=R2, act="gelu", stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])

    for X, W, b, R in cases:
        sx, sr = X.clone(), R.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            Y, Z = a.forward(sx, W, bias=b, act="gelu", save_z=True)
            grads = a.backward(sr, sx, W, Z=Z, act="gelu")
        for k in range(3):
            sx.copy_(X * (k + 1)), sr.copy_(R * (2 - k))
            g.replay()
            y, z = a.forward(sx, W, bias=b, act="gelu", save_z=True)
            assert torch.equal(Y, y) and torch.equal(Z, z)
            for p, q in zip(grads, a.backward(sr, sx, W, Z=z, act="gelu")):
                assert torch.equal(p, q)
    assert a.status() == 0 and c.status() == 0
    a.close(), c.close()


def test_mlp_of_two_dense_layers():
    """fc1 with GELU, fc2 with the residual, and both backward passes in a row,
    against 64-bit autograd of the same MLP. Each of the chain's stored values
    (h, Z, dh, dZ) is rounded once; the roundings are independent, so the whole
    is off by at most the root of their count, six, times u."""
    N, d, f = 201, 256, 1024
    g = gen(2)
    X, dY = rand(g, N, d), rand(g, N, d)
    W1, b1 = rand(g, f, d, scale=d ** -0.5), rand(g, f, scale=0.1)
    W2, b2 = rand(g, d, f, scale=f ** -0.5), rand(g, d, scale=0.1)
    l1, l2 = layers.DenseLinear(d, f), layers.DenseLinear(f, d)
    h, Z1 = l1.forward(X, W1, bias=b1, act="gelu", save_z=True)
    Y = l2.forward(h, W2, bias=b2, residual=X)
    dh, dW2, db2 = l2.backward(dY, h, W2)
    dX, dW1, db1 = l1.backward(dh, X, W1, Z=Z1, act="gelu")
    t = [v.double().requires_grad_(True) for v in (X, W1, b1, W2, b2)]
    y = act64(t[0] @ t[1].t() + t[2], "gelu") @ t[3].t() + t[4] + t[0]
    want = torch.autograd.grad(y, t, dY.double())
    pairs = [(Y, y), (dX.double() + dY.double(), want[0]), (dW1, want[1]), (db1, want[2]),
             (dW2, want[3]), (db2, want[4])]
    for got, w in pairs:
        rel = ((got.double() - w).norm() / w.norm()).item()
        assert rel <= math.sqrt(6.0) * U["bf16"], rel
    l1.close(), l2.close()


# ------------------------------------------------------------------ experts ----

def moe_case(N, d, f, E, K, dtype, seed=0):
    g = gen(seed + N + d + f + E)
    X = rand(g, N, d, dtype=dtype)
    Wr = rand(g, E, d, dtype=dtype, scale=d ** -0.5)
    Wgu = rand(g, E, 2 * f, d, dtype=dtype, scale=d ** -0.5)
    Wd = rand(g, E, d, f, dtype=dtype, scale=f ** -0.5)
    R = rand(g, N, d, dtype=dtype)
    return X, Wr, Wgu, Wd, R


def experts64(X, ids, w, Wgu, Wd, R, act, dtype):
    """(y, bound) in 64 bits, expert by expert."""
    N, K = ids.shape
    E, f = Wgu.shape[0], Wd.shape[2]
    u = U[dtype]
    x = X.double()
    y = torch.zeros_like(x) if R is None else R.double()
    off, mag = torch.zeros_like(x), y.abs()
    for e in range(E):
        n, slot = (ids == e).nonzero(as_tuple=True)
        if n.numel() == 0:
            continue
        A = Wgu[e].double()
        gu, ga = x[n] @ A.t(), x[n].abs() @ A.abs().t()
        k1 = (X.shape[1] + 8) * 2.0 ** -23
        a, b = act64(gu[:, :f], act), gu[:, f:]
        da = 1.2 * k1 * ga[:, :f] + 2.0 ** -20 * gu[:, :f].abs()
        h = a * b
        dh = da * b.abs() + a.abs() * k1 * ga[:, f:] + da * k1 * ga[:, f:] + u * h.abs()
        B = Wd[e].double()
        wk = w[n, slot].double()[:, None]
        y = y.index_add(0, n, wk * (h @ B.t()))
        part = wk.abs() * ((h.abs() + dh) @ B.abs().t())
        off = off.index_add(0, n, wk.abs() * (dh @ B.abs().t()) + (f + 8) * 2.0 ** -23 * part)
        mag = mag.index_add(0, n, part)
    return y, off + (K + 4) * 2.0 ** -23 * mag + u * y.abs() + 1e-30


def check_experts(layer, X, ids, w, Wgu, Wd, R, act, dtype):
    Y = layer.experts(X, ids, w, Wgu, Wd, residual=R)
    y, tol = experts64(X, ids, w, Wgu, Wd, R, act, dtype)
    assert_within(Y, y, tol, "Y")
    assert layer.status() == 0
    return Y


MOE_BF16 = [(1, 64, 64, 4, 1), (1, 512, 1024, 8, 2), (2, 128, 72, 8, 8), (3, 1000, 488, 17, 3),
            (7, 136, 200, 64, 4), (16, 256, 512, 8, 2), (17, 264, 136, 5, 2), (33, 2048, 128, 9, 3),
            (64, 512, 256, 128, 8), (64, 8, 8, 3, 3), (1, 4096, 2048, 2, 2), (48, 72, 1032, 300, 16),
            (33, 16, 24, 512, 16), (5, 1288, 8, 3, 1), (40, 8, 2056, 2, 2)]
MOE_F32 = [(1, 1, 1, 1, 1), (50, 136, 200, 3, 2), (61, 33, 70, 2, 2), (64, 5, 129, 1, 1),
           (3, 256, 512, 8, 2), (5, 33, 17, 6, 3), (64, 65, 70, 12, 4), (2, 1000, 251, 4, 2),
           (3, 133, 264, 5, 3), (50, 133, 264, 3, 2), (50, 132, 261, 3, 2)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,d,f,E,K", MOE_BF16)
def test_moe_bf16(N, d, f, E, K, renorm):
    check_moe(N, d, f, E, K, "bf16", renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("N,d,f,E,K", MOE_F32)
def test_moe_f32(N, d, f, E, K, renorm):
    check_moe(N, d, f, E, K, "f32", renorm)


def check_moe(N, d, f, E, K, dtype, renorm):
    layer = layers.MoeLayer(d, f, E, K, dtype, renorm=renorm)
    X, Wr, Wgu, Wd, R = moe_case(N, d, f, E, K, dtype)
    Y, ids, w = layer.forward(X, Wr, Wgu, Wd, residual=R)
    logits = X.double() @ Wr.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    # the router's sums are within a few 2^-24 of each eight products' size
    gap = (order.values[:, :K] - logits.gather(1, ids.long())).abs()
    assert (gap <= 2.0 ** -20 * (X.double().abs() @ Wr.double().abs().t()).amax(1, True)).all()
    assert all(len(set(r)) == K for r in ids.tolist())
    p = torch.softmax(logits, 1).gather(1, ids.long())
    w64 = p / p.sum(1, keepdim=True) if renorm else p
    # exp of a logit off by at most 2^-20, a sum of E terms, a quotient
    assert ((w.double() - w64).abs() <= (E + 8) * 2.0 ** -23 * w64 + 4 * 2.0 ** -20 * w64).all()
    i2, w2 = layer.route(X, Wr)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    assert torch.equal(layer.experts(X, ids, w, Wgu, Wd, residual=R), Y)
    check_experts(layer, X, ids, w, Wgu, Wd, R, "silu", dtype)
    check_experts(layer, X, ids, w, Wgu, Wd, None, "silu", dtype)
    layer.close()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_activations(act, dtype):
    layer = layers.MoeLayer(64, 96, 6, 2, dtype, act=act)
    X, Wr, Wgu, Wd, R = moe_case(20, 64, 96, 6, 2, dtype)
    ids, w = layer.route(X, Wr)
    check_experts(layer, X * 3, ids, w, Wgu, Wd, R, act, dtype)
    layer.close()


def test_route_ties_and_nan():
    """Equal logits: the lower index first. A NaN logit is the lowest."""
    d, E, K = 64, 40, 4
    layer = layers.MoeLayer(d, 8, E, K, "f32")
    X = torch.zeros(4, d, device="cuda")
    Wr = torch.zeros(E, d, device="cuda")
    Wr[:, 0] = torch.tensor([float(i % 5) for i in range(E)])
    Wr[7] = float("nan")
    X[:3, 0] = torch.tensor([1.0, -1.0, 0.0])
    X[3] = float("nan")
    ids, w = layer.route(X, Wr)
    # experts with value 4, then 0 (lowest value leads for -1); expert 7 is NaN for every token
    assert ids.tolist() == [[4, 9, 14, 19], [0, 5, 10, 15], [0, 1, 2, 3], [0, 1, 2, 3]]
    assert torch.equal(w[:3], torch.full((3, K), 0.25, device="cuda"))
    assert torch.isnan(w[3]).all()
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_masks_and_repeats(dtype):
    """Ids that name no expert, tokens without any, one expert named twice, all
    tokens on one expert, and no token on any."""
    N, d, f, E, K = 37, 136, 72, 11, 3
    layer = layers.MoeLayer(d, f, E, K, dtype)
    X, Wr, Wgu, Wd, R = moe_case(N, d, f, E, K, dtype)
    g = gen(9)
    w = torch.rand(N, K, generator=g, device="cuda")
    ids = torch.randint(0, E, (N, K), generator=g, device="cuda", dtype=torch.int32)
    ids[3], ids[5, 1], ids[6, 0], ids[7, 2] = -1, -1, E, 2 ** 31 - 1
    ids[8], ids[9, 0] = 4, -2 ** 31
    w[5, 1] = float("nan")  # the weight of a masked slot is not used
    for R_ in (R, None):
        Y = check_experts(layer, X, ids, w, Wgu, Wd, R_, "silu", dtype)
        assert torch.equal(Y[3], R[3] if R_ is not None else torch.zeros_like(Y[3]))
        check_experts(layer, X, torch.full_like(ids, 2), torch.rand_like(w), Wgu, Wd, R_, "silu",
                      dtype)
        none = layer.experts(X, torch.full_like(ids, -1), w, Wgu, Wd, residual=R_)
        assert torch.equal(none, R if R_ is not None else torch.zeros_like(none))
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_experts_do_not_leak(dtype):
    """An expert whose weights are not finite changes only the tokens that name
    it; a token whose inputs are not finite only itself."""
    N, d, f, E, K = 20, 64, 136, 6, 2
    layer = layers.MoeLayer(d, f, E, K, dtype)
    X, Wr, Wgu, Wd, R = moe_case(N, d, f, E, K, dtype)
    ids, w = layer.route(X, Wr)
    want = layer.experts(X, ids, w, Wgu, Wd, residual=R)
    Wgu2, Wd2 = Wgu.clone(), Wd.clone()
    Wgu2[2], Wd2[4] = float("inf"), float("nan")
    got = layer.experts(X, ids, w, Wgu2, Wd2, residual=R)
    clean = ~((ids == 2) | (ids == 4)).any(1)
    assert clean.any() and torch.equal(got[clean], want[clean])
    assert not torch.isfinite(got[(ids == 4).any(1)].float()).any()
    X2 = X.clone()
    X2[5] = float("nan")
    got = layer.experts(X2, ids, w, Wgu, Wd, residual=R)
    rows = torch.arange(N, device="cuda") != 5
    assert torch.equal(got[rows], want[rows]) and torch.isnan(got[5]).all()
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_moe_more_than_one_group(dtype):
    """Beyond 64 tokens the call runs in groups; rows behind the last token are
    left alone, and Y may be the residual."""
    N, d, f, E, K = 150, 72, 136, 7, 2
    layer = layers.MoeLayer(d, f, E, K, dtype)
    X, Wr, Wgu, Wd, R = moe_case(N + 9, d, f, E, K, dtype)
    ids, w = layer.route(X[:N], Wr)
    Y = check_experts(layer, X[:N], ids, w, Wgu, Wd, R[:N], "silu", dtype)
    Y2 = R.clone()
    layer.experts(X[:N], ids, w, Wgu, Wd, residual=Y2[:N], Y=Y2[:N])
    assert torch.equal(Y2[:N], Y) and torch.equal(Y2[N:], R[N:])
    one = layer.experts(X[100:101].clone(), ids[100:101].clone(), w[100:101].clone(), Wgu, Wd,
                        residual=R[100:101].clone())
    y, tol = experts64(X[100:101], ids[100:101], w[100:101], Wgu, Wd, R[100:101], "silu", dtype)
    assert_within(one, y, tol, "one token of the group")
    e = torch.empty(0, d, device="cuda", dtype=DT[dtype])
    assert layer.forward(e, Wr, Wgu, Wd)[0].shape == (0, d)
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_many_tokens(dtype):
    """More tokens than one launch of the router takes."""
    N, d, E, K = 2100, 72, 37, 5
    layer = layers.MoeLayer(d, 8, E, K, dtype, renorm=False)
    g = gen(4)
    X, Wr = rand(g, N, d, dtype=dtype), rand(g, E, d, dtype=dtype, scale=d ** -0.5)
    ids, w = layer.route(X, Wr)
    logits = X.double() @ Wr.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    gap = (order.values[:, :K] - logits.gather(1, ids.long())).abs()
    assert (gap <= 2.0 ** -20 * (X.double().abs() @ Wr.double().abs().t()).amax(1, True)).all()
    w64 = torch.softmax(logits, 1).gather(1, ids.long())
    assert ((w.double() - w64).abs() <= (E + 8) * 2.0 ** -23 * w64 + 4 * 2.0 ** -20 * w64).all()
    part, wp = layer.route(X[1500:1510].clone(), Wr)
    assert torch.equal(part, ids[1500:1510]) and torch.equal(wp, w[1500:1510])
    assert layer.status() == 0
    layer.close()


def test_moe_streams_graphs_and_bits():
    N, d, f, E, K = 13, 256, 392, 16, 4
    a, c = layers.MoeLayer(d, f, E, K), layers.MoeLayer(d, f, E, K)
    X, Wr, Wgu, Wd, R = moe_case(N, d, f, E, K, "bf16")
    want = a.forward(X, Wr, Wgu, Wd, residual=R)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append(a.forward(X, Wr, Wgu, Wd, residual=R, stream=s1))
        got.append(c.forward(X, Wr, Wgu, Wd, residual=R, stream=s2))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    sx = X.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = a.forward(sx, Wr, Wgu, Wd, residual=R)
    for k in range(4):
        sx.copy_(X.flip(0) * (k - 1.5))
        g.replay()
        again = a.forward(sx, Wr, Wgu, Wd, residual=R)
        assert all(torch.equal(x, y) for x, y in zip(out, again))
    assert a.status() == 0 and c.status() == 0
    a.close(), c.close()


def test_moe_refusals_on_the_device():
    layer = layers.MoeLayer(64, 64, 4, 2)
    X, Wr, Wgu, Wd, R = moe_case(4, 64, 64, 4, 2, "bf16")
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    w = torch.zeros(4, 2, device="cuda")
    Y = torch.full((4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    s = torch.cuda.current_stream().cuda_stream
    inv, al = dyra.DYRA_ERR_INVALID_ARG, dyra.DYRA_ERR_ALIGNMENT

    def refused(code, call, *a):
        with pytest.raises(dyra.DyraError) as e:
            call(layer.handle, *a)
        assert e.value.code == code

    full = [X, ids, w, Wgu, Wd, None, Y]
    for i in (0, 1, 2, 3, 4, 6):
        a = list(full)
        a[i] = None
        refused(inv, layers.dyra_moe_experts, *a, 4, s)
        a[i] = full[i].data_ptr() + 4
        refused(al, layers.dyra_moe_experts, *a, 3, s)
    refused(inv, layers.dyra_moe_experts, *full, -1, s)
    refused(inv, layers.dyra_moe_route, X, None, ids, w, 4, s)
    refused(inv, layers.dyra_moe_forward, X, Wr, None, Wd, None, Y, ids, w, 4, s)
    refused(al, layers.dyra_moe_forward, X, Wr, Wgu, Wd, R.data_ptr() + 2, Y, ids, w, 3, s)
    refused(inv, layers.dyra_moe_forward, X, Wr, Wgu, Wd, None, Y, None, w, 4, s)
    torch.cuda.synchronize()
    assert bool((Y == 7.0).all()) and layer.status() == 0
    layer.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 16, 300])
def test_calls_in_a_row(N, dtype):
    """A block's calls in a row, each reading what the one before wrote, over and
    over the same buffers: every kernel is set up while the one before it runs, so
    the chain's bits must be those of the same calls with a wait after each."""
    d, f, E, K = 256, 520, 9, 2
    fc1, fc2 = layers.DenseLinear(d, f, dtype), layers.DenseLinear(f, d, dtype)
    moe = layers.MoeLayer(d, 136, E, K, dtype)
    X, W1, b1, _ = dense_case(N, d, f, dtype, seed=1)
    _, W2, b2, _ = dense_case(N, f, d, dtype, seed=2)
    _, Wr, Wgu, Wd, _ = moe_case(N, d, 136, E, K, dtype)

    def chain(wait):
        x, out = X.clone(), []
        for _ in range(8):
            h, Z = fc1.forward(x, W1, bias=b1, act="gelu", save_z=True)
            wait()
            fc2.forward(h, W2, bias=b2, residual=x, Y=x)
            wait()
            y, ids, w = moe.forward(x, Wr, Wgu, Wd)
            wait()
            dx, dw, db = fc1.backward(h, y, W1, Z=Z, act="gelu")
            wait()
            torch.add(y, dx, alpha=0.01, out=x)
            wait()
            x.div_(x.float().std().to(x.dtype))
            wait()
            out += [ids, w, dw, db, x.clone()]
        return out

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        for a, c in zip(chain(lambda: None), want):
            assert torch.equal(a, c)
    assert fc1.status() == 0 and fc2.status() == 0 and moe.status() == 0
    fc1.close(), fc2.close(), moe.close()


@pytest.mark.parametrize("N", [1, 100])
def test_bf16_on_the_cuda_cores(N, monkeypatch):
    """DYRA_KERNELS=simt, read at creation, runs bf16 handles on the CUDA cores."""
    monkeypatch.setenv("DYRA_KERNELS", "simt")
    layer = layers.DenseLinear(136, 264, "bf16")
    X, W, b, R = dense_case(N, 136, 264, "bf16")
    _, Z = check_forward(layer, X, W, b, R, "gelu", "bf16")
    check_backward(layer, X, W, Z, R, "gelu", "bf16")
    layer.close()
    check_moe(min(N, 64), 136, 72, 9, 3, "bf16", True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_far_out(act, dtype):
    """Beyond |z| = 100 the activations are z or 0 and their slopes 1 or 0 to less
    than 1e-40, up to the largest finite values, and a NaN stays one."""
    z = torch.tensor([100.0, 1e4, 3e9, 2e19, 1e25, 2e30, 3e38, -100.0, -1e4, -3e9, -2e19, -1e25,
                      -2e30, -3e38, float("nan"), 0.0], device="cuda", dtype=DT[dtype])
    n = z.numel()
    layer = layers.DenseLinear(8, n, dtype)
    X = torch.zeros(1, 8, device="cuda", dtype=DT[dtype])
    W = torch.zeros(n, 8, device="cuda", dtype=DT[dtype])
    Y = layer.forward(X, W, bias=z, act=act)[0]
    ones = torch.ones(1, n, device="cuda", dtype=DT[dtype])
    _, _, slope = layer.backward(ones, None, None, Z=z.view(1, n), act=act, need_dX=False,
                                 need_dW=False)
    assert torch.isnan(Y[14]) and torch.isnan(slope[14])
    assert Y[15] == 0.0 and slope[15] == 0.5
    assert torch.equal(Y[:7], z[:7]) and bool((Y[7:14].abs() < 1e-37).all())
    assert bool((slope[:7] == 1.0).all()) and bool((slope[7:14].abs() < 1e-37).all())
    layer.close()


def test_overlapping_outputs_are_refused():
    n, d = 16, 64
    layer, moe = layers.DenseLinear(d, d), layers.MoeLayer(d, d, 4, 2)
    X, W, b, R = dense_case(n, d, d, "bf16")
    _, Wr, Wgu, Wd, _ = moe_case(n, d, d, 4, 2, "bf16")
    Y, Z, G, V = (torch.full((n, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    big = torch.full((2 * n, d), 7.0, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(n, 2, device="cuda", dtype=torch.int32)
    w = torch.zeros(n, 2, device="cuda")
    kept = [t.clone() for t in (X, W, b, R, Wr, Wgu, Wd, ids, w)]
    s = torch.cuda.current_stream().cuda_stream

    def refused(call, handle, *a):
        with pytest.raises(dyra.DyraError) as e:
            call(handle, *a)
        assert e.value.code == dyra.DYRA_ERR_INVALID_ARG

    fwd, bwd = layers.dyra_dense_forward, layers.dyra_dense_backward
    h, gelu = layer.handle, layers.DYRA_ACT_GELU
    for y in (X, W, b, Z):
        refused(fwd, h, X, W, b, R, gelu, y, Z, n, s)
    for z in (X, W, b, R):
        refused(fwd, h, X, W, b, R, gelu, Y, z, n, s)
    refused(fwd, h, X, W, b, big[:n], gelu, big[1:n + 1], None, n, s)  # not the same rows
    refused(fwd, h, big[:n], W, b, R, gelu, big[n - 1:2 * n - 1], None, n, s)
    for dz in (X, W, b):
        refused(bwd, h, R, X, W, Z, gelu, dz, Y, G, b if dz is not b else dz, n, s)
    refused(bwd, h, R, X, W, big[:n], gelu, big[2:n + 2], Y, G, b, n, s)
    for over in (R, X, W, Z, V, G, b):
        refused(bwd, h, R, X, W, Z, gelu, V, over, G, b, n, s)
    for over in (R, X, W, Z, V, b):
        refused(bwd, h, R, X, W, Z, gelu, V, Y, over, b, n, s)
    for over in (R, X, W, Z, V):
        refused(bwd, h, R, X, W, Z, gelu, V, Y, G, over, n, s)
    h = moe.handle
    for y in (X, ids, w, Wgu, Wd):
        refused(layers.dyra_moe_experts, h, X, ids, w, Wgu, Wd, R, y, n, s)
        refused(layers.dyra_moe_forward, h, X, Wr, Wgu, Wd, R, y, ids, w, n, s)
    refused(layers.dyra_moe_forward, h, X, Wr, Wgu, Wd, R, Wr, ids, w, n, s)
    refused(layers.dyra_moe_experts, h, X, ids, w, Wgu, Wd, big[:n], big[1:n + 1], n, s)
    for over in (X, Wr, ids):
        refused(layers.dyra_moe_route, h, X, Wr, ids, over, n, s)
    for over in (X, Wr, w):
        refused(layers.dyra_moe_route, h, X, Wr, over, w, n, s)
    for over in (Wgu, Wd, R):
        refused(layers.dyra_moe_forward, h, X, Wr, Wgu, Wd, R, Y, over, w, n, s)
        refused(layers.dyra_moe_forward, h, X, Wr, Wgu, Wd, R, Y, ids, over, n, s)
    torch.cuda.synchronize()
    for t, k in zip((X, W, b, R, Wr, Wgu, Wd, ids, w), kept):
        assert torch.equal(t, k)
    assert bool((Y == 7.0).all()) and bool((big == 7.0).all())
    # what is not read may be written over: X without dW, Z and dZ without an activation
    z0 = torch.zeros(n, d, device="cuda", dtype=torch.bfloat16)
    bwd(layer.handle, R, z0, W, z0, 0, z0, z0, None, None, n, s)
    dX, _, _ = layer.backward(R, None, W, need_dW=False, need_dbias=False)
    assert torch.equal(z0, dX)
    assert layer.status() == 0 and moe.status() == 0
    layer.close(), moe.close()


@pytest.mark.parametrize("graphs", ["0", "1"])
def test_between_approximated_layers(graphs, monkeypatch):
    """Exact layers before and behind an approximated one whose factors change from
    step to step, all on one stream without a wait: the bits of the same calls with
    a wait after each."""
    monkeypatch.setenv("DYRA_GRAPHS", graphs)
    B, T, d, f, r, k = 3, 67, 256, 512, 64, 32
    up, down = layers.DenseLinear(d, f), layers.DenseLinear(d, d)
    mid = dyra.DyraLinear(f, d, r, k)
    X, W1, b1, _ = dense_case(B * T, d, f, "bf16", seed=3)
    _, W2, b2, _ = dense_case(B * T, d, d, "bf16", seed=4)
    g = gen(5)
    factors = [(rand(g, d, r, scale=r ** -0.5), rand(g, f, r, scale=f ** -0.5),
                rand(g, f, k, scale=f ** -0.5), rand(g, d, f, scale=0.1 * f ** -0.5))
               for _ in range(2)]
    h, y = X.new_empty(B * T, f), X.new_empty(B * T, d)
    s = torch.cuda.Stream()

    def chain(wait):
        x, out = X.clone(), []
        for i in range(6):
            dyra.dyra_load_factors(mid.plan, *factors[i % 2], 0.1, s)
            wait()
            up.forward(x, W1, bias=b1, act="gelu", Y=h, stream=s)
            wait()
            mid.forward(h, B=B, T=T, Y=y, stream=s)
            wait()
            z = down.forward(y, W2, bias=b2, residual=x, act="silu", stream=s)
            wait()
            x.copy_(z / z.float().std().to(z.dtype))
            wait()
            out.append(x.clone())
        return out

    with torch.cuda.stream(s):
        want = chain(torch.cuda.synchronize)
        assert all(bool(torch.isfinite(t).all()) for t in want)
        for _ in range(3):
            for a, c in zip(chain(lambda: None), want):
                assert torch.equal(a, c)
    assert up.status() == 0 and down.status() == 0 and mid.status() == 0
    up.close(), down.close(), mid.close()
