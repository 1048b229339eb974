"""The router's choice against the exact logits. A product of two bf16 or f32 values
is exact in 64 bits, so logits summed there are off by at most d 2^-53 of the sum of
their products' magnitudes, and not at all where the products are multiples of one
step and their sums stay within 2^53 of it."""

import pytest
import torch

from rank_structured_matmul_b200 import layers

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def values(g, n, dtype):
    """Values of full mantissas, multiples of 2^-24, below 16: 256 of them, and as many
    products with powers of two, sum without a rounding in 64 bits but not in 32."""
    v = torch.randint(-(2 ** 28) + 1, 2 ** 28, (n,), generator=g, dtype=torch.int64)
    if dtype == "bf16":  # eight bits at 21 places: 2^-24 to 2^-4
        v = torch.randint(128, 256, (n,), generator=g, dtype=torch.int64)
        v = v << torch.randint(0, 21, (n,), generator=g, dtype=torch.int64)
        v = v * (1 - 2 * torch.randint(0, 2, (n,), generator=g, dtype=torch.int64))
    else:  # 24 bits: what f32 holds
        v = v >> 4 << 4
    out = (v.double() * 2.0 ** -24).to(DT[dtype])
    assert torch.equal(out.double() * 2.0 ** 24, v.double())
    return out


@pytest.mark.parametrize("d", [5, 16, 64, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_logits_in_any_order(dtype, d):
    """Rows that hold the same values in different orders: exactly equal logits, the
    lower index first, equal weights."""
    if dtype == "bf16":
        d = (d + 7) // 8 * 8
    E, K, N = 40, 6, 9
    g = torch.Generator().manual_seed(d)
    row = values(g, d, dtype)
    Wr = torch.stack([row[torch.randperm(d, generator=g)] for _ in range(E)]).cuda()
    X = torch.ones(N, d, dtype=DT[dtype]) * 2.0 ** torch.arange(-4, 5)[:, None].to(DT[dtype])
    layer = layers.MoeLayer(d, 8, E, K, dtype)
    ids, w = layer.route(X.cuda(), Wr)
    assert torch.equal(ids.cpu(), torch.arange(K, dtype=torch.int32).expand(N, K))
    assert bool((w == w[:, :1]).all())
    assert layer.status() == 0
    layer.close()


@pytest.mark.parametrize("dtype,N,d,E,K", [("f32", 200, 250, 128, 8), ("bf16", 200, 2048, 128, 8),
                                           ("f32", 64, 4096, 300, 16), ("bf16", 64, 72, 512, 16)])
def test_order_of_close_logits(dtype, N, d, E, K):
    """Experts in groups whose rows differ in single last places: the order is the
    64-bit one wherever its neighbours are further apart than both sums' errors."""
    g = torch.Generator().manual_seed(N + d)
    X = torch.randn(N, d, generator=g).to(DT[dtype])
    base = (torch.randn((E + 3) // 4, d, generator=g) * d ** -0.5).to(DT[dtype])
    Wr = base.repeat_interleave(4, dim=0)[:E].clone()
    at = torch.randint(0, d, (E,), generator=g)
    step = torch.finfo(DT[dtype]).eps
    Wr[torch.arange(E), at] = (Wr[torch.arange(E), at].double() * (1 + step)).to(DT[dtype])
    layer = layers.MoeLayer(d, 8, E, K, dtype)
    ids, _ = layer.route(X.cuda(), Wr.cuda())
    logits = X.double() @ Wr.double().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    gap = (order.values[:, :K] - logits.gather(1, ids.cpu().long())).abs()
    off = 2 * d * 2.0 ** -53 * (X.double().abs() @ Wr.double().abs().t()).amax(1, keepdim=True)
    assert bool((gap <= off).all())
    assert all(len(set(r)) == K for r in ids.tolist())
    layer.close()
