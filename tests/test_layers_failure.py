"""Waits of the exact layers that run out: the call returns, reports it, and the next
one is right. A diagnostic setter shortens the limit; nothing here traps, asserts on
the device or waits for good."""

import os
import re

import pytest
import torch

from rank_structured_matmul_b200 import dyra, layers

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "rank_structured_matmul_b200", "csrc")


@pytest.mark.parametrize("header", ["umma_gemm.cuh", "umma_gemm_pair.cuh", "stream_gemm.cuh"])
def test_epilogue_threads_stop_together(header):
    """The epilogue's threads meet at barriers, so none of them may leave alone: each
    wait for an accumulator is the argument of a vote."""
    text = open(os.path.join(CSRC, header)).read()
    code = re.sub(r"//[^\n]*", "", text)
    epilogue = code[code.index("struct EpiCtx") if "struct EpiCtx" in code else 0:]
    waits = [m.start() for m in re.finditer(r"mbar_wait\((tfull_bar|done_bar)", epilogue)]
    assert waits
    for at in waits:
        assert re.search(r"all_threads\([^;]*$", epilogue[:at]), epilogue[at - 80:at + 40]


def rand(*shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("N,d_in,d_out,pairs", [(64, 16384, 1024, False), (1, 16384, 14336, True),
                                                (40, 8192, 128, False), (1, 4096, 14336, False)])
def test_dense_wait_that_runs_out(N, d_in, d_out, pairs):
    """Tiles on clusters and on single CTAs; the forward and the gradients. A forward on
    CTA pairs keeps the default limit."""
    layer = layers.DenseLinear(d_in, d_out)
    X, W, dY = rand(N, d_in), rand(d_out, d_in, scale=d_in ** -0.5), rand(N, d_out)
    want = (layer.forward(X, W, act="gelu"), *layer.backward(dY, X, W))
    assert layer.status() == 0
    for _ in range(3):
        layers.dyra_debug_dense_set_wait_limit(layer.handle, 1)  # 1 ns
        layer.forward(X, W, act="gelu")
        status = layer.status()
        assert status == (0 if pairs else dyra.DYRA_STATUS_WAIT_TIMEOUT), status
        layer.backward(dY, X, W)
        layer.status()
        layers.dyra_debug_dense_set_wait_limit(layer.handle, 0)
        again = (layer.forward(X, W, act="gelu"), *layer.backward(dY, X, W))
        assert layer.status() == 0
        for a, c in zip(again, want):
            assert torch.equal(a, c)
    layer.close()


@pytest.mark.gpu
@pytest.mark.parametrize("N,d,f,E,K", [(64, 2048, 1024, 16, 4), (1, 4096, 4096, 4, 2),
                                       (150, 1024, 2048, 5, 2)])
def test_experts_wait_that_runs_out(N, d, f, E, K):
    """Counters of arrivals that a call left behind start again; 150 tokens are three
    groups, the second one behind a first that gave up."""
    layer = layers.MoeLayer(d, f, E, K)
    X, R = rand(N, d), rand(N, d)
    Wr, Wgu, Wd = (rand(E, d, scale=d ** -0.5), rand(E, 2 * f, d, scale=d ** -0.5),
                   rand(E, d, f, scale=f ** -0.5))
    want = layer.forward(X, Wr, Wgu, Wd, residual=R)
    assert layer.status() == 0
    for _ in range(3):
        layers.dyra_debug_moe_set_wait_limit(layer.handle, 1)
        layer.forward(X, Wr, Wgu, Wd, residual=R)
        status = layer.status()
        assert status == dyra.DYRA_STATUS_WAIT_TIMEOUT, status
        layers.dyra_debug_moe_set_wait_limit(layer.handle, 0)
        again = layer.forward(X, Wr, Wgu, Wd, residual=R)
        assert layer.status() == 0
        for a, c in zip(again, want):
            assert torch.equal(a, c)
    layer.close()


@pytest.mark.gpu
def test_no_waits_on_the_cuda_cores():
    dense, moe = layers.DenseLinear(8, 8, "f32"), layers.MoeLayer(8, 8, 2, 1, "f32")
    for call, h in ((layers.dyra_debug_dense_set_wait_limit, dense.handle),
                    (layers.dyra_debug_moe_set_wait_limit, moe.handle)):
        with pytest.raises(dyra.DyraError) as e:
            call(h, 1)
        assert e.value.code == dyra.DYRA_ERR_UNSUPPORTED
        with pytest.raises(dyra.DyraError) as e:
            call(None, 1)
        assert e.value.code == dyra.DYRA_ERR_INVALID_ARG
    dense.close(), moe.close()
