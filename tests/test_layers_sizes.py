"""Sizes beyond a C int: refused, not taken for their low 32 bits."""

import pytest

from rank_structured_matmul_b200 import dyra, layers

WRAP = [2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1, 2 ** 64 + 64]


def refused(call, *args):
    with pytest.raises(dyra.DyraError) as e:
        call(*args)
    assert e.value.code == dyra.DYRA_ERR_INVALID_ARG, args


@pytest.mark.parametrize("big", WRAP)
def test_sizes_beyond_a_c_int(big):
    for i in range(2):
        sizes = [64, 64]
        sizes[i] = big
        refused(layers.dyra_dense_create, *sizes, dyra.DYRA_BF16)
        refused(layers.DenseLinear, *sizes)
    for i in range(4):
        sizes = [64, 64, 8, 2]
        sizes[i] = big
        refused(layers.dyra_moe_create, *sizes, layers.DYRA_ACT_SILU, 1, dyra.DYRA_BF16)
        refused(layers.MoeLayer, *sizes)


def test_sizes_are_integers():
    for bad in (64.0, "64", None):
        with pytest.raises(TypeError):
            layers.DenseLinear(bad, 64)
        with pytest.raises(TypeError):
            layers.MoeLayer(64, 64, 8, bad)
