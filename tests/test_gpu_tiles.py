"""The feed-forward block and the adapters at sizes that reach the tile shapes
which the sizes of test_gpu_ffn.py and test_gpu_lora.py do not (test_tile_choice.py
holds the two lists together against the choice by size): the same checks
against the definitions in 64 bits, with the same bounds.  Most have row,
column and K tiles that are cut off."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_gpu_ffn as ffn  # noqa: E402
import test_gpu_lora as lora  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import dense_matmul_amd

    return dense_matmul_amd


# gate and up / down projection: few tokens with 16 waves / 8, 16 / 16; 128 / 128;
# 128D / 128; 128D / 128D; 256 / 256; 128D / 128D
@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("m,d,f", [(1, 2056, 1032), (13, 7168, 2048), (4775, 344, 264), (3649, 520, 264), (2197, 992, 528), (5965, 1464, 648), (1003, 2048, 2048)])
def test_forward(dmm, m, d, f, act):
    ffn.test_forward(dmm, m, d, f, act)


# dh / dx / the weights' gradients: 128 / 128D / 128D; 128D three times; 128D /
# 128 / 128D; 128D / 256 / 128D; 64 / 64 / 128; 256 / both in one launch; 256
# three times; 128D / 128D / 256
@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("m,d,f", [(4133, 592, 1064), (2390, 904, 880), (3726, 1328, 528), (5516, 1744, 344), (131, 2032, 1232),
                                   (3281, 264, 2472), (5832, 2080, 1944), (1003, 2048, 2048)])
def test_backward(dmm, m, d, f, act):
    ffn.test_backward(dmm, m, d, f, act)


@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("m,d,f", [(133, 288, 5664), (130, 1056, 5920)])
def test_fp8_up(dmm, m, d, f, act):
    ffn.test_fp8_up(dmm, m, d, f, act)


# few tokens, whose first product is a launch of its own (16 and 32 ranks a
# workgroup), beside one and several shares of the other; 128D tiles
@pytest.mark.parametrize("order", ("mixed", "runs"))
@pytest.mark.parametrize("m,n,k,r,adapters", [(160, 272, 1160, 8, 52), (33, 264, 5432, 16, 58), (34, 304, 5648, 32, 37), (147, 360, 1192, 24, 23),
                                              (650, 3184, 520, 32, 5), (5644, 336, 808, 248, 8), (1000, 4096, 4096, 16, 32)])
def test_against_the_definition(dmm, m, n, k, r, adapters, order):
    lora.test_against_the_definition(dmm, m, n, k, r, adapters, order)
