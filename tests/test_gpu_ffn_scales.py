"""Scales of the fp8 gate and up projections whose product is outside fp32's
range while g and u are not: h is its definition's all the same, as it is with
gemm_a8w8_ptpc, which applies one scale after the other.  Every kernel that
applies them: few tokens, K shared out over workgroups, whole tiles."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# (m, d, f): up to 16 tokens, K shared out, tiles
SHAPES = [(5, 272, 72), (64, 7168, 136), (300, 272, 264)]


@pytest.fixture(scope="module")
def dmm():
    import dense_matmul_amd

    return dense_matmul_amd


def codes(shape, seed):
    """The four values of the largest binade: 256, 320, 384, 448."""
    v = np.random.default_rng(seed).integers(4, 8, shape).astype(np.float32) * 64
    return torch.from_numpy(v).to(torch.float8_e4m3fn).cuda()


def full(n, v):
    return torch.full((n,), v, device="cuda")


def test_shapes_take_each_kernel(dmm):
    need = [dmm.lib().gated_up_a8w8_ptpc_workspace(*s) for s in SHAPES]
    assert need[0] == 0 and need[1] > 0 and need[2] == 0


@pytest.mark.parametrize("sg,su", [(2.0**-75, 2.0**60), (2.0**60, 2.0**-75)])
@pytest.mark.parametrize("m,d,f", SHAPES)
def test_scales_whose_product_underflows(dmm, m, d, f, sg, su):
    """2^-75 twice is half of the least fp32 value; times a sum of 2^24 and
    more it is a normal number.  The sums are whole multiples of 2^12 below
    2^24 of them, so exact but for the matrix op's own error, 2^-9 of the
    largest of its 128 products, none of which is under a third of another:
    3 2^-16 of the sum.  Two scalings and the activation are good to 2^-18 of
    g and of u, the rounding to bf16 is 2^-8."""
    a, wg, wu = codes((m, d), 1), codes((f, d), 2), codes((f, d), 3)
    sx = 2.0**-75
    h = dmm.gated_up_a8w8_ptpc(a, wg, wu, full(m, sx), full(f, sg), full(f, su))
    g, u = a.double() @ wg.double().t() * sx * sg, a.double() @ wu.double().t() * sx * su
    assert min(t.min().item() for t in (g, u)) > 2.0**-126
    ref = g / (1 + torch.exp(-g)) * u
    # silu's relative slope, z act'(z) / act(z), is at most 2 for z > 0
    bound = (2.0**-8 + 1.01 * 3 * (2.0**-18 + 3 * 2.0**-16)) * ref
    assert ((h.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("m,d,f", SHAPES)
def test_scales_whose_product_overflows(dmm, m, d, f):
    """Tokens of zeros under two scales whose product is past the largest fp32
    value: 0, not 0 times infinity."""
    a, wg, wu = codes((m, d), 1), codes((f, d), 2), codes((f, d), 3)
    a[::2] = 0.0
    h = dmm.gated_up_a8w8_ptpc(a, wg, wu, full(m, 2.0**70), full(f, 2.0**70), full(f, 2.0**70))
    assert not h[::2].any()
