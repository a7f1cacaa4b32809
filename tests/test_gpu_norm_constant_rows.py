"""Layer norm of rows of one value: the result is the bias, bit for bit.  The
sum of such a row is exact in fp32 (8 significant bits times 14 of the width), so
its mean is the value itself and nothing is left to be multiplied by rstd, which
is 1 / sqrt(eps) there and would make a residue of one last place visible."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_gpu_norm as norm  # noqa: E402

pytestmark = pytest.mark.gpu

# 8 significant bits at most
VALUES = (0.0, 1.0, -3.0, 100.0, 9984.0, -255 * 2.0**10, 171 * 2.0**13, 2.0**-20, -201 * 2.0**30)


@pytest.fixture(scope="module")
def dmm():
    import dense_matmul_amd

    return dense_matmul_amd


@pytest.mark.parametrize("kind", norm.TYPES)
@pytest.mark.parametrize("cols", norm.COLS + (24, 40, 56, 88, 168, 1000, 3000, 5000, 7000, 12000))
def test_constant_rows(dmm, cols, kind):
    dt = norm.TYPES[kind]
    x = torch.tensor(VALUES, dtype=dt, device="cuda")[:, None].expand(-1, cols).contiguous()
    assert torch.equal(x[:, 0].double().cpu(), torch.tensor(VALUES, dtype=torch.float64))
    w, b = norm.draw((cols,), 1, dt), norm.draw((cols,), 2, dt)
    y, mean, rstd = dmm.layer_norm(x, w, b, eps=2.0**-20, save=True)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(rstd, torch.full_like(rstd, 2.0**10))
    assert torch.equal(y, b.expand_as(y))
