"""NaN tokens of the feed-forward block reach their own rows and no others, at
every size of test_gpu_ffn.py and test_gpu_tiles.py, so in every kernel that is
chosen by size: a value read past a row's end, from a neighbour's row or from
memory that nothing wrote would turn other rows NaN or change their bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_gpu_ffn as ffn  # noqa: E402
import test_gpu_tiles as tiles  # noqa: E402
from test_tile_choice import sizes  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dmm():
    import dense_matmul_amd

    return dense_matmul_amd


def hit_rows(m):
    """The first, the last and one in the middle."""
    return torch.tensor(sorted({0, m // 2, m - 1}), device="cuda")


def check(got, want, rows):
    assert got[rows].isnan().all()
    keep = torch.ones(got.shape[0], dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], want[keep])


def poisoned(t, rows):
    t = t.clone()
    t[rows] = float("nan")
    return t


@pytest.mark.parametrize("m,d,f", sizes(ffn, "test_forward", "m,d,f") + sizes(tiles, "test_forward", "m,d,f"))
def test_forward(dmm, m, d, f):
    x, *w = ffn.block(m, d, f)
    rows = hit_rows(m)
    for got, want in zip(dmm.gated_ffn(poisoned(x, rows), *w, save=True), dmm.gated_ffn(x, *w, save=True)):
        check(got, want, rows)


@pytest.mark.parametrize("m,d,f", sizes(ffn, "test_backward", "m,d,f") + sizes(tiles, "test_backward", "m,d,f"))
def test_backward(dmm, m, d, f):
    args = ffn.block(m, d, f, 11)
    dy, gate, up = ffn.draw((m, d), 20, 0.1), ffn.draw((m, f), 21, 1.5), ffn.draw((m, f), 22, 1.5)
    rows = hit_rows(m)
    got = dmm.gated_ffn_backward(poisoned(dy, rows), *args, gate, up)
    check(got[0], dmm.gated_ffn_backward(dy, *args, gate, up)[0], rows)
    assert all(t.isnan().all() for t in got[1:])


@pytest.mark.parametrize("m,d,f", sizes(ffn, "test_fp8_up", "m,d,f") + sizes(tiles, "test_fp8_up", "m,d,f"))
def test_fp8_up(dmm, m, d, f):
    (a, sa), (wg, sg), (wu, su) = ffn.codes((m, d), 1), ffn.codes((f, d), 2), ffn.codes((f, d), 3)
    rows = hit_rows(m)
    want = dmm.gated_up_a8w8_ptpc(a, wg, wu, sa, sg, su)
    bad = a.clone()
    bad.view(torch.uint8)[rows] = 0x7F
    check(dmm.gated_up_a8w8_ptpc(bad, wg, wu, sa, sg, su), want, rows)
    check(dmm.gated_up_a8w8_ptpc(a, wg, wu, poisoned(sa, rows), sg, su), want, rows)
