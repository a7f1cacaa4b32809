"""The feed-forward block, the adapters and the norm's gradients on whole numbers,
bit for bit.

The inputs are small whole numbers, few enough per row that the magnitudes of
every sum's terms add up to less than 2^24 (of halves, in the backward pass and
with scales of a half), so that fp32 holds it in whatever order it is added.  Gates are 0 or far out, where silu and gelu are 0, a
half of the slope or the identity.  What is left are the documented roundings to
bf16, to the nearest even: of g, u, h and y forward, of the results backward
(dg, du and h fit bf16), of y with adapters (v fits bf16, so few and many tokens
agree).  Each result has one value, and a lost, doubled or misplaced product
shows wherever it is more than half of a last place; the bounds of the other
tests, which are over sums of magnitudes, leave room for a few.

The sizes of the block and the adapters are those of test_gpu_ffn.py, test_gpu_lora.py and test_gpu_tiles.py,
so every kernel that is chosen by size is run."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_gpu_ffn as ffn  # noqa: E402
import test_gpu_lora as lora  # noqa: E402
import test_gpu_norm as norm  # noqa: E402
import test_gpu_tiles as tiles  # noqa: E402
from test_tile_choice import sizes  # noqa: E402

BF = torch.bfloat16


@pytest.fixture(scope="module")
def dmm():
    import dense_matmul_amd

    return dense_matmul_amd


def signs(shape, seed, per_row=None):
    """-1, 0 and 1, with about per_row values other than 0 to a row."""
    rng = np.random.default_rng(seed)
    v = rng.integers(0, 2, shape, dtype=np.int8) * 2 - 1
    share = 2 / 3 if per_row is None else min(2 / 3, per_row / shape[-1])
    return torch.from_numpy(v * (rng.random(shape, dtype=np.float32) < share)).to(torch.float64)


def choice(shape, seed, values):
    return torch.from_numpy(np.random.default_rng(seed).choice(np.array(values, dtype=np.float64), shape))


def product(a, b, unit=0.5):
    """a b, whose terms are multiples of unit and exact in fp32 in any order."""
    terms = a.abs() @ b.abs()
    assert terms.numel() == 0 or terms.max() < 2.0**24 * unit and torch.equal(terms, (terms / unit).round() * unit)
    return a @ b


def rounded(t):
    """What fp32 holds exactly, rounded to bf16 and widened again."""
    assert torch.equal(t.to(torch.float32).to(torch.float64), t)
    return t.to(torch.float32).to(BF).to(torch.float64)


def fits(t):
    assert torch.equal(rounded(t), t)
    return t


def same(got, want):
    assert torch.equal(got.double(), want), f"{int((got.double() != want).sum())} of {want.numel()} values differ"


def on_gpu(*tensors):
    return [t.to(BF).cuda() for t in tensors]


# ------------------------------------------------------------------ block
def forward_inputs(m, d, f):
    x, wg, wu, wd = signs((m, d), 1, 400), signs((f, d), 2), signs((f, d), 3), signs((d, f), 4)
    x[:, 0], wg[:, 0] = 16, 16  # every gate is 256 and a sum of about 400 signs
    return x, wg, wu, wd


def forward(x, wg, wu, wd):
    g, u = product(x, wg.t(), 1), product(x, wu.t(), 1)
    assert g.min() > 100
    return rounded(product(rounded(g * u), wd.t(), 1)), rounded(g), rounded(u)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("m,d,f", sizes(ffn, "test_forward", "m,d,f") + sizes(tiles, "test_forward", "m,d,f"))
def test_forward(dmm, m, d, f, act):
    args = forward_inputs(m, d, f)
    got = dmm.gated_ffn(*on_gpu(*args), act=act, save=True)
    for a, b in zip(got, forward(*(t.cuda() for t in args))):
        same(a, b)


def backward_inputs(m, d, f):
    return (signs((m, d), 1, 200), signs((m, d), 2), signs((f, d), 3), signs((f, d), 4), signs((d, f), 5),
            choice((m, f), 6, (0, 32, 64, -256)), choice((m, f), 7, (-2, -1, 0, 1, 2)))


def backward(dy, x, wg, wu, wd, gate, up):
    val, slope = gate.clamp(min=0), (gate > 0) + 0.5 * (gate == 0)
    dh = product(dy, wd)
    dg, du, h = fits(dh * up * slope), fits(dh * val), fits(val * up)
    return [rounded(t) for t in (product(dg, wg) + product(du, wu), product(dg.t(), x), product(du.t(), x), product(dy.t(), h))]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ffn.ACTS)
@pytest.mark.parametrize("m,d,f", sizes(ffn, "test_backward", "m,d,f") + sizes(tiles, "test_backward", "m,d,f"))
def test_backward(dmm, m, d, f, act):
    args = backward_inputs(m, d, f)
    got = dmm.gated_ffn_backward(*on_gpu(*args), act=act)
    for a, b in zip(got, backward(*(t.cuda() for t in args))):
        same(a, b)


# --------------------------------------------------------------- adapters
def adapter_inputs(m, n, k, r, adapters, order):
    rng = np.random.default_rng(9)
    if order == "mixed":
        ids = rng.integers(-1, adapters, m)
    else:
        cuts = np.sort(rng.integers(0, m + 1, 2 * adapters))
        ids = rng.integers(-1, adapters, 2 * adapters + 1)[np.searchsorted(cuts, np.arange(m), side="right")]
    return {"x": signs((m, k), 1, 200), "w": signs((n, k), 2), "a": signs((adapters, r, k), 3), "b": signs((adapters, n, r), 4),
            "c": choice((m, n), 5, range(-100, 101)), "ids": torch.from_numpy(ids.astype(np.int64)), "s": choice((adapters,), 6, (0.5, 1, 2))}


def adapted(p, shared):
    y = product(p["x"], p["w"].t()) if shared else p["c"].clone()
    for i in range(p["a"].shape[0]):
        rows = (p["ids"] == i).nonzero()[:, 0]
        y[rows] += product(fits(p["s"][i] * product(p["x"][rows], p["a"][i].t())), p["b"][i].t())
    return rounded(y)


@pytest.mark.gpu
@pytest.mark.parametrize("order", ("mixed", "runs"))
@pytest.mark.parametrize("m,n,k,r,adapters", sizes(lora, "test_against_the_definition", "m,n,k,r,adapters") +
                         sizes(tiles, "test_against_the_definition", "m,n,k,r,adapters"))
def test_adapters(dmm, m, n, k, r, adapters, order):
    p = {q: t.cuda() for q, t in adapter_inputs(m, n, k, r, adapters, order).items()}
    g = {q: t.int() if q == "ids" else t.float() if q == "s" else t.to(BF) for q, t in p.items()}
    tail = (g["a"], g["b"], g["ids"], g["s"])
    y, z = dmm.lora_gemm_bf16(g["x"], g["w"], *tail), dmm.lora_add_bf16(g["c"], g["x"], *tail)
    same(y, adapted(p, True))
    same(z, adapted(p, False))
    few = min(m, 40)
    tail = (g["a"], g["b"], g["ids"][:few].contiguous(), g["s"])
    assert torch.equal(dmm.lora_gemm_bf16(g["x"][:few].contiguous(), g["w"], *tail), y[:few])
    assert torch.equal(dmm.lora_add_bf16(g["c"][:few].contiguous(), g["x"][:few].contiguous(), *tail), z[:few])


# ------------------------------------------------------------------- norm
@pytest.mark.gpu
@pytest.mark.parametrize("kind", norm.TYPES)
@pytest.mark.parametrize("rows", (1, 37, 2051, 9001))
@pytest.mark.parametrize("cols", norm.COLS)
def test_norm_gradients(dmm, rows, cols, kind):
    """With a mean of 0 and an rstd of 1, xh is x: the sums over the rows."""
    dt = norm.TYPES[kind]
    x, dy = signs((rows, cols), 1).cuda() * 3, signs((rows, cols), 2).cuda()
    zero, one = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    _, dw, db = dmm.layer_norm_backward(dy.to(dt), x.to(dt), torch.ones(cols, dtype=dt, device="cuda"), zero, one)
    for got, want in ((dw, (dy * x).sum(0)), (db, dy.sum(0))):
        same(got, rounded(want) if dt == BF else want)


# ---------------------------------------------------- what the checks see
def differ(a, b):
    return [not torch.equal(p, q) for p, q in zip(a, b)]


def test_a_lost_value_shows():
    """One token out of 8200 left out of the weights' gradients, one K value of
    one projection, one rank of one adapter: the expected values change."""
    args = backward_inputs(8200, 72, 136)
    lost = [t.clone() for t in args]
    lost[0][4096] = 0  # dy of one token
    assert all(differ(backward(*args), backward(*lost)))
    args = forward_inputs(64, 1024, 72)
    for which in (1, 2):
        lost = [t.clone() for t in args]
        lost[which][:, 777] = 0
        assert differ(forward(*args), forward(*lost))[which]
        assert differ(forward(*args), forward(*lost))[0]
    p = adapter_inputs(300, 136, 72, 40, 5, "mixed")
    q = dict(p, b=p["b"].clone())
    q["b"][3, :, 39] = 0
    assert not torch.equal(adapted(p, True), adapted(q, True)) and not torch.equal(adapted(p, False), adapted(q, False))
