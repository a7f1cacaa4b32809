"""The loops of the adapters' tile kernels in the emitted gfx950 code (no GPU),
which lie inside a loop over the adapters' ids that test_isa_dense.py's audit of
steady loops leaves out.  From this build's own object:

* the pipelined loop over K (the shared product's, and the first product's)
  waits for all loads only where a step's own wait count is 0, at its barrier:
  once a step with two stages, never with four;
* the loop over an adapter's rank loads a K tile, waits, and meets a barrier
  before and after it is read, and waits nowhere else;
* between the pipelined loop and the next use of its stages the first product's
  outer loop has a wait for all loads (the pipeline's last ones).

Each check must catch an edited disassembly."""
import os
import re
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_isa_dense as dense  # noqa: E402
import test_isa_schedule as isa  # noqa: E402


@pytest.fixture(scope="module")
def kernels():
    from dense_matmul_amd import build

    return {s: v for s, v in isa.parse(build.disassemble("lora.hip")).items() if "lora_tile" in s or "shrink_tile" in s}


def innermost(insns):
    spans = dense.loops(insns)
    return [p for p in spans if not any(q != p and q[0] >= p[0] and q[1] <= p[1] for q in spans)]


def full_waits(span):
    """Of every wait for all loads, whether a barrier comes next."""
    return [span[k + 1][1] == "s_barrier" for k, x in enumerate(span) if x[1] == "s_waitcnt" and "vmcnt(0)" in x[2]]


def faults(sym, insns):
    """What breaks a rule, and how many loops of each kind there are."""
    rows, cols, stages = map(int, re.search(r"CfgILi(\d+)ELi(\d+)ELi(\d+)E", sym).groups())
    tile = 2 * (rows // 32) * (cols // 32)  # a wave's matrix ops of one K tile
    bad, piped, ranks = [], 0, 0
    for lo, hi in innermost(insns):
        span = insns[lo:hi + 1]
        ops, waits, barriers = (sum(x[1].startswith("v_mfma") for x in span), full_waits(span),
                                sum(x[1] == "s_barrier" for x in span))
        if ops == stages * tile:
            piped += 1
            if barriers != stages or len(waits) != (2 if stages == 2 else 0) or not all(waits):
                bad.append(f"pipelined loop: {barriers} barriers, waits {waits}")
        else:
            ranks += 1
            if ops != tile or barriers != 2 or len(waits) != 2 or not all(waits):
                bad.append(f"rank loop: {ops} matrix ops, {barriers} barriers, waits {waits}")
    if "shrink_tile" in sym:
        lo, hi = innermost(insns)[0]
        outer = min((p for p in dense.loops(insns) if p[0] < lo and p[1] > hi), key=lambda p: p[1] - p[0])
        # the pipelined loop's stages are next written by the DMAs of the outer loop's next round
        if not full_waits(insns[hi + 1:outer[1] + 1]):
            bad.append("no wait for the pipeline's last loads")
    return bad, piped, ranks


def test_loops(kernels):
    assert len(kernels) == 6
    for sym, insns in sorted(kernels.items()):
        bad, piped, ranks = faults(sym, insns)
        assert not bad, f"{sym}: " + "; ".join(bad)
        beside_c = "lora_tile" in sym and "ELb0EEEvPKt" in sym
        assert (piped, ranks) == (0 if beside_c else 1, 0 if "shrink_tile" in sym else 1), sym


def test_edits_are_caught(kernels):
    for sym, insns in sorted(kernels.items()):
        lo, hi = innermost(insns)[0]
        stray = insns[:lo + 1] + [(insns[lo][0] + 1, "s_waitcnt", "vmcnt(0)", None)] + insns[lo + 1:]
        assert faults(sym, stray)[0]
        at = next(k for k in range(lo, hi) if insns[k][1] == "s_barrier")
        assert faults(sym, insns[:at] + insns[at + 1:])[0]
    sym = next(s for s in kernels if "shrink_tile" in s)
    insns, (_, hi) = kernels[sym], innermost(kernels[sym])[0]
    assert faults(sym, insns[:hi + 1] + [x for x in insns[hi + 1:] if "vmcnt(0)" not in x[2]])[0]
