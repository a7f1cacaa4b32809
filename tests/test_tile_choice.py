"""Every kernel that the feed-forward block and the adapters choose by size
(csrc/dense_pick.h) is run by a GPU test: the choice is computed on the host for
every size of test_gpu_ffn.py, test_gpu_lora.py and test_gpu_tiles.py.  A change
to the time model behind it that takes a kernel out of the tests' reach fails
here; so does one that makes the header need more than a C++ compiler."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_matmul_amd", "csrc")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import test_gpu_ffn as ffn  # noqa: E402
import test_gpu_lora as lora  # noqa: E402
import test_gpu_tiles as tiles  # noqa: E402

PROGRAM = r"""
#include "dense_pick.h"
#include <cstdio>
#include <cstring>
using namespace dmm;

// kb: bytes of a row, by which the kernels for few tokens are chosen
static const char* of(dense::Tile t, long kb) {
    static const char* names[] = {"256", "128", "128D", "64", "split"};
    const int w = thin::waves_for(kb);
    return t != dense::kThin ? names[t] : w == 16 ? "16w" : w == 8 ? "8w" : "4w";
}

int main() {
    char op[32];
    long m, k, n, r, a;
    while (scanf("%31s %ld %ld %ld %ld %ld", op, &m, &k, &n, &r, &a) == 6) {
        if (!strcmp(op, "forward")) {
            printf("up:%s ", of(ffn::up_choice(m, k, n, 2).tile, 2 * k));
            printf("down:%s", of(m <= ffn::kThinMost ? dense::kThin : ffn::product_choice(m, k, n, false).tile, 2 * n));
        } else if (!strcmp(op, "fp8")) {
            printf("up8:%s", of(ffn::up_choice(m, k, n, 1).tile, k));
        } else if (!strcmp(op, "backward")) {
            printf("dh:%s ", of(ffn::product_choice(m, n, k, false).tile, 0));
            if (ffn::grads_with_dx(m, k, n))
                printf("dx+dw");
            else
                printf("dx:%s dw:%s", of(ffn::product_choice(m, k, n, true).tile, 0), of(ffn::grads_choice(m, k, n), 0));
        } else if (m <= lora::kJoinMost) {
            printf("v:%d%s base:%s", lora::shrink_mb(r), lora::shrink_with_base(lora::shrink_blocks(m, k, r, a)) ? "+base" : "",
                   lora::base_plan(m, n, k).shares > 1 ? "shares" : "one");
        } else {
            printf("y:%s vshares:%s", of(lora::second_choice(m, n, k), 0), lora::shrink_plan(m, k, r).shares > 1 ? "many" : "one");
        }
        printf("\n");
    }
}
"""
TILES = ("256", "128", "128D", "64", "split")
EVERY = ({f"{p}:{t}" for p in ("up", "up8", "down") for t in TILES + ("16w", "8w", "4w")} | {f"{p}:{t}" for p in ("dh", "dx") for t in TILES} |
         {f"{p}:{t}" for p in ("dw", "y") for t in TILES[:4]} | {"dx+dw", "base:shares", "base:one", "vshares:many", "vshares:one"} |
         {f"v:{mb}{b}" for mb in (1, 2, 4) for b in ("", "+base")})


def sizes(module, name, names):
    """What the test of that name is parametrised with over these arguments."""
    for mark in getattr(module, name).pytestmark:
        if mark.name == "parametrize" and mark.args[0] == names:
            return mark.args[1]
    raise AssertionError(f"{name} has no parameters {names}")


def cases():
    out = []
    for module in (ffn, tiles):
        out += [("forward", *s, 0, 0) for s in sizes(module, "test_forward", "m,d,f")]
        out += [("backward", *s, 0, 0) for s in sizes(module, "test_backward", "m,d,f")]
        out += [("fp8", *s, 0, 0) for s in sizes(module, "test_fp8_up", "m,d,f")]
    for module in (lora, tiles):
        for m, n, k, r, adapters in sizes(module, "test_against_the_definition", "m,n,k,r,adapters"):
            out.append(("lora", m, k, n, r, adapters))
    return out


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    work = tmp_path_factory.mktemp("pick")
    (work / "t.cpp").write_text(PROGRAM)
    exe = str(work / "t")
    subprocess.run(["g++", "-std=c++20", "-O1", "-Wall", "-Werror", "-I", CSRC, str(work / "t.cpp"), "-o", exe], check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        return [set(line.split()) for line in subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()]

    return run


def test_every_choice_is_run_by_a_gpu_test(choose):
    made = choose(cases())
    assert len(made) == len(cases()) and set().union(*made) <= EVERY
    assert not EVERY - set().union(*made)


def test_dropped_sizes_are_missed(choose):
    """The check sees it when the sizes that reach a choice are gone."""
    all_cases = cases()
    made = choose(all_cases)
    keep = [c for c, branches in zip(all_cases, made) if "dh:256" not in branches]
    assert len(keep) < len(all_cases) and "dh:256" in EVERY - set().union(*choose(keep))
