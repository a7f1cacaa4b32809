"""The package imports on a torch that lacks the private call by which the
stream's handle is read in one step; the public way gives the same handle."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(program):
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_import_without_the_private_call():
    run("import torch\n"
        "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
        "import dense_matmul_amd as dmm\n"
        "class Stream:\n"
        "    def __init__(self, dev): self.cuda_stream = 1000 + dev\n"
        "torch.cuda.current_stream = Stream\n"
        "assert dmm._raw_stream(3) == 1003\n")


@pytest.mark.gpu
def test_operators_without_the_private_call():
    run("import torch\n"
        "x, w, b = torch.zeros(5, 64, device='cuda'), torch.randn(64, device='cuda'), torch.randn(64, device='cuda')\n"
        "side = torch.cuda.Stream()\n"
        "private = getattr(torch._C, '_cuda_getCurrentRawStream', None)\n"
        "if private is not None: del torch._C._cuda_getCurrentRawStream\n"
        "import dense_matmul_amd as dmm\n"
        "with torch.cuda.stream(side):\n"
        "    assert dmm._raw_stream(0) == side.cuda_stream\n"
        "    assert private is None or private(0) == side.cuda_stream\n"
        "torch.cuda.synchronize()\n"
        "assert torch.equal(dmm.layer_norm(x, w, b), b.expand(5, 64))\n")
