"""Workspace queries and refusals make no HIP call (include/dmm.h: argument
errors are returned before any), so a process may size its buffers before it
forks, and a size depends on the problem alone.  The HIP runtime's own log of
the calls made to it is the witness; a call to the runtime itself at the end
shows that the log is being written."""
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import ctypes
import sys
import dense_matmul_amd as dmm
L = dmm.lib()
P = 1 << 20  # an aligned address that is never dereferenced
def say(s):
    sys.stderr.write("=== " + s + "\\n")
    sys.stderr.flush()
say("queries")
for m in (0, 1, 16, 17, 64, 300, 1003, 8192):
    for d, f in ((64, 72), (1024, 896), (7168, 2048)):
        L.layer_norm_backward_workspace(m, d)
        L.gated_ffn_workspace(m, d, f)
        L.gated_ffn_backward_workspace(m, d, f)
        L.gated_up_a8w8_ptpc_workspace(m, d, f)
        L.lora_gemm_workspace(m, f, d, 16)
        L.lora_add_workspace(m, f, d, 16)
say("refusals")
assert L.gated_ffn_bf16(*[P] * 8, 1, 64, 7168, 2048, 0, None) == 1
assert L.gated_ffn_backward_bf16(*[P] * 12, 1, 64, 7168, 2048, 0, None) == 1
assert L.gated_up_a8w8_ptpc(*[P] * 8, 1, 64, 7168, 136, 0, None) == 1
for call in (L.lora_gemm_bf16, L.lora_add_bf16):
    for m in (64, 1000):
        assert call(*[P] * 8, 1, m, 2048, 4096, 16, 4, None) == 1
assert L.layer_norm_backward(*[P] * 9, 1, 4, 64, 1, None) == 1
say("device")
L.hipGetDevice(ctypes.byref(ctypes.c_int()))  # found in the library's own dependency
say("end")
"""


def calls(text):
    return re.findall(r"\b(hip[A-Z]\w*) \(", text)


def test_no_hip_call():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, env={**os.environ, "AMD_LOG_LEVEL": "3"}, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    part = dict(p.split("\n", 1) for p in r.stderr.split("=== ")[1:])
    assert not calls(part["queries"]) and not calls(part["refusals"])
    assert "hipGetDevice" in calls(part["device"])
