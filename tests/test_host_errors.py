"""What the tensor-core call of the linear attention reports where the host side of a launch
fails (no GPU needed: a process that sees no device)."""
import os
import subprocess
import sys

from gated_delta_rule_109_b200 import build as kbuild

PROGRAM = """
import ctypes
import gated_delta_rule_109_b200 as kda
lib, at = kda.load(), 0x100000
for call in range(2):
    st = lib.kda_la_forward(at, at, at, None, None, at, None, 1, 4096, 2, 128, 128, kda.KDA_BF16, ctypes.c_float(0), at, 1 << 40, None)
    print(st, lib.kda_last_cuda_error().decode())
st = lib.kda_la_forward(at, at, at, None, None, at, None, 1, 64, 2, 64, 64, kda.KDA_F32, ctypes.c_float(0), None, 0, None)
print(st, lib.kda_last_cuda_error().decode())
"""


def test_the_reason_is_reported_every_time():
    """Both kernels of the linear attention meet the same failure, so they name the same reason:
    neither the lookup of the tensor-map encoder nor the look at the kernel's registers hides it."""
    kbuild.build()
    run = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=600,
                         env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert run.returncode == 0, run.stderr
    lines = run.stdout.strip().splitlines()
    assert len(lines) == 3 and len(set(lines)) == 1, lines
    assert lines[0].startswith("4 cuda") and "NotSupported" not in lines[0], lines
