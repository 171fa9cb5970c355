"""A call that failed on the host leaves nothing behind that a later, good call would report, on
the GPU.  In a process of its own: the failure spoils a stream capture."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PROGRAM = """
import torch
import gated_delta_rule_109_b200 as kda
from gated_delta_rule_109_b200 import build
build.build()
g = torch.Generator(device="cuda").manual_seed(9)
r = lambda *s: torch.randn(s, generator=g, device="cuda")
decay = torch.tensor([-0.1, -0.01], device="cuda")
prompt = [(0.1 * r(1, 700, 2, 128)).bfloat16() for _ in range(3)]
small = [(0.1 * r(1, 700, 2, 64)) for _ in range(3)]
one = [x[:, 0].contiguous() for x in prompt]
state = r(1, 2, 128, 128)
cache = [r(4, 16, 2, 128).bfloat16() for _ in range(2)]
table = torch.arange(4, dtype=torch.int32, device="cuda").reshape(1, 4)
lengths = torch.tensor([50], dtype=torch.int32, device="cuda")
calls = [lambda: kda.la_decode_step(*one, decay, state), lambda: kda.la_forward(*prompt, decay, state),
         lambda: kda.la_forward(*small, decay), lambda: kda.paged_decode_step(*one, *cache, table, lengths),
         lambda: kda.forward(*prompt, -0.1 * torch.ones((1, 700, 2, 128), device="cuda"),
                             0.5 * torch.ones((1, 700, 2), device="cuda"), state)]
for call in calls:
    call()
    torch.cuda.synchronize()
    refused = False
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            try:
                kda.check_status()          # it synchronises, which a capture does not allow
            except kda.KDAError as e:
                refused = e.status == kda.KDA_ERR_CUDA
    except RuntimeError:
        pass                                # the capture is spoilt
    assert refused
    call()
    torch.cuda.synchronize()
    kda.check_status()
print("good")
"""


def test_a_good_call_after_a_failed_one_is_good():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    run = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0 and "good" in run.stdout, run.stderr[-2000:]
