"""The process's first linear-attention and paged calls made inside a stream capture, on the GPU."""
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
calls = []
for dt, d in ((torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128)):
    q, k, v, go = ((0.1 * r(1, 3001, 2, d)).to(dt) for _ in range(4))
    s = r(1, 2, d, d)
    one = [x[:, 0].contiguous() for x in (q, k, v)]
    calls.append(lambda q=q, k=k, v=v, s=s: kda.la_forward(q, k, v, decay, s))
    calls.append(lambda q=q, k=k, v=v, s=s, go=go: tuple(kda.la_backward(q, k, v, decay, go, s, s).values()))
    calls.append(lambda one=one, s=s: (kda.la_decode_step(*one, decay, s.clone()),))
    a = [x.to(dt) for x in (r(2, 8, d), r(2, 2, d), r(2, 2, d), r(400, 16, 2, d), r(400, 16, 2, d))]
    table = torch.arange(400, dtype=torch.int32, device="cuda").reshape(2, 200)
    lengths = torch.tensor([3000, 5], dtype=torch.int32, device="cuda")
    calls.append(lambda a=a, t=table, n=lengths: (kda.paged_decode_step(*a, t, n),))
torch.cuda.synchronize()
side = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    got = [c() for c in calls]
graph.replay()
torch.cuda.synchronize()
kda.check_status()
got = [[x.clone() for x in xs] for xs in got]
for xs, c in zip(got, calls):
    assert all(torch.equal(a, b) for a, b in zip(xs, c()))
print("equal")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    run = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]
