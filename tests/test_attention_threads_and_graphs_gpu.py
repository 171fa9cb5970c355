"""The linear-attention and paged calls from several host threads, and a training step through
LAFunction captured whole, on the GPU."""
import subprocess
import sys
import threading

import pytest
import torch

import gated_delta_rule_109_b200 as kda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_109_b200 import build
    build.build()


def _work(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    decay = torch.tensor([-0.1, -0.01, -0.001], device="cuda")
    calls = []
    for dt, d in ((torch.bfloat16, 128), (torch.float32, 64)):
        q, k, v, go = ((0.1 * r(1, 2000, 3, d)).to(dt) for _ in range(4))
        s, one = r(1, 3, d, d), [x[:, 7].contiguous() for x in (q, k, v)]
        a = [x.to(dt) for x in (r(2, 8, d), r(2, 2, d), r(2, 2, d), r(80, 16, 2, d), r(80, 16, 2, d))]
        table = torch.arange(80, dtype=torch.int32, device="cuda").reshape(2, 40)
        lengths = torch.tensor([600, 5], dtype=torch.int32, device="cuda")
        calls += [lambda q=q, k=k, v=v, s=s: kda.la_forward(q, k, v, decay, s),
                  lambda q=q, k=k, v=v, s=s, go=go: tuple(kda.la_backward(q, k, v, decay, go, s, s).values()),
                  lambda one=one, s=s: (kda.la_decode_step(*one, decay, s.clone()),),
                  lambda a=a, t=table, n=lengths: (kda.paged_decode_step(*a, t, n),)]
    return calls


def test_calls_from_several_threads():
    works = [_work(s) for s in range(4)]
    want = [[c() for c in calls] for calls in works]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = [c() for c in works[i]]
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for x, y in zip(got, want[i]) for a, b in zip(x, y)):
                        wrong.append(i)
        except Exception as e:                      # a thread's own error would be lost
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    kda.check_status()
    assert not wrong, wrong


STEP = """
import torch
import gated_delta_rule_109_b200 as kda
from gated_delta_rule_109_b200 import build
build.build()
g = torch.Generator(device="cuda").manual_seed(11)
r = lambda *s: torch.randn(s, generator=g, device="cuda")
decay = torch.tensor([-0.1, -0.001], device="cuda")
for dt, d in ((torch.bfloat16, 128), (torch.float32, 64)):
    data = [0.1 * r(1, 1500, 2, d).to(dt) for _ in range(3)] + [r(1, 2, d, d)]
    weight, other = r(1, 1500, 2, d).to(dt), [0.1 * r(1, 1500, 2, d).to(dt) for _ in range(3)] + [r(1, 2, d, d)]

    def step(leaves):
        out, last = kda.LAFunction.apply(*leaves[:3], decay, leaves[3])
        loss = (out * weight).float().sum() + (last * last).sum()
        loss.backward()
        return loss

    def eager(values):
        leaves = [x.clone().requires_grad_(True) for x in values]
        loss = step(leaves)
        return [loss.detach()] + [x.grad for x in leaves]

    leaves = [x.clone().requires_grad_(True) for x in data]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step(leaves)
            for x in leaves:
                x.grad = None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss = step(leaves)
    for values in (data, other):
        with torch.no_grad():
            for x, y in zip(leaves, values):
                x.copy_(y)
        for x in leaves:
            x.grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got, want = [loss.detach()] + [x.grad for x in leaves], eager(values)
        assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
kda.check_status()
print("equal")
"""


def test_a_captured_training_step():
    """In a process of its own: a capture that goes wrong spoils the ones after it."""
    run = subprocess.run([sys.executable, "-c", STEP], capture_output=True, text=True, timeout=600)
    assert run.returncode == 0 and "equal" in run.stdout, run.stderr[-2000:]
