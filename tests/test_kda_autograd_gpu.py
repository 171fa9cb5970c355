"""KDAFunction with gradients that begin between 16-byte boundaries, on the GPU."""
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


def test_gradients_that_begin_between_16_byte_boundaries():
    B, T, H, d = 1, 100, 2, 128
    g = torch.Generator(device="cuda").manual_seed(10)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()
    data = (unit(r(B, T, H, d)), unit(r(B, T, H, d)), r(B, T, H, d).bfloat16(), -0.1 * r(B, T, H, d).abs(),
            torch.sigmoid(r(B, T, H)), r(B, H, d, d))
    go, gs = r(B, T, H, d), r(B, H, d, d)
    want = kda.backward(*data[:5], go, data[5], gs)
    leaves = [x.clone().requires_grad_(True) for x in data]
    out, last = kda.KDAFunction.apply(*leaves)
    one = torch.zeros(1, device="cuda")
    joined = [torch.cat([one, x.flatten()]) for x in (out, last)]
    torch.autograd.backward(joined, [torch.cat([one, x.flatten()]) for x in (go, gs)])
    for x, n in zip(leaves, ("dq", "dk", "dv", "dlog_alpha", "dbeta", "dinitial_state")):
        assert torch.equal(x.grad, want[n].to(x.dtype)), n
