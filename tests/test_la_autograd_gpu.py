"""LAFunction with the gradients that autograd really hands over, on the GPU."""
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_that_begin_between_16_byte_boundaries(dtype):
    """Concatenated with one more element in front, outputs and states get back views of one
    gradient that start wherever that element leaves them."""
    B, T, H, d = 1, 150, 2, 128
    g = torch.Generator(device="cuda").manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    data = unit(r(B, T, H, d)), unit(r(B, T, H, d)), r(B, T, H, d).to(dtype), r(B, H, d, d)
    log_decay = torch.tensor([-0.1, -0.01], device="cuda")
    go, gs = r(B, T, H, d).to(dtype), r(B, H, d, d)
    want = kda.la_backward(*data[:3], log_decay, go, data[3], gs)
    leaves = [x.clone().requires_grad_(True) for x in data]
    out, last = kda.LAFunction.apply(*leaves[:3], log_decay, leaves[3])
    one = torch.zeros(1, device="cuda")
    joined = torch.cat([one.to(dtype), out.flatten()]), torch.cat([one, last.flatten()])
    torch.autograd.backward(joined, [torch.cat([one.to(dtype), go.flatten()]), torch.cat([one, gs.flatten()])])
    for x, n in zip(leaves, ("dq", "dk", "dv", "dinitial_state")):
        assert torch.equal(x.grad, want[n])
