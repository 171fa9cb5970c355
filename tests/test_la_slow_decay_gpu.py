"""Thousands of single-token steps of linear attention with slow decays, on the GPU.

Every step rounds the fp32 state once.  With the decay itself exact to well below 2^-24 the
roundings are independent, half a step (2^-24 of the value) at most and 0.41 of that in the root
mean square, so after N steps the 2-norm of a head's error is about 0.41 sqrt(N) 2^-24 of the
largest state on the way; 2 sqrt(N) 2^-24 is five times that.  A decay rounded to one fp32 number
is off by up to 2^-25 in the same direction at every step instead, up to N 2^-25 together.
(The tokens are new ones throughout: of a few that come again and again the roundings repeat, and
a step in exact arithmetic, rounded once, would be 3e-5 off at the slowest decay below.  And
products of two bf16 have 16 bits: added to the state they often leave nothing to round, so that a
decay below half a step of fp32, 2^-25, is lost there even in exact arithmetic: 1e-4 after these
steps at -2e-8, 7e-6 at -1e-6.  The bf16 decays begin at -1e-5.)
"""
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
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_the_state_of_many_steps(dk, dv, dtype):
    steps = 12000
    slowest = [-2e-8, -1e-6] if dtype == torch.float32 else []
    log_decay = torch.tensor(slowest + [-1e-5, -7e-5, -2.0 ** -12, -3.1e-4, -1e-3, -0.02], device="cuda")
    H = log_decay.numel()
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    state = 4 * r(1, H, dk, dv)
    want, decay = state.double(), torch.exp(log_decay.double())[:, None, None]
    most = want.flatten(2).norm(dim=-1)
    for t in range(steps):
        if t % 100 == 0:
            k, v = (0.125 * r(100, 1, H, dk)).to(dtype), r(100, 1, H, dv).to(dtype)
            terms = k.double().unsqueeze(-1) * v.double().unsqueeze(-2)
        kda.la_decode_step(k[t % 100], k[t % 100], v[t % 100], log_decay, state)
        want = decay * want + terms[t % 100]
        most = torch.maximum(most, want.flatten(2).norm(dim=-1))
    kda.check_status()
    err = (state.double() - want).flatten(2).norm(dim=-1) / most
    assert bool((err <= 2 * steps ** 0.5 * 2.0 ** -24).all()), err.tolist()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_end_where_the_prefill_does(dtype):
    B, T, H, d = 1, 4096, 4, 128
    g = torch.Generator(device="cuda").manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    log_decay = torch.tensor([-1e-5, -2.0 ** -12, -7e-5, -1e-3], device="cuda")
    q, k = ((x / x.norm(dim=-1, keepdim=True)).to(dtype) for x in (r(B, T, H, d), r(B, T, H, d)))
    v, state = r(B, T, H, d).to(dtype), 3 * r(B, H, d, d)
    _, last = kda.la_forward(q, k, v, log_decay, state)
    for t in range(T):
        kda.la_decode_step(*(x[:, t].contiguous() for x in (q, k, v)), log_decay, state)
    kda.check_status()
    # the prefill's states are within 1e-5 of the definition's, the steps' as above
    err = (state - last).double().flatten(2).norm(dim=-1) / last.double().flatten(2).norm(dim=-1)
    assert bool((err <= 1e-5 + 2 * T ** 0.5 * 2.0 ** -24).all()), err.tolist()
