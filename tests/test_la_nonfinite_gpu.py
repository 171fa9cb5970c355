"""Tokens that are not finite in a sequence that linear attention cuts into segments, on the GPU:
what the contract allows them to reach is their own chunk of 128 tokens and what comes after it in
the walk, never a chunk before it."""
import math

import pytest
import torch

import gated_delta_rule_109_b200 as kda

pytestmark = pytest.mark.gpu
CHUNK = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_109_b200 import build
    build.build()


def _inputs(T, H, d, dtype):
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    return dict(q=unit(r(1, T, H, d)), k=unit(r(1, T, H, d)), v=r(1, T, H, d).to(dtype), go=r(1, T, H, d).to(dtype),
                state=0.3 * r(1, H, d, d), gs=0.3 * r(1, H, d, d),
                log_decay=torch.full((H,), -0.003, device="cuda"))


def _rows(x):
    """Tokens of head 0 whose whole row is finite."""
    return torch.isfinite(x[0, :, 0]).all(-1)


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128), (torch.float32, 64)])
@pytest.mark.parametrize("name,bad", [("k", math.nan), ("v", math.inf), ("v", -math.inf)])
def test_earlier_chunks_of_the_segment_stay_finite(dtype, d, name, bad):
    T, H = 5003, 2
    assert kda.la_workspace_bytes(1, T, H, d, d, dtype) > 0         # it is cut
    clean = _inputs(T, H, d, dtype)
    whole, _ = kda.la_forward(clean["q"], clean["k"], clean["v"], clean["log_decay"], clean["state"])
    for t in range(100, T, 3 * CHUNK):
        x = dict(clean, **{name: clean[name].clone()})
        x[name][0, t, 0, 9] = bad
        out, last = kda.la_forward(x["q"], x["k"], x["v"], x["log_decay"], x["state"])
        first = t // CHUNK * CHUNK
        assert torch.equal(out[:, :first], whole[:, :first]), t     # nothing of an earlier chunk moves
        assert torch.equal(out[:, :, 1], whole[:, :, 1])            # nor of the other head
        assert not _rows(out)[t:].any() and not torch.isfinite(last[0, 0]).all()
    kda.check_status()


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 128)])
@pytest.mark.parametrize("name,bad", [("go", math.nan), ("q", math.inf), ("k", math.nan), ("v", math.inf)])
def test_gradients_of_the_chunks_that_the_walk_has_passed_stay_finite(dtype, d, name, bad):
    T, H = 5003, 2
    assert kda.la_workspace_bytes(1, T, H, d, d, dtype, backward=True) > 0
    clean = _inputs(T, H, d, dtype)
    call = lambda x: kda.la_backward(x["q"], x["k"], x["v"], x["log_decay"], x["go"], x["state"], x["gs"])
    whole = call(clean)
    for t in range(100, T, 3 * CHUNK):
        x = dict(clean, **{name: clean[name].clone()})
        x[name][0, t, 0, 9] = bad
        got = call(x)
        first, behind = t // CHUNK * CHUNK, (t // CHUNK + 1) * CHUNK
        # dq walks forwards over k and v, dk and dv walk backwards over q and grad_out
        assert torch.equal(got["dq"][:, :first], whole["dq"][:, :first]), t
        for n in ("dk", "dv"):
            assert torch.equal(got[n][:, behind:], whole[n][:, behind:]), (n, t)
        if name in ("go", "q"):
            assert not torch.isfinite(got["dinitial_state"][0, 0]).all()
        else:
            assert torch.equal(got["dinitial_state"], whole["dinitial_state"])
            assert not _rows(got["dq"])[t:].any()
    kda.check_status()
