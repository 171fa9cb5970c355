"""Linear attention with a 64-channel head or in fp32, held to what those kernels promise, on the GPU.

bf16 with a 64-channel head: operands go in as two parts or exactly, so the only rounding to bf16 is
the output's, half a step, 2^-8 of the value.  Before it an output is a sum whose accumulator cuts
what it adds off, at most 2^-23 of the terms' magnitudes a step: (dk / 8) steps for the scores, 3 dk / 8
and 16 for the output, 80 at most, 9.5e-6; the parts leave 2^-22 of a term, four times at most, 1e-6; the
state is within 1e-5.  Together 2e-5 of mag, the same sums over absolute values: |err| <=
2^-8 |ref| + 2e-5 mag.  (A lost second part, 2^-12 of every term, is 8e-5 to 1.6e-4 of mag off at
some of the elements.)

bf16 with 128-channel heads also rounds the scores and the entering state, 0.41 x 2^-8 of each term in
the root mean square; for independent terms that is the same share of the two halves of the output, so
with the output's own rounding sqrt(2) x 1.6e-3 = 2.3e-3 of its norm: held to 3e-3.
"""
import pytest
import torch

import gated_delta_rule_109_b200 as kda
from oracle import attention as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
MIXED = [(64, 64), (64, 128), (128, 64)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_109_b200 import build
    build.build()


def _inputs(B, T, H, dk, dv, dtype, seed, decays=(-0.004, -0.6, 0.0, -2.5e-4)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    return dict(q=unit(r(B, T, H, dk)), k=unit(r(B, T, H, dk)), v=r(B, T, H, dv).to(dtype), go=r(B, T, H, dv).to(dtype),
                log_decay=torch.tensor(decays, device="cuda")[torch.arange(H, device="cuda") % len(decays)].contiguous(),
                state=0.3 * r(B, H, dk, dv), gs=0.3 * r(B, H, dk, dv))


def _forward(x):
    return kda.la_forward(x["q"], x["k"], x["v"], x["log_decay"], x["state"])


def _backward(x):
    return kda.la_backward(x["q"], x["k"], x["v"], x["log_decay"], x["go"], x["state"], x["gs"])


def _within(got, want, mag):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= HALF * want.abs() + 2e-5 * mag).all()), float((err - HALF * want.abs()).div(mag).max())


@pytest.mark.parametrize("dk,dv", MIXED)
@pytest.mark.parametrize("B,T,H", [(2, 70, 4), (1, 129, 4), (1, 1000, 2)])
def test_one_rounding_of_a_64_channel_head(B, T, H, dk, dv):
    x = _inputs(B, T, H, dk, dv, torch.bfloat16, 40 + T + dk)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    out, last = _forward(x)
    want, wl = ref.la_forward(*a, x["state"])
    mag, ml = ref.la_forward(*(t.abs() for t in a[:3]), a[3], x["state"].abs())
    _within(out, want, mag)
    assert bool(((last.cpu().double() - wl).abs() <= 1e-5 * ml).all())
    g = _backward(x)
    want = ref.la_backward(*a, x["go"], x["state"], x["gs"])
    mag = ref.la_backward(*(t.abs() for t in a[:3]), a[3], *(x[n].abs() for n in ("go", "state", "gs")))
    for n in ("dq", "dk", "dv"):
        _within(g[n], want[n], mag[n])
    assert bool(((g["dinitial_state"].cpu().double() - want["dinitial_state"]).abs() <= 1e-5 * mag["dinitial_state"]).all())
    kda.check_status()


def test_three_roundings_of_a_128_channel_head():
    x = _inputs(1, 900, 4, 128, 128, torch.bfloat16, 50)
    out, _ = _forward(x)
    want, _ = ref.la_forward(x["q"], x["k"], x["v"], x["log_decay"], x["state"])
    assert float((out.cpu().double() - want).norm() / want.norm()) <= 3e-3
    g = _backward(x)
    want = ref.la_backward(x["q"], x["k"], x["v"], x["log_decay"], x["go"], x["state"], x["gs"])
    for n in ("dq", "dk", "dv"):
        assert float((g[n].cpu().double() - want[n]).norm() / want[n].norm()) <= 3e-3, n


def _same(a, b, tol):
    """Head by head: [B, T, H, d]."""
    a, b = a.double(), b.double()
    assert bool(torch.isfinite(a).all())
    assert bool(((a - b).pow(2).sum((1, 3)).sqrt() <= tol * b.pow(2).sum((1, 3)).sqrt() + 1e-30).all())


@pytest.mark.parametrize("dtype,dk,dv,B,T,H,at", [(torch.bfloat16, 64, 64, 1, 30011, 20, 4099), (torch.bfloat16, 64, 128, 2, 9001, 90, 2063),
                                                  (torch.bfloat16, 128, 64, 1, 20011, 8, 3001), (torch.float32, 64, 64, 1, 30011, 20, 4099),
                                                  (torch.float32, 128, 64, 2, 9001, 40, 2063)])
def test_a_long_call_equals_its_pieces(dtype, dk, dv, B, T, H, at):
    """The same sequence at once, cut into segments, and in pieces that carry the state (and, backwards,
    its gradient).  Outputs in bf16: each side is one rounding, 0.41 x 2^-8 of its norm, from nearly the
    same value; the rest within twice 1e-5 and 2e-5."""
    x = _inputs(B, T, H, dk, dv, dtype, 60 + dk)
    tol = 3.5e-3 if dtype == torch.bfloat16 else 4e-5
    heads = lambda y: y.transpose(1, 2)                     # states [B, H, dk, dv] as outputs are after this
    out, last = _forward(x)
    g = _backward(x)
    pieces = [slice(t, min(t + at, T)) for t in range(0, T, at)]
    cut = lambda s: {n: x[n][:, s].contiguous() for n in ("q", "k", "v", "go")}
    states, state = [], x["state"]
    for s in pieces:
        states.append(state)
        o, state = _forward(dict(x, **cut(s), state=state))
        _same(out[:, s], o, tol)
    _same(heads(last), heads(state), 4e-5)
    gs = x["gs"]
    for s, state in zip(reversed(pieces), reversed(states)):
        p = _backward(dict(x, **cut(s), state=state, gs=gs))
        gs = p["dinitial_state"]
        for n in ("dq", "dk", "dv"):
            _same(g[n][:, s], p[n], tol)
    _same(heads(g["dinitial_state"]), heads(gs), 4e-5)
    kda.check_status()


@pytest.mark.parametrize("dtype,dk,dv", [(torch.float32, 128, 128), (torch.float32, 64, 64), (torch.bfloat16, 64, 64), (torch.bfloat16, 64, 128)])
def test_calls_at_once_on_two_streams(dtype, dk, dv):
    """Cut sequences: each call is two launches (more for gradients), the second of which may begin
    while the first ends."""
    xs = [_inputs(1, 3001, 3, dk, dv, dtype, s) for s in (70, 71)]
    assert kda.la_workspace_bytes(1, 3001, 3, dk, dv, dtype) > 0
    want = [(*_forward(x), *_backward(x).values()) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((*_forward(xs[i]), *_backward(xs[i]).values()))
    torch.cuda.synchronize()
    for mine, w in zip(got, want):
        for run in mine:
            assert all(torch.equal(a, b) for a, b in zip(run, w))
    kda.check_status()
