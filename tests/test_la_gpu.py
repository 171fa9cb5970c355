"""Linear attention with a decay per head on the GPU against the fp64 token loops.

Tolerances, fixed before the first run.
fp32: |err| <= 1e-5 rms(ref) + 1e-5 |ref|.  A value is a chain of sums of at most 128 + 64 + 128
terms with fp32 products; rounding errors of random sign grow like sqrt(320) 2^-24 = 1.1e-6 of the
terms' size, whose sum of magnitudes stays within a few times the rms.  States (fp32 for both
types, inputs exact) are held to the same bound.
bf16: outputs are rounded once (half a step: 2^-8 of the value), and the kernel may round the
scores and the entering state to bf16 (2^-8 of each term).  With mag the same sums over absolute
values, |err| <= 2^-8 |ref| + 2^-8 (1 + 2^-8) mag + the fp32 bound, element by element; the errors of
the terms are independent, so the 2-norm of the error is also within 2 * 2^-8 of the reference's.
"""
import math

import pytest
import torch

import gated_delta_rule_109_b200 as kda
from oracle import attention as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_109_b200 import build
    build.build()


def _inputs(B, T, H, dk, dv, dtype, seed, state=True, decay="mixed"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-30)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    if decay == "mixed":       # from no memory at all to one that never fades
        kinds = torch.tensor([-0.004, -math.inf, -30.0, 0.0, -0.6, -2.5e-4], device="cuda")
        log_decay = kinds[torch.arange(H, device="cuda") % 6].contiguous()
    else:
        log_decay = None if decay is None else torch.full((H,), float(decay), device="cuda")
    return dict(q=unit(r(B, T, H, dk)).to(dt), k=unit(r(B, T, H, dk)).to(dt), v=r(B, T, H, dv).to(dt),
                log_decay=log_decay, state=0.3 * r(B, H, dk, dv) if state else None,
                go=r(B, T, H, dv).to(dt), gs=0.3 * r(B, H, dk, dv) if state else None)


def _close(got, want, mag=None):
    assert got.shape == want.shape and torch.isfinite(got).all()
    if got.numel() == 0:
        return
    got, rms = got.cpu().double(), float(want.square().mean().sqrt())
    tol = 1e-5 * rms + 1e-5 * want.abs()
    if mag is not None:
        tol = tol + HALF * want.abs() + HALF * (1 + HALF) * mag
        assert float((got - want).norm()) <= 2 * HALF * float(want.norm()) + 1e-30
    err = (got - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()), rms)


def _abs(x):
    return None if x is None else x.abs()


def _check_forward(x, out, last, scale=None):
    want, wl = ref.la_forward(x["q"], x["k"], x["v"], x["log_decay"], x["state"], scale)
    mag = None
    if x["q"].dtype == torch.bfloat16:
        mag, _ = ref.la_forward(x["q"].abs(), x["k"].abs(), x["v"].abs(), x["log_decay"], _abs(x["state"]),
                                None if scale is None else abs(scale))
    _close(out, want, mag)
    if last is not None:
        _close(last, wl)


def _check_backward(x, g, scale=None, state=True):
    a = (x["q"], x["k"], x["v"], x["log_decay"], x["go"], x["state"], x["gs"])
    want = ref.la_backward(*a, scale)
    mag = {n: None for n in want}
    if x["q"].dtype == torch.bfloat16:
        mag = ref.la_backward(*(t if n == 3 else _abs(t) for n, t in enumerate(a)), None if scale is None else abs(scale))
    for n in ("dq", "dk", "dv"):
        assert g[n].dtype == x["q"].dtype
        _close(g[n], want[n], mag[n])
    if state:
        _close(g["dinitial_state"], want["dinitial_state"])


def _forward(x, **kw):
    return kda.la_forward(x["q"], x["k"], x["v"], x["log_decay"], x["state"], **kw)


def _backward(x, **kw):
    return kda.la_backward(x["q"], x["k"], x["v"], x["log_decay"], x["go"], x["state"], x["gs"], **kw)


SHAPES = [(1, 1, 1, 128, 128), (2, 2, 3, 128, 128), (1, 63, 6, 128, 128), (1, 64, 2, 128, 128), (2, 65, 6, 128, 128),
          (1, 127, 2, 128, 128), (1, 128, 6, 128, 128), (2, 129, 3, 128, 128), (1, 300, 6, 128, 128), (3, 257, 2, 128, 128),
          (1, 700, 1, 128, 128), (1, 1, 2, 64, 64), (2, 70, 6, 64, 64), (1, 200, 3, 64, 128), (2, 130, 2, 128, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv", SHAPES)
def test_forward(B, T, H, dk, dv, dtype):
    for state in (False, True):
        x = _inputs(B, T, H, dk, dv, dtype, 100 + T + dk, state)
        out, last = _forward(x)
        kda.check_status()
        assert out.dtype == x["q"].dtype and last.dtype == torch.float32
        _check_forward(x, out, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,dk,dv", SHAPES)
def test_backward(B, T, H, dk, dv, dtype):
    for state in (False, True):
        x = _inputs(B, T, H, dk, dv, dtype, 200 + T + dk, state)
        g = _backward(x)
        kda.check_status()
        _check_backward(x, g)


@pytest.mark.parametrize("decay", [None, -1e-5, -0.05, -1.0, -20.0, -math.inf])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decays(dtype, decay):
    x = _inputs(1, 400, 2, 128, 128, dtype, 7, decay=decay)
    out, last = _forward(x)
    _check_forward(x, out, last)
    _check_backward(x, _backward(x))


@pytest.mark.parametrize("scale", [1.0, -0.37, 1e-3])
def test_scale(scale):
    x = _inputs(1, 150, 3, 128, 128, "bf16", 8)
    out, last = _forward(x, scale=scale)
    _check_forward(x, out, last, scale)
    _check_backward(x, _backward(x, scale=scale), scale)


def test_a_long_sequence_is_cut_into_segments():
    x = _inputs(1, 5003, 2, 128, 128, "bf16", 9, decay=-0.003)
    assert kda.la_workspace_bytes(1, 5003, 2, 128, 128) > 0 and kda.la_workspace_bytes(1, 5003, 2, 128, 128, backward=True) > 0
    out, last = _forward(x)
    _check_forward(x, out, last)
    _check_backward(x, _backward(x))


def test_a_split_call_carries_the_state():
    x = _inputs(2, 500, 3, 128, 128, "bf16", 10)
    whole, last = _forward(x)
    at = 193
    cut = lambda n, s: x[n][:, s].contiguous()
    first = {n: cut(n, slice(0, at)) for n in ("q", "k", "v")}
    second = {n: cut(n, slice(at, None)) for n in ("q", "k", "v")}
    state = x["state"].clone()
    o1, s1 = kda.la_forward(first["q"], first["k"], first["v"], x["log_decay"], state, final_state=state)
    assert s1 is state
    o2, _ = kda.la_forward(second["q"], second["k"], second["v"], x["log_decay"], state, final_state=state)
    _check_forward(x, torch.cat([o1, o2], 1), state)
    _check_forward(x, whole, last)


def test_in_place_state_of_a_cut_sequence():
    x = _inputs(1, 4000, 2, 128, 128, "bf16", 11, decay=-0.01)
    out, last = _forward(x)
    state = x["state"].clone()
    out2, _ = _forward(dict(x, state=state), final_state=state)
    assert torch.equal(out, out2) and torch.equal(last, state)


@pytest.mark.parametrize("dtype,B,T,H,at", [("bf16", 1, 65517, 32, 8191), ("bf16", 3, 9001, 61, 2063),
                                            ("f32", 1, 20011, 20, 3001)])
def test_a_long_call_equals_its_pieces(dtype, B, T, H, at):
    """More work items than the GPU has places for at once, against the same sequence in pieces
    that carry the state (and, backwards, its gradient).  Each side is within the tolerances at
    the top of the reference, so the two are within their sum, head by head."""
    x = _inputs(B, T, H, 128, 128, dtype, 21)
    out, last = _forward(x)
    g = _backward(x)
    pieces = [slice(t, min(t + at, T)) for t in range(0, T, at)]
    cut = lambda s: {n: x[n][:, s].contiguous() for n in ("q", "k", "v", "go")}
    states, state = [], x["state"]
    for s in pieces:
        states.append(state)
        o, state = _forward(dict(x, **cut(s), state=state))
        _same_heads(out[:, s], o, dtype, 2)
    _same_heads(last[:, None], state[:, None], "f32", 3)
    gs = x["gs"]
    for s, state in zip(reversed(pieces), reversed(states)):
        p = _backward(dict(x, **cut(s), state=state, gs=gs))
        gs = p["dinitial_state"]
        for n in ("dq", "dk", "dv"):
            _same_heads(g[n][:, s], p[n], dtype, 2)
    _same_heads(g["dinitial_state"][:, None], gs[:, None], "f32", 3)


def _same_heads(a, b, dtype, head_axis):
    tol = 4 * HALF if dtype == "bf16" else 4e-5
    if head_axis == 3:                      # states [B, 1, H, dk, dv]
        a, b = a.flatten(3), b.flatten(3)
    a, b = (y.transpose(1, 2).flatten(2).double() for y in (a, b))      # [B, H, all of a head]
    assert bool(torch.isfinite(a).all())
    assert bool(((a - b).norm(dim=-1) <= tol * b.norm(dim=-1) + 1e-30).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [0, 1, 100, 128, 300])
def test_a_sequence_padded_with_zeros(dtype, length):
    x = _inputs(2, 389, 6, 128, 128, dtype, 22)
    for n in ("q", "k", "v", "go"):
        x[n][0, length:] = 0
    out, last = _forward(x)
    g = _backward(x)
    assert not out[0, length:].any() and not any(g[n][0, length:].any() for n in ("dq", "dk", "dv"))
    _check_forward(x, out, last)
    _check_backward(x, g)
    short = {n: x[n][:1, :length].contiguous() for n in ("q", "k", "v")}
    y = dict(x, **short, state=x["state"][:1].contiguous(), log_decay=None)
    _, at_end = _forward(y)
    _, padded = _forward(dict(x, log_decay=None))
    assert float((at_end - padded[:1]).norm()) <= 2e-5 * float(at_end.norm())


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("bits", ["nan", "all ones", "inf"])
def test_what_is_not_finite_is_not_lost(dtype, d, bits):
    for n, after in (("q", False), ("k", True), ("v", True)):
        x = _inputs(1, 300, 1, d, d, dtype, 23, decay=-0.01)
        if bits == "all ones":
            x[n].view(torch.int32 if dtype == "f32" else torch.int16)[0, 200, 0, 5] = 0x7fffffff if dtype == "f32" else 0x7fff
        else:
            x[n][0, 200, 0, 5] = float(bits)
        out, last = _forward(x)
        lost = torch.isfinite(out[0, :, 0]).all(-1)
        assert not lost[200] and not (after and lost[200:].any())
        assert torch.isfinite(last).all() == (not after) and bool(lost[:128].all())


def test_no_tokens():
    x = _inputs(2, 0, 3, 128, 128, "bf16", 12)
    out, last = _forward(x)
    assert out.shape == (2, 0, 3, 128) and torch.equal(last, x["state"])
    assert torch.equal(_backward(x)["dinitial_state"], x["gs"])
    out, last = _forward(dict(x, state=None))
    assert not last.any()


def test_outputs_that_are_not_wanted():
    x = _inputs(1, 140, 2, 128, 128, "bf16", 13)
    out, last = _forward(x, return_final_state=False)
    assert last is None
    g = _backward(x, initial_state_grad=False)
    assert g["dinitial_state"] is None
    _check_forward(x, out, None)
    _check_backward(x, g, state=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_results_repeat_and_ignore_what_the_workspace_held(dtype):
    x = _inputs(1, 3000, 2, 128, 128, dtype, 14)
    dt = x["q"].dtype
    n, m = (kda.la_workspace_bytes(1, 3000, 2, 128, 128, dt, backward=b) for b in (False, True))
    ws = torch.full((max(n, m),), 255, dtype=torch.uint8, device="cuda")      # NaN
    out, last = _forward(x)
    out2, last2 = _forward(x, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(last, last2)
    g, g2 = _backward(x), _backward(x, workspace=ws.fill_(255))
    assert all(torch.equal(g[k], g2[k]) for k in g)
    with pytest.raises(kda.KDAError):
        _forward(x, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_rows_next_to_the_outputs_are_left_alone():
    x = _inputs(2, 131, 3, 128, 128, "bf16", 15)
    room = torch.full((2 * 131 * 3 * 128 + 2 * 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = room[4096:-4096].view(2, 131, 3, 128)
    _forward(x, out=out)
    assert bool((room[:4096] == 7).all()) and bool((room[-4096:] == 7).all())
    _check_forward(x, out, None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 128, 128), (3, 5, 128, 128), (40, 8, 128, 128), (2, 3, 64, 64),
                                       (200, 3, 64, 64), (2, 3, 64, 128), (90, 4, 64, 128), (2, 3, 128, 64),
                                       (90, 4, 128, 64)])
def test_decode_steps_follow_the_prefill(B, H, dk, dv, dtype):
    x = _inputs(B, 5, H, dk, dv, dtype, 300 + B + dk)
    state = x["state"].clone()
    outs = []
    for t in range(5):
        outs.append(kda.la_decode_step(*(x[n][:, t].contiguous() for n in ("q", "k", "v")), x["log_decay"], state))
        assert outs[-1].dtype == x["q"].dtype
    _check_forward(x, torch.stack(outs, 1), state)


def test_captured_calls_replay_on_new_data():
    x, y = _inputs(1, 3001, 2, 128, 128, "bf16", 16), _inputs(1, 3001, 2, 128, 128, "bf16", 17)
    hold = {n: t.clone() if t is not None else None for n, t in x.items()}
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        _forward(hold), _backward(hold)
        side.synchronize()
        for call in (_forward, _backward):          # two graphs, each with a workspace of its own
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                got = call(hold)
            graphs.append((graph, got))
    for src in (y, x):
        for n in hold:
            if hold[n] is not None:
                hold[n].copy_(src[n])
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want_f, want_b = _forward(src), _backward(src)
        assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want_f))
        assert all(torch.equal(graphs[1][1][n], want_b[n]) for n in want_b)
    kda.check_status()


def test_two_calls_at_once_on_two_streams():
    xs = [_inputs(1, 6000, 2, 128, 128, "bf16", s) for s in (18, 19)]
    want = [_forward(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _forward(xs[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd_function(dtype):
    x = _inputs(2, 150, 2, 128, 128, dtype, 20)
    leaves = {n: x[n].clone().requires_grad_(True) for n in ("q", "k", "v", "state")}
    out, last = kda.LAFunction.apply(leaves["q"], leaves["k"], leaves["v"], x["log_decay"], leaves["state"])
    torch.autograd.backward([out, last], [x["go"], x["gs"]])
    _check_backward(x, dict(dq=leaves["q"].grad, dk=leaves["k"].grad, dv=leaves["v"].grad,
                            dinitial_state=leaves["state"].grad))
    # the outputs alone, from a zero state
    leaves = {n: x[n].clone().requires_grad_(True) for n in ("q", "k", "v")}
    out, _ = kda.LAFunction.apply(leaves["q"], leaves["k"], leaves["v"], x["log_decay"], None)
    out.backward(x["go"])
    _check_backward(dict(x, state=None, gs=None), {"d" + n: t.grad for n, t in leaves.items()}, state=False)


def test_gradients_are_the_slopes_of_differences():
    x = _inputs(1, 90, 2, 64, 64, "f32", 21, decay=-0.05)
    g = _backward(x)
    gen = torch.Generator(device="cuda").manual_seed(22)

    def loss(y):
        out, last = _forward(y)
        return float((out.double() * x["go"].double()).sum() + (last.double() * x["gs"].double()).sum())

    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("state", "dinitial_state")):
        step = torch.randn(x[n].shape, generator=gen, device="cuda")
        # the loss is linear in each input alone: a wide step has no curvature, and drowns rounding
        slope = (loss(dict(x, **{n: x[n] + step})) - loss(dict(x, **{n: x[n] - step}))) / 2
        want = float((g[gn].double() * step.double()).sum())
        size = float(g[gn].double().norm() * step.double().norm())
        assert abs(slope - want) <= 1e-5 * size, n


def test_refusals_of_the_binding():
    x = _inputs(1, 20, 3, 128, 128, "bf16", 30)
    call = lambda **kw: _forward(dict(x, **kw))
    with pytest.raises(ValueError, match="contiguous"):
        call(k=x["k"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="shape"):
        call(k=x["k"][:, :19].contiguous())
    with pytest.raises(ValueError, match="log_decay"):
        call(log_decay=x["log_decay"][:2].contiguous())
    with pytest.raises(TypeError, match="v must be"):
        call(v=x["v"].float())
    with pytest.raises(TypeError):
        call(q=x["q"].half(), k=x["k"].half(), v=x["v"].half())
    with pytest.raises(ValueError, match="initial_state is on"):
        call(state=x["state"].cpu())
    with pytest.raises(TypeError, match="out must be"):
        _forward(x, out=torch.empty(x["v"].shape, device="cuda"))
    with pytest.raises(kda.KDAError, match="MISALIGNED"):
        room = torch.empty(x["q"].numel() + 1, dtype=torch.bfloat16, device="cuda")
        call(q=room[1:].view(x["q"].shape))
    with pytest.raises(kda.KDAError, match="UNSUPPORTED"):
        _forward({n: (t[..., :96].contiguous() if n in ("q", "k") else None if n in ("state", "gs") else t) for n, t in x.items()})


def test_no_second_derivative():
    x = _inputs(1, 20, 2, 64, 64, "f32", 31, state=False)
    q = x["q"].requires_grad_(True)
    out, _ = kda.LAFunction.apply(q, x["k"], x["v"], x["log_decay"], None)
    (g,) = torch.autograd.grad(out.square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
