"""The fp64 definitions of linear attention and paged attention, held against each other's
other forms on the CPU: autograd, differences, the closed form, dense softmax."""
import math

import pytest
import torch

from oracle import attention as ref


def _la_inputs(B, T, H, dk, dv, seed, state=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    return dict(q=r(B, T, H, dk), k=r(B, T, H, dk), v=r(B, T, H, dv),
                log_decay=torch.tensor([-0.7, -0.01, 0.0][:H], dtype=torch.float64),
                initial_state=r(B, H, dk, dv) if state else None)


def test_forward_is_the_decayed_sum_of_all_earlier_tokens():
    x = _la_inputs(2, 9, 3, 4, 5, 1)
    out, last = ref.la_forward(**x)
    a = torch.exp(x["log_decay"])
    for t in range(9):
        want = a[None, :, None] ** (t + 1) * torch.einsum("bhc,bhcd->bhd", x["q"][:, t], x["initial_state"])
        for j in range(t + 1):
            w = a ** (t - j) * (x["q"][:, t] * x["k"][:, j]).sum(-1)
            want = want + w[..., None] * x["v"][:, j]
        assert torch.allclose(out[:, t], want / math.sqrt(4), rtol=1e-12, atol=1e-12)
    want = a[None, :, None, None] ** 9 * x["initial_state"]
    for j in range(9):
        want = want + (a ** (8 - j))[None, :, None, None] * x["k"][:, j, :, :, None] * x["v"][:, j, :, None, :]
    assert torch.allclose(last, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("state", [True, False])
def test_backward_is_autograds(state):
    x = _la_inputs(2, 7, 3, 4, 5, 2, state)
    leaves = [n for n in ("q", "k", "v", "initial_state") if x[n] is not None]
    for n in leaves:
        x[n].requires_grad_(True)
    out, last = ref.la_forward(**x)
    g = torch.Generator().manual_seed(3)
    go, gs = torch.randn(out.shape, generator=g, dtype=torch.float64), torch.randn(last.shape, generator=g, dtype=torch.float64)
    want = torch.autograd.grad((out * go).sum() + (last * gs).sum(), [x[n] for n in leaves])
    got = ref.la_backward(x["q"], x["k"], x["v"], x["log_decay"], go, x["initial_state"], gs)
    for n, w in zip(leaves, want):
        assert torch.allclose(got["d" + n], w, rtol=1e-11, atol=1e-11), n


def test_backward_is_the_slope_of_differences():
    x = _la_inputs(1, 5, 2, 3, 4, 4)
    g = torch.Generator().manual_seed(5)
    go = torch.randn((1, 5, 2, 4), generator=g, dtype=torch.float64)
    gs = torch.randn((1, 2, 3, 4), generator=g, dtype=torch.float64)
    loss = lambda y: sum((a * b).sum() for a, b in zip(ref.la_forward(**y), (go, gs)))
    got = ref.la_backward(x["q"], x["k"], x["v"], x["log_decay"], go, x["initial_state"], gs)
    for n in ("q", "k", "v", "initial_state"):
        step = torch.randn(x[n].shape, generator=g, dtype=torch.float64)
        up, down = dict(x), dict(x)
        up[n], down[n] = x[n] + 1e-5 * step, x[n] - 1e-5 * step
        slope = (loss(up) - loss(down)) / 2e-5
        assert abs(slope - (got["d" + n] * step).sum()) < 1e-7 * (1 + abs(slope)), n


def test_paged_rows_are_dense_softmax():
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    q, k, v, kc, vc = r(4, 4, 8), r(4, 2, 8), r(4, 2, 8), r(9, 3, 2, 8), r(9, 3, 2, 8)
    table = torch.tensor([[0, 1, 2], [3, 4, 5], [6, 99, 7], [8, -1, 0]], dtype=torch.int32)
    lengths = torch.tensor([5, 0, 7, -1], dtype=torch.int32)
    out, _, kc2, _ = ref.paged_decode(q, k, v, kc, vc, table, lengths)
    assert torch.isnan(out[3]).all()                              # idle
    assert torch.equal(out[1, 3], v[1, 1])                        # its own key alone
    assert torch.equal(kc2[1, 2], k[0]) and torch.equal(kc2[3, 0], k[1]) and torch.equal(kc2[7, 1], k[2])
    kk = torch.cat([kc[0], kc[1][:2], k[:1]])[:, 1]
    vv = torch.cat([vc[0], vc[1][:2], v[:1]])[:, 1]
    assert torch.allclose(out[0, 2], torch.softmax(kk @ q[0, 2] / math.sqrt(8), 0) @ vv)
    kk, vv = torch.cat([kc[6], kc[7][:1], k[2:3]])[:, 0], torch.cat([vc[6], vc[7][:1], v[2:3]])[:, 0]
    assert torch.allclose(out[2, 1], torch.softmax(kk @ q[2, 1] / math.sqrt(8), 0) @ vv)     # page 99 is absent
    empty, _, _, _ = ref.paged_decode(q, None, None, kc, vc, table, torch.zeros(4, dtype=torch.int32))
    assert not empty.any()
