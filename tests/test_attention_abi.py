"""Refusals of the linear-attention and paged calls: every bad argument is turned into a
status on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import gated_delta_rule_109_b200 as kda
from gated_delta_rule_109_b200 import build as kbuild

FAKE = 0x100000          # 256-byte aligned, never dereferenced: every call below fails validation
INVALID, UNSUPPORTED, MISALIGNED = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load()


def _fwd(lib, q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, out=FAKE, sT=None, B=1, T=4096, H=2, dk=128, dv=128,
         dtype=kda.KDA_BF16, scale=0.0, ws=FAKE, nbytes=1 << 40):
    return lib.kda_la_forward(q, k, v, g, s0, out, sT, B, T, H, dk, dv, dtype, ctypes.c_float(scale), ws, nbytes, None)


def _bwd(lib, q=FAKE, k=FAKE, v=FAKE, g=FAKE, s0=None, go=FAKE, gs=None, gq=FAKE, gk=FAKE, gv=FAKE, gs0=FAKE,
         B=1, T=4096, H=2, dk=128, dv=128, dtype=kda.KDA_BF16, scale=0.0, ws=FAKE, nbytes=1 << 40):
    return lib.kda_la_backward(q, k, v, g, s0, go, gs, gq, gk, gv, gs0, B, T, H, dk, dv, dtype, ctypes.c_float(scale),
                               ws, nbytes, None)


def _dec(lib, q=FAKE, k=FAKE, v=FAKE, g=FAKE, st=FAKE, out=FAKE, B=1, H=2, dk=128, dv=128, dtype=kda.KDA_BF16,
         scale=0.0):
    return lib.kda_la_decode_step(q, k, v, g, st, out, B, H, dk, dv, dtype, ctypes.c_float(scale), None)


def _paged(lib, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lengths=FAKE, out=FAKE, B=2, H=8, Hkv=2, D=128,
           num_pages=4, page=16, max_pages=2, dtype=kda.KDA_BF16, scale=0.0, ws=FAKE, nbytes=1 << 40):
    return lib.kda_paged_decode_step(q, k, v, kc, vc, table, lengths, out, B, H, Hkv, D, num_pages, page, max_pages,
                                     dtype, ctypes.c_float(scale), ws, nbytes, None)


COMMON = [(dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(B=0), INVALID),
          (dict(H=-1), INVALID), (dict(dk=0), INVALID), (dict(dtype=7), INVALID), (dict(scale=float("nan")), INVALID),
          (dict(scale=float("inf")), INVALID), (dict(B=1 << 15, H=1 << 15), INVALID), (dict(dk=96), UNSUPPORTED),
          (dict(dv=256), UNSUPPORTED), (dict(q=FAKE + 8), MISALIGNED), (dict(v=FAKE + 2), MISALIGNED),
          (dict(g=FAKE + 2), MISALIGNED)]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(out=None), INVALID), (dict(T=-1), INVALID), (dict(T=2 ** 31 - 1), INVALID), (dict(ws=None), INVALID),
    (dict(nbytes=1), INVALID), (dict(out=FAKE + 4), MISALIGNED), (dict(s0=FAKE + 4), MISALIGNED),
    (dict(sT=FAKE + 8), MISALIGNED), (dict(ws=FAKE + 16), MISALIGNED)])
def test_la_forward_refuses(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(go=None), INVALID), (dict(gq=None), INVALID), (dict(gv=None), INVALID), (dict(T=-1), INVALID),
    (dict(ws=None), INVALID), (dict(nbytes=1), INVALID), (dict(gk=FAKE + 4), MISALIGNED),
    (dict(gs=FAKE + 4), MISALIGNED), (dict(gs0=FAKE + 4), MISALIGNED), (dict(ws=FAKE + 16), MISALIGNED)])
def test_la_backward_refuses(lib, kw, code):
    assert _bwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [(dict(st=None), INVALID), (dict(out=None), INVALID),
                                              (dict(st=FAKE + 4), MISALIGNED), (dict(out=FAKE + 2), MISALIGNED)])
def test_la_decode_refuses(lib, kw, code):
    assert _dec(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(table=None), INVALID), (dict(lengths=None), INVALID), (dict(out=None), INVALID),
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(H=7), INVALID), (dict(num_pages=0), INVALID),
    (dict(page=0), INVALID), (dict(max_pages=0), INVALID), (dict(page=1 << 16, max_pages=1 << 15), INVALID),
    (dict(dtype=2), INVALID), (dict(scale=float("inf")), INVALID), (dict(ws=None), INVALID), (dict(nbytes=64), INVALID),
    (dict(B=1 << 20, H=1 << 12, Hkv=1 << 12), INVALID), (dict(D=96), UNSUPPORTED), (dict(q=FAKE + 8), MISALIGNED),
    (dict(kc=FAKE + 8), MISALIGNED), (dict(table=FAKE + 2), MISALIGNED), (dict(lengths=FAKE + 1), MISALIGNED),
    (dict(out=FAKE + 8), MISALIGNED), (dict(ws=FAKE + 64), MISALIGNED)])
def test_paged_decode_refuses(lib, kw, code):
    assert _paged(lib, **kw) == code


def test_no_tokens_and_no_state_is_nothing_to_do(lib):
    none = dict(q=None, k=None, v=None, T=0, ws=None, nbytes=0)
    assert _fwd(lib, out=None, **none) == kda.KDA_OK
    assert _fwd(lib, out=None, s0=FAKE, sT=FAKE, **none) == kda.KDA_OK
    assert _bwd(lib, go=None, gq=None, gk=None, gv=None, gs0=None, **none) == kda.KDA_OK


def test_workspace_sizes(lib):
    fwd = lambda *a, **kw: kda.la_workspace_bytes(*a, **kw)
    state = 128 * 128 * 4
    assert fwd(1, 1, 32, 128, 128) == 0                           # one chunk: nothing to cut
    assert fwd(4, 1 << 16, 148, 128, 128) == 0                    # heads fill the device
    # few heads: many segments, a state for each (and for bf16 what the segments wait on)
    n = fwd(1, 65536, 4, 128, 128, dtype=torch.float32)
    assert n % (4 * state) == 0 and n // (4 * state) > 8
    n = fwd(1, 65536, 4, 128, 128)
    assert n % 256 == 0 and n // (4 * state) > 8
    assert fwd(1, 65536, 4, 128, 128, dtype=torch.float32, backward=True) % (3 * 4 * state) == 0
    assert fwd(0, 8, 2, 128, 128) == 0 and fwd(1, 8, 2, 96, 128) == 0 and fwd(1, 0, 2, 128, 128) == 0
    paged = kda.paged_decode_workspace_bytes
    assert paged(32, 8, 128) > 0 and paged(7, 2, 128) == 0 and paged(8, 2, 96) == 0
    assert paged(8, 8, 64) < paged(128, 8, 64)


def _host(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_refuses_host_tensors(lib):
    q = _host(1, 8, 2, 128)
    q1 = _host(1, 2, 128)
    st = torch.zeros((1, 2, 128, 128))
    cache = _host(3, 16, 2, 128)
    ints = torch.zeros((1, 2), dtype=torch.int32)
    for call in (lambda: kda.la_forward(q, q, q, torch.zeros(2)), lambda: kda.la_backward(q, q, q, None, q),
                 lambda: kda.la_decode_step(q1, q1, q1, None, st),
                 lambda: kda.paged_decode_step(q1, q1, q1, cache, cache, ints, ints[0, :1])):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


def test_log_decay_takes_no_gradient(lib):
    q = _host(1, 8, 2, 128)
    with pytest.raises(ValueError, match="constant"):
        kda.LAFunction.apply(q, q, q, torch.zeros(2, requires_grad=True), None)


def test_the_split_of_the_units_and_its_inverse():
    # paged rows: owner c of G has the units [c U / G, (c + 1) U / G); the joining kernel finds the
    # owner of unit x as ((x + 1) G - 1) / U.  Every owner has a unit, and the two agree.
    import random
    rng = random.Random(3)
    for _ in range(300):
        units, grid = rng.randint(1, 5000), rng.choice((1, 148, 296, 592))
        owners = min(units, grid)
        starts = [c * units // owners for c in range(owners + 1)]
        assert starts[0] == 0 and starts[-1] == units and all(a < b for a, b in zip(starts, starts[1:]))
        assert max(b - a for a, b in zip(starts, starts[1:])) - min(b - a for a, b in zip(starts, starts[1:])) <= 1
        for x in {0, units - 1} | {rng.randrange(units) for _ in range(20)}:
            c = ((x + 1) * owners - 1) // units
            assert starts[c] <= x < starts[c + 1]


def test_division_by_the_page_size():
    # the quotient t / d as (floor(m t / 2^32) + t) / 2^l, for every page size and position allowed
    import random
    rng = random.Random(4)
    for _ in range(20000):
        d = rng.choice((rng.randint(1, 300), rng.randint(1, 2 ** 31 - 1025), 1 << rng.randint(0, 30)))
        t = rng.choice((rng.randint(0, 2 ** 31 - 1), rng.randint(0, 5000), min(2 ** 31 - 1, max(0, d * rng.randint(0, 9) + rng.randint(-1, 1)))))
        l = (d - 1).bit_length()
        m = ((1 << 32) * ((1 << l) - d)) // d + 1
        high = (m * t) >> 32
        assert m < 1 << 32 and high + t < 1 << 32 and (high + t) >> l == t // d
