"""Paged decode attention on the GPU against the fp64 definition.

Tolerances, fixed before the first run: with mag = sum_j p_j |v_j|, fp32 scores of at most 128
products are off by a few 1e-6 at the sizes drawn here, which moves a probability by as much, and
the sums round like sqrt(keys) 2^-24: |err| <= 2e-5 mag.  bf16 adds the rounding of the output,
2^-8 |ref|, and allows probabilities rounded to bf16: 2^-8 mag.
"""
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


def _case(lengths, H, Hkv, D, page, dtype, seed, spare=3, new=True, hostile=True):
    """Rows of the given lengths on shuffled pages; everything that no key may come from is NaN
    or an infinity."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    B = len(lengths)
    per = max(max(lengths), 0) // page + 1
    pages = torch.randperm(B * per + spare, generator=g, device="cuda")[: B * per].to(torch.int32).reshape(B, per).contiguous()
    x = dict(q=r(B, H, D), k=r(B, Hkv, D) if new else None, v=r(B, Hkv, D) if new else None,
             k_cache=r(B * per + spare, page, Hkv, D), v_cache=r(B * per + spare, page, Hkv, D),
             block_table=pages, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    if hostile:
        used = torch.zeros(x["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(lengths):
            at = torch.arange(max(n, 0), device="cuda")
            used[pages[b, at // page].long(), at % page] = True
        x["k_cache"][~used] = float("nan")
        x["v_cache"][~used] = float("inf")
    return x


def _call(x, **kw):
    return kda.paged_decode_step(x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"], x["block_table"], x["lengths"], **kw)


def _check(x, before, out, scale=None):
    """`before`: the caches before the call."""
    want, mag, kc, vc = ref.paged_decode(x["q"], x["k"], x["v"], *before, x["block_table"], x["lengths"], scale)
    rows = ~torch.isnan(want).all(-1).all(-1)
    got, want, mag = out.cpu().double()[rows], want[rows], mag[rows]
    tol = 2e-5 * mag
    if out.dtype == torch.bfloat16:
        tol = tol + HALF * want.abs() + HALF * mag
    err = (got - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
    bits = lambda t: t.cpu().contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)
    assert torch.equal(bits(x["k_cache"]), bits(kc)) and torch.equal(bits(x["v_cache"]), bits(vc))


def _run(x, scale=0.0, **kw):
    before = (x["k_cache"].clone(), x["v_cache"].clone())
    out = _call(x, scale=scale, **kw)
    kda.check_status()
    assert out.dtype == x["q"].dtype
    _check(x, before, out, scale or None)
    return out


LENGTHS = [0, 1, 2, 14, 15, 16, 17, 47, 62, 63, 64, 65, 127, 128, 200, 511, 700]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 2), (6, 2), (7, 1), (8, 1), (18, 2), (32, 2), (40, 1)])
def test_groups_and_lengths(H, Hkv, D, dtype):
    _run(_case(LENGTHS, H, Hkv, D, 16, dtype, 1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("page", [1, 7, 8, 16, 64, 100, 256, 1000])
def test_page_sizes(page, dtype):
    _run(_case(LENGTHS, 8, 2, 128, page, dtype, 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[5000], [1], [0], [20000, 3], [3, 20000], [64 * 300 - 1] * 2, [40] * 300, [-1, 9000, -1]])
def test_splits(lengths, dtype):
    _run(_case(lengths, 8, 2, 128, 32, dtype, 3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_idle_and_empty_rows(dtype):
    x = _case([-1, 5, -7, 0, 300, -1], 8, 2, 128, 16, dtype, 4)
    out = torch.full_like(x["q"], 3.0)
    _run(x, out=out)
    assert bool((out[[0, 2, 5]] == 3).all())
    x = _case([-1, 5, 0, 300, 0], 8, 2, 128, 16, dtype, 5, new=False)
    out = torch.full_like(x["q"], 3.0)
    _run(x, out=out)
    assert bool((out[0] == 3).all()) and not out[[2, 4]].any()
    x = _case([-1, -1], 8, 2, 128, 16, dtype, 6)
    out = torch.full_like(x["q"], 3.0)
    _run(x, out=out)
    assert bool((out == 3).all())
    x = _case([0, 0], 8, 2, 128, 16, dtype, 6, new=False)
    assert not _run(x).any()


def test_reading_alone_leaves_the_cache():
    for dtype in ("f32", "bf16"):
        _run(_case([1, 17, 64, 3000], 8, 2, 64, 16, dtype, 7, new=False))


@pytest.mark.parametrize("scale", [1.0, -0.5, 4.0])
def test_scales_and_peaked_rows(scale):
    # 4.0 puts nearly all weight on single keys: the running maximum rises late and often
    x = _case([900, 33, 2000], 8, 2, 128, 16, "f32", 8)
    before = (x["k_cache"].clone(), x["v_cache"].clone())
    out = _call(x, scale=scale)
    want, mag, _, _ = ref.paged_decode(x["q"], x["k"], x["v"], *before, x["block_table"], x["lengths"], scale)
    # scores reach |s| ~ 4 * 5 * sqrt(128) = 230: an fp32 score is off by up to 230 * 2^-22, its weight by as much
    tol = (2e-5 + 230 * 2.0 ** -22 * abs(scale)) * mag
    assert bool(((out.cpu().double() - want).abs() <= tol).all())


def test_infinite_scores():
    # a key of -inf weighs nothing, whichever keys stand before it
    x = _case([70, 3], 2, 1, 64, 16, "f32", 9, hostile=False)
    x["q"] = x["q"].abs() + 0.1
    x["k_cache"][x["block_table"][0, 0].long(), :16] = -float("inf")
    x["k_cache"][x["block_table"][1, 0].long(), :3] = -float("inf")
    out = _call(x)
    want, _, _, _ = ref.paged_decode(x["q"], x["k"], x["v"], x["k_cache"], x["v_cache"], x["block_table"], x["lengths"])
    assert torch.allclose(out.cpu().double(), want, rtol=1e-5, atol=1e-5)


def test_rows_share_pages():
    x = _case([100, 100, 70], 8, 2, 128, 16, "bf16", 10, hostile=False)
    x["block_table"][1, :6] = x["block_table"][0, :6]           # a common prefix of 96 keys
    x["block_table"][2, :4] = x["block_table"][0, :4]
    _run(x)


@pytest.mark.parametrize("new", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (16, 16, 64), (7, 1, 64), (40, 1, 128), (18, 2, 64)])
def test_a_wider_table_changes_nothing(H, Hkv, D, dtype, new):
    # short tables: a CTA takes whole rows; wide ones: the CTAs share the keys
    for lengths in ([40, 0, -1, 33, 1, 16], [3] * 300, [250, 249, 0, 7]):
        x = _case(lengths, H, Hkv, D, 16, dtype, 18, new=new)
        B, n = x["block_table"].shape
        wide = torch.full((B, 5000), -7, dtype=torch.int32, device="cuda")
        wide[:, :n] = x["block_table"]
        y = dict(x, k_cache=x["k_cache"].clone(), v_cache=x["v_cache"].clone(), block_table=wide)
        out, out2 = (torch.full((B, H, D), 5.0, device="cuda").to(x["q"].dtype) for _ in range(2))
        before = (x["k_cache"].clone(), x["v_cache"].clone())
        _call(x, out=out)
        _call(y, out=out2)
        kda.check_status()
        _check(x, before, out)
        _check(y, before, out2)
        for b, m in enumerate(lengths):
            if m < 0:
                assert bool((out[b] == 5).all()) and bool((out2[b] == 5).all())
            elif m == 0 and not new:
                assert not out[b].any() and not out2[b].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [0, 31, 64, 700])
def test_rows_that_write_one_position_attend_to_their_own_key(n, dtype):
    x = _case([n, n], 8, 2, 128, 16, dtype, 17, hostile=False)
    x["block_table"][1] = x["block_table"][0]
    before = x["k_cache"].clone(), x["v_cache"].clone()
    out = _call(x)
    kda.check_status()
    for b in range(2):
        y = dict(x, q=x["q"][b:b + 1], k=x["k"][b:b + 1], v=x["v"][b:b + 1], block_table=x["block_table"][b:b + 1],
                 lengths=x["lengths"][b:b + 1], k_cache=before[0].clone(), v_cache=before[1].clone())
        alone = _call({m: t.contiguous() for m, t in y.items()})
        assert torch.allclose(out[b:b + 1].float(), alone.float(), rtol=2 * HALF if dtype == "bf16" else 1e-4,
                              atol=2 * HALF if dtype == "bf16" else 1e-4)
    for c, old, new in ((x["k_cache"], before[0], x["k"]), (x["v_cache"], before[1], x["v"])):
        page, row = int(x["block_table"][0, n // 16]), n % 16
        assert bool(((c[page, row] == new[0]) | (c[page, row] == new[1])).all())
        c[page, row] = old[page, row]
        assert torch.equal(c, old)


def test_a_run_of_steps_fills_the_cache():
    x = _case([14, -1, 0, 62], 8, 4, 128, 16, "bf16", 12, spare=12)
    every = torch.arange(x["k_cache"].shape[0], device="cuda", dtype=torch.int32)
    free = every[~torch.isin(every, x["block_table"])].reshape(4, 3)          # three more pages for every row
    x["block_table"] = torch.cat([x["block_table"], free], 1).contiguous()
    g = torch.Generator(device="cuda").manual_seed(13)
    for _ in range(20):
        for n in ("q", "k", "v"):
            x[n] = torch.randn(x[n].shape, generator=g, device="cuda").to(torch.bfloat16)
        _run(x)
        x["lengths"] += (x["lengths"] >= 0).int()


def test_offsets_past_32_bits():
    # 2^31 + elements in each cache: the last pages lie beyond what 32-bit offsets reach
    page, Hkv, D = 64, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 5
    kc = torch.zeros((pages, page, Hkv, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = torch.Generator(device="cuda").manual_seed(14)
    kc[-4:] = torch.randn((4, page, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    vc[-4:] = torch.randn((4, page, Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(pages - 4, pages, dtype=torch.int32, device="cuda").reshape(1, 4)
    lengths = torch.tensor([230], dtype=torch.int32, device="cuda")
    q, k, v = r(1, 16, D), r(1, Hkv, D), r(1, Hkv, D)
    small = dict(q=q, k=k, v=v, k_cache=kc[-4:].clone(), v_cache=vc[-4:].clone(), lengths=lengths,
                 block_table=torch.arange(4, dtype=torch.int32, device="cuda").reshape(1, 4))
    want = _run(small)
    out = kda.paged_decode_step(q, k, v, kc, vc, table, lengths)
    assert torch.equal(out, want) and torch.equal(kc[-4:], small["k_cache"]) and torch.equal(vc[-4:], small["v_cache"])
    assert not kc[:5].any() and not vc[:5].any()


def test_a_captured_step_replays_with_other_lengths():
    x = _case([900, 3, -1, 64], 8, 2, 128, 16, "bf16", 15, hostile=False)
    y = _case([900, 3, -1, 64], 8, 2, 128, 16, "bf16", 16, hostile=False)
    side = torch.cuda.Stream()
    out = torch.zeros_like(x["q"])
    with torch.cuda.stream(side):
        _call(x, out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            _call(x, out=out)
    for lengths in ([900, 3, -1, 64], [5, 600, 17, -3], [0, 0, 0, 0], [899, 899, 899, 899]):
        for n in ("q", "k", "v", "k_cache", "v_cache", "block_table"):
            x[n].copy_(y[n])
        x["lengths"].copy_(torch.tensor(lengths, dtype=torch.int32))
        before = (x["k_cache"].clone(), x["v_cache"].clone())
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        kda.check_status()
        torch.cuda.synchronize()
        _check(x, before, out)


def test_two_steps_at_once_on_two_streams():
    xs = [_case([3000, 10, 500], 8, 2, 128, 16, "bf16", s, hostile=False) for s in (17, 18)]
    want = [_call(x) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _call(xs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_steps_in_a_row_on_one_stream_share_a_workspace():
    xs = [_case([n, 10, 5 * n], 8, 2, 128, 16, "bf16", n, hostile=False) for n in (300, 1, 900)]
    ws = torch.full((kda.paged_decode_workspace_bytes(8, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    want = [_call(x) for x in xs]
    got = [_call(x, workspace=ws) for x in xs]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(kda.KDAError):
        _call(xs[0], workspace=ws[:1024])


def test_hybrid_step_runs_both_kinds_of_layers():
    """One token through a recurrent layer, a linear-attention layer and a cached layer, as a
    hybrid stack serves them, for several tokens; each against its own definition."""
    B, H, D = 3, 4, 128
    g = torch.Generator(device="cuda").manual_seed(19)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    log_decay = torch.tensor([-0.5, -0.1, -0.02, 0.0], device="cuda")
    prompt = dict(q=unit(r(B, 40, H, D)), k=unit(r(B, 40, H, D)), v=r(B, 40, H, D).to(torch.bfloat16))
    _, la_state = kda.la_forward(prompt["q"], prompt["k"], prompt["v"], log_decay)
    _, kda_state = kda.forward(prompt["q"], prompt["k"], prompt["v"], -0.1 * torch.ones((B, 40, H, D), device="cuda"),
                               0.5 * torch.ones((B, 40, H), device="cuda"))
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").reshape(B, 4)
    kc = torch.zeros((B * 4, 16, H, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    at = torch.arange(40, device="cuda")
    where = (table[:, at // 16].long(), (at % 16).expand(B, 40))
    kc[where], vc[where] = prompt["k"], prompt["v"]
    lengths = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    all_q, all_k, all_v = [prompt["q"]], [prompt["k"]], [prompt["v"]]
    outs = []
    for _ in range(10):
        q, k, v = unit(r(B, H, D)), unit(r(B, H, D)), r(B, H, D).to(torch.bfloat16)
        kda.decode_step(q, k, v, -0.1 * torch.ones((B, H, D), device="cuda"), 0.5 * torch.ones((B, H), device="cuda"), kda_state)
        outs.append(kda.la_decode_step(q, k, v, log_decay, la_state))
        x = dict(q=q, k=k, v=v, k_cache=kc, v_cache=vc, block_table=table, lengths=lengths)
        _run(x)
        lengths += 1
        for keep, t in ((all_q, q), (all_k, k), (all_v, v)):
            keep.append(t[:, None])
    kda.check_status()
    want, last = ref.la_forward(torch.cat(all_q, 1), torch.cat(all_k, 1), torch.cat(all_v, 1), log_decay)
    mag, _ = ref.la_forward(*(torch.cat(t, 1).abs() for t in (all_q, all_k, all_v)), log_decay)
    err = (torch.stack(outs, 1).cpu().double() - want[:, 40:]).abs()
    assert bool((err <= HALF * want[:, 40:].abs() + HALF * mag[:, 40:] + 1e-5).all())
    assert torch.allclose(la_state.cpu().double(), last, rtol=1e-5, atol=1e-5)


# the two below come last: what a bad page or length may touch is checked by the kernel itself
def test_bad_pages_are_absent_and_reported():
    for bad in (-1, 10 ** 6):
        x = _case([100, 40, 16], 8, 2, 128, 16, "bf16", 20, hostile=False)
        x["block_table"][0, 2] = bad                   # a page in the middle
        x["block_table"][1, 2] = bad                   # the page of the new key
        before = (x["k_cache"].clone(), x["v_cache"].clone())
        out = _call(x)
        with pytest.raises(kda.KDAError) as e:
            kda.check_status()
        assert e.value.status == kda.KDA_ERR_INVALID_ARG
        kda.check_status()                             # reported once
        _check(x, before, out)


def test_rows_longer_than_their_table_are_left_alone():
    x = _case([100, 40, 16], 8, 2, 128, 16, "bf16", 21, hostile=False)
    x["lengths"][1] = 16 * x["block_table"].shape[1]
    x["lengths"][2] = 2 ** 31 - 1
    before = (x["k_cache"].clone(), x["v_cache"].clone())
    out = torch.full_like(x["q"], 3.0)
    _call(x, out=out)
    with pytest.raises(kda.KDAError):
        kda.check_status()
    assert bool((out[1:] == 3).all())
    _check(x, before, out)
