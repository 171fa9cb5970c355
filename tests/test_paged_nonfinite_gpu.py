"""Paged decode attention with infinities and NaN among what a row attends to, on the GPU.

softmax(scale q K^T) V on such values, as IEEE arithmetic has it: a NaN or +inf score makes the
head's row NaN; an infinite value makes its channel infinite, a NaN value makes it NaN.  The fp64
definition says where; finite elements are held to the tolerances of the finite case: 2e-5
sum_j p_j |v_j|, and for bf16 2^-8 |ref| + 2^-8 sum_j p_j |v_j| more.
"""
import math

import pytest
import torch

import gated_delta_rule_109_b200 as kda
from oracle import attention as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_delta_rule_109_b200 import build
    build.build()


# Short rows on a table of their size (a CTA takes rows whole), short rows on a wide table (the
# device decides), one long row and long rows beside short ones (CTAs share rows).
LAYOUTS = [([70, 3, 16], 0), ([70, 3, 16], 5000), ([5000], 0), ([3000, 40, 2999], 0)]


def _case(lengths, spare_columns, dtype, D, seed, group=4, Hkv=2, page=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    B, per = len(lengths), max(lengths) // page + 1
    table = torch.full((B, per + spare_columns), -7, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.randperm(B * per, generator=g, device="cuda").reshape(B, per)
    return dict(q=r(B, Hkv * group, D), k=r(B, Hkv, D), v=r(B, Hkv, D), k_cache=r(B * per, page, Hkv, D),
                v_cache=r(B * per, page, Hkv, D), block_table=table,
                lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))


def _at(x, b, t):
    """Page and entry of position t of row b."""
    page = x["k_cache"].shape[1]
    return int(x["block_table"][b, t // page]), t % page


def _check(x):
    a = [x[n] for n in ("q", "k", "v", "k_cache", "v_cache", "block_table", "lengths")]
    want, mag, _, _ = ref.paged_decode(*a)
    got = kda.paged_decode_step(*a).cpu().double()
    kda.check_status()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    tol = 2e-5 * mag[fine] + (HALF * (want[fine].abs() + mag[fine]) if x["q"].dtype == torch.bfloat16 else 0)
    assert bool(((got - want)[fine].abs() <= tol).all())
    return want


@pytest.mark.parametrize("lengths,spare", LAYOUTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_that_are_not_finite_make_the_row_nan(dtype, D, lengths, spare):
    n = lengths[0]
    for bad in (NAN, INF):
        x = _case(lengths, spare, dtype, D, 1)              # in one head's query
        x["q"][0, 5, 7] = bad
        want = _check(x)
        assert bool(torch.isnan(want[0, 5]).all()) and bool(torch.isfinite(want[0, :5]).all())
        for t in (0, 17, n // 2, n - 1):                    # in one key of one key-value head
            x = _case(lengths, spare, dtype, D, 2)
            x["q"][0, :, 7] = x["q"][0, :, 7].abs() + 0.5   # +inf, not -inf
            x["k_cache"][(*_at(x, 0, t), 1, 7)] = bad
            want = _check(x)
            assert bool(torch.isnan(want[0, 4:]).all()) and bool(torch.isfinite(want[0, :4]).all())
        x = _case(lengths, spare, dtype, D, 3)              # in the new key
        x["q"][0, :, 7] = x["q"][0, :, 7].abs() + 0.5
        x["k"][0, 0, 7] = bad
        want = _check(x)
        assert bool(torch.isnan(want[0, :4]).all()) and bool(torch.isfinite(want[0, 4:]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_of_nan_keys_alone(dtype):
    x = _case([20, 300], 0, dtype, 128, 4)
    x["k_cache"][:] = NAN
    x["k"][:] = NAN
    assert bool(torch.isnan(_check(x)).all())


@pytest.mark.parametrize("lengths,spare", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_that_all_score_minus_infinity_weigh_nothing(dtype, lengths, spare):
    x = _case(lengths, spare, dtype, 64, 8)
    x["q"] = x["q"].abs() + 0.5
    x["k_cache"][:, :, 0, 3] = -INF
    x["k"][:, 0, 3] = -INF
    a = [x[n] for n in ("q", "k", "v", "k_cache", "v_cache", "block_table", "lengths")]
    got = kda.paged_decode_step(*a)
    kda.check_status()
    assert not got[:, :4].any() and bool(torch.isfinite(got).all()) and bool((got[:, 4:] != 0).any())


@pytest.mark.parametrize("lengths,spare", LAYOUTS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_that_are_not_finite_stay_what_they_are(dtype, D, lengths, spare):
    n = lengths[0]
    for t in (0, 17, n // 2, n - 1):
        x = _case(lengths, spare, dtype, D, 5)
        x["q"] = 0.25 * x["q"]                              # weights that fp32 holds for every key
        page, entry = _at(x, 0, t)
        x["v_cache"][page, entry, 1, 3] = INF
        x["v_cache"][page, entry, 1, 4] = -INF
        x["v_cache"][page, entry, 1, 5] = NAN
        x["v"][0, 0, 6] = -INF
        want = _check(x)
        assert bool((want[0, 4:, 3] == INF).all()) and bool((want[0, 4:, 4] == -INF).all())
        assert bool(torch.isnan(want[0, 4:, 5]).all()) and bool((want[0, :4, 6] == -INF).all())
        assert int(torch.isfinite(want[0]).sum()) == 8 * D - 16
    x = _case(lengths, spare, dtype, D, 6)                  # +inf and -inf in one channel
    x["q"] = 0.25 * x["q"]
    x["v_cache"][(*_at(x, 0, 1), 0, 2)], x["v"][0, 0, 2] = INF, -INF
    assert bool(torch.isnan(_check(x)[0, :4, 2]).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_only_key_with_an_infinite_value(dtype):
    # its probability is 1, which one bf16 holds: nothing is left for a second part
    x = _case([0, 0], 0, dtype, 64, 7)
    x["v"][0, 0, 2] = INF
    assert bool((_check(x)[0, :4, 2] == INF).all())
