"""GPU: rows of q have nothing to do with each other in window attention, whatever one of them
holds: values that are not finite, values far above the others, the ends of the types' ranges."""
import math

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests import window_ref as ref
from tests.test_gpu_window import _built, make, wanted  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def largest_of_the_row(want, s):
    """window_ref's results with the last, the largest |q| of the request's rows of a KV head times
    the largest sum of |k|, formed with the row's own largest |q| instead."""
    *front, floor = want
    q = s["q"].cpu().double().abs()
    G = q.shape[1] // s["k_cache"].shape[1]
    ptr = s["qo_indptr"].tolist()
    for r0, r1 in zip(ptr[:-1], ptr[1:]):
        for h in range(q.shape[1]):
            block = q[r0:r1, h // G * G:(h // G + 1) * G].max()
            floor[r0:r1, h] *= q[r0:r1, h].amax(-1) / block
    return (*front, floor)


def check_rows(got, want, s):
    out, lse = want[0], want[1]
    b, z = ref.attention_bounds(*largest_of_the_row(want, s), s["q"].dtype, s["q"].shape[2], two_parts=False)
    o, l = got["out"].cpu().double(), got["lse"].cpu().double()
    assert ((l - lse).abs() <= z).all(), ((l - lse).abs() - z).max()
    far = (o - out).abs() - b
    assert far.max() <= 0, (far.max(), (o - out).abs().max())


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Hq", [8, 32])  # head_dim 128: blocks of 32 rows, of 64
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("mask", ["chain", "tree", "none"])
def test_a_value_that_is_not_finite_stays_in_its_row_128(value, Hq, dtype, mask):
    stays_in_its_row(make(51, [6, 3], [700, 10], Hq, 2, 128, 16, dtype, mask), value)


def stays_in_its_row(s, value):
    s["q"] = s["q"].contiguous()
    clean = tv.window_attention(**s, lse=True)
    rest = torch.ones(s["q"].shape[:2], dtype=torch.bool)
    for r, h, d in ((1, 2, 77 % s["q"].shape[2]), (4, 0, 0), (8, s["q"].shape[1] - 1, 5)):
        s["q"][r, h, d] = value
        rest[r, h] = False
    got = tv.window_attention(**s, lse=True)
    assert torch.equal(got["out"].cpu()[rest], clean["out"].cpu()[rest])
    assert torch.equal(got["lse"].cpu()[rest], clean["lse"].cpu()[rest])
    assert torch.isnan(got["out"].cpu()[~rest]).all() and torch.isnan(got["lse"].cpu()[~rest]).all()


@pytest.mark.parametrize("Hq", [8, 32])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_of_very_different_sizes(D, Hq, dtype):
    # one head and one row 2^12 times the rest (fp16: up to 32000): a score of a row errs by 2^-17 of
    # the row's own largest |q|
    windows, lens = [4, 3], [300, 77]
    s = make(52, windows, lens, Hq, 2, D, 32, dtype)
    s["q"] = s["q"].contiguous()
    s["q"][:, 1] *= 4096
    s["q"][5] = (s["q"][5].float() * 4096).clamp(-32000, 32000).to(dtype)
    check_rows(tv.window_attention(**s, lse=True), wanted(s, windows, lens), s)


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("Hq", [4, 8, 32])  # blocks of 16, 32 and 64 rows
@pytest.mark.parametrize("mask", ["chain", "none"])
def test_a_value_that_is_not_finite_stays_in_its_row_64(value, Hq, mask):
    for dtype in (BF16, F16):
        stays_in_its_row(make(53, [6, 3], [700, 10], Hq, 2, 64, 16, dtype, mask), value)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,mask", [([20], "none"), ([0], "chain"), ([20], "chain"), ([0], "none")])
def test_an_infinity_whose_scores_are_all_minus_infinity(D, lens, mask):
    # K is negative everywhere, one query +inf: each of its scores is -inf, and it is NaN all the
    # same (without a token to see: 0)
    for dtype in (BF16, F16):
        s = make(54, [3], lens, 4, 2, D, 16, dtype, mask, garbage=False)
        s["q"] = s["q"].contiguous()
        s["k_cache"] = (-s["k_cache"].float().abs() - 1).to(ref.F8)
        if mask != "none":
            s["k_new"] = -s["k_new"].abs() - 1
        s["q"][1, 2, 3] = math.inf
        got = tv.window_attention(**s, lse=True)
        rest = torch.ones((3, 4), dtype=torch.bool)
        rest[1, 2] = False
        if lens == [0] and mask == "none":
            assert (got["out"] == 0).all() and torch.isneginf(got["lse"]).all()
            continue
        assert torch.isnan(got["out"][1, 2]).all() and torch.isnan(got["lse"][1, 2])
        assert torch.isfinite(got["out"].cpu()[rest].float()).all() and torch.isfinite(got["lse"].cpu()[rest]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [4, 32])
@pytest.mark.parametrize("by", [2.0 ** 104, 2.0 ** -104])
def test_queries_near_the_ends_of_bf16(D, Hq, by):
    windows, lens = [4, 3], [200, 33]
    s = make(55, windows, lens, Hq, 2, D, 16, BF16)
    s["q"] = (s["q"].float() * by).to(BF16)
    scale = 0.1 / by
    check_rows(tv.window_attention(**s, sm_scale=scale, lse=True), wanted(s, windows, lens, scale), s)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq", [2, 64])
@pytest.mark.parametrize("n,own", [(1, False), (40, False), (0, True), (40, True)])
def test_scores_far_below_zero(D, Hq, n, own):
    # every score is -D 1e30, which fp32 holds: the softmax is the mean of V all the same
    q = torch.ones((1, Hq, D), dtype=BF16, device="cuda")
    pages = 3
    k = torch.full((pages, 1, 16, D), -1.0).to(ref.F8).cuda()
    v = torch.randn((pages, 1, 16, D), generator=torch.Generator().manual_seed(56)).to(ref.F8).cuda()
    ones = torch.ones((pages, 1), device="cuda")
    new = dict(k_new=-q[:, :1], v_new=torch.full((1, 1, D), 0.5, dtype=BF16, device="cuda")) if own else {}
    got = tv.window_attention(q, k, v, ones, ones.clone(), torch.arange(pages, dtype=torch.int32)[None].cuda(),
                              torch.tensor([n], dtype=torch.int32).cuda(), sm_scale=1e30, lse=True, **new)
    x = v.float().double().view(-1, D)[:n]
    if own:
        x = torch.cat([x, torch.full((1, D), 0.5, dtype=torch.float64, device="cuda")])
    # equal scores: each is one product, the same for all, so that every probability is exact; sums and
    # the output are rounded
    assert ((got["out"].double() - x.mean(0)).abs() <= 2.0 ** -8 * x.mean(0).abs() + 2.0 ** -14 * x.abs().max()).all()
    assert ((got["lse"].double() / (-D * 1e30) - 1).abs() <= 2.0 ** -18).all()
