"""GPU: window attention where one token outweighs each of the others and they, many and alike, weigh
together as much: what is lost of each small probability is lost to the same side, and shows.

Token `at` has score a, every other one 0, so with n tokens the exact result is
out = (e^a v_at + (n - 1) v) / (e^a + n - 1). Enough requests name the same pages for each to be worked on
from its first token to its last by one multiprocessor (a piece that begins behind the large
token has references of its own)."""
import math

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built  # noqa: F401 (a fixture)
from tests.window_ref import F8

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


def large_and_small(n, at, rows, D, dtype, page=128):
    """out, lse of the call and the exact ones, per row of a window; rows: (window rows, heads)."""
    T, Hq = rows
    B = torch.cuda.get_device_properties(0).multi_processor_count * (1 if D == 128 else 2)
    pages = -(-n // page)
    k = torch.zeros((pages, 1, page, D), dtype=torch.float32)
    k[at // page, 0, at % page, 0] = 1.0
    # V by dims: (large, small) = (1, 1), (0, 1), (1, 0), (-1, 1)
    large = torch.tensor([1.0, 0.0, 1.0, -1.0]).repeat(D // 4)
    small = torch.tensor([1.0, 1.0, 0.0, 1.0]).repeat(D // 4)
    v = small.expand(pages, 1, page, D).clone()
    v[at // page, 0, at % page] = large
    ones = torch.ones((pages, 1)).cuda()
    # 4 to 20 in steps that bf16 holds
    a = 4 + torch.arange(T * Hq, dtype=torch.float64) * (128 // (T * Hq)) / 8
    q = torch.zeros((T, Hq, D), dtype=torch.float64)
    q[:, :, 0] = a.view(T, Hq)
    assert torch.equal(q.to(dtype).double(), q)
    got = tv.window_attention(
        q.to(dtype).repeat(B, 1, 1).cuda(), k.to(F8).cuda(), v.to(F8).cuda(), ones, ones.clone(),
        torch.arange(pages, dtype=torch.int32).repeat(B, 1).cuda(),
        torch.full((B,), n, dtype=torch.int32).cuda(), sm_scale=1.0, lse=True)
    w = torch.exp(a)[:, None]
    out = (w * large + (n - 1) * small) / (w + n - 1)
    absv = (w * large.abs() + (n - 1) * small) / (w + n - 1)
    lse = a + torch.log1p((n - 1) * torch.exp(-a))
    view = (B, T * Hq, D)
    return got["out"].cpu().double().view(view), got["lse"].cpu().double().view(view[:2]), out, absv, lse


def check(n, at, rows, D, dtype):
    """Bounds. Scores: one product, exact, then an exponent of at most 30 and its reference, rounded
    (2^-19 each), and 2^x to 2^-22: d = 2^-17. Probabilities: 2^-11 of each for its rounding to 11
    bits; and what small ones lose beyond that, a fixed step each, 2^-11 of the row's whole sum
    together, times |v| <= 1 (of the sum, not of the small ones' part of it: 8191 of 2^-28 of
    the largest may vanish). Sums: no chain is longer than a 32nd of the tokens (a warp's or a
    product's share) plus 64 steps of joining, each rounded or truncated by 2^-23 of the whole. The quotient
    doubles what its sums share; the output is rounded by eps / 2."""
    o, l, out, absv, lse = large_and_small(n, at, rows, D, dtype)
    d, sums = 2.0 ** -17, (n / 32 + 64) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    far = (o - out).abs() - half * out.abs() - (1 + half) * (absv * (2.0 ** -11 + 2 * d + 2 * sums) + 2.0 ** -11)
    assert far.max() <= 0, (far.max(), (o - out).abs().amax((0, 2)))
    assert ((l - lse).abs() <= d + sums + 2.0 ** -22 * (lse + 1)).all(), (l - lse).abs().max()


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [1000, 8192])
@pytest.mark.parametrize("rows", [(1, 8), (8, 8)])  # blocks of 32 rows, of 64
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_probabilities_behind_a_large_one_128(dtype, rows, n, at):
    check(n, {"first": 0, "middle": n // 2, "last": n - 1}[at], rows, 128, dtype)


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [32768, 131072])
@pytest.mark.parametrize("rows", [(1, 8), (8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_small_probabilities_behind_a_large_one_128(dtype, rows, n, at):
    check(n, {"first": 0, "middle": n // 2, "last": n - 1}[at], rows, 128, dtype)


def test_references_that_rise_and_fall_again():
    # large tokens at the beginning, in the middle and at the end of a long context of small ones, which
    # are larger in its second half: against the softmax in 64 bits
    n, page, D, T, Hq = 70001, 128, 128, 2, 4
    for dtype in (BF16, F16):
        B = torch.cuda.get_device_properties(0).multi_processor_count
        score = torch.zeros(n, dtype=torch.float64)
        score[n // 2:] = 0.5
        score[[3, 20011, 35000, 35001, 69999]] = torch.tensor([1.0, 0.875, 1.125, 0.75, 1.0], dtype=torch.float64)
        v = torch.randn(n, generator=torch.Generator().manual_seed(1)).to(F8).double()
        pages = -(-n // page)
        k_cache, v_cache = torch.zeros((2, pages * page, D))
        k_cache[:n, 0] = score.float()
        v_cache[:n] = v.float()[:, None]
        a = torch.arange(8, 24, 2, dtype=torch.float64)  # a row's scores: a times those
        q = torch.zeros((T, Hq, D), dtype=torch.float64)
        q[:, :, 0] = a.view(T, Hq)
        ones = torch.ones((pages, 1)).cuda()
        got = tv.window_attention(
            q.to(dtype).repeat(B, 1, 1).cuda(), k_cache.view(pages, 1, page, D).to(F8).cuda(),
            v_cache.view(pages, 1, page, D).to(F8).cuda(), ones, ones.clone(),
            torch.arange(pages, dtype=torch.int32).repeat(B, 1).cuda(),
            torch.full((B,), n, dtype=torch.int32).cuda(), sm_scale=1.0, lse=True)
        w = torch.softmax(a[:, None] * score, -1)
        out, absv = w @ v, w @ v.abs()
        o = got["out"].cpu().double().view(B, T * Hq, D)
        # as in check, with |v| below 5
        half, share = torch.finfo(dtype).eps / 2, 2.0 ** -11 + 2.0 ** -16 + 2 * (n / 32 + 64) * 2.0 ** -23
        far = (o - out[:, None]).abs() - (half * out.abs() + (1 + half) * (absv * share + 5 * 2.0 ** -11))[:, None]
        assert far.max() <= 0, far.max()


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [1000, 131072, 524288])
@pytest.mark.parametrize("rows", [(1, 8), (4, 8), (8, 8)])  # blocks of 16, 32 and 64 rows
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_small_probabilities_behind_a_large_one_64(dtype, rows, n, at):
    check(n, {"first": 0, "middle": n // 2, "last": n - 1}[at], rows, 64, dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [(1, 8), (8, 8)])
@pytest.mark.parametrize("large_first", [True, False])
@pytest.mark.parametrize("vscale", [2.0 ** -100, 2.0 ** -80, 1.0, 2.0 ** 80])
def test_sums_stay_in_range(vscale, large_first, rows, D):
    # half of the tokens have score a, half 0, V is vscale everywhere. Sums hold probabilities over V's
    # scale (2^-80 at least): references that rise late or fall must not take them out of fp32's range
    n, page, (T, Hq) = 131072, 128, rows
    B = torch.cuda.get_device_properties(0).multi_processor_count * (1 if D == 128 else 2)
    pages = n // page
    k = torch.zeros((pages, 1, page, D))
    k[:pages // 2 if large_first else pages, 0, :, 0] = 1.0
    if not large_first:
        k[:pages // 2] = 0.0
    a = 4 + torch.arange(T * Hq, dtype=torch.float64) * (128 // (T * Hq)) / 8
    q = torch.zeros((T, Hq, D), dtype=torch.float64)
    q[:, :, 0] = a.view(T, Hq)
    ones = torch.ones((pages, 1)).cuda()
    got = tv.window_attention(
        q.to(BF16).repeat(B, 1, 1).cuda(), k.to(F8).cuda(), torch.ones_like(k).to(F8).cuda(), ones, ones * vscale,
        torch.arange(pages, dtype=torch.int32).repeat(B, 1).cuda(),
        torch.full((B,), n, dtype=torch.int32).cuda(), sm_scale=1.0, lse=True)
    sums = (n / 32 + 64) * 2.0 ** -23  # as in check
    o = got["out"].cpu().double() / max(vscale, 2.0 ** -80)
    assert ((o - 1).abs() <= 2.0 ** -8 + (1 + 2.0 ** -8) * (2.0 ** -10 + 2.0 ** -16 + 2 * sums)).all(), (o - 1).abs().max()
    lse = a + math.log(n // 2) + torch.log1p(torch.exp(-a))
    z = (got["lse"].cpu().double().view(B, T * Hq) - lse).abs()
    assert (z <= 2.0 ** -17 + sums + 2.0 ** -22 * (lse + 1)).all(), z.max()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [(1, 8), (8, 8)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_a_token_that_outweighs_the_rest_comes_out_as_it_is(dtype, rows, D):
    # two tokens, scores a and 0, V with a scale of any value: the large one's probability must not be rounded in
    # the products alone. Its exponent and 2^x to 2^-18, the small one's rounding 2^-11 e^-6
    T, Hq = rows
    B = 64
    g = torch.Generator().manual_seed(81)
    k = torch.zeros((B, 1, 16, D))
    k[:, 0, 0, 0] = 1.0
    v = (torch.randn((B, 1, 16, D), generator=g) * 50).to(F8)
    vs = torch.rand((B, 1), generator=g) + 0.5
    a = 6 + torch.arange(T * Hq, dtype=torch.float64) / 16
    q = torch.zeros((T, Hq, D), dtype=torch.float64)
    q[:, :, 0] = a.view(T, Hq)
    assert torch.equal(q.to(dtype).double(), q)
    got = tv.window_attention(q.to(dtype).repeat(B, 1, 1).cuda(), k.to(F8).cuda(), v.cuda(), torch.ones((B, 1)).cuda(),
                              vs.cuda(), torch.arange(B, dtype=torch.int32)[:, None].cuda(),
                              torch.full((B,), 2, dtype=torch.int32).cuda(), sm_scale=1.0)["out"]
    x = v.float().double()[:, 0, :2] * vs.double()[:, :, None]         # [B, 2, D]
    w = torch.sigmoid(a)[None, :, None]
    out = w * x[:, None, 0] + (1 - w) * x[:, None, 1]
    off = (got.cpu().double().view(B, T * Hq, D) - out).abs()
    top = x.abs().amax(1)[:, None]
    far = off - (torch.finfo(dtype).eps / 2 * out.abs() + 1.01 * (2.0 ** -16 + 2.0 ** -11 * math.exp(-6)) * top)
    assert far.max() <= 0, far.max()
