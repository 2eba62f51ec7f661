"""GPU: shared attention where one token outweighs each of the others and they, many and alike, weigh
together as much (what is lost of each small probability is lost to the same side, and shows), and
where references rise and fall. Every group is one request, and there are as many groups as
multiprocessors, all with the same pages: each is worked on from its first token to its last by one."""
import math

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built  # noqa: F401 (a fixture)
from tests.window_ref import F8

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
PAGE = 128
ROWS = [(1, 8), (32, 8)]  # (window rows, heads): both slots at one block's tiles in turn; a slot each


def attend(q, k, v, k_scale, v_scale, n):
    """shared_attention of requests that all have q [T, Hq, D] and the pages' n tokens, all of them shared."""
    B = torch.cuda.get_device_properties(0).multi_processor_count
    pages, T = k.shape[0], q.shape[0]
    got = tv.shared_attention(
        q.repeat(B, 1, 1), k, v, k_scale, v_scale, torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1),
        torch.full((B,), n, dtype=torch.int32, device="cuda"), group_indptr=torch.arange(B + 1, dtype=torch.int32, device="cuda"),
        shared_lens=torch.full((B,), n, dtype=torch.int32, device="cuda"), sm_scale=1.0, lse=True)
    Hq, D = q.shape[1:]
    return got["out"].double().view(B, T * Hq, D), got["lse"].double().view(B, T * Hq)


def queries(a, T, D, dtype):
    """Row t, head h asks for a[h] in dim 0."""
    q = torch.zeros((T, len(a), D), dtype=torch.float64, device="cuda")
    q[:, :, 0] = a
    assert torch.equal(q.to(dtype).double(), q)
    return q.to(dtype)


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [1 << 15, 1 << 18, 1 << 20])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_probabilities_behind_a_large_one(dtype, D, rows, n, at):
    """Token `at` has score a, every other one 0: out = (e^a v_at + (n - 1) v) / (e^a + n - 1).

    Bounds, as window attention's for the same tokens (test_gpu_window_tails.py): scores, one exact
    product, an exponent of at most 30 and its reference, rounded (2^-19 each), 2^x to 2^-22 and the join
    with the (empty) rest, 2^-18: d = 2^-17. Probabilities: 2^-11 of each for its rounding to 11 bits,
    and what small ones lose beyond that, 2^-11 of the row's whole sum together. Sums: no chain is longer than
    a 16th of the tokens (a product takes 16) plus 64 steps of joining, 2^-23 of the whole each."""
    T, Hq = rows
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[at]
    pages = n // PAGE
    k = torch.zeros((pages, 1, PAGE, D), dtype=torch.uint8, device="cuda")
    k[at // PAGE, 0, at % PAGE, 0] = 0x38  # 1
    # V by dims: (large, small) = (1, 1), (0, 1), (1, 0), (-1, 1)
    large = torch.tensor([1.0, 0.0, 1.0, -1.0], device="cuda").repeat(D // 4)
    small = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda").repeat(D // 4)
    v = small.to(F8).view(torch.uint8).expand(pages, 1, PAGE, D).contiguous()
    v[at // PAGE, 0, at % PAGE] = large.to(F8).view(torch.uint8)
    ones = torch.ones((pages, 1), device="cuda")
    a = torch.tensor([4.0, 12.0, 17.0, 19.0, 19.75, 20.0, 20.125, 21.0], dtype=torch.float64, device="cuda")
    o, l = attend(queries(a, T, D, dtype), k.view(F8), v.view(F8), ones, ones.clone(), n)
    a = a.repeat(T)
    w = torch.exp(a)[:, None]
    out = (w * large + (n - 1) * small) / (w + n - 1)
    absv = (w * large.abs() + (n - 1) * small) / (w + n - 1)
    lse = a + torch.log1p((n - 1) * torch.exp(-a))
    d, sums = 2.0 ** -17, (n / 16 + 64) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    far = (o - out).abs() - half * out.abs() - (1 + half) * (absv * (2.0 ** -11 + 2 * d + 2 * sums) + 2.0 ** -11)
    assert far.max() <= 0, (far.max(), (o - out).abs().amax((0, 2)))
    assert ((l - lse).abs() <= d + sums + 2.0 ** -22 * (lse + 1)).all(), (l - lse).abs().max()


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_references_that_rise_and_fall_again(dtype, D, rows):
    # large tokens here and there in a long context of small ones that come in steps, up and down: against
    # the softmax in 64 bits, as in test_gpu_window_tails.py (|v| below 5)
    T, Hq = rows
    n = 1 << 19
    score = torch.zeros(n, dtype=torch.float64, device="cuda")
    step = n // 8
    for i, s in enumerate([0.0, 0.25, 0.5, 0.25, 0.75, 0.0, 0.5, 0.125]):
        score[i * step:(i + 1) * step] = s
    score[[3, 200011, 350000, 350001, n - 1]] = torch.tensor([1.0, 0.875, 1.125, 0.75, 1.0], dtype=torch.float64, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    v = torch.randn(n, generator=g, device="cuda").to(F8)
    k = torch.zeros((n, D), dtype=torch.uint8, device="cuda")
    k[:, 0] = score.float().to(F8).view(torch.uint8)
    v_cache = v.view(torch.uint8)[:, None].expand(n, D).contiguous().view(F8)
    pages = n // PAGE
    ones = torch.ones((pages, 1), device="cuda")
    a = torch.arange(8, 24, 2, dtype=torch.float64, device="cuda")
    o, _ = attend(queries(a, T, D, dtype), k.view(F8).view(pages, 1, PAGE, D), v_cache.view(pages, 1, PAGE, D), ones, ones.clone(), n)
    w = torch.softmax(a[:, None] * score, -1)
    out, absv = (w @ v.double()).repeat(T), (w @ v.double().abs()).repeat(T)
    half, share = torch.finfo(dtype).eps / 2, 2.0 ** -11 + 2.0 ** -16 + 2 * (n / 16 + 64) * 2.0 ** -23
    far = (o - out[:, None]).abs() - (half * out.abs() + (1 + half) * (absv * share + 5 * 2.0 ** -11))[:, None]
    assert far.max() <= 0, far.max()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("large_first", [True, False])
@pytest.mark.parametrize("vscale", [2.0 ** -100, 2.0 ** -80, 1.0, 2.0 ** 80])
def test_sums_stay_in_range(vscale, large_first, rows, D):
    # half of the tokens have score a, half 0, V is vscale everywhere: references that rise late or fall
    # must not take the sums (over V's scale, 2^-80 at least) out of fp32's range
    T, Hq = rows
    n = 1 << 18
    pages = n // PAGE
    k = torch.zeros((pages, 1, PAGE, D), dtype=torch.uint8, device="cuda")
    k[slice(0, pages // 2) if large_first else slice(pages // 2, pages), 0, :, 0] = 0x38
    ones = torch.ones((pages, 1), device="cuda")
    a = torch.tensor([4.0, 6.0, 9.0, 13.0, 17.0, 20.0, 30.0, 60.0], dtype=torch.float64, device="cuda")
    o, l = attend(queries(a, T, D, BF16), k.view(F8), torch.full_like(k, 0x38).view(F8), ones, ones * vscale, n)
    a = a.repeat(T)
    sums = (n / 16 + 64) * 2.0 ** -23  # as above
    o = o / max(vscale, 2.0 ** -80)
    assert ((o - 1).abs() <= 2.0 ** -8 + (1 + 2.0 ** -8) * (2.0 ** -10 + 2.0 ** -15 + 2 * sums)).all(), (o - 1).abs().max()
    lse = a + math.log(n // 2) + torch.log1p(torch.exp(-a))
    z = (l - lse).abs()
    # an exponent of at most 2^8 here: 2^-16
    assert (z <= 2.0 ** -15 + sums + 2.0 ** -22 * (lse + 1)).all(), z.max()


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_small_probabilities_of_a_requests_own_tokens(dtype, D, at):
    """The same where nothing is shared: 2^24 tokens of each request, which three CTAs a multiprocessor
    work on. All pages but one are the same few; a product takes 16 tokens of every 64."""
    n, Hq, few = 1 << 24, 8, 64
    B = 3 * torch.cuda.get_device_properties(0).multi_processor_count
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[at]
    k = torch.zeros((few + 1, 1, PAGE, D), dtype=torch.uint8, device="cuda")
    k[few, 0, at % PAGE, 0] = 0x38
    large = torch.tensor([1.0, 0.0, 1.0, -1.0], device="cuda").repeat(D // 4)
    small = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda").repeat(D // 4)
    v = small.to(F8).view(torch.uint8).expand(few + 1, 1, PAGE, D).contiguous()
    v[few, 0, at % PAGE] = large.to(F8).view(torch.uint8)
    row = torch.arange(n // PAGE, dtype=torch.int32, device="cuda") % few
    row[at // PAGE] = few
    ones = torch.ones((few + 1, 1), device="cuda")
    a = torch.tensor([12.0, 20.0, 21.0, 22.0, 22.125, 22.25, 22.5, 23.0], dtype=torch.float64, device="cuda")
    got = tv.shared_attention(
        queries(a, 1, D, dtype).repeat(B, 1, 1), k.view(F8), v.view(F8), ones, ones.clone(), row.repeat(B, 1),
        torch.full((B,), n, dtype=torch.int32, device="cuda"), group_indptr=torch.tensor([0, B], dtype=torch.int32, device="cuda"),
        shared_lens=torch.zeros(1, dtype=torch.int32, device="cuda"), sm_scale=1.0)
    w = torch.exp(a)[:, None]
    out = (w * large + (n - 1) * small) / (w + n - 1)
    absv = (w * large.abs() + (n - 1) * small) / (w + n - 1)
    d, sums = 2.0 ** -17, (n / 64 + 64) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    far = (got["out"].double() - out).abs() - half * out.abs() - (1 + half) * (absv * (2.0 ** -11 + 2 * d + 2 * sums) + 2.0 ** -11)
    assert far.max() <= 0, (far.max(), (got["out"].double() - out).abs().amax((0, 2)))
