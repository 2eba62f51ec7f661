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
