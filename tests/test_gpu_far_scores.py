"""GPU: scores of any size are scores. Tokens whose scores are all the same, however large, weigh the same."""
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built  # noqa: F401 (a fixture)
from tests.window_ref import F8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [(1, 4), (8, 8), (40, 8)])
@pytest.mark.parametrize("size", [2.0 ** 4, 2.0 ** 20, 2.0 ** 30, 2.0 ** 60, 2.0 ** 106])
@pytest.mark.parametrize("sign", [-1, 1])
def test_equal_scores(sign, size, rows, dtype, D, shared):
    """K is one code everywhere, so a row's scores are the same number for each of its tokens (q is a multiple
    of 1/8, so that its products and their sums are exact in any order), and out the mean of V. Bounds:
    2^-11 for the probability (its rounding is the same for all), sums of n, n 2^-23, twice, 2^-16 for what
    joins the parts, the output's rounding. For lse the score's own rounding too, (D + 8) 2^-23 of it."""
    T, Hq = rows
    B, n, page, H = 3, 1500, 16, 2
    pages = -(-n // page)
    g = torch.Generator("cuda").manual_seed(3)
    k = torch.full((pages, H, page, D), 0x38, dtype=torch.uint8, device="cuda").view(F8)
    v = torch.randn((pages, H, page, D), generator=g, device="cuda").to(F8)
    scale = torch.full((pages, H), 2.0 ** 20, device="cuda")
    q = (torch.randint(4, 13, (B * T, Hq, D), generator=g, device="cuda") / 8).to(dtype) * sign
    sm = size / (2.0 ** 20 * D)  # scores about sign * size
    table = torch.randperm(pages, generator=g, device="cuda").int().repeat(B, 1)
    args = (q, k, v, scale, torch.ones_like(scale), table, torch.full((B,), n, dtype=torch.int32, device="cuda"))
    kw = dict(group_indptr=torch.tensor([0, B], dtype=torch.int32, device="cuda"),
              shared_lens=torch.tensor([n - 100], dtype=torch.int32, device="cuda")) if shared else {}
    got = (tv.shared_attention if shared else tv.window_attention)(*args, **kw, sm_scale=sm, lse=True)
    tokens = v[table[0].long()].permute(0, 2, 1, 3).reshape(-1, H, D)[:n].double()
    mean, absv = (x.mean(0).repeat_interleave(Hq // H, 0) for x in (tokens, tokens.abs()))
    half = torch.finfo(dtype).eps / 2
    share = 2.0 ** -11 + 2 * n * 2.0 ** -23 + 2.0 ** -16
    far = (got["out"].double() - mean).abs() - half * mean.abs() - (1 + half) * absv * share - torch.finfo(dtype).tiny
    assert far.max() <= 0, far.max()
    x = q.double().sum(-1) * 2.0 ** 20 * sm
    lse = x + torch.log(torch.tensor(float(n), dtype=torch.float64))
    assert ((got["lse"].double() - lse).abs() <= x.abs() * (D + 8) * 2.0 ** -23 + n * 2.0 ** -23 + 2.0 ** -17).all()
