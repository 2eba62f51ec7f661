"""GPU: window attention with head_dim 64 over 2^24 tokens, one of which outweighs each of the others by 2^32 and
more: what each of them loses must not add up. As test_gpu_window_tails.py, whose bounds these are."""
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built  # noqa: F401 (a fixture)
from tests.window_ref import F8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("T", [1, 4])  # blocks of 16 rows, of 32
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_small_probabilities_behind_a_large_one(dtype, T, at):
    """Two CTAs a multiprocessor, a request each; all pages but one are the same few. A product takes 16 tokens of
    every 64, so no chain of sums is longer than a 64th of the tokens."""
    D, n, few, page = 64, 1 << 24, 64, 128
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[at]
    k = torch.zeros((few + 1, 1, page, D), dtype=torch.uint8, device="cuda")
    k[few, 0, at % page, 0] = 0x38  # 1
    # V by dims: (large, small) = (1, 1), (0, 1), (1, 0), (-1, 1)
    large = torch.tensor([1.0, 0.0, 1.0, -1.0], device="cuda").repeat(D // 4)
    small = torch.tensor([1.0, 1.0, 0.0, 1.0], device="cuda").repeat(D // 4)
    v = small.to(F8).view(torch.uint8).expand(few + 1, 1, page, D).contiguous()
    v[few, 0, at % page] = large.to(F8).view(torch.uint8)
    row = torch.arange(n // page, dtype=torch.int32, device="cuda") % few
    row[at // page] = few
    ones = torch.ones((few + 1, 1), device="cuda")
    a = torch.tensor([12.0, 20.0, 21.0, 22.0, 22.125, 22.25, 22.5, 23.0], dtype=torch.float64, device="cuda")
    q = torch.zeros((B * T, 8, D), dtype=dtype, device="cuda")
    q[:, :, 0] = a.to(dtype)
    assert torch.equal(q[0, :, 0].double(), a)
    got = tv.window_attention(q, k.view(F8), v.view(F8), ones, ones.clone(), row.repeat(B, 1),
                              torch.full((B,), n, dtype=torch.int32, device="cuda"), sm_scale=1.0)["out"].double()
    w = torch.exp(a)[:, None]
    out = (w * large + (n - 1) * small) / (w + n - 1)
    absv = (w * large.abs() + (n - 1) * small) / (w + n - 1)
    d, sums = 2.0 ** -17, (n / 64 + 64) * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    far = (got - out).abs() - half * out.abs() - (1 + half) * (absv * (2.0 ** -11 + 2 * d + 2 * sums) + 2.0 ** -11)
    assert far.max() <= 0, (far.max(), (got - out).abs().amax((0, 2)))
