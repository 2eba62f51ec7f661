"""GPU: block scales of the cache that are not finite, in window attention."""
import math

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built, make  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("D,Hq", [(64, 4), (64, 32), (128, 4), (128, 32)])
@pytest.mark.parametrize("where", [0, 3, 18])  # the block's place among the request's 19
def test_a_scale_that_is_not_finite_reaches_the_rows_that_see_its_block(name, value, D, Hq, where):
    for dtype in (torch.bfloat16, torch.float16):
        s = make(91, [4, 3], [300, 40], Hq, 2, D, 16, dtype)
        clean = tv.window_attention(**s, lse=True)
        s[name][s["page_table"][0, where].long(), 1] = value
        got = tv.window_attention(**s, lse=True)
        hit = torch.zeros((7, Hq), dtype=torch.bool)
        hit[:4, Hq // 2:] = True
        assert torch.isnan(got["out"].cpu()[hit]).all() and torch.isnan(got["lse"].cpu()[hit]).all()
        for n in ("out", "lse"):
            assert torch.equal(got[n].cpu()[~hit], clean[n].cpu()[~hit])
