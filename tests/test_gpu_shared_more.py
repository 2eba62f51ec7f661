"""GPU: shared attention at edges of its own."""
import pytest
import torch

from tests.test_gpu_shared import case, reference, tv  # noqa: F401 (tv: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("where", ["window", "cached", "pieces"])
def test_a_prefix_that_weighs_nothing_passes_nan_on(tv, where, rows, D):  # noqa: F811
    """0 times a value that is not finite is NaN, as in window attention: a row's own tokens outweigh the
    whole prefix by more than fp32's range (scores of 256 against 0, so 2^-369)."""
    own = {"window": 5, "cached": 20, "pieces": 9000}[where]
    c = case(31, [(400, [(own, rows)] * 5), (300, [(own, rows)] * 2)], 8, 2, D, 16, mask="none" if where != "window" else "chain")
    c["q"][:] = 16
    c["k_cache"].view(torch.uint8)[:] = 0
    c["k_scale"][:] = 1
    if where == "window":
        c["k_new"][:] = 16.0 / D
    else:  # the first of the request's own pages
        for b, s in enumerate([400] * 5 + [300 // 16 * 16] * 2):
            c["k_cache"].view(torch.uint8)[c["page_table"][b, s // 16].long(), :, 1] = {64: 0x28, 128: 0x20}[D]  # 16 / D
    before = tv.shared_attention(**c, sm_scale=1.0, lse=True)
    assert torch.isfinite(before["out"]).all()
    assert ((before["lse"].double() - reference(c, 1.0)[1]).abs() < 1e-3).all()
    page = int(c["page_table"][0, 3])
    for code in (0x7F, 0xFF):
        c["v_cache"].view(torch.uint8)[page, 1, 2, 11] = code
        got = tv.shared_attention(**c, sm_scale=1.0, lse=True)
        want = torch.zeros_like(before["out"], dtype=torch.bool)
        want[:5 * rows, 4:, 11] = True
        assert torch.equal(torch.isnan(got["out"]), want)
        assert torch.equal(got["out"][~want], before["out"][~want]) and torch.equal(got["lse"], before["lse"])
        old = tv.window_attention(**{k: v for k, v in c.items() if k not in ("group_indptr", "shared_lens")}, sm_scale=1.0)
        assert torch.equal(torch.isnan(old["out"]), want)
