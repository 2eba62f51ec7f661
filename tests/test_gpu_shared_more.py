"""GPU: shared attention at edges of its own."""
import pytest
import torch

from tests.test_gpu_shared import case, check, reference, tv  # noqa: F401 (tv: a fixture)

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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [3, 60])
def test_scores_that_are_all_very_negative(tv, rows, D):  # noqa: F811
    """Shared tokens of scores near -2^107 and the window's own of ordinary ones: out is the window's alone,
    as if nothing were cached (their weights are 2^-(2^107))."""
    c = case(9, [(128 * 24, [(20, 2)] * rows)], 8, 2, D, 128)
    c["k_scale"][:] = 2.0 ** 100
    c["k_cache"].view(torch.uint8)[:] = 0x38          # ones
    c["q"] = -c["q"].abs()
    got = tv.shared_attention(**c, lse=True)
    alone = dict(c, seq_lens=torch.zeros_like(c["seq_lens"]))
    check(alone, got)


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_v_that_are_nothing(tv, D):  # noqa: F811
    """Scales of V of the shared tokens below 2^-80 count as 2^-80: out is what the other tokens give, and all of
    the sum."""
    c = case(10, [(16 * 40, [(20, 2)] * 40)], 8, 2, D, 16)
    pages = c["page_table"][0, :40].long()
    c["v_scale"][pages] = 0
    c["v_scale"][pages[:20]] = 2.0 ** -140
    check(c, tv.shared_attention(**c, lse=True))
    # the same, its V's codes the largest there are: 448 * 2^-80 a token at most
    c["v_cache"].view(torch.uint8)[pages] = 0x7E
    check(c, tv.shared_attention(**c, lse=True))


@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_v_that_are_nothing_everywhere(tv, D):  # noqa: F811
    # what is left is 2^-80 times the codes' mean, which bf16 holds
    c = case(10, [(16 * 40, [(0, 2)] * 40)], 8, 2, D, 16, mask="none")
    c["v_scale"][:] = 0
    got = tv.shared_attention(**c, lse=True)
    check(dict(c, v_scale=torch.full_like(c["v_scale"], 2.0 ** -80)), got)


def busy(stream, buffers, n):
    """Copies that keep DRAM busy meanwhile."""
    with torch.cuda.stream(stream):
        for _ in range(n):
            buffers[0].copy_(buffers[1])


def test_a_wait_that_runs_out_with_head_dim_64(tv):  # noqa: F811
    """As in test_gpu_shared.py, where DRAM is busy with other work, so that what is waited for takes longer than a
    wait's first tries."""
    c = case(19, [(30000, [(20, 4)] * 50), (17000, [(20, 9)] * 30)], 64, 8, 64, 128)
    want = tv.shared_attention(**c, lse=True)
    assert tv.device_error() == 0
    guard = torch.full((c["q"].shape[0] + 2, 64, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    buffers = torch.empty((2, 1 << 30), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    word = 0
    for _ in range(20):
        busy(side, buffers, 20)
        tv.set_wait_cycles(1)
        try:
            tv.shared_attention(**c, out=guard[1:-1])
            torch.cuda.synchronize()
        finally:
            tv.set_wait_cycles(0)
        word |= tv.device_error(clear=True)
        if word:
            break
    assert word == 1 << 28, hex(word)
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()
    got = tv.shared_attention(**c, lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    assert tv.device_error() == 0
