"""GPU: a wait of window attention (head_dim 128) that runs out is reported and does not reach the
next call. With a budget of one cycle waits give up before their copies land: nothing faults or
hangs (the block issues nothing more, runs to its end, and waits there for what is in flight), the
call's outputs are unspecified, ts_device_error reports it (bit 27)."""
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_gpu_window import _built, make  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("windows,lens,Hq,mask", [
    ([2], [300], 8, "chain"),                                       # blocks of 32 rows
    ([9] * 40, [(i * 211) % 3000 for i in range(40)], 16, "tree"),  # of 64; several units a block
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_wait_that_runs_out(windows, lens, Hq, mask, dtype):
    s = make(61, windows, lens, Hq, 2, 128, 16, dtype, mask)
    want = tv.window_attention(**s, lse=True)
    assert tv.device_error(clear=True) == 0
    rows = sum(windows)
    guard = torch.full((rows + 2, Hq, 128), 7.0, dtype=dtype, device="cuda")
    tv.set_wait_cycles(1)
    try:
        tv.window_attention(**s, out=guard[1:-1])
        torch.cuda.synchronize()
    finally:
        tv.set_wait_cycles(0)
    word = tv.device_error(clear=True)
    assert word == 1 << 27, hex(word)
    assert (guard[0] == 7.0).all() and (guard[-1] == 7.0).all()
    got = tv.window_attention(**s, lse=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])
    assert tv.device_error(clear=True) == 0
