"""Refusals of held_lens in the calls on the cache's pages, on the host (no GPU needed)."""
import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_pages_host import B, C, D, WS, args, refused
from tests.test_window_host import lib, tensors  # noqa: F401


@pytest.mark.parametrize("call,held", [
    ("ts_kv_free", B + 36), ("ts_kv_reserve", B), ("ts_kv_reserve", C + 28), ("ts_kv_reserve", D + 4),
    ("ts_kv_reserve", WS + 64), ("ts_kv_compact", B + 4), ("ts_kv_compact", C), ("ts_kv_compact", D - 4), ("ts_kv_compact", WS)])
def test_arrays_that_overlap(lib, call, held):  # noqa: F811
    refused(lib, call, args(call, held_lens=held), "apart", ws=WS)


def test_binding():
    c = tensors()
    i, two = torch.zeros(5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call, kw in ((tv.kv_free, {}), (tv.kv_reserve, dict(new_lens=two)), (tv.kv_compact, {})):
        with pytest.raises(ValueError, match="CUDA"):
            call(*c, refcount=i, held_lens=two, **kw)
    for call, kw in ((tv.kv_reserve, dict(new_lens=two)), (tv.kv_compact, {})):
        for bad in (i, two.long(), torch.zeros((2, 1), dtype=torch.int32)):
            with pytest.raises(ValueError, match="held_lens"):
                call(*c, refcount=i, held_lens=bad, **kw)
