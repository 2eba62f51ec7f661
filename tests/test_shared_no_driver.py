"""Shared attention where the driver's encoder of tensor maps is not found: refused as window attention refuses
it, before anything is launched."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_window_host import FAKE, attn, cache, lib  # noqa: F401


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only where nothing can run")
@pytest.mark.parametrize("D", [64, 128])
def test_without_a_driver(lib, D):  # noqa: F811
    a = attn(cache(head_dim=D))
    s = tv.SharedArgs(attn=ctypes.pointer(a), group_indptr=FAKE, shared_lens=FAKE, groups=2)
    st = lib.ts_shared_attention(ctypes.byref(s), ctypes.c_void_p(FAKE), 1 << 40, None)
    msg = lib.ts_last_error_message().decode()
    if D == 128:
        assert lib.ts_window_attention(ctypes.byref(a), ctypes.c_void_p(FAKE), 1 << 40, None) == st
        assert lib.ts_last_error_message().decode().replace("window", "shared") == msg
    # before the plan was launched: not that there is no device to launch it on
    assert st == 3 and "operation not supported" in msg, (st, msg)
