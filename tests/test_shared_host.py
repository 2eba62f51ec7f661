"""Refusals of shared attention, on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_window_host import FAKE, attn, cache, lib, tensors  # noqa: F401


def refused(lib, a, word, status=1, ws=FAKE, size=1 << 40, **kw):  # noqa: F811
    s = dict(attn=ctypes.pointer(a), group_indptr=FAKE, shared_lens=FAKE, groups=2)
    s.update(kw)
    st = lib.ts_shared_attention(ctypes.byref(tv.SharedArgs(**s)), ctypes.c_void_p(ws), size, None)
    msg = lib.ts_last_error_message().decode()
    assert st == status and word in msg, (st, msg)


def test_what_window_attention_refuses(lib):  # noqa: F811
    refused(lib, attn(cache(head_dim=96)), "head_dim")
    refused(lib, attn(cache(page_size=24)), "page_size")
    refused(lib, attn(dtype=tv.TS_F32), "bf16 or fp16", 2)
    refused(lib, attn(heads_q=12), "multiple")
    refused(lib, attn(k_new=0), "together")
    refused(lib, attn(k_new=0, v_new=0, parents=FAKE), "parents")
    refused(lib, attn(q=0), "required")
    refused(lib, attn(q_row_stride=8), "16-byte")
    refused(lib, attn(total_rows=257), "total_rows")
    refused(lib, attn(total_rows=5), "multiple of batch")


def test_groups(lib):  # noqa: F811
    for n in (0, -1, 65537):
        refused(lib, attn(), "groups", groups=n)
    refused(lib, attn(), "group_indptr", group_indptr=0)
    refused(lib, attn(), "shared_lens", shared_lens=0)
    assert lib.ts_shared_attention(None, ctypes.c_void_p(FAKE), 1 << 40, None) == 1
    assert lib.ts_shared_attention(ctypes.byref(tv.SharedArgs(group_indptr=FAKE, shared_lens=FAKE, groups=1)),
                                   ctypes.c_void_p(FAKE), 1 << 40, None) == 1


def test_workspace(lib):  # noqa: F811
    size = lib.ts_shared_attention_workspace_size
    need = size(2, 2, 6, 32, 8, 128)
    assert need > lib.ts_attention_workspace_size(2, 6, 32, 8, 128)
    refused(lib, attn(), "workspace", ws=0)
    refused(lib, attn(), "workspace", ws=FAKE + 8)
    refused(lib, attn(), "workspace", size=need - 1)
    assert size(2, 0, 6, 32, 8, 128) == size(2, 65537, 6, 32, 8, 128) == size(0, 1, 6, 32, 8, 128) == 0
    assert size(2, 2, 6, 30, 8, 128) == size(2, 2, 257, 32, 8, 128) == size(2, 2, 6, 32, 8, 96) == 0


def test_binding():
    c = tensors()
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    ok = dict(group_indptr=i, shared_lens=i[:2])
    with pytest.raises(ValueError, match="CUDA"):
        tv.shared_attention(x, *c, **ok)
    with pytest.raises(ValueError, match="group_indptr"):
        tv.shared_attention(x, *c, group_indptr=i[:2], shared_lens=i[:2])
    with pytest.raises(ValueError, match="shared_lens"):
        tv.shared_attention(x, *c, group_indptr=i, shared_lens=i[:2].long())
    with pytest.raises(ValueError, match="shared_lens|group_indptr"):
        tv.shared_attention(x, *c, group_indptr=i, shared_lens=i[:2].view(1, 2))
    with pytest.raises(ValueError, match="rows and the dtype"):
        tv.shared_attention(x, *c, **ok, k_new=x[:2], v_new=x)
