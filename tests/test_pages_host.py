"""Refusals of the calls on the cache's pages, on the host (no GPU needed)."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv
from tests.test_window_host import FAKE, cache, lib, tensors  # noqa: F401

A, B, C, D = (FAKE * (i + 1000) for i in range(4))  # apart from each other and from FAKE


def args(call, c=None, **kw):
    c = c or cache()
    a = {"ts_kv_fork": dict(sources=A, n=3, refcount=B, refcount_out=B, table_out=C, ld_out=4, lens_out=D),
         "ts_kv_free": dict(release=A, refcount=B, refcount_out=B),
         "ts_kv_reserve": dict(new_lens=A, refcount=B, refcount_out=B, table_out=C, ld_out=4, reserved=D),
         "ts_kv_compact": dict(refcount=B, refcount_out=B, table_out=C, ld_out=4, live=D)}[call]
    a.update(kw)
    kind = {"ts_kv_fork": tv.KvForkArgs, "ts_kv_free": tv.KvFreeArgs, "ts_kv_reserve": tv.KvReserveArgs,
            "ts_kv_compact": tv.KvCompactArgs}[call]
    return kind(cache=ctypes.pointer(c), **a)


def refused(lib, call, a, word, ws=A, size=1 << 40):  # noqa: F811
    more = (ctypes.c_void_p(ws), size) if call in ("ts_kv_reserve", "ts_kv_compact") else ()
    st = getattr(lib, call)(ctypes.byref(a), *more, None)
    msg = lib.ts_last_error_message().decode()
    assert st == 1 and word in msg, (st, msg)


CALLS = ["ts_kv_fork", "ts_kv_free", "ts_kv_reserve", "ts_kv_compact"]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,word", [
    (dict(head_dim=96), "head_dim"), (dict(page_size=8), "page_size"), (dict(batch=0), "batch"),
    (dict(k=0), "required"), (dict(ld_table=3), "ld_table"), (dict(k_token_stride=8), "16-byte"),
])
def test_caches(lib, call, kw, word):  # noqa: F811
    refused(lib, call, args(call, cache(**kw)), word)


@pytest.mark.parametrize("call", CALLS)
def test_counts(lib, call):  # noqa: F811
    refused(lib, call, args(call, refcount=0), "refcount")
    refused(lib, call, args(call, refcount_out=0), "refcount")
    refused(lib, call, args(call, refcount_out=B + 36), "apart")  # 10 pages: 40 bytes


@pytest.mark.parametrize("call", ["ts_kv_fork", "ts_kv_reserve", "ts_kv_compact"])
def test_tables(lib, call):  # noqa: F811
    refused(lib, call, args(call, table_out=0), "table_out")
    refused(lib, call, args(call, ld_out=3), "ld_out")
    refused(lib, call, args(call, table_out=FAKE + 16), "apart")  # 2 requests of 4 entries at FAKE
    refused(lib, call, args(call, table_out=FAKE, ld_out=5), "apart")


def test_the_rest(lib):  # noqa: F811
    refused(lib, "ts_kv_fork", args("ts_kv_fork", table_out=FAKE), "apart")
    for n in (0, -1, 65537):
        refused(lib, "ts_kv_fork", args("ts_kv_fork", n=n), "n must")
    refused(lib, "ts_kv_fork", args("ts_kv_fork", sources=0), "sources")
    refused(lib, "ts_kv_fork", args("ts_kv_fork", lens_out=0), "lens_out")
    refused(lib, "ts_kv_fork", args("ts_kv_fork", lens_out=FAKE + 4), "seq_lens")
    refused(lib, "ts_kv_fork", args("ts_kv_fork", lens_out=A + 8), "sources")
    refused(lib, "ts_kv_reserve", args("ts_kv_reserve", new_lens=0), "new_lens")
    refused(lib, "ts_kv_reserve", args("ts_kv_reserve", reserved=0), "reserved")
    refused(lib, "ts_kv_reserve", args("ts_kv_reserve", reserved=A), "apart")
    refused(lib, "ts_kv_reserve", args("ts_kv_reserve", reserved=FAKE), "apart")
    refused(lib, "ts_kv_compact", args("ts_kv_compact", live=0), "live")
    for call in ("ts_kv_reserve", "ts_kv_compact"):
        refused(lib, call, args(call), "workspace", ws=0)
        refused(lib, call, args(call), "workspace", ws=A + 8)
        refused(lib, call, args(call), "workspace", size=lib.ts_kv_pages_workspace_size(2, 10) - 1)
    for call in CALLS:
        more = (ctypes.c_void_p(A), 1 << 40) if call in ("ts_kv_reserve", "ts_kv_compact") else ()
        assert getattr(lib, call)(None, *more, None) == 1


WS = FAKE << 20  # far from the rest


@pytest.mark.parametrize("call,kw", [
    ("ts_kv_fork", dict(lens_out=C + 44)), ("ts_kv_fork", dict(lens_out=B + 8)),          # 3 rows of 4 entries at C
    ("ts_kv_fork", dict(table_out=B)), ("ts_kv_fork", dict(table_out=A + 8)),
    ("ts_kv_fork", dict(refcount=B, refcount_out=FAKE)), ("ts_kv_fork", dict(refcount=B, refcount_out=C, table_out=B)),
    ("ts_kv_free", dict(refcount_out=A + 4)), ("ts_kv_free", dict(refcount_out=FAKE)),
    ("ts_kv_reserve", dict(reserved=C + 28)), ("ts_kv_reserve", dict(reserved=B + 36)),
    ("ts_kv_reserve", dict(table_out=A)), ("ts_kv_reserve", dict(refcount=C, refcount_out=B)),
    ("ts_kv_reserve", dict(refcount=WS, refcount_out=WS)), ("ts_kv_reserve", dict(new_lens=WS + 64)),
    ("ts_kv_compact", dict(live=B)), ("ts_kv_compact", dict(live=C + 28)), ("ts_kv_compact", dict(live=FAKE + 4)),
    ("ts_kv_compact", dict(live=WS)), ("ts_kv_compact", dict(table_out=B + 36)),
])
def test_arrays_that_overlap(lib, call, kw):  # noqa: F811
    refused(lib, call, args(call, **kw), "apart", ws=WS)


def test_workspace(lib):  # noqa: F811
    size = lib.ts_kv_pages_workspace_size
    assert 0 < size(1, 0) <= size(1, 10) < size(1, 10 ** 6) < size(1, 2 ** 31 - 1)
    assert size(0, 10) == size(65537, 10) == size(1, -1) == size(1, 2 ** 31) == 0
    assert size(1, 10) % 16 == 0


def test_binding():
    c = tensors()
    i = torch.zeros(5, dtype=torch.int32)
    two = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_fork(*c, sources=two, refcount=i)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_free(*c, refcount=i)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_reserve(*c, new_lens=two, refcount=i)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_compact(*c, refcount=i)
    for call, kw in ((tv.kv_fork, dict(sources=two)), (tv.kv_free, {}), (tv.kv_reserve, dict(new_lens=two)), (tv.kv_compact, {})):
        with pytest.raises(ValueError, match="refcount"):
            call(*c, refcount=i[:4], **kw)
        with pytest.raises(ValueError, match="refcount"):
            call(*c, refcount=i.long(), **kw)
        with pytest.raises(ValueError, match="refcount_out"):
            call(*c, refcount=i, refcount_out=i[:3], **kw)
    with pytest.raises(ValueError, match="sources"):
        tv.kv_fork(*c, sources=two.long(), refcount=i)
    with pytest.raises(ValueError, match="sources"):
        tv.kv_fork(*c, sources=table, refcount=i)
    with pytest.raises(ValueError, match="new_lens"):
        tv.kv_reserve(*c, new_lens=i, refcount=i)
    for call, kw in ((tv.kv_reserve, dict(new_lens=two)), (tv.kv_compact, {})):
        for bad in (table.long(), table[:1], table.t(), table[:1].expand(2, 2)):
            with pytest.raises(ValueError, match="page_table_out"):
                call(*c, refcount=i, page_table_out=bad, **kw)
