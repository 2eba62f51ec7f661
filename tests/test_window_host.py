"""Refusals of the calls around the verify step, on the host (no GPU needed): the C ABI on
arguments that are never dereferenced, the binding on CPU tensors."""
import ctypes

import pytest
import torch

from speculative_decoding_verify_temp_gb300 import tsverify as tv

FAKE = 1 << 12


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verify_temp_gb300 import build

    build.build()
    return tv.load()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_page_stride=16384, k_head_stride=2048, k_token_stride=128,
             v_page_stride=16384, v_head_stride=2048, v_token_stride=128, k_scale=FAKE,
             v_scale=FAKE, num_pages=10, heads=8, head_dim=128, page_size=16, max_pages=4,
             page_table=FAKE, ld_table=4, seq_lens=FAKE, batch=2)
    a.update(kw)
    return tv.KvCache(**a)


def attn(c=None, **kw):
    a = dict(q=FAKE, q_row_stride=8192, q_head_stride=256, dtype=tv.TS_BF16, heads_q=32,
             k_new=FAKE, v_new=FAKE, k_row_stride=2048, k_head_stride=256, v_row_stride=2048,
             v_head_stride=256, total_rows=6, sm_scale=0.1, out=FAKE)
    a.update(kw)
    return tv.AttnArgs(cache=ctypes.pointer(c or cache()), **a)


def append(c=None, **kw):
    a = dict(k=FAKE, v=FAKE, k_row_stride=2048, k_head_stride=256, v_row_stride=2048,
             v_head_stride=256, dtype=tv.TS_BF16, total_rows=6)
    a.update(kw)
    return tv.KvAppendArgs(cache=ctypes.pointer(c or cache()), **a)


def read(c=None, **kw):
    a = dict(out_indptr=FAKE, total_rows=6, dtype=tv.TS_BF16, k_out=FAKE, v_out=FAKE)
    a.update(kw)
    return tv.KvReadArgs(cache=ctypes.pointer(c or cache()), **a)


def tree(**kw):
    a = dict(target_probs=FAKE, vocab=100, ld=100, batch=2, total_rows=6, tokens=FAKE,
             parents=FAKE, uniforms=FAKE, D=2, accepted_tokens=FAKE, accept_length=FAKE)
    a.update(kw)
    return tv.TreeArgs(**a)


def refused(lib, call, args, word, status=1):
    if call == "ts_window_attention":
        st = lib.ts_window_attention(ctypes.byref(args), ctypes.c_void_p(FAKE), 1 << 40, None)
    else:
        st = getattr(lib, call)(ctypes.byref(args), None)
    msg = lib.ts_last_error_message().decode()
    assert st == status and word in msg, (st, msg)


BAD_CACHES = [
    (dict(head_dim=96), "head_dim"), (dict(page_size=24), "page_size"), (dict(page_size=8), "page_size"),
    (dict(heads=0), "heads"), (dict(batch=0), "batch"), (dict(batch=1 << 17), "batch"),
    (dict(num_pages=-1), "num_pages"), (dict(max_pages=-1), "max_pages"),
    (dict(max_pages=1 << 27, ld_table=1 << 27), "max_pages"), (dict(ld_table=3), "ld_table"),
    (dict(k=FAKE + 8), "aligned"), (dict(v_token_stride=100), "aligned"), (dict(k_head_stride=24), "aligned"),
    (dict(k_page_stride=-16384), "positive"), (dict(v_head_stride=0), "positive"), (dict(k_token_stride=1 << 41), "positive"),
    (dict(k=None), "required"), (dict(v_scale=None), "required"), (dict(seq_lens=None), "required"),
    (dict(page_table=None), "required"),
]


@pytest.mark.parametrize("kw,word", BAD_CACHES)
@pytest.mark.parametrize("call,make", [("ts_window_attention", attn), ("ts_kv_append", append),
                                       ("ts_kv_read", read)])
def test_bad_caches(lib, call, make, kw, word):
    refused(lib, call, make(cache(**kw)), word)


@pytest.mark.parametrize("kw,word,status", [
    (dict(dtype=tv.TS_F32), "bf16 or fp16", 2), (dict(dtype=9), "bf16 or fp16", 2),
    (dict(heads_q=12), "multiple", 1), (dict(heads_q=0), "multiple", 1),
    (dict(total_rows=0), "total_rows", 1), (dict(total_rows=131, qo_indptr=FAKE), "total_rows", 1),
    (dict(total_rows=5), "multiple of batch", 1), (dict(q=None), "required", 1), (dict(out=None), "required", 1),
    (dict(v_new=None), "together", 1), (dict(k_new=None, v_new=None, parents=FAKE), "parents", 1),
    (dict(q_row_stride=8200), "aligned", 1), (dict(k_new=FAKE + 2), "aligned", 1), (dict(out=FAKE + 4), "aligned", 1),
])
def test_attention_refusals(lib, kw, word, status):
    refused(lib, "ts_window_attention", attn(**kw), word, status)


def test_attention_workspace(lib):
    need = lib.ts_attention_workspace_size(2, 6, 32, 8, 128)
    assert need > lib.ts_attention_workspace_size(2, 6, 32, 8, 64) > 0 and need % 256 == 0
    assert lib.ts_attention_workspace_size(2, 130, 32, 8, 128) > need
    for bad in ((2, 6, 32, 8, 96), (0, 6, 32, 8, 128), (2, 131, 32, 8, 128), (2, 0, 32, 8, 128), (2, 6, 32, 7, 128),
                (2, 6, 32, 0, 128), (1 << 17, 6, 32, 8, 128)):
        assert lib.ts_attention_workspace_size(*bad) == 0
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 4, need)):
        a = attn()
        assert lib.ts_window_attention(ctypes.byref(a), ctypes.c_void_p(ws), n, None) == 1
        assert "workspace" in lib.ts_last_error_message().decode()
    assert lib.ts_window_attention(None, ctypes.c_void_p(FAKE), need, None) == 1


@pytest.mark.parametrize("kw,word,status", [
    (dict(dtype=5), "dtype", 2), (dict(k=None), "required", 1), (dict(total_rows=0), "total_rows", 1),
    (dict(total_rows=5), "multiple of batch", 1), (dict(src_index=FAKE), "together", 1),
    (dict(src_index=FAKE, src_len=FAKE, qo_indptr=FAKE, ld_src=4), "together", 1),
    (dict(src_index=FAKE, src_len=FAKE, ld_src=0), "ld_src", 1), (dict(v=FAKE + 8), "aligned", 1),
])
def test_append_refusals(lib, kw, word, status):
    refused(lib, "ts_kv_append", append(**kw), word, status)


@pytest.mark.parametrize("kw,word,status", [
    (dict(dtype=7), "dtype", 2), (dict(out_indptr=None), "required", 1), (dict(k_out=None), "required", 1),
    (dict(total_rows=0), "total_rows", 1), (dict(v_out=FAKE + 8), "aligned", 1),
])
def test_read_refusals(lib, kw, word, status):
    refused(lib, "ts_kv_read", read(**kw), word, status)


@pytest.mark.parametrize("kw,word", [
    (dict(D=-1), "D must"), (dict(D=65), "D must"), (dict(vocab=0), "vocab"), (dict(ld=99), "ld"),
    (dict(batch=0), "batch"), (dict(total_rows=0), "total_rows"), (dict(total_rows=131, qo_indptr=FAKE), "total_rows"),
    (dict(total_rows=5), "multiple of batch"), (dict(tokens=None), "required"),
    (dict(uniforms=None), "required"), (dict(accept_length=None), "required"),
])
def test_tree_refusals(lib, kw, word):
    refused(lib, "ts_tree_spec_sampling", tree(**kw), word)


def test_null_arguments(lib):
    for call in ("ts_kv_append", "ts_kv_read", "ts_tree_spec_sampling"):
        assert getattr(lib, call)(None, None) == 1
    a = append()
    a.cache = None
    refused(lib, "ts_kv_append", a, "cache is NULL")


# ---- the binding's own checks

def tensors(B=2, H=2, D=64, size=16, pages=5, P=2):
    k = torch.zeros((pages, H, size, D), dtype=torch.uint8)
    s = torch.ones((pages, H))
    return [k, k.clone(), s, s.clone(), torch.zeros((B, P), dtype=torch.int32), torch.zeros(B, dtype=torch.int32)]


def replaced(i, t):
    c = tensors()
    c[i] = t
    return c


@pytest.mark.parametrize("c,error", [
    (replaced(0, torch.zeros((5, 2, 16, 32), dtype=torch.uint8)), ValueError),
    (replaced(0, torch.zeros((5, 2, 16, 64))), TypeError),
    (replaced(1, torch.zeros((5, 2, 16, 128), dtype=torch.uint8)[..., ::2]), ValueError),
    (replaced(2, torch.ones((5, 3))), ValueError),
    (replaced(3, torch.ones((5, 2), dtype=torch.float16)), ValueError),
    (replaced(4, torch.zeros((2, 2), dtype=torch.int64)), ValueError),
    (replaced(4, torch.zeros((2, 2), dtype=torch.int32).t()), ValueError),
    (replaced(5, torch.zeros(3, dtype=torch.int32)), ValueError),
    (replaced(5, torch.zeros(2, dtype=torch.int64)), ValueError),
])
def test_binding_refuses_bad_caches(c, error):
    with pytest.raises(error):
        tv.kv_append(torch.zeros((2, 2, 64)), torch.zeros((2, 2, 64)), *c)


def test_binding_refuses_bad_rows():
    c = tensors()
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_append(x, x, *c)
    with pytest.raises(ValueError, match="v must"):
        tv.kv_append(x, x.half(), *c)
    with pytest.raises(ValueError, match="k must"):
        tv.kv_append(x[:, :1], x, *c)
    with pytest.raises(ValueError, match="rows and the dtype"):
        tv.window_attention(x, *c, k_new=x[:2], v_new=x)
    with pytest.raises(ValueError, match="CUDA"):
        tv.window_attention(x, *c, k_new=x, v_new=x)
    with pytest.raises(ValueError, match="CUDA"):
        tv.kv_read(*c, out_indptr=torch.zeros(3, dtype=torch.int32), total_rows=4)
    p = torch.zeros((4, 10))
    i = torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        tv.tree_spec_sampling(p, 1, i, i, torch.zeros((2, 2)))
    with pytest.raises(ValueError, match="one row"):
        tv.tree_spec_sampling(p[:3], 1, i, i, torch.zeros((2, 2)))
    with pytest.raises(ValueError, match="uniforms"):
        tv.tree_spec_sampling(p, 1, i, i, torch.zeros((2, 3)))
    with pytest.raises(TypeError):
        tv.tree_spec_sampling(p.half(), 1, i, i, torch.zeros((2, 2)))


def test_binding_refuses_overlapping_page_tables():
    # requests that share a prefix have tables of their own that name the same pages
    c = replaced(4, torch.zeros((1, 2), dtype=torch.int32).expand(2, 2))
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: tv.kv_append(x, x, *c), lambda: tv.window_attention(x, *c),
                 lambda: tv.kv_read(*c, out_indptr=torch.zeros(3, dtype=torch.int32), total_rows=4)):
        with pytest.raises(ValueError, match="overlap"):
            call()


def test_attention_refuses_heads_past_its_indices(lib):
    refused(lib, "ts_window_attention", attn(heads_q=1 << 17), "multiple", 1)
    assert lib.ts_attention_workspace_size(2, 6, 1 << 17, 8, 128) == 0
