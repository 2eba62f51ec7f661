"""Thin ctypes binding over libtsverify.so.

Argument marshalling only: each function takes torch tensors, passes their device
pointers, sizes and the current CUDA stream to the C call of the same name, and
raises ``TsError`` on a non-zero status. No computation happens here and there is
no fallback: if the library is missing or a call fails, the call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtsverify.so")

TS_F32, TS_BF16, TS_F16 = 0, 1, 2
GREEDY_T = 1e-5
MAX_DRAFT = 64
MAX_WINDOW = MAX_DRAFT + 1
_lib = None


class TsError(RuntimeError):
    def __init__(self, call: str, status: int, message: str):
        super().__init__(f"{call} failed with status {status}: {message}")
        self.status = status


class ChainArgs(ctypes.Structure):
    _fields_ = [
        ("target", ctypes.c_void_p),
        ("target_dtype", ctypes.c_int32),
        ("target_is_logits", ctypes.c_int32),
        ("batch", ctypes.c_int64),
        ("D", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("vocab", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("temperature", ctypes.c_void_p),
        ("top_k", ctypes.c_void_p),
        ("top_p", ctypes.c_void_p),
        ("draft_probs", ctypes.c_void_p),
        ("ld_draft", ctypes.c_int64),
        ("draft_tokens", ctypes.c_void_p),
        ("seed", ctypes.c_void_p),
        ("offset", ctypes.c_void_p),
        ("uniforms", ctypes.c_void_p),
        ("accepted_tokens", ctypes.c_void_p),
        ("accept_length", ctypes.c_void_p),
        ("accept_index", ctypes.c_void_p),
        ("logprobs", ctypes.c_void_p),
        ("min_p", ctypes.c_void_p),
        ("threshold_single", ctypes.c_float),
        ("threshold_acc", ctypes.c_float),
        ("qo_indptr", ctypes.c_void_p),
        ("total_rows", ctypes.c_int64),
    ]


TS_FILTER_TOP_K_FIRST = 0
TS_FILTER_JOINT = 1


class SampleArgs(ctypes.Structure):
    """ts_sample_args of include/ts_verify.h."""
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("n_per_req", ctypes.c_int32),
        ("batch", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("temperature", ctypes.c_void_p),
        ("top_k", ctypes.c_void_p),
        ("top_p", ctypes.c_void_p),
        ("min_p", ctypes.c_void_p),
        ("filter_order", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("seed", ctypes.c_void_p),
        ("offset", ctypes.c_void_p),
        ("uniforms", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p),
        ("logprobs", ctypes.c_void_p),
        ("probs", ctypes.c_void_p),
        ("ld_probs", ctypes.c_int64),
        ("probs_row", ctypes.c_void_p),
    ]


class KvCache(ctypes.Structure):
    """ts_kv_cache of include/ts_verify.h."""
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_page_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("k_token_stride", ctypes.c_int64),
        ("v_page_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("v_token_stride", ctypes.c_int64),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("page_table", ctypes.c_void_p),
        ("ld_table", ctypes.c_int64),
        ("seq_lens", ctypes.c_void_p),
        ("batch", ctypes.c_int64),
    ]


class AttnArgs(ctypes.Structure):
    """ts_attn_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("q", ctypes.c_void_p),
        ("q_row_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("heads_q", ctypes.c_int32),
        ("k_new", ctypes.c_void_p),
        ("v_new", ctypes.c_void_p),
        ("k_row_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("total_rows", ctypes.c_int64),
        ("qo_indptr", ctypes.c_void_p),
        ("parents", ctypes.c_void_p),
        ("sm_scale", ctypes.c_float),
        ("reserved0", ctypes.c_float),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
    ]


class SharedArgs(ctypes.Structure):
    """ts_shared_args of include/ts_verify.h."""
    _fields_ = [
        ("attn", ctypes.POINTER(AttnArgs)),
        ("group_indptr", ctypes.c_void_p),
        ("shared_lens", ctypes.c_void_p),
        ("groups", ctypes.c_int64),
    ]


class KvAppendArgs(ctypes.Structure):
    """ts_kv_append_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_row_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("total_rows", ctypes.c_int64),
        ("src_index", ctypes.c_void_p),
        ("src_len", ctypes.c_void_p),
        ("ld_src", ctypes.c_int64),
        ("qo_indptr", ctypes.c_void_p),
    ]


class KvReadArgs(ctypes.Structure):
    """ts_kv_read_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("out_indptr", ctypes.c_void_p),
        ("start", ctypes.c_void_p),
        ("total_rows", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("k_out", ctypes.c_void_p),
        ("v_out", ctypes.c_void_p),
    ]


class KvForkArgs(ctypes.Structure):
    """ts_kv_fork_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("sources", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("refcount", ctypes.c_void_p),
        ("refcount_out", ctypes.c_void_p),
        ("table_out", ctypes.c_void_p),
        ("ld_out", ctypes.c_int64),
        ("lens_out", ctypes.c_void_p),
    ]


class KvFreeArgs(ctypes.Structure):
    """ts_kv_free_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("release", ctypes.c_void_p),
        ("refcount", ctypes.c_void_p),
        ("refcount_out", ctypes.c_void_p),
        ("held_lens", ctypes.c_void_p),
    ]


class KvReserveArgs(ctypes.Structure):
    """ts_kv_reserve_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("new_lens", ctypes.c_void_p),
        ("refcount", ctypes.c_void_p),
        ("refcount_out", ctypes.c_void_p),
        ("table_out", ctypes.c_void_p),
        ("ld_out", ctypes.c_int64),
        ("reserved", ctypes.c_void_p),
        ("held_lens", ctypes.c_void_p),
    ]


class KvCompactArgs(ctypes.Structure):
    """ts_kv_compact_args of include/ts_verify.h."""
    _fields_ = [
        ("cache", ctypes.POINTER(KvCache)),
        ("refcount", ctypes.c_void_p),
        ("refcount_out", ctypes.c_void_p),
        ("table_out", ctypes.c_void_p),
        ("ld_out", ctypes.c_int64),
        ("live", ctypes.c_void_p),
        ("held_lens", ctypes.c_void_p),
    ]


class TreeArgs(ctypes.Structure):
    """ts_tree_args of include/ts_verify.h."""
    _fields_ = [
        ("target_probs", ctypes.c_void_p),
        ("vocab", ctypes.c_int64),
        ("ld", ctypes.c_int64),
        ("batch", ctypes.c_int64),
        ("total_rows", ctypes.c_int64),
        ("qo_indptr", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p),
        ("parents", ctypes.c_void_p),
        ("uniforms", ctypes.c_void_p),
        ("D", ctypes.c_int32),
        ("reserved0", ctypes.c_int32),
        ("accepted_tokens", ctypes.c_void_p),
        ("accept_length", ctypes.c_void_p),
        ("accept_index", ctypes.c_void_p),
        ("logprobs", ctypes.c_void_p),
    ]


def load():
    """Loads libtsverify.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    st = ctypes.c_int
    L.ts_workspace_size.argtypes = [i64, i32, i64]
    L.ts_workspace_size.restype = ctypes.c_size_t
    L.ts_workspace_init.argtypes = [P, ctypes.c_size_t, P]
    L.ts_workspace_init.restype = st
    L.ts_last_error_message.argtypes = []
    L.ts_last_error_message.restype = ctypes.c_char_p
    L.ts_device_error.argtypes = [P, ctypes.c_int]
    L.ts_device_error.restype = st
    L.ts_set_wait_cycles.argtypes = [ctypes.c_uint64]
    L.ts_set_wait_cycles.restype = st
    L.ts_softmax_temp.argtypes = [P, ctypes.c_int, i64, i64, i64, P, P, P]
    L.ts_softmax_temp.restype = st
    L.ts_topk_topp_renorm.argtypes = [P, i64, i64, i64, P, P, P, P]
    L.ts_topk_topp_renorm.restype = st
    L.ts_verify_chain_greedy.argtypes = [P, ctypes.c_int, i64, i32, i64, i64, P, P, P, P, P, P,
                                         ctypes.c_size_t, P]
    L.ts_verify_chain_greedy.restype = st
    L.ts_chain_spec_sampling.argtypes = [ctypes.POINTER(ChainArgs), P, ctypes.c_size_t, P]
    L.ts_chain_spec_sampling.restype = st
    L.ts_gumbel_max_sample.argtypes = [P, ctypes.c_int, i64, i32, i64, i64, P, P, P, P, P,
                                       ctypes.c_size_t, P]
    L.ts_gumbel_max_sample.restype = st
    L.ts_gather_logprobs.argtypes = [P, ctypes.c_int, i32, i64, i64, i64, P, P, P,
                                     ctypes.c_size_t, P]
    L.ts_gather_logprobs.restype = st
    L.ts_sample_from_logits.argtypes = [ctypes.POINTER(SampleArgs), P, ctypes.c_size_t, P]
    L.ts_verify_chain_greedy_ragged.argtypes = [P, ctypes.c_int, i64, i32, i64, i64, P, i64, P,
                                                P, P, P, P, P, ctypes.c_size_t, P]
    L.ts_verify_chain_greedy_ragged.restype = st
    L.ts_sample_from_logits.restype = st
    L.ts_attention_workspace_size.argtypes = [i64, i64, i32, i32, i32]
    L.ts_attention_workspace_size.restype = ctypes.c_size_t
    L.ts_window_attention.argtypes = [ctypes.POINTER(AttnArgs), P, ctypes.c_size_t, P]
    L.ts_window_attention.restype = st
    L.ts_shared_attention_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    L.ts_shared_attention_workspace_size.restype = ctypes.c_size_t
    L.ts_shared_attention.argtypes = [ctypes.POINTER(SharedArgs), P, ctypes.c_size_t, P]
    L.ts_shared_attention.restype = st
    for name, args in (("ts_kv_append", KvAppendArgs), ("ts_kv_read", KvReadArgs),
                       ("ts_kv_fork", KvForkArgs), ("ts_kv_free", KvFreeArgs),
                       ("ts_tree_spec_sampling", TreeArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args), P]
        getattr(L, name).restype = st
    for name, args in (("ts_kv_reserve", KvReserveArgs), ("ts_kv_compact", KvCompactArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args), P, ctypes.c_size_t, P]
        getattr(L, name).restype = st
    L.ts_kv_pages_workspace_size.argtypes = [i64, i64]
    L.ts_kv_pages_workspace_size.restype = ctypes.c_size_t
    _lib = L
    return L


def _check(call: str, status: int):
    if status != 0:
        msg = load().ts_last_error_message().decode(errors="replace")
        raise TsError(call, status, msg)


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _dtype(t) -> int:
    if t.dtype == torch.float32:
        return TS_F32
    if t.dtype == torch.bfloat16:
        return TS_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _rows(x):
    """(rows, vocab, ld) of a 2-D row-major tensor whose rows may be padded."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride in the last dimension")
    return x.shape[0], x.shape[1], x.stride(0)


def workspace_size(batch: int, rows_per_req: int, vocab: int) -> int:
    return int(load().ts_workspace_size(batch, rows_per_req, vocab))


def make_workspace(batch: int, rows_per_req: int, vocab: int, device=None, stream=None):
    """A zero-filled workspace for calls of this size (reusable: calls leave it zeroed)."""
    n = workspace_size(batch, rows_per_req, vocab)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    _check("ts_workspace_init", load().ts_workspace_init(_p(ws), n, _stream(stream)))
    return ws


def device_error(clear: bool = True) -> int:
    """The device error word (0: no bounded wait gave up). Synchronises the device."""
    w = ctypes.c_uint32(0)
    st = load().ts_device_error(ctypes.byref(w), int(clear))
    if st not in (0, 4):
        _check("ts_device_error", st)
    return int(w.value)


def set_wait_cycles(cycles: int) -> None:
    """Sets the budget in SM clock cycles of the chain kernel's stage waits and of window
    attention's waits (0: the default)."""
    _check("ts_set_wait_cycles", load().ts_set_wait_cycles(int(cycles)))


def _dense_out(out, rows, V, device):
    """A [rows, V] contiguous fp32 output (the C ABI writes rows of V floats back to back)."""
    if out is None:
        return torch.empty((rows, V), dtype=torch.float32, device=device)
    if out.dtype != torch.float32 or tuple(out.shape) != (rows, V) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous fp32 tensor of shape ({rows}, {V})")
    return out


def softmax_temp(logits, temperature=None, out=None, stream=None):
    rows, V, ld = _rows(logits)
    out = _dense_out(out, rows, V, logits.device)
    _check("ts_softmax_temp", load().ts_softmax_temp(
        _p(logits), _dtype(logits), rows, V, ld, _p(temperature), _p(out), _stream(stream)))
    return out


def topk_topp_renorm(probs, top_k=None, top_p=None, out=None, stream=None):
    rows, V, ld = _rows(probs)
    out = _dense_out(out, rows, V, probs.device)
    _check("ts_topk_topp_renorm", load().ts_topk_topp_renorm(
        _p(probs), rows, V, ld, _p(top_k), _p(top_p), _p(out), _stream(stream)))
    return out


def _chain_outputs(B, R, device, accept_index, logprobs):
    acc = torch.empty((B, R), dtype=torch.int32, device=device)
    alen = torch.empty((B,), dtype=torch.int32, device=device)
    aidx = torch.empty((B, R), dtype=torch.int32, device=device) if accept_index else None
    lp = torch.empty((B, R), dtype=torch.float32, device=device) if logprobs else None
    return acc, alen, aidx, lp


def verify_chain_greedy(target_logits, D: int, draft_tokens, workspace=None, *,
                        accept_index: bool = True, logprobs: bool = True, outputs=None,
                        stream=None):
    rows, V, ld = _rows(target_logits)
    R = D + 1
    B = rows // R
    if workspace is None:
        workspace = make_workspace(B, R, V, target_logits.device, stream)
    acc, alen, aidx, lp = outputs or _chain_outputs(B, R, target_logits.device, accept_index,
                                                    logprobs)
    _check("ts_verify_chain_greedy", load().ts_verify_chain_greedy(
        _p(target_logits), _dtype(target_logits), B, D, V, ld, _p(draft_tokens), _p(acc),
        _p(alen), _p(aidx), _p(lp), _p(workspace), workspace.numel(), _stream(stream)))
    return dict(accepted_tokens=acc, accept_length=alen, accept_index=aidx, logprobs=lp)


def verify_chain_greedy_ragged(target_logits, D: int, qo_indptr, draft_tokens, workspace=None,
                               *, accept_index: bool = True, logprobs: bool = True,
                               outputs=None, stream=None):
    """Greedy verification of packed rows (request b owns rows qo_indptr[b] ..
    qo_indptr[b+1] - 1, qo_indptr int32 [B+1] on the device); outputs [B, D+1]."""
    rows, V, ld = _rows(target_logits)
    R = D + 1
    B = qo_indptr.numel() - 1
    if workspace is None:
        workspace = make_workspace(B, R, V, target_logits.device, stream)
    acc, alen, aidx, lp = outputs or _chain_outputs(B, R, target_logits.device, accept_index,
                                                    logprobs)
    _check("ts_verify_chain_greedy_ragged", load().ts_verify_chain_greedy_ragged(
        _p(target_logits), _dtype(target_logits), B, D, V, ld, _p(qo_indptr), rows,
        _p(draft_tokens), _p(acc), _p(alen), _p(aidx), _p(lp), _p(workspace), workspace.numel(),
        _stream(stream)))
    return dict(accepted_tokens=acc, accept_length=alen, accept_index=aidx, logprobs=lp)


def chain_spec_sampling(target, target_is_logits: bool, D: int, draft_tokens, *,
                        draft_probs=None, temperature=None, top_k=None, top_p=None,
                        seed=None, offset=None, uniforms=None, workspace=None,
                        accept_index: bool = True, logprobs: bool = True, outputs=None,
                        stream=None, min_p=None, threshold_single: float = 1.0,
                        threshold_acc: float = 1.0, qo_indptr=None):
    """Chain sampling of [B*(D+1), V] rows, or, with qo_indptr (int32 [B+1] on the
    device), of packed rows: request b owns rows qo_indptr[b] .. qo_indptr[b+1] - 1."""
    rows, V, ld = _rows(target)
    R = D + 1
    B = rows // R if qo_indptr is None else qo_indptr.numel() - 1
    if workspace is None:
        workspace = make_workspace(B, R, V, target.device, stream)
    acc, alen, aidx, lp = outputs or _chain_outputs(B, R, target.device, accept_index, logprobs)
    a = ChainArgs()
    a.target = target.data_ptr()
    a.target_dtype = _dtype(target)
    a.target_is_logits = int(bool(target_is_logits))
    a.batch, a.D, a.vocab, a.ld = B, D, V, ld
    a.temperature = None if temperature is None else temperature.data_ptr()
    a.top_k = None if top_k is None else top_k.data_ptr()
    a.top_p = None if top_p is None else top_p.data_ptr()
    if draft_probs is not None:
        q = draft_probs.reshape(-1, draft_probs.shape[-1]) if draft_probs.dim() == 3 else draft_probs
        a.draft_probs = q.data_ptr()
        a.ld_draft = q.stride(0)
    a.draft_tokens = None if draft_tokens is None else draft_tokens.data_ptr()
    a.seed = None if seed is None else seed.data_ptr()
    a.offset = None if offset is None else offset.data_ptr()
    a.uniforms = None if uniforms is None else uniforms.data_ptr()
    a.accepted_tokens = acc.data_ptr()
    a.accept_length = alen.data_ptr()
    a.accept_index = None if aidx is None else aidx.data_ptr()
    a.logprobs = None if lp is None else lp.data_ptr()
    a.min_p = None if min_p is None else min_p.data_ptr()
    a.threshold_single = float(threshold_single)
    a.threshold_acc = float(threshold_acc)
    if qo_indptr is not None:
        a.qo_indptr = qo_indptr.data_ptr()
        a.total_rows = rows
    _check("ts_chain_spec_sampling", load().ts_chain_spec_sampling(
        ctypes.byref(a), _p(workspace), workspace.numel(), _stream(stream)))
    return dict(accepted_tokens=acc, accept_length=alen, accept_index=aidx, logprobs=lp)


def sample_from_logits(logits, n_per_req: int = 1, *, temperature=None, top_k=None, top_p=None,
                       min_p=None, joint: bool = False, seed=None, offset=None, uniforms=None,
                       workspace=None, logprobs: bool = False, probs=None, probs_row=None,
                       out=None, stream=None):
    """Single-step sampling of each row. probs: True for a new [rows, V] fp32 tensor of
    the kept distributions, or a 2-D fp32 tensor that probs_row (int64 [rows]) indexes."""
    rows, V, ld = _rows(logits)
    B = rows // n_per_req
    dev = logits.device
    if workspace is None:
        workspace = make_workspace(rows, 1, V, dev, stream)
    tok = out if out is not None else torch.empty((rows,), dtype=torch.int32, device=dev)
    lp = torch.empty((rows,), dtype=torch.float32, device=dev) if logprobs else None
    if probs is True:
        probs = torch.empty((rows, V), dtype=torch.float32, device=dev)
    a = SampleArgs()
    a.logits = logits.data_ptr()
    a.dtype = _dtype(logits)
    a.n_per_req = n_per_req
    a.batch, a.vocab, a.ld = B, V, ld
    for name, t in (("temperature", temperature), ("top_k", top_k), ("top_p", top_p),
                    ("min_p", min_p), ("seed", seed), ("offset", offset),
                    ("uniforms", uniforms), ("probs_row", probs_row)):
        setattr(a, name, None if t is None else t.data_ptr())
    a.filter_order = TS_FILTER_JOINT if joint else TS_FILTER_TOP_K_FIRST
    a.tokens = tok.data_ptr()
    a.logprobs = None if lp is None else lp.data_ptr()
    if probs is not None:
        a.probs = probs.data_ptr()
        a.ld_probs = probs.stride(0)
    _check("ts_sample_from_logits", load().ts_sample_from_logits(
        ctypes.byref(a), _p(workspace), workspace.numel(), _stream(stream)))
    return dict(tokens=tok, logprobs=lp, probs=probs)


def gumbel_max_sample(logits, n_per_req: int, temperature, seed, offset, workspace=None,
                      out=None, stream=None):
    rows, V, ld = _rows(logits)
    B = rows // n_per_req
    if workspace is None:
        workspace = make_workspace(B, n_per_req, V, logits.device, stream)
    if out is None:
        out = torch.empty((rows,), dtype=torch.int32, device=logits.device)
    _check("ts_gumbel_max_sample", load().ts_gumbel_max_sample(
        _p(logits), _dtype(logits), B, n_per_req, V, ld, _p(temperature), _p(seed), _p(offset),
        _p(out), _p(workspace), workspace.numel(), _stream(stream)))
    return out


def gather_logprobs(x, tokens, is_probs: bool = False, workspace=None, out=None, stream=None):
    rows, V, ld = _rows(x)
    if workspace is None and not is_probs:
        workspace = make_workspace(rows, 1, V, x.device, stream)
    if out is None:
        out = torch.empty((rows,), dtype=torch.float32, device=x.device)
    nbytes = 0 if workspace is None else workspace.numel()
    _check("ts_gather_logprobs", load().ts_gather_logprobs(
        _p(x), _dtype(x), int(bool(is_probs)), rows, V, ld, _p(tokens), _p(out), _p(workspace),
        nbytes, _stream(stream)))
    return out


# ---- around the verify step: a window's attention over the 8-bit cache, the cache, trees ----

_CODES = (torch.float8_e4m3fn, torch.uint8)
_KV_DTYPES = {torch.float32: TS_F32, torch.bfloat16: TS_BF16, torch.float16: TS_F16}


def _kv_dtype(dtype) -> int:
    if dtype not in _KV_DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    return _KV_DTYPES[dtype]


class _On:
    """The device and stream of a call that names a stream or is not on the current device: its
    outputs and scratch come from that stream's pool, its kernels go to that stream."""

    def __init__(self, device, stream):
        self.contexts = [torch.cuda.device(device)]
        if stream is not None:
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


class _Here:
    """The usual case: the current stream of the current device."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        return self.stream

    def __exit__(self, *exc):
        pass


def _on(device: int, stream):
    if device < 0:
        raise ValueError("expected CUDA tensors")
    if stream is None and device == torch.cuda.current_device():
        return _Here(torch._C._cuda_getCurrentRawStream(device))
    return _On(device, stream)


def _same_device(device: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor is on {t.device}, the first one on device {device}")


def _int32(name, t, *shape):
    """The address of a contiguous int32 tensor of this shape (None: not given)."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens):
    """The ts_kv_cache of the tensors (pages, heads, page_size, head_dim) and their device."""
    shape = k_cache.shape
    if len(shape) != 4 or shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must be [pages, heads, page_size, head_dim]")
    n, H, size, D = shape
    k0, k1, k2, k3 = k_cache.stride()
    v0, v1, v2, v3 = v_cache.stride()
    if k_cache.dtype not in _CODES or v_cache.dtype not in _CODES:
        raise TypeError("the cache holds float8_e4m3fn (or its bytes as uint8)")
    if k3 != 1 or v3 != 1:
        raise ValueError("the cache needs unit stride in the last dimension")
    for t in (k_scale, v_scale):
        if t.dtype != torch.float32 or t.shape != (n, H) or not t.is_contiguous():
            raise ValueError(f"scales must be contiguous fp32 tensors of shape ({n}, {H})")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be a 2-D int32 tensor with unit stride in the last dimension")
    B, P = page_table.shape
    ld = page_table.stride(0) if B > 1 and P > 0 else P
    if ld < P:
        raise ValueError("the rows of page_table must not overlap")
    device = k_cache.get_device()
    _same_device(device, v_cache, k_scale, v_scale, page_table, seq_lens)
    return KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k0, k1, k2, v0, v1, v2,
                   k_scale.data_ptr(), v_scale.data_ptr(), n, H, D, size, P, page_table.data_ptr(),
                   ld, _int32("seq_lens", seq_lens, B), B), device


def _heads(name, t, heads, D):
    """(rows, row stride, head stride) in bytes of a [rows, heads, D] tensor."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != D or stride[2] != 1:
        raise ValueError(f"{name} must be [rows, {heads}, {D}] with unit stride in the last dimension")
    size = t.element_size()
    return shape[0], stride[0] * size, stride[1] * size


def attention_workspace_size(batch: int, rows: int, heads_q: int, heads: int, head_dim: int) -> int:
    return int(load().ts_attention_workspace_size(batch, rows, heads_q, heads, head_dim))


def make_attention_workspace(batch: int, rows: int, heads_q: int, heads: int, head_dim: int, device=None):
    """Scratch for window_attention calls of this size that do not overlap."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return torch.empty(attention_workspace_size(batch, rows, heads_q, heads, head_dim),
                           dtype=torch.uint8, device="cuda")


def window_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, k_new=None,
                     v_new=None, qo_indptr=None, parents=None, sm_scale=None, lse: bool = False,
                     out=None, workspace=None, stream=None):
    """Attention of each request's window over its cached tokens and itself.

    q [rows, Hq, D] and the window's own k_new, v_new [rows, H, D] (bf16 or fp16; without them:
    the cached tokens only); k_cache, v_cache [pages, H, page_size, D] e4m3 with k_scale,
    v_scale fp32 [pages, H]; page_table int32 [B, max_pages], seq_lens int32 [B]. Rows are
    packed by qo_indptr (int32 [B+1]) or rows / B a request; parents (int32 [rows], window
    row numbers) makes each window a tree. sm_scale: 1/sqrt(D) by default. Returns
    dict(out=[rows, Hq, D], lse=[rows, Hq] fp32 or None)."""
    cache = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    return _attend(cache, None, q, k_new, v_new, qo_indptr, parents, sm_scale, lse, out, workspace, stream)


def _attend(cache, shared, q, k_new, v_new, qo_indptr, parents, sm_scale, lse, out, workspace, stream):
    """Window attention, or, with shared = (group_indptr, shared_lens), shared attention."""
    c, device = cache
    D, H, B = c.head_dim, c.heads, c.batch
    if q.dim() != 3:
        raise ValueError("q must be [rows, heads, head_dim]")
    Hq = q.shape[1]
    rows, qr, qh = _heads("q", q, Hq, D)
    _same_device(device, q, k_new, v_new, qo_indptr, parents, out, workspace, *(shared or ()))
    if shared:
        groups = shared[1].shape[0] if shared[1].dim() == 1 else 0
        shared = _int32("group_indptr", shared[0], groups + 1), _int32("shared_lens", shared[1], groups), groups
    k_ptr = v_ptr = None
    kr = kh = vr = vh = 0
    if k_new is not None and v_new is not None:
        nk, kr, kh = _heads("k_new", k_new, H, D)
        nv, vr, vh = _heads("v_new", v_new, H, D)
        if nk != rows or nv != rows or k_new.dtype != q.dtype or v_new.dtype != q.dtype:
            raise ValueError("k_new and v_new must have the rows and the dtype of q")
    if k_new is not None:
        k_ptr = k_new.data_ptr()
    if v_new is not None:
        v_ptr = v_new.data_ptr()
    with _on(device, stream) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous, with the shape and dtype of q")
        z = torch.empty((rows, Hq), dtype=torch.float32, device=q.device) if lse else None
        if workspace is None:
            size = shared_attention_workspace_size(B, groups, rows, Hq, H, D) if shared else \
                attention_workspace_size(B, rows, Hq, H, D)
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
        elif not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        a = AttnArgs(ctypes.pointer(c), q.data_ptr(), qr, qh, _kv_dtype(q.dtype), Hq, k_ptr, v_ptr,
                     kr, kh, vr, vh, rows, _int32("qo_indptr", qo_indptr, B + 1),
                     _int32("parents", parents, rows), D ** -0.5 if sm_scale is None else sm_scale,
                     0.0, out.data_ptr(), None if z is None else z.data_ptr())
        if shared:
            st = load().ts_shared_attention(SharedArgs(ctypes.pointer(a), *shared), workspace.data_ptr(),
                                            workspace.nbytes, s)
        else:
            st = load().ts_window_attention(a, workspace.data_ptr(), workspace.nbytes, s)
        if st:
            _check("ts_shared_attention" if shared else "ts_window_attention", st)
    return dict(out=out, lse=z)


def shared_attention_workspace_size(batch: int, groups: int, rows: int, heads_q: int, heads: int,
                                    head_dim: int) -> int:
    return int(load().ts_shared_attention_workspace_size(batch, groups, rows, heads_q, heads, head_dim))


def make_shared_attention_workspace(batch: int, groups: int, rows: int, heads_q: int, heads: int, head_dim: int,
                                    device=None):
    """Scratch for shared_attention calls of this size that do not overlap."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return torch.empty(shared_attention_workspace_size(batch, groups, rows, heads_q, heads, head_dim),
                           dtype=torch.uint8, device="cuda")


def shared_attention(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, group_indptr, shared_lens,
                     k_new=None, v_new=None, qo_indptr=None, parents=None, sm_scale=None, lse: bool = False,
                     out=None, workspace=None, stream=None):
    """window_attention of requests that continue common prefixes: group g is the requests
    group_indptr[g] .. group_indptr[g+1] - 1 (int32 [groups+1]); the whole pages among the first
    shared_lens[g] tokens (int32 [groups]) must be the same in all of its tables (kv_fork leaves
    them so) and are read once for the group. Everything else as for window_attention."""
    cache = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    return _attend(cache, (group_indptr, shared_lens), q, k_new, v_new, qo_indptr, parents, sm_scale, lse, out,
                   workspace, stream)


def kv_append(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, qo_indptr=None,
              src_index=None, src_len=None, stream=None):
    """Quantises rows of k, v [rows, H, D] (bf16, fp16 or fp32) into the cache, in place, behind
    each request's seq_lens tokens (which it does not update): the rows src_index[b, :src_len[b]]
    (a verify call's accept_index and accept_length), or the packed rows of qo_indptr, or
    rows / B a request."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    H, D, B = c.heads, c.head_dim, c.batch
    rows, kr, kh = _heads("k", k, H, D)
    nv, vr, vh = _heads("v", v, H, D)
    if nv != rows or v.dtype != k.dtype:
        raise ValueError("v must have the rows and the dtype of k")
    _same_device(device, k, v, qo_indptr, src_index, src_len)
    n = 0
    if src_index is not None:
        if src_index.dim() != 2:
            raise ValueError("src_index must be [B, n]")
        n = src_index.shape[1]
    with _on(device, stream) as s:
        a = KvAppendArgs(ctypes.pointer(c), k.data_ptr(), v.data_ptr(), kr, kh, vr, vh,
                         _kv_dtype(k.dtype), 0, rows, _int32("src_index", src_index, B, n),
                         _int32("src_len", src_len, B), n, _int32("qo_indptr", qo_indptr, B + 1))
        st = load().ts_kv_append(a, s)
        if st:
            _check("ts_kv_append", st)


def kv_read(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, out_indptr, total_rows: int,
            start=None, dtype=torch.bfloat16, out=None, stream=None):
    """Reads tokens back: request b's tokens from start[b] (0) on into rows out_indptr[b] ..
    out_indptr[b+1] - 1 of k and v [total_rows, H, D] (out: a pair of such tensors)."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    B, shape = c.batch, (total_rows, c.heads, c.head_dim)
    with _on(device, stream) as s:
        if out is None:
            k = torch.empty(shape, dtype=dtype, device=k_cache.device)
            v = torch.empty(shape, dtype=dtype, device=k_cache.device)
        else:
            k, v = out
            for t in (k, v):
                if t.dtype != k.dtype or t.shape != shape or not t.is_contiguous():
                    raise ValueError(f"outputs must be contiguous tensors of shape {shape} and one dtype")
        _same_device(device, out_indptr, start, k, v)
        a = KvReadArgs(ctypes.pointer(c), _int32("out_indptr", out_indptr, B + 1),
                       _int32("start", start, B), total_rows, _kv_dtype(k.dtype), 0, k.data_ptr(),
                       v.data_ptr())
        st = load().ts_kv_read(a, s)
        if st:
            _check("ts_kv_read", st)
    return dict(k=k, v=v)


def _counts(c, refcount, refcount_out):
    """The addresses of the counts, and the tensor that the call's go to (in place by default)."""
    if refcount_out is None:
        refcount_out = refcount
    return (_int32("refcount", refcount, c.num_pages), _int32("refcount_out", refcount_out, c.num_pages),
            refcount_out)


def _table_out(name, t, rows, P):
    """The ld of a table that a call writes."""
    if t.dtype != torch.int32 or t.shape != (rows, P) or (P > 1 and t.stride(1) != 1) or \
            (rows > 1 and t.stride(0) < P):
        raise ValueError(f"{name} must be an int32 tensor of shape ({rows}, {P}) with unit stride in the last "
                         "dimension and rows that do not overlap")
    return t.stride(0) if rows > 1 and P > 0 else P


def pages_workspace_size(batch: int, num_pages: int) -> int:
    return int(load().ts_kv_pages_workspace_size(batch, num_pages))


def make_pages_workspace(batch: int, num_pages: int, device=None):
    """Scratch for kv_reserve and kv_compact calls of this size that do not overlap."""
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        return torch.empty(pages_workspace_size(batch, num_pages), dtype=torch.uint8, device="cuda")


def _pages_workspace(workspace, c, device):
    if workspace is None:
        return torch.empty(pages_workspace_size(c.batch, c.num_pages), dtype=torch.uint8, device=device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def kv_fork(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, sources, refcount,
            refcount_out=None, out=None, stream=None):
    """Continuations of requests that share their pages: request i of the result continues
    request sources[i] (int32 [n]; outside the batch: an empty one). refcount (int32 [pages],
    holders of each page) counts each entry of the result, in place or into refcount_out.
    Returns dict(page_table [n, max_pages], seq_lens [n], refcount); out: a pair of tensors for the
    first two."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    count, count_out, refcount_out = _counts(c, refcount, refcount_out)
    n = sources.shape[0] if sources.dim() == 1 else 0
    src = _int32("sources", sources, n)
    _same_device(device, sources, refcount, refcount_out, *(out or ()))
    with _on(device, stream) as s:
        if out is None:
            table = torch.empty((n, c.max_pages), dtype=torch.int32, device=k_cache.device)
            lens = torch.empty((n,), dtype=torch.int32, device=k_cache.device)
        else:
            table, lens = out
        a = KvForkArgs(ctypes.pointer(c), src, n, count, count_out, table.data_ptr(),
                       _table_out("page_table of out", table, n, c.max_pages), _int32("seq_lens of out", lens, n))
        st = load().ts_kv_fork(a, s)
        if st:
            _check("ts_kv_fork", st)
    return dict(page_table=table, seq_lens=lens, refcount=refcount_out)


def kv_free(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, refcount, release=None,
            held_lens=None, refcount_out=None, stream=None):
    """Releases the pages of the requests with release[b] != 0 (int32 [B]; without it: of all):
    each of their entries counts one holder less in refcount (int32 [pages]), in place or into
    refcount_out, which is returned. Tables and lengths stay as they are. held_lens: as for
    kv_reserve."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    count, count_out, refcount_out = _counts(c, refcount, refcount_out)
    _same_device(device, refcount, refcount_out, release, held_lens)
    with _on(device, stream) as s:
        a = KvFreeArgs(ctypes.pointer(c), _int32("release", release, c.batch), count, count_out,
                       _int32("held_lens", held_lens, c.batch))
        st = load().ts_kv_free(a, s)
        if st:
            _check("ts_kv_free", st)
    return refcount_out


def kv_reserve(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, new_lens, refcount,
               held_lens=None, refcount_out=None, page_table_out=None, workspace=None, stream=None):
    """Room for new_lens (int32 [B]) tokens, ready for kv_append: fresh pages, and a copy of a
    last page that others hold too. refcount and page_table are updated in place, or into
    refcount_out and page_table_out. Returns dict(page_table, refcount, reserved): reserved[b]
    is new_lens[b], or seq_lens[b] where the pool had too few pages left: no more than that
    may be appended. held_lens (int32 [B]): tokens that requests have pages for already, the
    largest `reserved` each was given; without it pages behind those of seq_lens are lost.
    Layers with a pool each under one table: a call a layer, all from the same page_table and
    refcount into the same page_table_out and refcount_out."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    count, count_out, refcount_out = _counts(c, refcount, refcount_out)
    table = page_table if page_table_out is None else page_table_out
    ld = _table_out("page_table_out", table, c.batch, c.max_pages)
    new, held = _int32("new_lens", new_lens, c.batch), _int32("held_lens", held_lens, c.batch)
    _same_device(device, new_lens, held_lens, refcount, refcount_out, table, workspace)
    with _on(device, stream) as s:
        reserved = torch.empty((c.batch,), dtype=torch.int32, device=k_cache.device)
        workspace = _pages_workspace(workspace, c, k_cache.device)
        a = KvReserveArgs(ctypes.pointer(c), new, count, count_out, table.data_ptr(), ld, reserved.data_ptr(),
                          held)
        st = load().ts_kv_reserve(a, workspace.data_ptr(), workspace.nbytes, s)
        if st:
            _check("ts_kv_reserve", st)
    return dict(page_table=table, refcount=refcount_out, reserved=reserved)


def kv_compact(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, *, refcount,
               held_lens=None, refcount_out=None, page_table_out=None, workspace=None, stream=None):
    """Moves the live pages (refcount above 0) to the lowest ids, and the tables with them, in
    place or into refcount_out and page_table_out. Returns dict(page_table, refcount, live):
    live int32 [1], the number of live pages. held_lens, and layers: as for kv_reserve."""
    c, device = _cache(k_cache, v_cache, k_scale, v_scale, page_table, seq_lens)
    count, count_out, refcount_out = _counts(c, refcount, refcount_out)
    table = page_table if page_table_out is None else page_table_out
    ld = _table_out("page_table_out", table, c.batch, c.max_pages)
    held = _int32("held_lens", held_lens, c.batch)
    _same_device(device, held_lens, refcount, refcount_out, table, workspace)
    with _on(device, stream) as s:
        live = torch.empty((1,), dtype=torch.int32, device=k_cache.device)
        workspace = _pages_workspace(workspace, c, k_cache.device)
        a = KvCompactArgs(ctypes.pointer(c), count, count_out, table.data_ptr(), ld, live.data_ptr(), held)
        st = load().ts_kv_compact(a, workspace.data_ptr(), workspace.nbytes, s)
        if st:
            _check("ts_kv_compact", st)
    return dict(page_table=table, refcount=refcount_out, live=live)


def tree_spec_sampling(target_probs, D: int, tokens, parents, uniforms, *, qo_indptr=None,
                       accept_index: bool = True, logprobs: bool = True, outputs=None, stream=None):
    """Verifies drafted trees against fp32 probability rows [rows, V] (one a node) with given
    coins: tokens, parents (int32) and uniforms (fp32) are [B, N], or [rows] packed by
    qo_indptr (int32 [B+1]). At most D drafts are accepted; outputs [B, D+1]."""
    rows, V, ld = _rows(target_probs)
    if target_probs.dtype != torch.float32:
        raise TypeError("target_probs must be fp32")
    if qo_indptr is None and tokens.dim() != 2:
        raise ValueError("tokens must be [B, N] without qo_indptr")
    B = tokens.shape[0] if qo_indptr is None else qo_indptr.numel() - 1
    if tokens.numel() != rows:
        raise ValueError("target_probs must have one row for each token")
    if uniforms.dtype != torch.float32 or uniforms.numel() != rows or not uniforms.is_contiguous():
        raise ValueError("uniforms must be a contiguous fp32 tensor with one coin for each token")
    device = target_probs.get_device()
    _same_device(device, tokens, parents, uniforms, qo_indptr)
    with _on(device, stream) as s:
        acc, alen, aidx, lp = outputs or _chain_outputs(B, D + 1, target_probs.device, accept_index,
                                                        logprobs)
        if outputs:
            _same_device(device, acc, alen, aidx, lp)
            if lp is not None and (lp.dtype != torch.float32 or lp.shape != (B, D + 1) or
                                   not lp.is_contiguous()):
                raise ValueError(f"logprobs must be a contiguous fp32 tensor of shape ({B}, {D + 1})")
        a = TreeArgs(target_probs.data_ptr(), V, ld, B, rows, _int32("qo_indptr", qo_indptr, B + 1),
                     _int32("tokens", tokens, *tokens.shape),
                     _int32("parents", parents, *tokens.shape), uniforms.data_ptr(), D, 0,
                     _int32("accepted_tokens", acc, B, D + 1), _int32("accept_length", alen, B),
                     _int32("accept_index", aidx, B, D + 1), None if lp is None else lp.data_ptr())
        st = load().ts_tree_spec_sampling(a, s)
        if st:
            _check("ts_tree_spec_sampling", st)
    return dict(accepted_tokens=acc, accept_length=alen, accept_index=aidx, logprobs=lp)
