"""Thin ctypes binding of libls, one Python function per C entry point, with
the same names.  Only argument marshalling happens here (torch tensors to
device pointers, structs, the current CUDA stream); every step of the replay
path runs in the library's kernels.  A missing library is an error: there is
no fallback.
"""
from __future__ import annotations

import ctypes
import os
from pathlib import Path

__all__ = [
    "LsError", "lib", "library_path", "AttnDesc", "PromptKV", "Member",
    "LS_DTYPE_F32", "LS_DTYPE_BF16",
    "ls_kv_page_write", "ls_replay_workspace_size", "ls_replay_fwd", "ls_lse_merge",
    "ls_replay_bwd_preprocess", "ls_replay_bwd", "ls_replay_group",
    "ls_read_device_status", "ls_clear_device_status", "ls_status_string", "ls_last_error",
    "ls_trace_enable", "ls_trace_reset", "ls_trace_read", "ls_num_kernel_ids",
    "ls_kernel_name", "ls_launch_count", "ls_uses_tensor_cores", "kernel_trace",
    "desc_for", "prompt_from", "EXPORTED_SYMBOLS", "ls_replay_fwd_noalloc",
    "ls_replay_fwd_noalloc_scratch_bytes", "ls_prompt_prefill", "ls_prompt_prefill_workspace_size",
    "ls_replay_fwd_part", "ls_replay_bwd_part", "ls_sum_parts",
    "GdnDesc", "LS_GDN_EXACT", "LS_GDN_TENSOR_CORE", "LS_GDN_BWD_REUSES_FORWARD", "ls_gdn_workspace_size", "ls_gdn_replay_fwd",
    "ls_gdn_replay_bwd", "ls_stage_pages",
    "LS_CACHE_F32", "LS_CACHE_BF16", "LS_CACHE_E4M3", "KvCache", "CachedAttnDesc", "VocabDesc",
    "kv_cache_from", "cached_attn_desc", "vocab_desc", "ls_cache_write", "ls_cache_read",
    "ls_cached_attn_workspace_size", "ls_cached_attn", "ls_vocab_logprob_workspace_size",
    "ls_vocab_logprob_fwd", "ls_vocab_logprob_bwd",
]

LS_DTYPE_F32 = 0
LS_DTYPE_BF16 = 1

EXPORTED_SYMBOLS = [
    "ls_kv_page_write", "ls_replay_workspace_size", "ls_replay_fwd", "ls_lse_merge",
    "ls_replay_bwd_preprocess", "ls_replay_bwd", "ls_replay_group", "ls_read_device_status",
    "ls_clear_device_status", "ls_status_string", "ls_last_error", "ls_trace_enable",
    "ls_trace_reset", "ls_trace_read", "ls_num_kernel_ids", "ls_kernel_name",
    "ls_launch_count", "ls_uses_tensor_cores", "ls_replay_fwd_noalloc",
    "ls_replay_fwd_noalloc_scratch_bytes", "ls_prompt_prefill", "ls_prompt_prefill_workspace_size",
    "ls_replay_fwd_part", "ls_replay_bwd_part", "ls_sum_parts",
    "ls_gdn_workspace_size", "ls_gdn_replay_fwd", "ls_gdn_replay_bwd", "ls_stage_pages",
    "ls_cache_write", "ls_cache_read", "ls_cached_attn_workspace_size", "ls_cached_attn",
    "ls_vocab_logprob_workspace_size", "ls_vocab_logprob_fwd", "ls_vocab_logprob_bwd",
]


class LsError(RuntimeError):
    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name}: {detail}")
        self.status = status
        self.name = name


class AttnDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float)]


class PromptKV(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("pool_pages", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("prompt_len", ctypes.c_int64)]


class Member(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("d_o", ctypes.c_void_p), ("resp_len", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("o", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("delta", ctypes.c_void_p), ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p),
                ("dv", ctypes.c_void_p)]


LS_GDN_EXACT = 0
LS_GDN_TENSOR_CORE = 1
LS_GDN_BWD_REUSES_FORWARD = 1  # ls_gdn_desc.flags


class GdnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("dk", ctypes.c_int32),
                ("dv", ctypes.c_int32), ("precision", ctypes.c_int32), ("flags", ctypes.c_int32)]


LS_CACHE_F32 = 0
LS_CACHE_BF16 = 1
LS_CACHE_E4M3 = 2


class KvCache(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pool_pages", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_exp", ctypes.c_void_p),
                ("v_exp", ctypes.c_void_p)]
    on_gpu = True  # kv_cache_from clears it for pools in host memory, which the calls refuse


class CachedAttnDesc(ctypes.Structure):
    _fields_ = [("q_dtype", ctypes.c_int32), ("o_dtype", ctypes.c_int32), ("hq", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("total_q", ctypes.c_int64), ("max_q", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("max_kv", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("softmax_scale", ctypes.c_float)]


class VocabDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("hidden", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("piece", ctypes.c_int32), ("n_rows", ctypes.c_int64), ("h_stride", ctypes.c_int64),
                ("w_stride", ctypes.c_int64), ("ignore_index", ctypes.c_int64),
                ("logit_scale", ctypes.c_float)]


def library_path() -> Path:
    return Path(os.environ.get("LS_LIBRARY",
                               Path(__file__).resolve().parent / "_lib" / "libls.so"))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libls; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not path.exists():
        raise RuntimeError(
            f"libls not found at {path}; build it first (python -c 'import __graft_entry__ as g; "
            "g.build()' or python long_context_grpo_replay_gb300/build.py)")
    L = ctypes.CDLL(str(path))
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "ls_kv_page_write": [ctypes.POINTER(AttnDesc), P, P, I64, P, I64, I64, I64, P, P, P, SZ, P],
        "ls_replay_workspace_size": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), I32,
                                     ctypes.POINTER(SZ)],
        "ls_replay_fwd": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), P, P, P, I32, P, P,
                          P, SZ, P],
        "ls_lse_merge": [I32, I64, I32, P, P, I32, P, P, P],
        "ls_replay_bwd_preprocess": [ctypes.POINTER(AttnDesc), P, P, I32, P, P],
        "ls_replay_bwd": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), P, P, P, P, P, P,
                          I32, P, P, P, P, SZ, P],
        "ls_replay_group": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), I32,
                            ctypes.POINTER(Member), P, SZ, P],
        "ls_prompt_prefill": [ctypes.POINTER(AttnDesc), P, P, P, I32, P, P, P, P, I64, P, I64, P,
                              SZ, P],
        "ls_prompt_prefill_workspace_size": [ctypes.POINTER(AttnDesc), I32, ctypes.POINTER(SZ)],
        "ls_sum_parts": [I32, I64, P, I32, P, P],
        "ls_replay_fwd_part": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), P, P, P, I32, I32,
                               P, P, P, SZ, P],
        "ls_replay_bwd_part": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), P, P, P, P, P, P,
                               I32, I32, P, P, P, P, SZ, P],
        "ls_gdn_workspace_size": [ctypes.POINTER(GdnDesc), I32, ctypes.POINTER(SZ)],
        "ls_gdn_replay_fwd": [ctypes.POINTER(GdnDesc), P, P, P, P, P, P, I32, P, P, P, SZ, P],
        "ls_gdn_replay_bwd": [ctypes.POINTER(GdnDesc), P, P, P, P, P, P, P, I32, P, P, P, P, P, P,
                              SZ, P],
        "ls_stage_pages": [ctypes.POINTER(AttnDesc), P, P, I64, P, I64, I32, P, P, P, SZ, P],
        "ls_cache_write": [ctypes.POINTER(KvCache), I32, P, P, I64, I64, P, I64, P, SZ, P],
        "ls_cache_read": [ctypes.POINTER(KvCache), P, I64, I32, P, P, P, SZ, P],
        "ls_cached_attn_workspace_size": [ctypes.POINTER(CachedAttnDesc), ctypes.POINTER(KvCache),
                                          ctypes.POINTER(SZ)],
        "ls_cached_attn": [ctypes.POINTER(CachedAttnDesc), ctypes.POINTER(KvCache), P, P, P, P, I64,
                           P, P, P, SZ, P],
        "ls_vocab_logprob_workspace_size": [ctypes.POINTER(VocabDesc), I32, ctypes.POINTER(SZ)],
        "ls_vocab_logprob_fwd": [ctypes.POINTER(VocabDesc), P, P, P, P, P, P, SZ, P],
        "ls_vocab_logprob_bwd": [ctypes.POINTER(VocabDesc), P, P, P, P, P, P, P, P, SZ, P],
        "ls_read_device_status": [P, SZ, P],
        "ls_clear_device_status": [P, SZ, P],
        "ls_trace_enable": [I32],
        "ls_trace_reset": [],
        "ls_trace_read": [I32, ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_double)],
        "ls_uses_tensor_cores": [ctypes.POINTER(AttnDesc)],
        "ls_replay_fwd_noalloc": [ctypes.POINTER(AttnDesc), ctypes.POINTER(PromptKV), P, P, P,
                                  I32, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int32
    for name, res, args in [("ls_status_string", ctypes.c_char_p, [I32]),
                            ("ls_last_error", ctypes.c_char_p, []),
                            ("ls_num_kernel_ids", I32, []),
                            ("ls_kernel_name", ctypes.c_char_p, [I32]),
                            ("ls_launch_count", I64, []),
                            ("ls_replay_fwd_noalloc_scratch_bytes", SZ, [])]:
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        L = lib()
        raise LsError(status, L.ls_status_string(status).decode(), L.ls_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        # torch.cuda.current_stream().cuda_stream without the Stream object in
        # between, which costs as much as a small call's launch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_CODES = {}  # torch dtype -> LS_DTYPE_*


def _dtype_code(dt) -> int:
    if not _CODES:
        import torch
        _CODES.update({torch.float32: LS_DTYPE_F32, torch.bfloat16: LS_DTYPE_BF16})
    code = _CODES.get(dt)
    if code is None:
        raise ValueError(f"unsupported dtype {dt}")
    return code


def desc_for(hq, hkv, head_dim, page_size, dtype, softmax_scale=None) -> AttnDesc:
    """Build an AttnDesc; dtype may be a torch dtype or an LS_DTYPE_* code."""
    code = dtype if isinstance(dtype, int) else _dtype_code(dtype)
    scale = softmax_scale if softmax_scale is not None else head_dim ** -0.5
    return AttnDesc(code, hq, hkv, head_dim, page_size, scale)


def prompt_from(k_pool, v_pool, page_table, prompt_len) -> PromptKV:
    """PromptKV over device tensors (pools [pool_pages, Hkv, S_p, d], int32 table)."""
    if prompt_len == 0:
        return PromptKV(None, None, 0, None, 0, 0)
    return PromptKV(_ptr(k_pool), _ptr(v_pool), k_pool.shape[0], _ptr(page_table),
                    page_table.shape[0], prompt_len)


# ------------------------------------------------------------------ entry points
def ls_kv_page_write(desc, k_pool, v_pool, page_table, start_pos, k, v, ws=None, stream=None):
    _want_dtype(desc, k_pool, v_pool, k, v)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().ls_kv_page_write(ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool),
                                  k_pool.shape[0], _ptr(page_table), page_table.shape[0],
                                  start_pos, k.shape[0], _ptr(k), _ptr(v), _ptr(ws), ws_bytes,
                                  _stream(stream)))


def ls_replay_workspace_size(desc, prompt, max_resp_len) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ls_replay_workspace_size(ctypes.byref(desc), ctypes.byref(prompt),
                                          max_resp_len, ctypes.byref(out)))
    return out.value


def _nbytes(t):
    return t.numel() * t.element_size()


def _want_f32(*ts):
    import torch
    for t in ts:
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"expected a float32 tensor, got {t.dtype}")


def _want_dtype(desc, *ts):
    for t in ts:
        if t is not None and _dtype_code(t.dtype) != desc.dtype:
            raise TypeError(f"tensor dtype {t.dtype} does not match the descriptor dtype")


def ls_replay_fwd(desc, prompt, q, k_resp, v_resp, o, lse, ws, stream=None):
    _want_f32(lse)
    _want_dtype(desc, q, k_resp, v_resp, o)
    _check(lib().ls_replay_fwd(ctypes.byref(desc), ctypes.byref(prompt), _ptr(q), _ptr(k_resp),
                               _ptr(v_resp), q.shape[0], _ptr(o), _ptr(lse), _ptr(ws),
                               _nbytes(ws), _stream(stream)))


def ls_prompt_prefill_workspace_size(desc, n_tok) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ls_prompt_prefill_workspace_size(ctypes.byref(desc), n_tok, ctypes.byref(out)))
    return out.value


def ls_prompt_prefill(desc, q, k, v, o, lse, k_pool, v_pool, page_table, ws, stream=None):
    """Capture a prompt: write its K/V into the pool pages and compute its
    causal self-attention o, lse (see ls.h)."""
    _want_f32(lse)
    _want_dtype(desc, q, k, v, o, k_pool, v_pool)
    _check(lib().ls_prompt_prefill(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), q.shape[0],
                                   _ptr(o), _ptr(lse), _ptr(k_pool), _ptr(v_pool), k_pool.shape[0],
                                   _ptr(page_table), page_table.shape[0], _ptr(ws), _nbytes(ws),
                                   _stream(stream)))


def ls_replay_fwd_part(desc, prompt, q, k_resp, v_resp, with_response, o_part, lse_part, ws,
                       stream=None):
    """One rank's exact float32 partial of the replay forward (see ls.h)."""
    _want_f32(o_part, lse_part)
    _want_dtype(desc, q, k_resp, v_resp)
    _check(lib().ls_replay_fwd_part(ctypes.byref(desc), ctypes.byref(prompt), _ptr(q), _ptr(k_resp),
                                    _ptr(v_resp), q.shape[0], 1 if with_response else 0,
                                    _ptr(o_part), _ptr(lse_part), _ptr(ws), _nbytes(ws),
                                    _stream(stream)))


def ls_replay_bwd_part(desc, prompt, q, k_resp, v_resp, d_o, lse, delta, with_response, dq_part,
                       dk=None, dv=None, ws=None, stream=None):
    """One rank's float32 share of dQ (and the response dK/dV on the rank
    that holds the response keys; see ls.h)."""
    _want_f32(lse, delta, dq_part)
    _want_dtype(desc, q, k_resp, v_resp, d_o, dk, dv)
    _check(lib().ls_replay_bwd_part(ctypes.byref(desc), ctypes.byref(prompt), _ptr(q), _ptr(k_resp),
                                    _ptr(v_resp), _ptr(d_o), _ptr(lse), _ptr(delta), q.shape[0],
                                    1 if with_response else 0, _ptr(dq_part), _ptr(dk), _ptr(dv),
                                    _ptr(ws), _nbytes(ws), _stream(stream)))


def ls_sum_parts(parts, out, stream=None):
    """out = parts.sum(0) in float32 accumulation (parts float32 [n, ...])."""
    _want_f32(parts)
    n = parts.shape[0]
    _check(lib().ls_sum_parts(n, out.numel(), _ptr(parts), _dtype_code(out.dtype), _ptr(out),
                              _stream(stream)))


def _gdn_desc(s0, q, precision, flags=0):
    """q [B, R, H, dk] (a group) or [R, H, dk] (one member)."""
    return GdnDesc(q.shape[0] if q.dim() == 4 else 1, s0.shape[0], s0.shape[2], s0.shape[1],
                   precision, flags)


def _resp_len(q):
    return q.shape[1] if q.dim() == 4 else q.shape[0]


def ls_gdn_workspace_size(desc, resp_len) -> int:
    """desc: GdnDesc(batch, heads, dk, dv, precision)."""
    out = ctypes.c_size_t(0)
    _check(lib().ls_gdn_workspace_size(ctypes.byref(desc), resp_len, ctypes.byref(out)))
    return out.value


def ls_gdn_replay_fwd(s0, q, k, v, g, beta, o, s_final=None, ws=None, stream=None,
                      precision=LS_GDN_EXACT):
    """Gated-DeltaNet replay from the captured state s0 [H, dv, dk] of one
    member (q [R, H, dk]) or a group (q [B, R, H, dk]); see ls.h.  float32
    buffers; precision LS_GDN_EXACT (ws may be None) or LS_GDN_TENSOR_CORE
    (ws of ls_gdn_workspace_size bytes)."""
    _want_f32(s0, q, k, v, g, beta, o, s_final)
    _check(lib().ls_gdn_replay_fwd(ctypes.byref(_gdn_desc(s0, q, precision)), _ptr(s0), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(g), _ptr(beta), _resp_len(q), _ptr(o), _ptr(s_final),
                                   _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def ls_gdn_replay_bwd(s0, q, k, v, g, beta, d_o, dq, dk, dv, dg, dbeta, ws, stream=None,
                      precision=LS_GDN_EXACT, reuse_forward=False):
    """Gradients of the replay for q, k, v, g, beta (none for s0; see ls.h).
    reuse_forward: ws holds the scratch of ls_gdn_replay_fwd on these same
    inputs (LS_GDN_BWD_REUSES_FORWARD)."""
    _want_f32(s0, q, k, v, g, beta, d_o, dq, dk, dv, dg, dbeta)
    desc = _gdn_desc(s0, q, precision, LS_GDN_BWD_REUSES_FORWARD if reuse_forward else 0)
    _check(lib().ls_gdn_replay_bwd(ctypes.byref(desc), _ptr(s0), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(g), _ptr(beta), _ptr(d_o), _resp_len(q), _ptr(dq), _ptr(dk),
                                   _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(ws), _nbytes(ws),
                                   _stream(stream)))


def ls_stage_pages(desc, k_src, v_src, page_table, first_page, n_pages, k_dst, v_dst, ws=None,
                   stream=None):
    """Logical pages first_page .. first_page+n_pages-1 (slots from the
    device page_table) of pinned-host or device pools into staging pools;
    see ls.h."""
    _want_dtype(desc, k_src, v_src, k_dst, v_dst)
    _check(lib().ls_stage_pages(ctypes.byref(desc), _ptr(k_src), _ptr(v_src), k_src.shape[0],
                                _ptr(page_table), first_page, n_pages, _ptr(k_dst), _ptr(v_dst),
                                _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def ls_replay_fwd_noalloc(desc, prompt, q, k_resp, v_resp, o, lse, stream=None):
    """ls_replay_fwd without a workspace: for callers that cannot allocate
    device memory; uses the library's fixed device scratch (see ls.h)."""
    _want_f32(lse)
    _want_dtype(desc, q, k_resp, v_resp, o)
    _check(lib().ls_replay_fwd_noalloc(ctypes.byref(desc), ctypes.byref(prompt), _ptr(q),
                                       _ptr(k_resp), _ptr(v_resp), q.shape[0], _ptr(o), _ptr(lse),
                                       _stream(stream)))


def ls_replay_fwd_noalloc_scratch_bytes() -> int:
    return lib().ls_replay_fwd_noalloc_scratch_bytes()


def ls_lse_merge(o_parts, lse_parts, o, lse=None, stream=None):
    n_parts, n_rows, d = o_parts.shape
    _want_f32(o_parts, lse_parts, lse)
    _check(lib().ls_lse_merge(n_parts, n_rows, d, _ptr(o_parts), _ptr(lse_parts),
                              _dtype_code(o.dtype), _ptr(o), _ptr(lse), _stream(stream)))


def ls_replay_bwd_preprocess(desc, o, d_o, delta, stream=None):
    _want_f32(delta)
    _want_dtype(desc, o, d_o)
    _check(lib().ls_replay_bwd_preprocess(ctypes.byref(desc), _ptr(o), _ptr(d_o), o.shape[0],
                                          _ptr(delta), _stream(stream)))


def ls_replay_bwd(desc, prompt, q, k_resp, v_resp, d_o, lse, delta, dq, dk, dv, ws, stream=None):
    _want_f32(lse, delta)
    _want_dtype(desc, q, k_resp, v_resp, d_o, dq, dk, dv)
    _check(lib().ls_replay_bwd(ctypes.byref(desc), ctypes.byref(prompt), _ptr(q), _ptr(k_resp),
                               _ptr(v_resp), _ptr(d_o), _ptr(lse), _ptr(delta), q.shape[0],
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws), _nbytes(ws),
                               _stream(stream)))


def ls_replay_group(desc, prompt, members, ws, stream=None):
    """members: sequence of dicts with tensors q, k, v, d_o, o, lse, delta, dq, dk, dv."""
    arr = (Member * max(1, len(members)))()
    for i, m in enumerate(members):
        _want_f32(m["lse"], m["delta"])
        _want_dtype(desc, m["q"], m["k"], m["v"], m["d_o"], m["o"], m["dq"], m["dk"], m["dv"])
        arr[i] = Member(_ptr(m["q"]), _ptr(m["k"]), _ptr(m["v"]), _ptr(m["d_o"]),
                        m["q"].shape[0], 0, _ptr(m["o"]), _ptr(m["lse"]), _ptr(m["delta"]),
                        _ptr(m["dq"]), _ptr(m["dk"]), _ptr(m["dv"]))
    _check(lib().ls_replay_group(ctypes.byref(desc), ctypes.byref(prompt), len(members), arr,
                                 _ptr(ws), _nbytes(ws), _stream(stream)))


def _want(t, dtype, shape, name):
    """Shape, dtype and contiguity of a tensor the library takes by its address alone."""
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _refuse_host():
    """The kernels read addresses: a tensor of the host's must not reach them."""
    raise ValueError("all tensors, and a cache's pools, must be on the GPU")


def _token_stride(t, name):
    """Elements from one token to the next of a [n, heads, d] tensor whose heads are contiguous."""
    n, heads, d = t.shape
    s = t.stride()
    if (s[2] != 1 or (heads > 1 and s[1] != d)) and t.numel():
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s[0] if n > 1 else heads * d


def kv_cache_from(k, v, k_exp=None, v_exp=None) -> KvCache:
    """A cache over pools [pages, Hkv, S_p, d]: float32, bfloat16, or float8_e4m3fn with
    int8 exponents [pages, Hkv, S_p].  The cache holds addresses: keep the tensors alive."""
    import torch
    fmt = {torch.float32: LS_CACHE_F32, torch.bfloat16: LS_CACHE_BF16,
           torch.float8_e4m3fn: LS_CACHE_E4M3}.get(k.dtype)
    if fmt is None or k.dim() != 4:
        raise TypeError(f"cache pools are 4-D float32, bfloat16 or float8_e4m3fn, got {k.dtype}")
    _want(k, k.dtype, k.shape, "k")
    _want(v, k.dtype, k.shape, "v")
    if fmt == LS_CACHE_E4M3:
        if k_exp is None or v_exp is None:
            raise ValueError("an e4m3 cache needs k_exp and v_exp")
        _want(k_exp, torch.int8, k.shape[:3], "k_exp")
        _want(v_exp, torch.int8, k.shape[:3], "v_exp")
    pages, hkv, page, d = k.shape
    cache = KvCache(fmt, hkv, d, page, pages, _ptr(k), _ptr(v), _ptr(k_exp), _ptr(v_exp))
    cache.on_gpu = all(t is None or t.is_cuda for t in (k, v, k_exp, v_exp))
    return cache


def _cache_rows(cache, slots, k, v):
    import torch
    n = k.shape[0]
    _want(slots, torch.int64, (n,), "slots")
    want = (n, cache.hkv, cache.head_dim)
    if k.shape != want or v.shape != want or v.dtype != k.dtype:
        raise ValueError(f"k and v must be {want} of one dtype")
    return n


def ls_cache_write(cache, k, v, slots, ws=None, stream=None):
    """Token t's rows of k, v [n, Hkv, d] (any token stride) into slot slots[t] (see ls.h)."""
    n = _cache_rows(cache, slots, k, v)
    k_stride, v_stride = _token_stride(k, "k"), _token_stride(v, "v")
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and cache.on_gpu and (ws is None or ws.is_cuda)):
        _refuse_host()
    _check(lib().ls_cache_write(cache, _dtype_code(k.dtype), k.data_ptr(), v.data_ptr(),
                                k_stride, v_stride, slots.data_ptr(),
                                n, _ptr(ws), 0 if ws is None else _nbytes(ws), _stream(stream)))


def ls_cache_read(cache, slots, k, v, ws=None, stream=None):
    """Slot slots[t] into token t of k, v [n, Hkv, d] (see ls.h)."""
    n = _cache_rows(cache, slots, k, v)
    if not (k.is_contiguous() and v.is_contiguous()):
        raise ValueError("k and v must be contiguous")
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and cache.on_gpu and (ws is None or ws.is_cuda)):
        _refuse_host()
    _check(lib().ls_cache_read(cache, slots.data_ptr(), n, _dtype_code(k.dtype), k.data_ptr(),
                               v.data_ptr(), _ptr(ws), 0 if ws is None else _nbytes(ws),
                               _stream(stream)))


def cached_attn_desc(q, o, batch, max_q, max_kv, causal=True, softmax_scale=None) -> CachedAttnDesc:
    """Desc of ls_cached_attn for q [total_q, Hq, d] and o of q's dtype or float32."""
    total, hq, d = q.shape
    scale = softmax_scale if softmax_scale is not None else d ** -0.5
    return CachedAttnDesc(_dtype_code(q.dtype), _dtype_code(o.dtype), hq, batch, total, max_q,
                          1 if causal else 0, max_kv, _token_stride(q, "q"), scale)


def ls_cached_attn_workspace_size(desc, cache) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ls_cached_attn_workspace_size(ctypes.byref(desc), ctypes.byref(cache),
                                               ctypes.byref(out)))
    return out.value


def ls_cached_attn(desc, cache, q, q_start, kv_len, page_table, o, lse, ws, stream=None):
    """Attention of each sequence's new tokens over its pages (see ls.h)."""
    import torch
    shape = (desc.total_q, desc.hq, cache.head_dim)
    if q.shape != shape or _dtype_code(q.dtype) != desc.q_dtype or \
            _token_stride(q, "q") != desc.q_stride:
        raise ValueError(f"q is not the {shape} tensor of the desc")
    _want(o, torch.float32 if desc.o_dtype == LS_DTYPE_F32 else torch.bfloat16, shape, "o")
    _want(lse, torch.float32, shape[:2], "lse")
    _want(q_start, torch.int32, (desc.batch + 1,), "q_start")
    _want(kv_len, torch.int64, (desc.batch,), "kv_len")
    pages = page_table.shape[-1]
    _want(page_table, torch.int32, (desc.batch, pages), "page_table")
    if not (q.is_cuda and q_start.is_cuda and kv_len.is_cuda and page_table.is_cuda and o.is_cuda and lse.is_cuda and
            ws.is_cuda and cache.on_gpu):
        _refuse_host()
    _check(lib().ls_cached_attn(desc, cache, q.data_ptr(), q_start.data_ptr(), kv_len.data_ptr(),
                                page_table.data_ptr(), pages, o.data_ptr(), lse.data_ptr(),
                                ws.data_ptr(), _nbytes(ws), _stream(stream)))


def _rows(t, name):
    if t.dim() != 2 or (t.numel() and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def vocab_desc(h, w, logit_scale=1.0, ignore_index=-100, piece=0) -> VocabDesc:
    """Desc of ls_vocab_logprob_* for h [n, hidden] and w [vocab, hidden] of one dtype."""
    if h.dtype != w.dtype or h.shape[1] != w.shape[1]:
        raise ValueError("h and w must share dtype and hidden")
    return VocabDesc(_dtype_code(h.dtype), h.shape[1], w.shape[0], piece, h.shape[0], _rows(h, "h"),
                     _rows(w, "w"), ignore_index, logit_scale)


def ls_vocab_logprob_workspace_size(desc, with_grad=True) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ls_vocab_logprob_workspace_size(ctypes.byref(desc), 1 if with_grad else 0,
                                                 ctypes.byref(out)))
    return out.value


def _vocab_check(desc, h, w, targets, *rows):
    import torch
    for t, n, stride, name in ((h, desc.n_rows, desc.h_stride, "h"), (w, desc.vocab, desc.w_stride, "w")):
        if t.shape != (n, desc.hidden) or _dtype_code(t.dtype) != desc.dtype or \
                _rows(t, name) != stride:
            raise ValueError(f"{name} is not the tensor of the desc")
    _want(targets, torch.int64, (desc.n_rows,), "targets")
    for t in rows:
        _want(t, torch.float32, (desc.n_rows,), "a per-row tensor")


def ls_vocab_logprob_fwd(desc, h, w, targets, logp, lse, ws, stream=None):
    """logp of targets [n] and the rows' lse, without the logits (see ls.h)."""
    _vocab_check(desc, h, w, targets, logp, lse)
    if not all(t.is_cuda for t in (h, w, targets, logp, lse, ws)):
        _refuse_host()
    _check(lib().ls_vocab_logprob_fwd(ctypes.byref(desc), _ptr(h), _ptr(w), _ptr(targets), _ptr(logp),
                                      _ptr(lse), _ptr(ws), _nbytes(ws), _stream(stream)))


def ls_vocab_logprob_bwd(desc, h, w, targets, lse, d_logp, dh, dw, ws, stream=None):
    """dh, dw (either may be None) from d_logp [n] (see ls.h)."""
    _vocab_check(desc, h, w, targets, lse, d_logp)
    for t, like, name in ((dh, h, "dh"), (dw, w, "dw")):
        if t is not None:
            _want(t, like.dtype, like.shape, name)
    if not all(t is None or t.is_cuda for t in (h, w, targets, lse, d_logp, dh, dw, ws)):
        _refuse_host()
    _check(lib().ls_vocab_logprob_bwd(ctypes.byref(desc), _ptr(h), _ptr(w), _ptr(targets), _ptr(lse),
                                      _ptr(d_logp), _ptr(dh), _ptr(dw), _ptr(ws), _nbytes(ws),
                                      _stream(stream)))


def ls_read_device_status(ws, stream=None):
    _check(lib().ls_read_device_status(_ptr(ws), _nbytes(ws), _stream(stream)))


def ls_clear_device_status(ws, stream=None):
    _check(lib().ls_clear_device_status(_ptr(ws), _nbytes(ws), _stream(stream)))


def ls_status_string(status: int) -> str:
    return lib().ls_status_string(status).decode()


def ls_last_error() -> str:
    return lib().ls_last_error().decode()


def ls_trace_enable(on: bool = True):
    _check(lib().ls_trace_enable(1 if on else 0))


def ls_trace_reset():
    _check(lib().ls_trace_reset())


def ls_trace_read(kernel_id: int):
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(lib().ls_trace_read(kernel_id, ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value


def ls_num_kernel_ids() -> int:
    return lib().ls_num_kernel_ids()


def ls_kernel_name(kernel_id: int) -> str:
    return lib().ls_kernel_name(kernel_id).decode()


def ls_launch_count() -> int:
    return lib().ls_launch_count()


def ls_uses_tensor_cores(desc) -> bool:
    return lib().ls_uses_tensor_cores(ctypes.byref(desc)) != 0


def kernel_trace() -> dict:
    """{kernel name: (launches, total ms)} accumulated since the last reset."""
    out = {}
    for k in range(ls_num_kernel_ids()):
        n, ms = ls_trace_read(k)
        if n:
            out[ls_kernel_name(k)] = (n, ms)
    return out
