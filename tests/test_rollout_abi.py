"""Refusals of the rollout and scoring entry points, before any launch (no GPU)."""
import ctypes

import pytest
import torch

A = 1 << 24  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def ls():
    from long_context_grpo_replay_gb300 import build

    build.build()
    import long_context_grpo_replay_gb300.binding as b

    b.lib()
    return b


def cache(ls, **kw):
    d = dict(format=ls.LS_CACHE_E4M3, hkv=4, head_dim=256, page_size=256, pool_pages=16, k=A, v=A, k_exp=A, v_exp=A)
    d.update(kw)
    return ls.KvCache(*(d[n] for n, _ in ls.KvCache._fields_))


def attn(ls, **kw):
    d = dict(q_dtype=1, o_dtype=1, hq=24, batch=2, total_q=4, max_q=2, causal=1, max_kv=1000, q_stride=24 * 256,
             softmax_scale=0.0625)
    d.update(kw)
    return ls.CachedAttnDesc(*(d[n] for n, _ in ls.CachedAttnDesc._fields_))


def vocab(ls, **kw):
    d = dict(dtype=1, hidden=64, vocab=1000, piece=0, n_rows=10, h_stride=64, w_stride=64, ignore_index=-100,
             logit_scale=1.0)
    d.update(kw)
    return ls.VocabDesc(*(d[n] for n, _ in ls.VocabDesc._fields_))


BAD_CACHES = [(dict(format=3), 1), (dict(head_dim=96), 2), (dict(hkv=0), 1), (dict(page_size=0), 1),
              (dict(pool_pages=0), 1), (dict(k=None), 1), (dict(v=A + 8), 1), (dict(k_exp=None), 1),
              (dict(pool_pages=1 << 40), 2)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches(ls, bad, status):
    c = cache(ls, **bad)
    L = ls.lib()
    assert L.ls_cache_write(ctypes.byref(c), 1, A, A, 1024, 1024, A, 3, None, 0, None) == status
    assert L.ls_cache_read(ctypes.byref(c), A, 3, 1, A, A, None, 0, None) == status
    n = ctypes.c_size_t(0)
    assert L.ls_cached_attn_workspace_size(ctypes.byref(attn(ls)), ctypes.byref(c), ctypes.byref(n)) == status
    assert ls.ls_last_error()


def test_cache_calls(ls):
    L, c = ls.lib(), cache(ls)
    w = lambda src=1, k=A, v=A, ks=1024, vs=1024, slots=A, n=3, ws=None, nb=0: L.ls_cache_write(  # noqa: E731
        ctypes.byref(c), src, k, v, ks, vs, slots, n, ws, nb, None)
    assert w(n=0, k=None, v=None, slots=None) == 0
    assert w(n=-1) == 1 and w(src=5) == 1 and w(k=None) == 1 and w(slots=None) == 1
    assert w(ks=1023) == 1 and w(vs=1028) == 1 and w(k=A + 2) == 1 and w(slots=A + 4) == 1
    assert w(ws=A, nb=16) == 3 and w(ws=A + 8, nb=1 << 20) == 1
    r = lambda dst=1, k=A, slots=A, n=3: L.ls_cache_read(ctypes.byref(c), slots, n, dst, k, A, None, 0, None)  # noqa: E731
    assert r(n=0, k=None) == 0 and r(n=-2) == 1 and r(dst=2) == 1 and r(k=None) == 1 and r(slots=A + 1) == 1
    assert L.ls_cache_write(None, 1, A, A, 1024, 1024, A, 3, None, 0, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(q_dtype=2), 1), (dict(o_dtype=2), 1), (dict(q_dtype=0, o_dtype=1), 1), (dict(hq=26), 1), (dict(hq=0), 1),
    (dict(batch=-1), 1), (dict(total_q=-1), 1), (dict(max_q=5), 1), (dict(total_q=5), 1), (dict(max_kv=-1), 1),
    (dict(max_kv=1 << 31), 2), (dict(batch=70000, total_q=2), 2), (dict(q_stride=24 * 256 - 8), 1),
    (dict(q_stride=24 * 256 + 4), 1), (dict(softmax_scale=0.0), 1), (dict(softmax_scale=float("inf")), 1)])
def test_bad_attention_descs(ls, bad, status):
    n = ctypes.c_size_t(0)
    c = cache(ls)
    assert ls.lib().ls_cached_attn_workspace_size(ctypes.byref(attn(ls, **bad)), ctypes.byref(c), ctypes.byref(n)) == status


def test_attention_calls(ls):
    L, c, d = ls.lib(), cache(ls), attn(ls)
    call = lambda d=d, q=A, qs=A, kv=A, pt=A, pps=8, o=A, lse=A, ws=A, nb=1 << 40: L.ls_cached_attn(  # noqa: E731
        ctypes.byref(d), ctypes.byref(c), q, qs, kv, pt, pps, o, lse, ws, nb, None)
    assert call(attn(ls, total_q=0, max_q=0), q=None, ws=None) == 0  # nothing to do
    assert call(attn(ls, batch=0, total_q=0, max_q=0), q=None, ws=None) == 0
    for name in ("q", "qs", "kv", "pt", "o", "lse", "ws"):
        assert call(**{name: None}) == 1, name
    assert call(q=A + 8) == 1 and call(o=A + 2) == 1 and call(kv=A + 4) == 1 and call(pps=-1) == 1
    assert call(pps=1 << 30) == 2
    need = ls.ls_cached_attn_workspace_size(d, c)
    assert call(nb=need - 1) == 3
    assert L.ls_cached_attn(None, ctypes.byref(c), A, A, A, A, 8, A, A, A, 1 << 40, None) == 1


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(hidden=0), 1), (dict(vocab=0), 1), (dict(n_rows=-1), 1), (dict(h_stride=63), 1),
    (dict(w_stride=8), 1), (dict(piece=-1), 1), (dict(ignore_index=5), 1), (dict(logit_scale=float("nan")), 1),
    (dict(n_rows=1 << 40), 2)])
def test_bad_vocab_descs(ls, bad, status):
    n = ctypes.c_size_t(0)
    assert ls.lib().ls_vocab_logprob_workspace_size(ctypes.byref(vocab(ls, **bad)), 1, ctypes.byref(n)) == status


def test_vocab_calls(ls):
    L, d = ls.lib(), vocab(ls)
    f = lambda d=d, h=A, w=A, t=A, logp=A, lse=A, ws=A, nb=1 << 40: L.ls_vocab_logprob_fwd(  # noqa: E731
        ctypes.byref(d), h, w, t, logp, lse, ws, nb, None)
    assert f(vocab(ls, n_rows=0), h=None, ws=None) == 0
    for name in ("h", "w", "t", "logp", "lse", "ws"):
        assert f(**{name: None}) == 1, name
    assert f(h=A + 1) == 1 and f(t=A + 4) == 1 and f(nb=255) == 3 and f(ws=A + 16) == 1
    b = lambda d=d, h=A, lse=A, dl=A, dh=A, dw=A, ws=A, nb=1 << 40: L.ls_vocab_logprob_bwd(  # noqa: E731
        ctypes.byref(d), h, A, A, lse, dl, dh, dw, ws, nb, None)
    assert b(dh=None, dw=None) == 0 and b(vocab(ls, n_rows=0), dw=None) == 0
    assert b(h=None) == 1 and b(lse=None) == 1 and b(dl=None) == 1 and b(dh=A + 4) == 1 and b(dw=A + 8) == 1
    assert b(nb=ls.ls_vocab_logprob_workspace_size(d, True) - 1) == 3
    assert ls.ls_vocab_logprob_workspace_size(d, False) <= ls.ls_vocab_logprob_workspace_size(d, True)


def test_binding_checks_tensors(ls):
    k = torch.zeros(2, 4, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ls.kv_cache_from(k.half(), k.half())
    with pytest.raises(ValueError):
        ls.kv_cache_from(k.to(torch.float8_e4m3fn), k.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError):
        ls.kv_cache_from(k.transpose(1, 2), k.transpose(1, 2))
    c = ls.kv_cache_from(k, k.clone())
    rows = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ls.ls_cache_write(c, rows, rows, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        ls.ls_cache_write(c, rows[:, :2], rows, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        ls.ls_cache_write(c, rows.transpose(0, 1).contiguous().transpose(0, 1), rows, torch.zeros(3, dtype=torch.int64))
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    d = ls.cached_attn_desc(q, q, 3, 1, 32)
    args = [torch.arange(4, dtype=torch.int32), torch.ones(3, dtype=torch.int64), torch.zeros(3, 2, dtype=torch.int32)]
    with pytest.raises(TypeError):
        ls.ls_cached_attn(d, c, q, args[0], args[1].int(), args[2], q, torch.zeros(3, 8), torch.zeros(1))
    with pytest.raises(ValueError):
        ls.ls_cached_attn(d, c, q[:2], *args, q, torch.zeros(3, 8), torch.zeros(1))
    h = torch.zeros(3, 64)
    with pytest.raises(ValueError):
        ls.vocab_desc(h, torch.zeros(10, 32))
    vd = ls.vocab_desc(h, torch.zeros(10, 64))
    with pytest.raises(TypeError):
        ls.ls_vocab_logprob_fwd(vd, h, torch.zeros(10, 64), torch.zeros(3, dtype=torch.int32), torch.zeros(3),
                                torch.zeros(3), torch.zeros(1))


def test_binding_refuses_host_tensors(ls):
    """Calls that are right but for tensors in host memory raise before anything is launched."""
    bf, i64 = torch.bfloat16, torch.int64
    k = torch.zeros(2, 4, 16, 64, dtype=bf)
    c = ls.kv_cache_from(k, k.clone())
    rows, slots = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, dtype=i64)
    q, ws = torch.zeros(3, 8, 64, dtype=bf), torch.zeros(1 << 20, dtype=torch.uint8)
    d = ls.cached_attn_desc(q, q, 3, 1, 32)
    h, w, n = torch.zeros(3, 64), torch.zeros(10, 64), lambda: torch.zeros(3)
    vd = ls.vocab_desc(h, w)
    attn = (q, torch.arange(4, dtype=torch.int32), torch.ones(3, dtype=i64), torch.zeros(3, 2, dtype=torch.int32),
            q.clone(), torch.zeros(3, 8), ws)
    on_gpu = ls.KvCache(*(getattr(c, f) for f, _ in ls.KvCache._fields_))  # the caller's word for its addresses
    for cache in (c, on_gpu):
        for call in (lambda: ls.ls_cache_write(cache, rows, rows, slots), lambda: ls.ls_cache_read(cache, slots, rows, rows),
                     lambda: ls.ls_cached_attn(d, cache, *attn)):
            with pytest.raises(ValueError, match="GPU"):
                call()
    with pytest.raises(ValueError, match="GPU"):
        ls.ls_vocab_logprob_fwd(vd, h, w, slots, n(), n(), ws)
    with pytest.raises(ValueError, match="GPU"):
        ls.ls_vocab_logprob_bwd(vd, h, w, slots, n(), n(), h.clone(), w.clone(), ws)
