"""Refusals of the entry points of a rollout with drafted tokens, before any launch (no GPU)."""
import ctypes

import pytest
import torch

A = 1 << 24  # an aligned address that is never dereferenced
I32, I64, F32 = torch.int32, torch.int64, torch.float32


@pytest.fixture(scope="module")
def ls():
    from long_context_grpo_replay_gb300 import build

    build.build()
    import long_context_grpo_replay_gb300.binding as b

    b.lib()
    return b


def fields(cls, given, **kw):
    d = dict(given)
    d.update(kw)
    return cls(*(d[n] for n, _ in cls._fields_))


def book(ls, **kw):
    return fields(ls.PageBook, dict(page_size=16, n_seqs=4, pages_per_seq=8, pool_pages=32, refs=A, page_table=A, kv_len=A), **kw)


def verify(ls, **kw):
    return fields(ls.VerifyDesc, dict(dtype=1, vocab=100, batch=3, max_q=2, total_q=5, logits_stride=100, draft_stride=100,
                                      logit_scale=1.0), **kw)


def decode(ls, **kw):
    return fields(ls.GdnDecodeDesc, dict(dtype=1, heads=4, key_heads=2, dk=128, dv=128, batch=3, max_q=2, reserved=0, total_q=5,
                                         q_stride=1024, k_stride=1024, v_stride=1024, n_states=6), **kw)


def cache(ls, **kw):
    return fields(ls.KvCache, dict(format=ls.LS_CACHE_E4M3, hkv=4, head_dim=256, page_size=256, pool_pages=16, k=A, v=A, k_exp=A,
                                   v_exp=A), **kw)


@pytest.mark.parametrize("bad,status", [
    (dict(page_size=0), 1), (dict(n_seqs=0), 1), (dict(pages_per_seq=0), 1), (dict(pool_pages=0), 1), (dict(refs=None), 1),
    (dict(page_table=None), 1), (dict(kv_len=None), 1), (dict(kv_len=A + 4), 1), (dict(refs=A + 2), 1),
    (dict(page_size=1 << 20, pages_per_seq=1 << 20), 2), (dict(pool_pages=(1 << 29) + 1), 2)])
def test_bad_books(ls, bad, status):
    L, b, n = ls.lib(), ctypes.byref(book(ls, **bad)), ctypes.c_size_t(0)
    assert L.ls_pages_workspace_size(b, ctypes.byref(n)) == status
    assert L.ls_pages_advance(b, 1, A, A, A, 1, A, A, A, 1 << 30, None) == status
    assert L.ls_pages_release(b, 1, A, A, 1 << 30, None) == status
    assert L.ls_pages_fork(b, 1, A, A, A, A, 1 << 30, None) == status
    assert L.ls_pages_compact(b, A, A, A, A, 1 << 30, None) == status
    assert ls.ls_last_error()


def test_pages_calls(ls):
    L, b = ls.lib(), book(ls)
    need = ls.ls_pages_workspace_size(b)
    adv = lambda n=2, seqs=A, keep=A, qs=A, total=3, slots=A, copies=A, ws=A, nb=need: L.ls_pages_advance(  # noqa: E731
        ctypes.byref(b), n, seqs, keep, qs, total, slots, copies, ws, nb, None)
    assert adv(n=0, total=0) == 0 and adv(n=0, seqs=None, keep=None, qs=None, total=0, slots=None, copies=None) == 0
    assert adv(n=-1) == 1 and adv(n=5) == 1                  # a call names each sequence at most once
    assert adv(total=-1) == 1 and adv(total=1 << 31) == 2 and adv(total=(1 << 29) + 1) == 2
    assert adv(qs=None) == 1 and adv(slots=None) == 1 and adv(copies=None) == 1 and adv(n=0) == 1
    assert adv(seqs=A + 2) == 1 and adv(keep=A + 4) == 1 and adv(qs=A + 1) == 1 and adv(slots=A + 4) == 1 and adv(copies=A + 2) == 1
    assert adv(ws=None) == 1 and adv(ws=A + 64) == 1 and adv(nb=need - 1) == 3
    rel = lambda n=2, seqs=A, ws=A, nb=need: L.ls_pages_release(ctypes.byref(b), n, seqs, ws, nb, None)  # noqa: E731
    assert rel(n=0) == 0 and rel(n=5) == 1 and rel(seqs=A + 2) == 1 and rel(nb=need - 1) == 3 and rel(ws=None) == 1
    fork = lambda n=2, src=A, dst=A, lens=A, nb=need: L.ls_pages_fork(ctypes.byref(b), n, src, dst, lens, A, nb, None)  # noqa: E731
    assert fork(n=0, src=None, dst=None) == 0 and fork(n=-1) == 1 and fork(n=5) == 1 and fork(src=None) == 1 and fork(dst=None) == 1
    assert fork(lens=A + 4) == 1 and fork(nb=need - 1) == 3
    comp = lambda t=A, r=A, c=A, nb=need: L.ls_pages_compact(ctypes.byref(b), t, r, c, A, nb, None)  # noqa: E731
    assert comp(t=None) == 1 and comp(r=None) == 1 and comp(c=None) == 1 and comp(c=A + 2) == 1 and comp(nb=need - 1) == 3
    c = cache(ls)
    cp = lambda c=c, copies=A, n=3, ws=None, nb=0: L.ls_cache_copy_pages(ctypes.byref(c), copies, n, ws, nb, None)  # noqa: E731
    assert cp(n=0, copies=None) == 0 and cp(n=-1) == 1 and cp(n=1 << 31) == 2 and cp(copies=None) == 1 and cp(copies=A + 2) == 1
    assert cp(ws=A, nb=16) == 3 and cp(cache(ls, head_dim=96)) == 2 and cp(cache(ls, k=None)) == 1
    assert L.ls_pages_advance(None, 1, A, A, A, 1, A, A, A, 1 << 30, None) == 1
    assert ls.ls_status_string(7) == "LS_ERR_OUT_OF_PAGES"


def test_results_of_the_pages_over_lists_and_book(ls):
    """What is read while other blocks write, and the results among each other.  (Calls that are right are made by the GPU's
    tests: nothing stops them before the launch.)"""
    L = ls.lib()
    at = lambda i: A + (i << 40)  # noqa: E731
    size = dict(refs=128, page_table=128, kv_len=32, seqs=12, keep=24, q_start=16, slots=56, copies=36, src=12, dst=12, lens=24,
                table_out=128, refs_out=128, moves=16 * 12)
    need = ls.ls_pages_workspace_size(book(ls))

    def call(kind, **kw):
        d = {n: at(i) for i, n in enumerate(size)} | kw
        bk = ctypes.byref(book(ls, refs=d["refs"], page_table=d["page_table"], kv_len=d["kv_len"]))
        if kind == "advance":
            st = L.ls_pages_advance(bk, 3, d["seqs"], d["keep"], d["q_start"], 7, d["slots"], d["copies"], at(20), need, None)
        elif kind == "release":
            st = L.ls_pages_release(bk, 3, d["seqs"], at(20), need, None)
        elif kind == "fork":
            st = L.ls_pages_fork(bk, 3, d["src"], d["dst"], d["lens"], at(20), need, None)
        else:
            st = L.ls_pages_compact(bk, d["table_out"], d["refs_out"], d["moves"], at(20), need, None)
        assert st == 1 and b"overlap" in L.ls_last_error(), (kind, kw)

    book_of = ("refs", "page_table", "kv_len")
    pairs = dict(
        advance=[(a, x) for a in ("slots", "copies") + book_of for x in ("seqs", "q_start", "keep") if (a, x) != ("kv_len", "keep")] +
                [(a, x) for a in ("slots", "copies") for x in book_of] + [("slots", "copies")],
        release=[(a, "seqs") for a in book_of],
        fork=[(a, x) for a in book_of for x in ("src", "dst")] + [("refs", "lens"), ("page_table", "lens")],
        compact=[("refs_out", x) for x in ("page_table", "kv_len", "table_out")] + [("table_out", x) for x in ("refs", "kv_len")] +
                [("moves", x) for x in book_of + ("table_out", "refs_out")])
    for kind, which in pairs.items():
        for a, x in which:
            for off in (0, 8 * ((size[x] - 1) // 8), -8 * ((size[a] - 1) // 8)):
                call(kind, **{a: 2 * A + off, x: 2 * A})
    call("advance", kv_len=2 * A, keep=2 * A + 8)            # a part of it
    call("fork", kv_len=2 * A, lens=2 * A + 8)
    call("compact", refs=2 * A, refs_out=2 * A + 4)
    call("compact", page_table=2 * A, table_out=2 * A - 4)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 30) + 1, logits_stride=1 << 31), 2), (dict(batch=-1), 1),
    (dict(batch=70000, max_q=1), 2), (dict(total_q=-1), 1), (dict(total_q=7), 1), (dict(max_q=6), 1), (dict(max_q=1), 1),
    (dict(logits_stride=99), 1), (dict(logit_scale=0.0), 1), (dict(logit_scale=float("nan")), 1), (dict(logit_scale=-1.0), 1),
    (dict(logit_scale=float("inf")), 1), (dict(logit_scale=3e38), 2), (dict(logit_scale=1e-31), 2), (dict(total_q=1 << 30, max_q=1 << 30, vocab=1 << 20, logits_stride=1 << 20), 2)])
def test_bad_verify_descs(ls, bad, status):
    n = ctypes.c_size_t(0)
    assert ls.lib().ls_draft_verify_workspace_size(ctypes.byref(verify(ls, **bad)), ctypes.byref(n)) == status


def test_vocabularies(ls):
    n = ctypes.c_size_t(0)
    for vocab, status in ((1 << 24, 0), ((1 << 24) + 1, 2), (1 << 30, 2)):
        d = verify(ls, vocab=vocab, logits_stride=vocab, draft_stride=vocab)
        assert ls.lib().ls_draft_verify_workspace_size(ctypes.byref(d), ctypes.byref(n)) == status


def test_verify_calls(ls):
    L = ls.lib()
    need = ls.ls_draft_verify_workspace_size(verify(ls))
    names = ("logits", "probs", "tokens", "q_start", "u", "u_next", "kv_len", "count", "out", "logp", "keep")

    def call(desc=None, ws=A, nb=need, **kw):
        d = {n: A + (i << 40) for i, n in enumerate(names)} | kw  # apart
        return L.ls_draft_verify(ctypes.byref(desc or verify(ls)), *(d[n] for n in names), ws, nb, None)

    assert call(verify(ls, batch=0, total_q=0, max_q=0), ws=None, **dict.fromkeys(names)) == 0
    for name in ("logits", "tokens", "q_start", "u", "u_next", "count", "out", "kv_len"):
        assert call(**{name: None}) == 1, name
    for name, off in (("logits", 1), ("probs", 2), ("tokens", 4), ("q_start", 2), ("u", 1), ("keep", 4), ("out", 4)):
        assert call(**{name: A + off}) == 1, name
    for name, other in (("out", "tokens"), ("logp", "u")):   # n tokens of 8 and of 4 bytes from either side
        each = 8 if name == "out" else 4
        for off in (0, 4 * each, -4 * each):
            assert call(**{name: 2 * A + off, other: 2 * A}) == 1, name
            assert b"overlap" in L.ls_last_error()
    assert call(verify(ls, draft_stride=99)) == 1 and call(nb=need - 1) == 3 and call(ws=None) == 1 and call(ws=A + 16) == 1


def test_results_of_a_verification_over_its_inputs(ls):
    """Blocks write results while others still read: every result against every small input, touching ends aside."""
    L = ls.lib()
    desc = verify(ls)                                        # 5 rows of 3 sequences
    need = ls.ls_draft_verify_workspace_size(desc)
    names = ("logits", "probs", "tokens", "q_start", "u", "u_next", "kv_len", "count", "out", "logp", "keep")
    size = dict(tokens=40, q_start=16, u=20, u_next=12, kv_len=24, count=12, out=40, logp=20, keep=24)

    def call(**kw):
        d = {n: A + (i << 40) for i, n in enumerate(names)} | kw  # apart
        return L.ls_draft_verify(ctypes.byref(desc), *(d[n] for n in names), None, need, None)

    assert call() == 1 and b"overlap" not in L.ls_last_error()  # ws is NULL: nothing is launched here
    for result in ("count", "out", "logp", "keep"):
        for given in ("tokens", "q_start", "u", "u_next", "kv_len"):
            for off, bad in ((0, (result, given) != ("keep", "kv_len")), (8 * ((size[given] - 1) // 8), True), (-8 * ((size[result] - 1) // 8), True),
                             (8 * (size[given] // 8 + 1), False), (-8 * (size[result] // 8 + 1), False)):
                assert call(**{result: 2 * A + off, given: 2 * A}) == 1
                assert (b"overlap" in L.ls_last_error()) == bad, (result, given, off)
    assert call(keep=None, kv_len=2 * A, out=2 * A) == 1 and b"overlap" not in L.ls_last_error()  # kv_len is not read then


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(heads=0), 1), (dict(key_heads=3), 1), (dict(key_heads=0), 1), (dict(dk=64), 2), (dict(dv=256), 2),
    (dict(heads=131072), 2), (dict(batch=-1), 1), (dict(batch=65536), 2), (dict(total_q=9), 1), (dict(max_q=6), 1), (dict(n_states=0), 1),
    (dict(q_stride=255), 1), (dict(q_stride=260), 1), (dict(k_stride=248), 1), (dict(v_stride=504), 1)])
def test_bad_decode_descs(ls, bad, status):
    args = [A] * 11 + [A, 256, None]
    assert ls.lib().ls_gdn_decode(ctypes.byref(decode(ls, **bad)), *args) == status


def test_decode_calls(ls):
    L = ls.lib()
    names = ("states", "q", "k", "v", "g", "beta", "q_start", "n_use", "state_in", "state_out", "o")

    def call(desc=None, ws=None, nb=0, **kw):
        d = {n: A + (i << 40) for i, n in enumerate(names)} | kw  # apart
        return L.ls_gdn_decode(ctypes.byref(desc or decode(ls)), *(d[n] for n in names), ws, nb, None)

    assert call(decode(ls, batch=0, total_q=0, max_q=0), **dict.fromkeys(names)) == 0
    assert call(o=None, state_out=None) == 0                # nothing asked for
    for name in ("states", "q", "k", "v", "g", "beta", "q_start", "state_in"):
        assert call(**{name: None}) == 1, name
    for name, off in (("states", 8), ("q", 8), ("o", 2), ("g", 2), ("state_out", 2), ("n_use", 1)):
        assert call(**{name: A + off}) == 1, name
    for name in ("q", "k", "v"):
        for off in (0, 1024, -1024):
            assert call(o=2 * A + off, **{name: 2 * A}) == 1, name
            assert b"overlap" in L.ls_last_error()
    assert call(ws=A, nb=255) == 3 and call(ws=A + 8, nb=256) == 1


def test_results_of_a_recurrent_step_over_its_inputs(ls):
    """Blocks write rows of o and of the states while others still read."""
    L = ls.lib()
    names = ("states", "q", "k", "v", "g", "beta", "q_start", "n_use", "state_in", "state_out", "o")
    size = dict(states=6 * 4 * 128 * 128 * 4, q=2 * (4 * 1024 + 256), k=2 * (4 * 1024 + 256), v=2 * (4 * 1024 + 512), g=80, beta=80, q_start=16,
                n_use=12, state_in=12, state_out=12, o=5 * 4 * 128 * 2)

    def call(**kw):
        d = {n: A + (i << 40) for i, n in enumerate(names)} | kw  # apart
        return L.ls_gdn_decode(ctypes.byref(decode(ls)), *(d[n] for n in names), A + 8, 256, None)

    assert call() == 1 and b"overlap" not in L.ls_last_error()  # ws is not aligned: nothing is launched here
    for result in ("o", "states"):
        for other in names:
            if other == result:
                continue
            for off, bad in ((0, True), (16 * ((size[other] - 1) // 16), True), (-16 * ((size[result] - 1) // 16), True),
                             (16 * (size[other] // 16 + 1), False), (-16 * (size[result] // 16 + 1), False)):
                assert call(**{result: 2 * A + off, other: 2 * A}) == 1
                assert (b"overlap" in L.ls_last_error()) == bad, (result, other, off)


def test_binding_checks_tensors(ls):
    z = lambda *s, dt=I32: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError):
        ls.page_book(z(4, dt=I64), z(2, 3), z(2, dt=I64), 16)
    with pytest.raises(ValueError):
        ls.page_book(z(4), z(3, 3), z(2, dt=I64), 16)
    with pytest.raises(ValueError):
        ls.page_book(z(4), z(3, 2).T, z(2, dt=I64), 16)
    b = ls.page_book(z(4), z(2, 3), z(2, dt=I64), 16)
    ws = z(4096, dt=torch.uint8)
    good = dict(q_start=z(3), slots=z(2, dt=I64), copies=z(2, 3))
    for bad in (dict(q_start=z(3, dt=I64)), dict(slots=z(2)), dict(copies=z(2, 2)), dict(copies=z(3, 3)), dict(seqs=z(3)),
                dict(keep=z(2)), dict(q_start=None), dict(slots=None), dict(copies=None)):
        kw = good | bad
        with pytest.raises((TypeError, ValueError)):
            ls.ls_pages_advance(b, kw.pop("q_start"), kw.pop("slots"), kw.pop("copies"), ws, **kw)
    logits, toks = z(5, 100, dt=F32), z(5, dt=I64)
    with pytest.raises(TypeError):
        ls.verify_desc(logits, 3, 2, draft_probs=logits.double())
    with pytest.raises(ValueError):
        ls.verify_desc(logits, 3, 2, draft_probs=logits[:, :50])
    with pytest.raises(ValueError):
        ls.verify_desc(logits.T, 3, 2)
    d = ls.verify_desc(logits, 3, 2)
    args = [d, logits, toks, z(4), z(5, dt=F32), z(3, dt=F32), z(3), toks.clone(), z(5, dt=F32), ws]
    for at, bad in ((1, logits[:4]), (1, logits.bfloat16()), (2, z(5)), (3, z(3)), (4, toks), (5, z(5, dt=F32)), (6, z(3, dt=I64)),
                    (7, z(4, dt=I64)), (8, z(5, dt=torch.bfloat16))):
        with pytest.raises((TypeError, ValueError)) as e:
            ls.ls_draft_verify(*(args[:at] + [bad] + args[at + 1:]))
        assert "GPU" not in str(e.value)
    with pytest.raises(ValueError, match="keep"):
        ls.ls_draft_verify(*args, keep=z(3, dt=I64))
    changed = ls.verify_desc(logits, 3, 2)
    changed.total_q = 4                                     # by hand: the tensors are no longer the desc's
    with pytest.raises(ValueError, match="desc"):
        ls.ls_draft_verify(changed, *args[1:])
    with pytest.raises(ValueError, match="draft_probs"):
        ls.ls_draft_verify(*args, draft_probs=logits[:, :99])
    q, v, s = z(5, 2, 128, dt=F32), z(5, 4, 128, dt=F32), z(6, 4, 128, 128, dt=F32)
    with pytest.raises(ValueError):
        ls.gdn_decode_desc(q, q[:4], v, s, 3, 2)
    with pytest.raises(ValueError):
        ls.gdn_decode_desc(q, q, v, s[:, :3], 3, 2)
    with pytest.raises(TypeError):
        ls.gdn_decode_desc(q, q, v, s.bfloat16(), 3, 2)
    d = ls.gdn_decode_desc(q, q, v, s, 3, 2)
    args = [d, s, q, q, v, z(5, 4, dt=F32), z(5, 4, dt=F32), z(4), z(3), z(3), v.clone()]
    changed = ls.gdn_decode_desc(q, q, v, s, 3, 2)
    changed.heads = 2
    with pytest.raises(ValueError, match="desc"):
        ls.ls_gdn_decode(changed, *args[1:])
    for at, bad in ((1, s[:5]), (2, q[:4]), (2, q.bfloat16()), (3, z(5, 4, 128, dt=F32)[:, ::2]), (4, v[:, :3]), (5, z(5, 3, dt=F32)),
                    (6, z(5, 4)), (7, z(3)), (8, z(3, dt=I64)), (9, z(4)), (10, v.bfloat16())):
        with pytest.raises((TypeError, ValueError)) as e:
            ls.ls_gdn_decode(*(args[:at] + [bad] + args[at + 1:]))
        assert "GPU" not in str(e.value)


def test_binding_refuses_host_tensors(ls):
    """Calls that are right but for tensors in host memory raise before anything is launched."""
    z = lambda *s, dt=I32: torch.zeros(*s, dtype=dt)  # noqa: E731
    ws = z(1 << 16, dt=torch.uint8)
    b = ls.page_book(z(4), z(2, 3), z(2, dt=I64), 16)
    k = z(4, 1, 16, 64, dt=torch.bfloat16)
    logits, toks = z(5, 100, dt=F32), z(5, dt=I64)
    q, v, s = z(5, 2, 128, dt=F32), z(5, 4, 128, dt=F32), z(6, 4, 128, 128, dt=F32)
    bare = ls.PageBook(*(getattr(b, n) for n, _ in ls.PageBook._fields_))  # the caller's word for its addresses
    calls = [lambda: ls.ls_cache_copy_pages(ls.kv_cache_from(k, k.clone()), z(2, 3)),
             lambda: ls.ls_draft_verify(ls.verify_desc(logits, 3, 2), logits, toks, z(4), z(5, dt=F32), z(3, dt=F32), z(3), toks.clone(),
                                        z(5, dt=F32), ws),
             lambda: ls.ls_gdn_decode(ls.gdn_decode_desc(q, q, v, s, 3, 2), s, q, q, v, z(5, 4, dt=F32), z(5, 4, dt=F32), z(4), z(3), z(3),
                                      v.clone())]
    for x in (b, bare):
        calls += [lambda x=x: ls.ls_pages_advance(x, z(3), z(2, dt=I64), z(2, 3), ws), lambda x=x: ls.ls_pages_release(x, ws),
                  lambda x=x: ls.ls_pages_advance(x, None, None, None, ws, keep=z(2, dt=I64)),
                  lambda x=x: ls.ls_pages_fork(x, z(1), z(1), ws), lambda x=x: ls.ls_pages_compact(x, z(2, 3), z(4), z(2, 3), ws)]
    for call in calls:
        with pytest.raises(ValueError, match="GPU"):
            call()
