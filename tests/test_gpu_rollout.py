"""GPU parity of the quantised cache, cached attention and vocabulary
log-probabilities with their float64 definitions.

Tolerances, element by element.  u is half a step of a type relative to the
value (float32 2^-24, f16 2^-11, bf16 2^-8).  A product of d terms summed in
float32 is off by at most d 2^-23 sum|q||k| (2^-23 covers sums that cut instead
of rounding); a score is off by dx of that, times the scale; an exponential by
2^-21 and its argument's rounding, |x| 2^-22.  An output o = sum p v is then off
by (2 dx + u_P + n 2^-23 + 2^-20) sum p|v| + u_out |o|, where u_P is the rounding of
the weights to their product's operand type: bf16 on a bf16 cache, f16 on an
e4m3 cache (with f16 queries, 2^-22 of the row's largest element more per term),
none in float32."""
import math

import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from oracle import rollout as ref

pytestmark = pytest.mark.gpu
F64 = torch.float64
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    return torch.device("cuda:0")


def make_cache(pages, hkv, page, d, fmt, dev, poison=True):
    shape = (pages, hkv, page, d)
    fill = math.nan if poison else 0.0
    k = torch.full(shape, fill, dtype=BF, device=dev).to(fmt)
    v = k.clone()
    if fmt != E4:
        return dict(k=k, v=v, k_exp=None, v_exp=None)
    return dict(k=k, v=v, k_exp=torch.zeros(shape[:3], dtype=torch.int8, device=dev),
                v_exp=torch.zeros(shape[:3], dtype=torch.int8, device=dev))


def cache_of(c):
    return ls.kv_cache_from(c["k"], c["v"], c["k_exp"], c["v_exp"])


def status_ws(dev, n=256):
    return torch.zeros(n, dtype=torch.uint8, device=dev)


def rows_of(pool, slots):
    """[n, Hkv, ...] rows of a pool [pages, Hkv, page, ...] by slot (on the host)."""
    page = pool.shape[2]
    return torch.stack([pool[int(s) // page, :, int(s) % page] for s in slots]) if len(slots) else pool[:0, :, 0]


# ------------------------------------------------------------------ cache
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("src", [BF, F32])
@pytest.mark.parametrize("fmt", [E4, BF, F32])
def test_write_and_read(d, src, fmt, dev):
    n, hkv, page, pages = 37, 3, 5, 11
    g = torch.Generator().manual_seed(d)
    wide = torch.randn(n, 2 * hkv * d + 24, generator=g)
    wide *= torch.exp2(torch.randint(-130, 100, (n, 1), generator=g).float())
    wide[3] = 0
    wide[4, :d] = 448 * 2.0 ** -20
    wide[5, 0], wide[5, d] = 449.0, -448.5
    if fmt == E4:
        wide[6, 1], wide[7, 2] = math.inf, math.nan
        wide[8, :d] = 2.0 ** -133  # below the least exponent's normal codes
    wide = wide.to(src)
    k, v = (wide[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[9], slots[10] = -1, -7
    c = make_cache(pages, hkv, page, d, fmt, dev)
    before = {x: t.clone() for x, t in c.items() if t is not None}
    w = wide.to(dev)
    kd, vd = (w[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    ws = status_ws(dev)
    ls.ls_cache_write(cache_of(c), kd, vd, slots.to(dev), ws)
    ls.ls_read_device_status(ws)
    there = slots >= 0
    for name, x in (("k", k), ("v", v)):
        got = rows_of(c[name].view(torch.uint8).reshape(pages, hkv, page, -1).cpu(), slots[there])
        if fmt == E4:
            codes, exps = ref.quantise(x[there])
            assert torch.equal(got, codes), name
            assert torch.equal(rows_of(c[name + "_exp"].cpu(), slots[there]), exps), name
        else:
            assert torch.equal(got, x[there].to(fmt).contiguous().view(torch.uint8).reshape(got.shape)), name
        # nothing else changed
        mask = torch.ones(pages * page, dtype=torch.bool)
        mask[slots[there]] = False
        rest = mask.reshape(pages, 1, page).expand(pages, hkv, page)
        assert torch.equal(c[name].view(torch.uint8).reshape(pages, hkv, page, -1).cpu()[rest],
                           before[name].view(torch.uint8).reshape(pages, hkv, page, -1).cpu()[rest])
    for dst in (BF, F32):
        ko = torch.full((n, hkv, d), 7.0, dtype=dst, device=dev)
        vo = ko.clone()
        ls.ls_cache_read(cache_of(c), slots.to(dev), ko, vo, ws)
        ls.ls_read_device_status(ws)
        for got, x in ((ko, k), (vo, v)):
            if fmt == E4:
                want = ref.dequantise(*ref.quantise(x))
            else:
                want = x.to(fmt).to(F64)
            want[~there] = 0
            # exact where the type holds the value
            want = want.to(F32).to(dst)
            assert torch.equal(got.cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))
            assert torch.equal(got.cpu().isnan(), want.isnan())


def test_write_nothing_and_bad_slots(dev):
    c = make_cache(4, 2, 8, 64, E4, dev)
    before = c["k"].view(torch.uint8).clone()
    x = torch.randn(3, 2, 64, device=dev).to(BF)
    ls.ls_cache_write(cache_of(c), x[:0], x[:0], torch.zeros(0, dtype=torch.int64, device=dev))
    ws = status_ws(dev)
    slots = torch.tensor([32, -1, 1 << 40], device=dev)
    ls.ls_cache_write(cache_of(c), x, x, slots, ws)
    with pytest.raises(ls.LsError) as e:
        ls.ls_read_device_status(ws)
    assert e.value.status == 5
    ls.ls_read_device_status(ws)  # cleared
    assert torch.equal(before, c["k"].view(torch.uint8))
    out = torch.ones_like(x)
    ls.ls_cache_read(cache_of(c), slots, out, out.clone(), ws)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    assert (out == 0).all()
    ls.ls_cache_write(cache_of(c), x, x, slots)  # without a workspace: skipped, not reported
    torch.cuda.synchronize()


# ------------------------------------------------------------------ attention
class Case:
    """Sequences' keys quantised (or not) by the definition, in scattered pages of a poisoned pool."""

    def __init__(self, q_lens, kv_lens, dev, hq=6, hkv=2, d=64, page=16, fmt=E4, qd=BF, wide=1.0, seed=0, pad=0,
                 q_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.fmt, self.d, self.hq, self.dev = q_lens, kv_lens, fmt, d, hq, dev
        t = sum(q_lens)
        wide_q = torch.randn(t, hq * d + pad, generator=g).mul(q_scale).to(qd)
        self.q_host = wide_q[:, :hq * d].unflatten(1, (hq, d))
        self.q = wide_q.to(dev)[:, :hq * d].unflatten(1, (hq, d))
        used = [-(-m // page) for m in kv_lens]
        self.pages = sum(used) + 2
        self.c = make_cache(self.pages, hkv, page, d, fmt, dev)
        host = {n: (x.view(torch.uint8).cpu() if x is not None and x.dtype == E4 else x.cpu() if x is not None else None)
                for n, x in self.c.items()}
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        width = max(1, max(used)) + 1
        self.table = torch.full((len(kv_lens), width), -5, dtype=torch.int32)  # never read past a length
        self.keys, self.values = [], []
        at = 0
        for b, m in enumerate(kv_lens):
            self.table[b, :used[b]] = order[at:at + used[b]]
            sides = []
            for name in ("k", "v"):
                x = torch.randn(m, hkv, d, generator=g) * wide
                x *= torch.exp2(torch.randint(-2, 3, (m, 1, 1), generator=g).float())
                if fmt == E4:
                    codes, exps = ref.quantise(x)
                    sides.append(ref.dequantise(codes, exps))
                else:
                    codes = x.to(fmt)
                    exps = None
                    sides.append(codes.to(F64))
                for j in range(m):
                    p, r = int(self.table[b, j // page]), j % page
                    host[name][p, :, r] = codes[j]
                    if exps is not None:
                        host[name + "_exp"][p, :, r] = exps[j]
            self.keys.append(sides[0])
            self.values.append(sides[1])
            at += used[b]
        for n, x in host.items():
            if x is not None:
                self.c[n].view(x.dtype).copy_(x)
        self.scale = d ** -0.5

    def q_start(self):
        return [sum(self.q_lens[:i]) for i in range(len(self.q_lens) + 1)]

    def run(self, causal=True, max_kv=None, o_dtype=None, table=None, kv_len=None, max_q=None, stream=None, ws=None):
        dev = self.dev
        o = torch.full(self.q.shape, 9.0, dtype=o_dtype or self.q.dtype, device=dev)
        lse = torch.full(self.q.shape[:2], 9.0, device=dev)
        desc = ls.cached_attn_desc(self.q, o, len(self.kv_lens), max(self.q_lens) if max_q is None else max_q,
                                   max(self.kv_lens) if max_kv is None else max_kv, causal, self.scale)
        cache = cache_of(self.c)
        if ws is None:
            ws = torch.full((ls.ls_cached_attn_workspace_size(desc, cache),), 0xA5, dtype=torch.uint8, device=dev)
            ws[:256] = 0
        qs = torch.tensor(self.q_start(), dtype=torch.int32, device=dev)
        kv = torch.tensor(kv_len or self.kv_lens, dtype=torch.int64, device=dev)
        pt = (self.table if table is None else table).to(dev)
        self.args = (desc, cache, self.q, qs, kv, pt, o, lse, ws)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        ls.ls_cached_attn(*self.args, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return o, lse, ws

    def check(self, o, lse, causal=True, key_ok=None, kv_len=None):
        kv = kv_len or self.kv_lens
        keys = [k[:m] for k, m in zip(self.keys, kv)]
        values = [v[:m] for v, m in zip(self.values, kv)]
        wo, wl, a, sx = ref.cached_attention(self.q_host, keys, values, self.q_start(), kv, causal, self.scale, key_ok)
        n = max(kv)
        dx = (self.d * 2.0 ** -23 + 2.0 ** -20) * sx
        u_p = 0.0
        if self.q.dtype == BF:
            u_p = 2.0 ** -11 if self.fmt == E4 else 2.0 ** -8
            if self.fmt == E4:  # f16 queries
                top = self.q_host.to(F64).abs().amax(-1)
                big = max(float(k.abs().sum(-1).max()) if k.numel() else 0.0 for k in keys)
                dx = dx + 2.0 ** -22 * top * big * self.scale
        u_o = 2.0 ** -8 if o.dtype == BF else 2.0 ** -24
        tol = (2 * dx + u_p + n * 2.0 ** -23 + 2.0 ** -20)[..., None] * a + u_o * wo.abs() + 1e-30
        err = (o.cpu().to(F64) - wo).abs()
        assert (err <= tol).all(), f"o off by {float((err / tol).max())} of the tolerance"
        some = wl > -math.inf
        assert (lse.cpu()[~some] == -math.inf).all() and (o.cpu()[~some] == 0).all()
        tol = dx + n * 2.0 ** -23 + 2.0 ** -20 + wl.abs() * 2.0 ** -21
        err = (lse.cpu().to(F64) - wl).abs()[some]
        assert (err <= tol[some]).all(), f"lse off by {float((err / tol[some]).max())} of the tolerance"


FORMS = [(E4, BF), (BF, BF), (F32, F32), (E4, F32), (BF, F32), (F32, BF)]


@pytest.mark.parametrize("fmt,qd", FORMS)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_ragged(fmt, qd, d, dev):
    c = Case([1, 0, 3, 5, 2, 1], [300, 40, 3, 2, 0, 1], dev, d=d, page=16, fmt=fmt, qd=qd, seed=d)
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    c.check(o, lse)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (24, 4), (12, 1), (8, 8), (32, 8), (20, 1)])
@pytest.mark.parametrize("fmt", [E4, BF])
def test_attention_heads(hq, hkv, fmt, dev):
    c = Case([1, 4, 2], [129, 64, 70], dev, hq=hq, hkv=hkv, d=128, page=16, fmt=fmt, seed=hq)
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    c.check(o, lse)


@pytest.mark.parametrize("page", [1, 3, 48, 64, 256])
@pytest.mark.parametrize("fmt", [E4, BF])
def test_attention_pages(page, fmt, dev):
    c = Case([2, 1], [257, 33], dev, hq=6, hkv=1, d=256, page=page, fmt=fmt, seed=page)
    for causal in (True, False):
        o, lse, ws = c.run(causal)
        ls.ls_read_device_status(ws)
        c.check(o, lse, causal)


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 33, 127, 128, 129, 200])
def test_attention_chunk_lengths(fmt, qd, n, dev):
    c = Case([n], [n + 77], dev, hq=6, hkv=1, d=256, page=64, fmt=fmt, qd=qd, seed=n, pad=40)
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    c.check(o, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", [E4, BF])
def test_attention_chunk_other_heads(d, fmt, dev):
    c = Case([150, 9, 64], [190, 700, 64], dev, hq=8, hkv=2, d=d, page=48, fmt=fmt, seed=d)
    for causal in (True, False):
        o, lse, ws = c.run(causal)
        ls.ls_read_device_status(ws)
        c.check(o, lse, causal)


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_wide_logits(fmt, n, dev):
    """Scores of size 60: few keys matter, and a missing key or tile shows."""
    c = Case([n], [900], dev, hq=6, hkv=1, d=256, page=256, fmt=fmt, seed=5, q_scale=40.0)
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    c.check(o, lse)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_scales_far_apart(n, dev):
    """Value rows whose scales span 2^-40 .. 2^40 of one another, and keys likewise with small queries."""
    c = Case([n], [400], dev, hq=6, hkv=1, d=256, page=16, seed=8)
    g = torch.Generator().manual_seed(1)
    shift = torch.randint(-40, 41, (400,), generator=g)
    for j in range(400):
        p, r = int(c.table[0, j // 16]), j % 16
        c.c["v_exp"][p, :, r] += int(shift[j])
    c.values[0] = c.values[0] * 2.0 ** shift.to(F64)[:, None, None]
    o, lse, ws = c.run()
    c.check(o, lse)
    small = Case([n], [400], dev, hq=6, hkv=1, d=256, page=16, seed=9, q_scale=2.0 ** -60)
    small.c["k_exp"] += 60
    small.keys[0] = small.keys[0] * 2.0 ** 60
    o, lse, ws = small.run()
    small.check(o, lse)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_one_key_above_many(n, dev):
    """One key whose weight is e^17 of the others': the others' sum still counts."""
    c = Case([n], [3000], dev, hq=6, hkv=1, d=256, page=256, seed=4, q_scale=0.0)
    q = torch.zeros_like(c.q_host)
    q[..., 0] = 16.0
    c.q_host = q
    c.q = q.to(dev)
    k = torch.zeros(3000, 1, 256, dtype=F64)
    k[7, 0, 0] = 17.0
    codes, exps = ref.quantise(k)
    for j in range(3000):
        p, r = int(c.table[0, j // 256]), j % 256
        if j % 256 == 0:
            m = min(256, 3000 - j)
            c.c["k"].view(torch.uint8)[p, :, :m] = codes[j:j + m].transpose(0, 1).to(dev)
            c.c["k_exp"][p, :, :m] = exps[j:j + m].transpose(0, 1).to(dev)
    c.keys[0] = ref.dequantise(codes, exps)
    o, lse, ws = c.run(False)
    c.check(o, lse, False)


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_split_and_float_parts(fmt, qd, n, dev):
    """A long cache is cut into parts; the number of parts (by max_kv) changes only rounding, and a
    float32 o is the unrounded result."""
    c = Case([n, n], [5000, 1200], dev, hq=6, hkv=1, d=256, page=256, fmt=fmt, qd=qd, seed=2)
    for max_kv in (5000, 0, 100000):
        o, lse, ws = c.run(max_kv=max_kv)
        ls.ls_read_device_status(ws)
        c.check(o, lse)
        of, lf, _ = c.run(max_kv=max_kv, o_dtype=F32)
        c.check(of, lf)
        assert torch.equal(of.to(o.dtype), o) and torch.equal(lf, lse)


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_not_finite(fmt, qd, n, dev):
    """A NaN query gives NaN rows, a NaN key or value row NaN to those that see it, and nothing else
    changes, but for the sequence's other rows where a bf16 or float32 value is NaN (its product with a weight of 0)."""
    c = Case([n, n], [700, 600], dev, hq=6, hkv=1, d=256, page=64, fmt=fmt, qd=qd, seed=3)
    o, lse, _ = c.run()
    q = c.q.clone()
    q[0, 1, 3] = math.nan
    c.q = q
    for side in ("k", "v"):
        # key 599 of the second sequence: only its last token sees it
        p, r = int(c.table[1, 599 // 64]), 599 % 64
        if fmt == E4:
            keep = c.c[side + "_exp"][p, 0, r].clone()
            c.c[side + "_exp"][p, 0, r] = -128
        else:
            keep = c.c[side][p, 0, r].clone()
            c.c[side][p, 0, r] = math.nan
        o2, lse2, ws = c.run()
        ls.ls_read_device_status(ws)
        assert o2[0, 1].isnan().all() and lse2[0, 1].isnan()
        assert o2[2 * n - 1].isnan().all()
        if side == "k":
            assert lse2[2 * n - 1].isnan().all()
        rest = torch.ones(o.shape[:2], dtype=torch.bool, device=dev)
        rest[0, 1] = False
        rest[2 * n - 1] = False
        if side == "v" and fmt != E4:
            rest[n:] = False  # an earlier row's weight of 0 times this NaN: the header leaves these open
        assert torch.equal(o2[rest], o[rest]) and torch.equal(lse2[rest], lse[rest])
        if fmt == E4:
            c.c[side + "_exp"][p, 0, r] = keep
        else:
            c.c[side][p, 0, r] = keep


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_bad_pages(fmt, qd, n, dev):
    """A page id outside the pool holds no keys and is reported; ids past a length are not looked at."""
    c = Case([n, n], [300, 130], dev, hq=6, hkv=1, d=256, page=64, fmt=fmt, qd=qd, seed=6)
    table = c.table.clone()
    table[0, 1], table[0, 3], table[1, :] = c.pages, -1, 1 << 30
    o, lse, ws = c.run(table=table)
    with pytest.raises(ls.LsError) as e:
        ls.ls_read_device_status(ws)
    assert e.value.status == 5
    ok = [torch.ones(300, dtype=torch.bool), torch.zeros(130, dtype=torch.bool)]
    ok[0][64:128] = False
    ok[0][192:256] = False
    c.check(o, lse, key_ok=ok)


def test_attention_lengths_out_of_range(dev):
    c = Case([1, 1], [100, 60], dev, hq=6, hkv=1, d=256, page=64, seed=7)
    o, lse, ws = c.run(kv_len=[-4, 60])
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    c.check(o, lse, kv_len=[0, 60])
    one = Case([1], [128], dev, hq=6, hkv=1, d=256, page=64, seed=7)
    one.table = one.table[:, :2]
    o, lse, ws = one.run(kv_len=[1 << 40])  # cut to the 128 keys that the table's row has pages for
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    one.check(o, lse)
    c3 = Case([3, 1], [100, 60], dev, hq=6, hkv=1, d=256, page=64, seed=7)
    o, lse, ws = c3.run(max_q=2)  # the first sequence has three tokens
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    assert (o[:3] == 9).all() and (lse[:3] == 9).all()


def test_attention_stream_and_graph(dev):
    c = Case([1, 2, 1], [700, 90, 33], dev, hq=24, hkv=4, d=256, page=64, seed=10)
    o, lse, ws = c.run(stream=torch.cuda.Stream())
    c.check(o, lse)
    args = c.args
    want, want_l = o.clone(), lse.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ls.ls_cached_attn(*args)
    args[6].zero_(), args[7].zero_()
    graph.replay()
    assert torch.equal(args[6], want) and torch.equal(args[7], want_l)
    # the lengths are read on the device: the same graph serves shorter caches
    args[4].copy_(torch.tensor([650, 80, 1]))
    graph.replay()
    torch.cuda.synchronize()
    c.check(args[6], args[7], kv_len=[650, 80, 1])


def test_attention_over_a_captured_prompt(dev):
    """Pages written by the prompt capture are a bf16 cache as they stand; its rows quantised are an
    e4m3 one; members decode together and the parts are merged with their own tokens'."""
    hq, hkv, d, page, n, members = 24, 4, 256, 64, 333, 3
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(n, hkv, d, generator=g).to(BF) for _ in range(2))
    pages = 8
    table = torch.randperm(pages, generator=g).to(torch.int32)[:6]
    c = make_cache(pages, hkv, page, d, BF, dev)
    desc = ls.desc_for(hq, hkv, d, page, BF)
    ls.ls_kv_page_write(desc, c["k"], c["v"], table.to(dev), 0, k.to(dev), v.to(dev))
    q = torch.randn(members, hq, d, generator=g).to(BF)
    own_k, own_v = (torch.randn(members, hkv, d, generator=g).to(BF) for _ in range(2))
    parts = torch.empty(2, members, hq, d, device=dev)
    lses = torch.empty(2, members, hq, device=dev)

    def call(cc, batch, kv, tab, i, causal):
        cd = ls.cached_attn_desc(q, parts[i], batch, members // batch, max(kv), causal)
        ch = cache_of(cc)
        ws = torch.zeros(ls.ls_cached_attn_workspace_size(cd, ch), dtype=torch.uint8, device=dev)
        starts = torch.arange(0, members + 1, members // batch, dtype=torch.int32, device=dev)
        ls.ls_cached_attn(cd, ch, q.to(dev), starts, torch.tensor(kv, device=dev), tab.to(dev), parts[i], lses[i], ws)
        ls.ls_read_device_status(ws)

    call(c, 1, [n], table[None], 0, False)
    own = make_cache(members, hkv, page, d, BF, dev)
    ls.ls_cache_write(cache_of(own), own_k.to(dev), own_v.to(dev), torch.arange(members, device=dev) * page)
    call(own, members, [1] * members, torch.arange(members, dtype=torch.int32)[:, None], 1, True)
    o = torch.empty(members, hq, d, dtype=BF, device=dev)
    lse = torch.empty(members, hq, device=dev)
    ls.ls_lse_merge(parts.view(2, members * hq, d), lses.view(2, -1), o.view(-1, d), lse.view(-1))
    want, wl, a, sx = ref.cached_attention(
        q, [torch.cat([k, own_k[i:i + 1]]).to(F64) for i in range(members)],
        [torch.cat([v, own_v[i:i + 1]]).to(F64) for i in range(members)], range(members + 1), [n + 1] * members, True, d ** -0.5)
    tol = (2.0 ** -8 + 4 * d * 2.0 ** -23 * float(sx.max()) + 2.0 ** -14) * a + 2.0 ** -8 * want.abs()
    assert ((o.cpu().to(F64) - want).abs() <= tol).all()
    assert ((lse.cpu().to(F64) - wl).abs() <= 2 * d * 2.0 ** -23 * float(sx.max()) + 1e-4).all()


def test_attention_past_32_bit_offsets(dev):
    """A pool of more than 2^32 bytes a side in bf16: rows at its far end."""
    hkv, d, page, pages = 4, 256, 256, 8300
    pools = [torch.empty((pages, hkv, page, d), dtype=BF, device=dev) for _ in range(2)]
    g = torch.Generator().manual_seed(0)
    n = 2 * page + 5
    k, v = (torch.randn(n, hkv, d, generator=g).to(BF) for _ in range(2))
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32)
    slots = torch.tensor([int(table[0, j // page]) * page + j % page for j in range(n)], device=dev)
    cache = ls.kv_cache_from(*pools)
    ls.ls_cache_write(cache, k.to(dev), v.to(dev), slots)
    ko, vo = torch.empty(n, hkv, d, dtype=BF, device=dev), torch.empty(n, hkv, d, dtype=BF, device=dev)
    ls.ls_cache_read(cache, slots, ko, vo)
    assert torch.equal(ko.cpu(), k) and torch.equal(vo.cpu(), v)
    for rows in (1, 30):
        q = torch.randn(rows, 24, d, generator=g).to(BF)
        o, lse = torch.empty(rows, 24, d, dtype=BF, device=dev), torch.empty(rows, 24, device=dev)
        desc = ls.cached_attn_desc(q, o, 1, rows, n)
        ws = torch.zeros(ls.ls_cached_attn_workspace_size(desc, cache), dtype=torch.uint8, device=dev)
        ls.ls_cached_attn(desc, cache, q.to(dev), torch.tensor([0, rows], dtype=torch.int32, device=dev),
                          torch.tensor([n], device=dev), table.to(dev), o, lse, ws)
        ls.ls_read_device_status(ws)
        want, wl, a, sx = ref.cached_attention(q, [k.to(F64)], [v.to(F64)], [0, rows], [n], True, d ** -0.5)
        tol = (2 * d * 2.0 ** -23 * sx + 2.0 ** -8 + n * 2.0 ** -23 + 2.0 ** -19)[..., None] * a + 2.0 ** -8 * want.abs()
        assert ((o.cpu().to(F64) - want).abs() <= tol).all()


# ------------------------------------------------------------------ vocabulary
def vocab_case(n, d, v, dtype, seed=0, h_pad=0, w_pad=0, shift=0):
    """h, w as views of wider rows; shift moves their first element off 16-byte alignment."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(n, d + h_pad, generator=g).to(dtype)[:, shift:shift + d] if h_pad else torch.randn(n, d, generator=g).to(dtype)
    w = torch.randn(v, d + w_pad, generator=g).mul(2 / math.sqrt(d)).to(dtype)
    w = w[:, shift:shift + d] if w_pad else w
    t = torch.randint(0, v, (n,), generator=g)
    if n > 2:
        t[1] = -100
        t[0], t[2] = 0, v - 1
    return h, w, t, torch.randn(n, generator=g)


def device_like(x, dev):
    """The same view on the device: strides and the offset of its first element."""
    base = torch.empty(0, dtype=x.dtype)
    base.set_(x.untyped_storage())
    y = base.to(dev)
    return y.as_strided(x.shape, x.stride(), x.storage_offset())


def run_vocab(h, w, t, dl, dev, scale=1.0, piece=0, need=("dh", "dw"), stream=None):
    hd, wd, td, gd = device_like(h, dev), device_like(w, dev), t.to(dev), dl.to(dev)
    desc = ls.vocab_desc(hd, wd, scale, -100, piece)
    ws = torch.full((ls.ls_vocab_logprob_workspace_size(desc, True),), 0xA5, dtype=torch.uint8, device=dev)
    ws[:256] = 0
    n = h.shape[0]
    logp, lse = torch.full((n,), 9.0, device=dev), torch.full((n,), 9.0, device=dev)
    dh = torch.full(h.shape, 9.0, dtype=h.dtype, device=dev) if "dh" in need else None
    dw = torch.full(w.shape, 9.0, dtype=w.dtype, device=dev) if "dw" in need else None
    ls.ls_vocab_logprob_fwd(desc, hd, wd, td, logp, lse, ws, stream=stream)
    ls.ls_vocab_logprob_bwd(desc, hd, wd, td, lse, gd, dh, dw, ws, stream=stream)
    return logp, lse, dh, dw, ws


def check_vocab(h, w, t, dl, scale, logp, lse, dh, dw):
    """Bounds: a logit is off by dx = hidden 2^-23 sum|h||w| |scale|, lse by that and V 2^-23 of a
    sum, D by |c| p (dx + dlse + 2^-20) + u_D |D| (bf16 operands), the products by their inner
    length times 2^-23, the gradients rounded once."""
    wp, wl, x, on, _ = ref.vocab_logprob(h, w, t, scale, -100)
    hh, ww = h.to(F64), w.to(F64)
    dx = (h.shape[1] * 2.0 ** -23 + 2.0 ** -22) * (hh.abs() @ ww.abs().T) * abs(scale)
    dlse = dx.amax(1) + w.shape[0] * 2.0 ** -23 + 2.0 ** -20 + 2.0 ** -21 * wl.abs()
    assert ((lse.cpu().to(F64) - wl).abs() <= dlse).all()
    assert ((logp.cpu().to(F64) - wp).abs() <= 2 * dlse + 2.0 ** -22 * wp.abs()).all()
    assert (logp.cpu()[~on] == 0).all()
    u = 2.0 ** -8 if h.dtype == BF else 2.0 ** -24
    rdh, rdw, slope, cp = ref.vocab_gradients(h, w, t, dl, scale, -100)
    ds = cp * (dx + dlse[:, None] + 2.0 ** -19 + 2.0 ** -21 * x.abs()) + u * slope.abs()
    if dh is not None:
        tol = ds @ ww.abs() + (w.shape[0] * 2.0 ** -23) * (slope.abs() @ ww.abs()) + u * rdh.abs() + 1e-30
        err = (dh.cpu().to(F64) - rdh).abs()
        assert (err <= tol).all(), float((err / tol).max())
        assert (dh.cpu()[~on] == 0).all()
    if dw is not None:
        tol = ds.T @ hh.abs() + (h.shape[0] * 2.0 ** -23) * (slope.abs().T @ hh.abs()) + u * rdw.abs() + 1e-30
        err = (dw.cpu().to(F64) - rdw).abs()
        assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d,v", [(1, 8, 1), (1, 64, 100), (3, 72, 257), (37, 64, 1000), (128, 128, 256),
                                   (129, 200, 513), (300, 264, 777), (130, 1032, 2049)])
def test_vocab(dtype, n, d, v, dev):
    h, w, t, dl = vocab_case(n, d, v, dtype, seed=n)
    got = run_vocab(h, w, t, dl, dev, 0.8)
    ls.ls_read_device_status(got[4])
    check_vocab(h, w, t, dl, 0.8, *got[:4])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,h_pad,w_pad,shift", [(64, 16, 40, 8), (64, 16, 40, 3), (63, 0, 0, 0), (65, 7, 1, 0), (64, 3, 5, 0),
                                                 (1, 0, 0, 0)])
def test_vocab_strides_and_alignment(dtype, d, h_pad, w_pad, shift, dev):
    h, w, t, dl = vocab_case(70, d, 300, dtype, seed=d, h_pad=h_pad, w_pad=w_pad, shift=shift)
    got = run_vocab(h, w, t, dl, dev)
    ls.ls_read_device_status(got[4])
    check_vocab(h, w, t, dl, 1.0, *got[:4])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("piece", [1, 100, 128, 300, 512, 5000])
def test_vocab_pieces(dtype, piece, dev):
    h, w, t, dl = vocab_case(130, 72, 1000, dtype, seed=piece)
    got = run_vocab(h, w, t, dl, dev, 1.5, piece)
    check_vocab(h, w, t, dl, 1.5, *got[:4])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_one_gradient_at_a_time(dtype, dev):
    h, w, t, dl = vocab_case(50, 64, 400, dtype)
    both = run_vocab(h, w, t, dl, dev)
    for need in (("dh",), ("dw",)):
        got = run_vocab(h, w, t, dl, dev, need=need)
        for a, b in zip(both[:4], got[:4]):
            assert b is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-1.0, 0.0, 30.0])
def test_vocab_scales(dtype, scale, dev):
    h, w, t, dl = vocab_case(40, 64, 300, dtype, seed=2)
    got = run_vocab(h, w, t, dl, dev, scale)
    check_vocab(h, w, t, dl, scale, *got[:4])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_targets(dtype, dev):
    """All rows ignored; a target out of range is ignored and reported."""
    h, w, t, dl = vocab_case(40, 64, 300, dtype)
    got = run_vocab(h, w, torch.full_like(t, -100), dl, dev)
    ls.ls_read_device_status(got[4])
    assert (got[0] == 0).all() and (got[2] == 0).all() and (got[3] == 0).all()
    bad = t.clone()
    bad[5], bad[6] = 300, -1
    got = run_vocab(h, w, bad, dl, dev)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(got[4])
    check_vocab(h, w, bad, dl, 1.0, *got[:4])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_ignored_rows_may_hold_anything(dtype, dev):
    h, w, t, dl = vocab_case(40, 64, 300, dtype)
    clean = run_vocab(h, w, t, dl, dev)
    h2, dl2 = h.clone(), dl.clone()
    h2[1], dl2[1] = math.nan, math.nan
    got = run_vocab(h2, w, t, dl2, dev)
    keep = torch.arange(40) != 1
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1][keep], clean[1][keep])
    assert torch.equal(got[2], clean[2])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_no_rows(dtype, dev):
    h, w, t, dl = vocab_case(0, 64, 300, dtype)
    _, _, _, dw, _ = run_vocab(h, w, t, dl, dev)
    assert (dw == 0).all()


def test_vocab_gradient_against_differences(dev):
    h, w, t, dl = vocab_case(20, 64, 200, F32, seed=4)
    _, _, dh, dw, _ = run_vocab(h, w, t, dl, dev, 1.2)

    def loss(hh, ww):
        logp = run_vocab(hh, ww, t, dl, dev, 1.2)[0]
        return float((logp.cpu().to(F64) * dl.to(F64)).sum())

    g = torch.Generator().manual_seed(9)
    for x, dx, f in ((h, dh, lambda z: loss(z, w)), (w, dw, lambda z: loss(h, z))):
        step = torch.randn(x.shape, generator=g)
        eps = 1e-2
        slope = (f(x + eps * step) - f(x - eps * step)) / (2 * eps)
        want = float((dx.cpu().to(F64) * step.to(F64)).sum())
        # the third derivative's share is eps^2; float32 losses of about 100 are off by 1e-5 / eps
        assert abs(slope - want) <= 2e-2 * abs(want) + 5e-2


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_stream_and_graph(dtype, dev):
    h, w, t, dl = vocab_case(140, 128, 600, dtype)
    want = run_vocab(h, w, t, dl, dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run_vocab(h, w, t, dl, dev)
    s.synchronize()
    for a, b in zip(want[:4], got[:4]):
        assert torch.equal(a, b)
    hd, wd, td, gd = h.to(dev), w.to(dev), t.to(dev), dl.to(dev)
    desc = ls.vocab_desc(hd, wd)
    ws = torch.zeros(ls.ls_vocab_logprob_workspace_size(desc, True), dtype=torch.uint8, device=dev)
    logp, lse, dh, dw = (torch.empty_like(x) for x in want[:4])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ls.ls_vocab_logprob_fwd(desc, hd, wd, td, logp, lse, ws)
        ls.ls_vocab_logprob_bwd(desc, hd, wd, td, lse, gd, dh, dw, ws)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want[:4], (logp, lse, dh, dw)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_vocab_many_rows(dtype, dev):
    """More rows than the forward takes at a time."""
    h, w, t, dl = vocab_case(65536 + 300, 8, 40, dtype)
    got = run_vocab(h, w, t, dl, dev)
    ls.ls_read_device_status(got[4])
    check_vocab(h, w, t, dl, 1.0, *got[:4])


@pytest.mark.parametrize("fmt", [E4, BF])
@pytest.mark.parametrize("q_lens,kv_lens", [([40, 3, 21], [700, 650, 90]), ([45], [3000]), ([22, 1, 2], [5, 0, 2000])])
def test_attention_pair_with_an_empty_second_half(fmt, q_lens, kv_lens, dev):
    """Calls planned for pairs of CTAs (more than 128 rows at most) in which a pair's second CTA has no
    rows of its own: sequences of up to 128 rows, and last tiles with that many left."""
    c = Case(q_lens, kv_lens, dev, hq=6, hkv=1, d=256, page=16, fmt=fmt, seed=len(q_lens))
    first = None
    for _ in range(5):
        o, lse, ws = c.run()
        ls.ls_read_device_status(ws)
        if first is None:
            c.check(o, lse)
            first = o, lse
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("n,d,v", [(300, 8, 777), (257, 512, 257), (40, 64, 90000)])
def test_vocab_repeats(n, d, v, dev):
    """Fewer blocks of the inner dimension than stages, more, and many tiles a pair of CTAs: every call ends with
    nothing on its way to a CTA that has left, and repeats itself bit for bit."""
    h, w, t, dl = vocab_case(n, d, v, BF, seed=d)
    first = run_vocab(h, w, t, dl, dev)
    check_vocab(h, w, t, dl, 1.0, *first[:4])
    for _ in range(10):
        got = run_vocab(h, w, t, dl, dev)
        ls.ls_read_device_status(got[4])
        for a, b in zip(first[:4], got[:4]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("n", [1, 40, 150])
def test_attention_parts_are_this_call_s(fmt, qd, n, dev):
    """Calls one after another in one workspace, with other queries each time and the parts' place overwritten in
    between: the joining kernel, which is launched before the parts are written, reads what this call wrote."""
    c = Case([n], [6000], dev, hq=6, hkv=1, d=256, page=256, fmt=fmt, qd=qd, seed=n)
    qs = [c.q, (c.q.float() * -0.5).to(qd).as_strided(c.q.shape, c.q.stride())]
    want = []
    for q in qs:
        c.q = q
        o, lse, ws = c.run(o_dtype=F32)
        want.append((o, lse))
    assert ws.numel() > 2 * (n * 6 * 256 * 4 + 512), "cut into parts"
    args, outs = c.args, []
    for i in range(40):
        ws[256:] = 0xFF  # NaN
        o, lse = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
        ls.ls_cached_attn(args[0], args[1], qs[i % 2], *args[3:6], o, lse, ws)
        outs.append((o, lse))
    ls.ls_read_device_status(ws)
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


@pytest.mark.parametrize("qd", [BF, F32])
@pytest.mark.parametrize("n", [2, 12, 40])
def test_attention_nan_e4m3_rows_reach_only_their_readers(qd, n, dev):
    """An e4m3 row marked NaN (key or value) makes the rows that see it NaN and changes no other."""
    c = Case([n, n], [700, 600], dev, hq=6, hkv=1, d=256, page=64, fmt=E4, qd=qd, seed=3)
    o, lse, _ = c.run()
    p, r = int(c.table[1, 599 // 64]), 599 % 64  # only the second sequence's last token sees it
    for side in ("k", "v"):
        keep = c.c[side + "_exp"][p, 0, r].clone()
        codes = c.c[side].view(torch.uint8)[p, 0, r].clone()
        c.c[side + "_exp"][p, 0, r] = -128
        c.c[side].view(torch.uint8)[p, 0, r] = 0
        o2, lse2, ws = c.run()
        ls.ls_read_device_status(ws)
        assert o2[-1].isnan().all() and lse2[-1].isnan().all()
        assert torch.equal(o2[:-1], o[:-1]) and torch.equal(lse2[:-1], lse[:-1])
        c.c[side + "_exp"][p, 0, r] = keep
        c.c[side].view(torch.uint8)[p, 0, r] = codes


def shift_values(c, b, shift, rows=None):
    """Moves the exponents of sequence b's value rows by shift [kv_len] (all heads), in the cache and the oracle."""
    page = c.c["v"].shape[2]
    for j in range(len(shift)):
        c.c["v_exp"][int(c.table[b, j // page]), :, j % page] += int(shift[j])
    c.values[b] = c.values[b] * 2.0 ** shift.to(F64)[:, None, None]


def check_times(c, o, lse, factor, causal=True):
    """c.check of results times a power of two, so that its absolute term stays out of it."""
    keep = c.values
    c.values = [v * factor for v in keep]
    c.check((o.double() * factor).to(o.dtype), lse, causal)
    c.values = keep


@pytest.mark.parametrize("fmt,qd", [(E4, BF), (E4, F32)])
@pytest.mark.parametrize("n", [1, 12, 40])
@pytest.mark.parametrize("at", [-126, -118, -97, -60, 100])
def test_attention_value_scales_at_their_ends(fmt, qd, n, at, dev):
    """All value rows near one far exponent (down to the least that the cache holds), in one part and in several."""
    for m in (1, 90, 4000):
        c = Case([n], [m], dev, hq=6, hkv=1, d=256, page=256, fmt=fmt, qd=qd, seed=m)
        low = min(int(c.c["v_exp"][int(c.table[0, j // 256]), 0, j % 256]) for j in range(m))
        shift_values(c, 0, torch.full((m,), at - low))
        o, lse, ws = c.run()
        ls.ls_read_device_status(ws)
        check_times(c, o, lse, 2.0 ** -(at + 8))


@pytest.mark.parametrize("n", [1, 12, 40])
@pytest.mark.parametrize("where", ["a part", "every other", "the first tile", "the last tile"])
def test_attention_least_value_scales_beside_ordinary_ones(n, where, dev):
    """Value rows at the least exponent beside ordinary rows: in a part of their own, mixed, first, last."""
    m = 4000
    c = Case([n], [m], dev, hq=6, hkv=1, d=256, page=256, seed=5)
    j = torch.arange(m)
    tiny = {"a part": j < 2000, "every other": j % 2 == 0, "the first tile": j < 128, "the last tile": j >= m - 160}[where]
    exps = torch.tensor([int(c.c["v_exp"][int(c.table[0, x // 256]), 0, x % 256]) for x in range(m)])
    shift_values(c, 0, torch.where(tiny, -126 - exps, torch.zeros_like(exps)))
    for causal in (True, False):
        o, lse, ws = c.run(causal)
        ls.ls_read_device_status(ws)
        c.check(o, lse, causal)


@pytest.mark.parametrize("n", [1, 12, 40])
def test_attention_value_scales_160_binades_apart(n, dev):
    """Rows around 2^100 and rows around 2^-60 of like weight: the small rows' weights count in the sum all the same."""
    m = 1500
    c = Case([n], [m], dev, hq=6, hkv=1, d=256, page=256, seed=6)
    shift_values(c, 0, torch.where(torch.arange(m) % 3 == 0, 100, -60))
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    check_times(c, o, lse, 2.0 ** -100)


def one_loud_key(c, at, loud):
    """Queries 16 in dimension 0; keys 0 but for key `at`, which is `loud` there: its score is loud, the others' 0."""
    m, page, d = c.keys[0].shape[0], c.c["k"].shape[2], c.d
    q = torch.zeros_like(c.q_host)
    q[..., 0] = 16.0
    c.q_host, c.q = q, q.to(c.dev)
    k = torch.zeros(m, 1, d, dtype=F64)
    k[at, 0, 0] = loud
    codes, exps = ref.quantise(k)
    for j in range(m):
        p, r = int(c.table[0, j // page]), j % page
        c.c["k"].view(torch.uint8)[p, :, r] = codes[j].to(c.dev)
        c.c["k_exp"][p, :, r] = exps[j].to(c.dev)
    c.keys[0] = ref.dequantise(codes, exps)


def zero_values(c, which):
    """Value rows `which` of the first sequence as the cache writes zeros."""
    page = c.c["v"].shape[2]
    for j in which:
        p, r = int(c.table[0, j // page]), j % page
        c.c["v"].view(torch.uint8)[p, :, r] = 128 if j % 2 else 0  # -0 and 0
        c.c["v_exp"][p, :, r] = 0
        c.values[0][j] = 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 12, 50])
def test_attention_a_zero_value_row_above_many(n, d, dev):
    """A key whose weight is e^17 of the others' and whose value row is zeros: the output is the others' small
    sum, whatever the scale of their values."""
    for at, shift in ((7, -5), (1999, -20), (700, 0)):
        c = Case([n], [2000], dev, hq=6, hkv=1, d=d, page=256, seed=4, q_scale=0.0)
        one_loud_key(c, at, 17.0 * 16 / 16 * math.sqrt(d) / 16)
        shift_values(c, 0, torch.full((2000,), shift))
        zero_values(c, [at])
        o, lse, ws = c.run(False)
        ls.ls_read_device_status(ws)
        check_times(c, o, lse, 2.0 ** -(shift - 24), False)


@pytest.mark.parametrize("n", [1, 12, 50])
@pytest.mark.parametrize("where", ["all", "the first tiles", "the last tiles", "every other"])
def test_attention_zero_value_rows(n, where, dev):
    """Value rows of zeros: all of them (o is 0, lse as ever), whole tiles, every other; the others far below 1."""
    m = 1400
    c = Case([n], [m], dev, hq=6, hkv=1, d=256, page=256, seed=7)
    shift_values(c, 0, torch.full((m,), -30))
    zero_values(c, {"all": range(m), "the first tiles": range(300), "the last tiles": range(1100, m),
                    "every other": range(0, m, 2)}[where])
    o, lse, ws = c.run()
    ls.ls_read_device_status(ws)
    check_times(c, o, lse, 2.0 ** 30)


@pytest.mark.parametrize("n", [1, 12, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("down", [-4, -8, -10, -12, -20, -40, -100])
def test_attention_quiet_keys_beside_zero_rows(n, d, down, dev):
    """Keys 2^down of ordinary ones, with queries that make up for it, in tiles that also hold key rows of zeros
    (written with exponent 0): the quiet keys' scores stay as they are."""
    m = 700
    c = Case([n], [m], dev, hq=8, hkv=1, d=d, page=256, seed=d, q_scale=2.0 ** -down)
    page = 256
    for j in range(m):
        p, r = int(c.table[0, j // page]), j % page
        if j % 7 == 0:
            c.c["k"].view(torch.uint8)[p, :, r] = 0
            c.c["k_exp"][p, :, r] = 0
            c.keys[0][j] = 0
        else:
            c.c["k_exp"][p, :, r] += down
            c.keys[0][j] *= 2.0 ** down
    for causal in (True, False):
        o, lse, ws = c.run(causal)
        ls.ls_read_device_status(ws)
        c.check(o, lse, causal)


@pytest.mark.parametrize("n,d,v", [(20, 4, 65535 * 64 + 70), (1, 1, 65535 * 256 + 300)])
def test_vocab_of_many_tiles(n, d, v, dev):
    """More tiles of the vocabulary than a grid's second dimension holds."""
    g = torch.Generator(device=dev).manual_seed(0)
    h, w = torch.randn(n, d, generator=g, device=dev), torch.randn(v, d, generator=g, device=dev)
    t = torch.randint(0, v, (n,), generator=g, device=dev)
    t[0] = v - 1
    dl = torch.randn(n, generator=g, device=dev)
    desc = ls.vocab_desc(h, w)
    ws = torch.zeros(ls.ls_vocab_logprob_workspace_size(desc, True), dtype=torch.uint8, device=dev)
    logp, lse, dh, dw = torch.empty(n, device=dev), torch.empty(n, device=dev), torch.empty_like(h), torch.empty_like(w)
    ls.ls_vocab_logprob_fwd(desc, h, w, t, logp, lse, ws)
    ls.ls_vocab_logprob_bwd(desc, h, w, t, lse, dl, dh, dw, ws)
    ls.ls_read_device_status(ws)
    x = h.double() @ w.double().T
    wl = torch.logsumexp(x, 1)
    p = torch.exp(x - wl[:, None])
    top = float(x.abs().max())
    # a logit of d terms, and a sum of v terms of which each partial sum is rounded
    dlse = (d + 4) * 2.0 ** -23 * top + 2.0 ** -16
    assert (lse.double() - wl).abs().max() <= dlse
    assert (logp.double() - (x.gather(1, t[:, None])[:, 0] - wl)).abs().max() <= 2 * dlse
    slope = -p * dl.double()[:, None]
    slope[torch.arange(n), t] += dl.double()
    del x
    mags = slope.abs()
    err = (dh.double() - slope @ w.double()).abs()
    assert (err <= 4 * dlse * (mags @ w.double().abs()) + 1e-30).all()
    err = (dw.double() - slope.T @ h.double()).abs()
    assert (err <= 4 * dlse * (mags.T @ h.double().abs()) + 1e-30).all()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [1, 12, 40])
@pytest.mark.parametrize("values", ["ordinary", "zero", "least", "large"])
def test_attention_lse_of_a_few_keys(n, d, values, dev):
    """One to five keys with scores near 0: lse is the logarithm of their number, whatever the values' scale."""
    for m in (1, 2, 3, 5):
        c = Case([n], [m], dev, hq=8, hkv=1, d=d, page=4, seed=m, q_scale=2.0 ** -20)
        at = {"ordinary": 0, "zero": 0, "least": -116, "large": 100}[values]
        shift_values(c, 0, torch.full((m,), at))
        if values == "zero":
            zero_values(c, range(m))
        for causal in (True, False):
            o, lse, ws = c.run(causal)
            ls.ls_read_device_status(ws)
            check_times(c, o, lse, 2.0 ** -at, causal)
