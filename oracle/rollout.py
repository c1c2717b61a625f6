"""Float64 definitions of the rollout and scoring operators, written from their
formulas (torch on the CPU; no code shared with the CUDA path): the e4m3 cache,
attention of new tokens over paged keys, and vocabulary log-probabilities with
their gradients.  Each also gives the magnitudes its error bounds are made of."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def e4m3_values():
    """The non-negative finite e4m3 values by code 0..126 (bias 7; exponent 0 is subnormal)."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=F64)


def quantise(x):
    """(codes uint8, exponents int8) of the rows (last axis) of x: the least e >= -126 with
    max|row| <= 448 * 2^e, codes rounded to nearest, ties to the even code; a row that is not
    finite gives codes 0 and exponent -128."""
    x = x.to(F64)
    flat = x.reshape(-1, x.shape[-1])
    table = e4m3_values()
    codes = torch.zeros(flat.shape, dtype=torch.uint8)
    exps = torch.zeros(flat.shape[0], dtype=torch.int8)
    for r in range(flat.shape[0]):
        top = float(flat[r].abs().max()) if flat.shape[1] else 0.0
        if not math.isfinite(top):
            exps[r] = -128
            continue
        e = 0
        if top > 0:
            e = max(-126, math.frexp(top)[1] - 10)
            while top > 448.0 * 2.0 ** e:
                e += 1
        y = flat[r] * 2.0 ** -e
        a = y.abs()
        hi = torch.searchsorted(table, a).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = a - table[lo], table[hi] - a
        pick = torch.where(dl < dh, lo, torch.where(dh < dl, hi, torch.where(lo % 2 == 0, lo, hi)))
        sign = torch.signbit(flat[r]).to(torch.uint8) << 7
        codes[r] = pick.to(torch.uint8) | sign
        exps[r] = e
    return codes.reshape(x.shape), exps.reshape(x.shape[:-1])


def dequantise(codes, exps):
    code = codes.to(torch.int64)
    v = torch.cat([e4m3_values(), torch.tensor([math.nan], dtype=F64)])[code & 127]
    v = torch.where(code >= 128, -v, v)
    scale = torch.where(exps == -128, torch.tensor(math.nan, dtype=F64), 2.0 ** exps.to(F64))
    return v * scale[..., None]


def cached_attention(q, keys, values, q_start, kv_len, causal, scale, key_ok=None):
    """q [T, Hq, d]; keys, values: per sequence float64 [kv_len, Hkv, d]; key_ok: per sequence a
    mask of keys that exist.  Returns o, lse, and per row the bound terms (a: sum_j p_j |v_j|,
    sx: the largest scale * sum |q||k| of a key it sees)."""
    t, hq, d = q.shape
    o = torch.zeros((t, hq, d), dtype=F64)
    a = torch.zeros((t, hq, d), dtype=F64)
    lse = torch.full((t, hq), -math.inf, dtype=F64)
    sx = torch.zeros((t, hq), dtype=F64)
    for b in range(len(kv_len)):
        first, last = int(q_start[b]), int(q_start[b + 1])
        n, m = last - first, int(kv_len[b])
        if n == 0 or m == 0:
            continue
        hkv = keys[b].shape[1]
        k = keys[b].repeat_interleave(hq // hkv, 1)
        v = values[b].repeat_interleave(hq // hkv, 1)
        qq = q[first:last].to(F64)
        see = torch.ones((n, m), dtype=torch.bool)
        if causal:
            see &= torch.arange(m)[None] <= (m - n + torch.arange(n))[:, None]
        if key_ok is not None:
            see &= key_ok[b][None]
        for i in range(n):
            at = see[i].nonzero()[:, 0]
            if len(at) == 0:
                continue
            x = torch.einsum("hd,jhd->hj", qq[i], k[at]) * scale
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            lse[first + i] = z
            o[first + i] = torch.einsum("hj,jhd->hd", p, v[at])
            a[first + i] = torch.einsum("hj,jhd->hd", p, v[at].abs())
            sx[first + i] = (torch.einsum("hd,jhd->hj", qq[i].abs(), k[at].abs()) * scale).amax(1)
    return o, lse, a, sx


def vocab_logprob(h, w, targets, scale, ignore_index):
    """logp, lse and the logits in float64."""
    x = h.to(F64) @ w.to(F64).T * scale
    lse = torch.logsumexp(x, 1)
    on = (targets != ignore_index) & (targets >= 0) & (targets < w.shape[0])
    t = torch.where(on, targets, torch.zeros_like(targets))
    logp = torch.where(on, x.gather(1, t[:, None])[:, 0] - lse, torch.zeros_like(lse))
    return logp, lse, x, on, t


def vocab_gradients(h, w, targets, d_logp, scale, ignore_index):
    """dh, dw, and the gradient's matrix over the logits' products (scale included)."""
    _, lse, x, on, t = vocab_logprob(h, w, targets, scale, ignore_index)
    c = torch.where(on, d_logp.to(F64) * scale, torch.zeros_like(lse))
    p = torch.exp(x - lse[:, None])
    slope = -c[:, None] * p
    slope[torch.arange(len(t)), t] += c
    return slope @ w.to(F64), slope.T @ h.to(F64), slope, p * c[:, None].abs()
