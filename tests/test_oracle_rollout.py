"""Pins of oracle/rollout.py (CPU): library functions, autograd, central
differences, closed forms, and planted mistakes that the pins must reject."""
import math

import pytest
import torch

from oracle import rollout as ref

F64 = torch.float64


def test_e4m3_table_is_the_type():
    codes = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(codes.view(torch.float8_e4m3fn).to(F64), ref.e4m3_values())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -100, 2.0 ** 100, 2.0 ** -126])
def test_quantise_against_the_library_type(dtype, scale):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(50, 64, generator=g, dtype=F64) * torch.rand(50, 1, generator=g, dtype=F64) * 4 * scale).to(dtype)
    x[3] = 0
    x[4] = 448 * scale
    x[5, 0] = 449 * scale
    codes, exps = ref.quantise(x)
    top = x.to(F64).abs().amax(1)
    e = exps.to(F64)
    assert (top <= 448 * 2.0 ** e).all()
    tight = (top > 448 * 2.0 ** (e - 1)) | (exps == -126)
    tight[3] = True
    assert tight.all() and exps[3] == 0
    want = (x.to(F64) * 2.0 ** -e[:, None]).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(want, codes)
    back = ref.dequantise(codes, exps)
    # half a step of 3 mantissa bits, or of the smallest code
    assert ((back - x.to(F64)).abs() <= torch.maximum(x.to(F64).abs() * 2.0 ** -4, 2.0 ** (e[:, None] - 10))).all()


def test_quantise_not_finite():
    x = torch.ones(3, 64)
    x[0, 5] = math.inf
    x[1, 6] = math.nan
    codes, exps = ref.quantise(x)
    assert exps.tolist() == [-128, -128, -8] and ref.dequantise(codes, exps)[:2].isnan().all()
    assert torch.equal(ref.dequantise(codes, exps)[2], torch.ones(64, dtype=F64))


def _attn_case(n, m, hq=4, hkv=2, d=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, hq, d, generator=g, dtype=F64), torch.randn(m, hkv, d, generator=g, dtype=F64),
            torch.randn(m, hkv, d, generator=g, dtype=F64))


@pytest.mark.parametrize("n,m", [(1, 1), (1, 9), (5, 5), (4, 30), (7, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_against_library(n, m, causal):
    q, k, v = _attn_case(n, m)
    o, lse, a, sx = ref.cached_attention(q, [k], [v], [0, n], [m], causal, 0.25)
    mask = torch.arange(m)[None] <= (m - n + torch.arange(n))[:, None] if causal else torch.ones(n, m, dtype=torch.bool)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.repeat_interleave(2, 1).transpose(0, 1), v.repeat_interleave(2, 1).transpose(0, 1),
        attn_mask=mask, scale=0.25).transpose(0, 1)
    some = mask.any(1)
    assert torch.allclose(o[some], want[some], atol=1e-12)
    assert (o[~some] == 0).all() and (lse[~some] == -math.inf).all()
    assert (a >= o.abs() - 1e-12).all() and (sx[some] > 0).all()


def test_attention_rejects_an_exclusive_diagonal():
    q, k, v = _attn_case(4, 4)
    o, *_ = ref.cached_attention(q, [k], [v], [0, 4], [4], True, 0.25)
    wrong, *_ = ref.cached_attention(q[1:], [k[:3]], [v[:3]], [0, 3], [3], True, 0.25)
    assert (o[1:] - wrong).abs().max() > 1e-3


def test_attention_key_mask_is_a_shorter_cache():
    q, k, v = _attn_case(3, 12)
    ok = torch.ones(12, dtype=torch.bool)
    ok[4:8] = False
    got = ref.cached_attention(q, [k], [v], [0, 3], [12], False, 0.5, [ok])
    want = ref.cached_attention(q, [k[ok]], [v[ok]], [0, 3], [8], False, 0.5)
    assert torch.allclose(got[0], want[0], atol=1e-13) and torch.allclose(got[1], want[1], atol=1e-13)


def _vocab_case(n=6, d=10, v=17):
    g = torch.Generator().manual_seed(1)
    h = torch.randn(n, d, generator=g, dtype=F64)
    w = torch.randn(v, d, generator=g, dtype=F64)
    t = torch.randint(0, v, (n,), generator=g)
    t[2] = -100
    return h, w, t, torch.randn(n, generator=g, dtype=F64)


def test_vocab_against_library_and_autograd():
    h, w, t, dl = _vocab_case()
    h.requires_grad_(), w.requires_grad_()
    logp, lse, *_ = ref.vocab_logprob(h.detach(), w.detach(), t, 0.7, -100)
    want = -torch.nn.functional.cross_entropy(h @ w.T * 0.7, t, reduction="none", ignore_index=-100)
    assert torch.allclose(logp, want, atol=1e-12)
    assert torch.allclose(lse, torch.logsumexp(h @ w.T * 0.7, 1), atol=1e-12)
    (want * dl).sum().backward()
    dh, dw, _, _ = ref.vocab_gradients(h.detach(), w.detach(), t, dl, 0.7, -100)
    assert torch.allclose(dh, h.grad, atol=1e-12) and torch.allclose(dw, w.grad, atol=1e-12)
    assert (dh[2] == 0).all()


def test_vocab_gradients_against_differences():
    h, w, t, dl = _vocab_case()
    dh, dw, _, _ = ref.vocab_gradients(h, w, t, dl, 1.3, -100)
    f = lambda: float((ref.vocab_logprob(h, w, t, 1.3, -100)[0] * dl).sum())  # noqa: E731
    for x, dx in ((h, dh), (w, dw)):
        for i in ((0, 0), (2, 3), (5, 9)):
            keep = float(x[i])
            x[i] = keep + 1e-5
            up = f()
            x[i] = keep - 1e-5
            down = f()
            x[i] = keep
            assert abs((up - down) / 2e-5 - float(dx[i])) < 1e-7


def test_vocab_pins_reject_a_missing_scale():
    h, w, t, dl = _vocab_case()
    dh, *_ = ref.vocab_gradients(h, w, t, dl, 1.3, -100)
    _, _, slope, _ = ref.vocab_gradients(h, w, t, dl, 1.3, -100)
    assert (slope / 1.3 @ w - dh).abs().max() > 1e-2
