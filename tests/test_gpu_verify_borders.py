"""Verification of drafts where a decision can go wrong."""
import math

import pytest
import torch

from test_gpu_verify import LOW, check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 1.25, 1e10, 1e12, 3e20, 2.0 ** 100])
def test_masked_drafts_at_any_scale(cuda_device, dtype, probs, scale):
    """A draft whose logit is -infinity or the type's lowest value has probability 0: it is rejected, by whatever the
    logits are multiplied (the product with the low part of scale * log2(e) passes float32's range from about 1e9 on)."""
    m = make([2] * 8, 777, dtype, probs, scale, seed=31)
    m["u"][:] = 0.5
    for b in range(8):
        r = m["q_start"][b]
        m["wide"][r, int(m["tokens"][r + 1])] = -math.inf if b % 2 else LOW[dtype]
        if probs:
            m["probs"][r, int(m["tokens"][r + 1])] = 0.25
    got = run(m)
    assert got[0].tolist() == [1] * 8
    for b in range(8):
        assert int(got[1][2 * b]) != int(m["tokens"][2 * b + 1]) and math.isfinite(float(got[2][2 * b]))
    if scale >= 1:
        check(m, got)
    else:                                              # all tokens but the masked one alike, to 2^-90
        for b in range(8):
            d = int(m["tokens"][2 * b + 1])
            q = m["probs"][2 * b].double() if probs else torch.zeros(777, dtype=torch.float64)
            p = torch.full((777,), 1 / 776, dtype=torch.float64)
            p[d] = 0.0
            upto = torch.cumsum((p - q).clamp(min=0), 0)
            edge = float(m["u_next"][b]) * float(upto[-1])
            if float((upto - edge).abs().min() / upto[-1]) > 2.0 ** -20:   # the excess is 2^-9.6 of the row, good to 2^-30 of it
                assert int(got[1][2 * b]) == int((upto <= edge).sum())


@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("by", [2 ** 32, -2 ** 32, 2 ** 40, -2 ** 40, 2 ** 63 - 512, -2 ** 63])
def test_drafts_whose_lower_half_is_a_token(cuda_device, probs, by):
    """An id outside the vocabulary is rejected as it is, and the next token comes from p: the token that its lower 32
    bits name is drawn like any other."""
    m = make([2] * 4, 512, torch.float32, probs, seed=33)
    m["u"][:] = 0.0
    for b, t in enumerate((0, 3, 300, 511)):
        r = m["q_start"][b]
        m["wide"][r, t] = m["wide"][r].max() + 3       # most of the row
        if probs:
            m["probs"][r, t] = 0.0
        m["u_next"][b] = float(torch.softmax(m["wide"][r].double(), 0)[:t].sum()) + 0.1
        m["tokens"][r + 1] = t + by
    got = run(m, status=5)
    check(m, got)
    assert got[0].tolist() == [1] * 4
    if not probs:
        assert got[1][::2].tolist() == [0, 3, 300, 511]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("masked", ["inf", "low"])
def test_a_segment_that_holds_the_rejected_draft_alone(cuda_device, dtype, masked):
    """Around the rejected draft all tokens are masked: nothing can be drawn there, whatever its weight leaves of the sums
    it was in.  The first or the last token that is left comes out."""
    n = 64
    m = make([2] * n, 8191, dtype, False, seed=35)
    low = -math.inf if masked == "inf" else LOW[dtype]
    m["u"][:] = 1.0 - 2.0 ** -24
    for b in range(n):
        r = m["q_start"][b]
        first = b % 4 < 2
        d = 7 + b if first else 8180 - b               # before all others, or behind them
        m["wide"][r] = low
        m["wide"][r, d] = -7.0 - 0.13 * b               # 2^-12 to 2^-23 of the others: its lower part is rounded with the rest of the sum
        m["wide"][r, 4000:4011] = torch.linspace(0, 1, 11).to(dtype)
        m["tokens"][r + 1] = d
        m["u_next"][b] = 0.0 if first else 1.0 - 2.0 ** -24
    got = run(m)
    assert got[0].tolist() == [1] * n
    assert got[1][::2].tolist() == [4000 if b % 4 < 2 else 4010 for b in range(n)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("drafts", [0, 1])
def test_tokens_too_small_to_be_drawn(cuda_device, dtype, drafts):
    """Tokens below 2^-61 of the row (2^-60 where its sum is a power of two) count as none one by one, whatever they are together: the first token that is drawn
    is the first of the others, never a masked one."""
    n = 6
    m = make([1 + drafts] * n, 5000, dtype, False, seed=37)
    m["u"][:] = 0.0                                    # the draft passes
    m["u_next"][:] = 0.0
    for b in range(n):
        r = m["q_start"][b] + drafts
        m["wide"][r] = -math.inf
        m["wide"][r, 10 + b:1024] = -42.5              # 2^-61.3 each, 2^-51.3 together
        m["wide"][r, 3000 + b] = 0.0
        m["wide"][r, 4000] = -42.5
    count, out, _, _ = run(m)
    assert count.tolist() == [1 + drafts] * n
    assert out[drafts::1 + drafts].tolist() == [3000 + b for b in range(n)]
    m["u_next"][:] = 1.0 - 2.0 ** -24
    assert run(m)[1][drafts::1 + drafts].tolist() == [3000 + b for b in range(n)]


def test_what_a_rejection_leaves_at_its_threshold(cuda_device):
    """max(p - q, 0) is taken for 0 everywhere where its sum is at most 2^-30 of p's, whatever p's sum is: just above the
    next token is the one that it has, just below it comes from p.  (The excess is good to float32's q of 2^-28, 2^-53.)"""
    n, v, j = 24, 1000, 417
    m = make([2] * n, v, torch.float32, True, seed=41)
    m["u"][:] = 0.9
    m["u_next"][:] = 0.5
    sums = []
    for b in range(n):
        r = m["q_start"][b]
        m["wide"][r, j] = -math.inf
        z = m["wide"][r].double()
        m["wide"][r, j] = float(torch.logsumexp(z, 0)) - 28 * math.log(2.0)
        z = m["wide"][r].double()
        sums.append(float(torch.exp(z - z.max()).sum()))
        p = torch.softmax(z, 0)
        m["probs"][r] = (1.5 * p).float()
        m["probs"][r, j] = (p[j] - (1.25 if b % 2 else 0.75) * 2.0 ** -30).float()
        m["tokens"][r + 1] = int(p.argmax())
    assert min(math.frexp(s)[0] for s in sums) < 0.6 and max(math.frexp(s)[0] for s in sums) > 0.9
    got = run(m)
    assert got[0].tolist() == [1] * n
    assert got[1][2::4].tolist() == [j] * (n // 2)
    assert j not in got[1][::4].tolist()
    check(m, got)
