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
