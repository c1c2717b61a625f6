"""Verification of drafts where a decision can go wrong.

Bounds.  An acceptance: a 2 KB piece's exponentials are 4 roundings of 2^-24 each (ex2's 2^-22), at most 23 additions
on their way, then up to 8 joins in a lane and 5 between lanes at 2^17 float32 logits, 6 roundings each (an addition,
two of the argument, ex2); the arguments' own roundings are 2.5 2^-24 of the mean of -log2 p over the row, at most 13
there, times ln 2: in all 4 + 23 + 78 + 22 = 127 roundings of 2^-24, and with the products and exp2f of the test
itself and 1.4 roundings for each bit that the draft is below the largest, under 256 for p down to 2^-80: 2^-16.  The
joins in a lane double with the vocabulary.  A draw's bounds stand at its tests."""
import math

import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from oracle import drafts as ref
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


def test_draws_from_millions_of_tokens(cuda_device):
    """A row of one large and V - 1 equal logits: the steps of the draw are known.  All lower parts of a thread's weights
    are alike, so that the roundings of their float32 sum add up: over 64 of them at most 2^-20 (1 + 1/4 + ...) / 2 of
    the sum, 2^-20.6, and as a block's warp holds a sixteenth of the row here (160 sequences, two blocks each), a border
    moves by 2^-24.6 of the whole.  The random numbers are float32 and lie in the middle of a token, 2^-23 from its
    borders but for their rounding of 2^-25."""
    v, b, x = 4_000_003, 160, 1.296875
    g = torch.Generator().manual_seed(39)
    row = torch.zeros(v, dtype=torch.bfloat16, device="cuda")
    row[0] = x
    logits = row.expand(2 * b, v).contiguous()
    top = math.exp(x)
    total = top + v - 1
    want = torch.randint(1, v, (b,), generator=g)
    ends = (torch.arange(1, 17) * (v // 16)).clamp(max=v - 1)   # about the last tokens of the segments
    want[:16] = ends - 1
    u_next = ((top + want.double() - 0.5) / total).float()
    i32, i64 = torch.int32, torch.int64
    desc = ls.verify_desc(logits, b, 2)
    ws = torch.zeros(ls.ls_draft_verify_workspace_size(desc), dtype=torch.uint8, device="cuda")
    count, out = torch.empty(b, dtype=i32, device="cuda"), torch.empty(2 * b, dtype=i64, device="cuda")
    ls.ls_draft_verify(desc, logits, torch.ones(2 * b, dtype=i64, device="cuda"), torch.arange(0, 2 * b + 1, 2, dtype=i32, device="cuda"),
                       torch.zeros(2 * b, device="cuda"), u_next.cuda(), count, out, None, ws)
    ls.ls_read_device_status(ws)
    assert (count == 2).all()
    got = out.cpu()[1::2]
    assert torch.equal(got, want), (got - want)[got != want]


@pytest.mark.parametrize("dtype,probs", [(torch.float32, True), (torch.bfloat16, True), (torch.bfloat16, False)])
def test_draws_from_a_million_tokens(cuda_device, dtype, probs):
    """Rejected and accepted drafts over a long row with a tail.  Some 10^6 lower parts are added in float32, each rounding
    within 2^-42 of the row (half a step of a sum of 64 below 2^-17): where they fall as they may 2^-32 in all, and the
    weights' own 2^-30 of each add 2^-40.  Draws within 2^-28 of the row of a border are left out."""
    v, b = 1_000_003, 48
    m = make([2] * b, v, dtype, probs, spread=1.5, seed=45, device="cuda")
    m["u"][::4] = 0.0
    count, out, _, _ = run(m)
    left_out = 0
    for i in range(b):
        r = 2 * i + int(count[i]) - 1
        z = m["wide"][2 * i:2 * i + 2].double()
        p = torch.softmax(z, 1)
        d = int(m["tokens"][2 * i + 1])
        q = m["probs"][2 * i].double() if probs else torch.nn.functional.one_hot(m["tokens"][2 * i + 1], v).double()
        side = float(m["u"][2 * i]) * float(q[d]), float(p[0, d])
        if abs(side[0] - side[1]) > 2.0 ** -13 * max(side):   # 2^-16, doubled three times
            assert int(count[i]) == 1 + (side[0] < side[1])
        w = p[1] if r % 2 else (p[0] - q).clamp(min=0)
        upto = torch.cumsum(w, 0)
        edge = float(m["u_next"][i]) * float(upto[-1])
        if float((upto - edge).abs().min()) < 2.0 ** -28:
            left_out += 1
            continue
        assert int(out[r]) == int((upto <= edge).sum())
    assert left_out <= 3


@pytest.mark.parametrize("value", [-math.inf, math.nan])
def test_caches_go_on_together(cuda_device, value):
    """keep - kv_len + n is how many of a sequence's n tokens have their keys kept, and how many the recurrent state takes:
    also behind a row without a distribution, where it is one more than n_emitted."""
    counts = [3, 2, 1, 0, 4]
    m = make(counts, 1031, torch.float32, probs=False, seed=43)
    m["u"][:] = 0.0                                    # every draft passes
    m["wide"][2] = value                               # the first's last row, the second's first
    m["wide"][3] = value
    b, n, page = len(counts), sum(counts), 4
    i32, i64 = torch.int32, torch.int64
    dev = lambda t: t.cuda()  # noqa: E731
    refs, table = torch.zeros(64, dtype=i32, device="cuda"), torch.zeros((b, 16), dtype=i32, device="cuda")
    kv_len = torch.zeros(b, dtype=i64, device="cuda")
    book = ls.page_book(refs, table, kv_len, page)
    pws = torch.zeros(ls.ls_pages_workspace_size(book), dtype=torch.uint8, device="cuda")
    slots, copies = torch.empty(5 * b + n, dtype=i64, device="cuda"), torch.empty((b, 3), dtype=i32, device="cuda")
    grown = torch.tensor([5 + c for c in counts])
    starts = torch.cat([torch.zeros(1, dtype=i64), grown.cumsum(0)]).to(i32)
    ls.ls_pages_advance(book, dev(starts), slots, copies, pws)
    logits, q_start = dev(m["wide"]), torch.tensor(m["q_start"], dtype=i32, device="cuda")
    desc = ls.verify_desc(logits, b, max(counts))
    ws = torch.zeros(ls.ls_draft_verify_workspace_size(desc), dtype=torch.uint8, device="cuda")
    count, out, keep = torch.empty(b, dtype=i32, device="cuda"), torch.empty(n, dtype=i64, device="cuda"), torch.empty(b, dtype=i64, device="cuda")
    ls.ls_draft_verify(desc, logits, dev(m["tokens"]), q_start, dev(m["u"]), dev(m["u_next"]), count, out, None, ws, kv_len=kv_len, keep=keep)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    n_use = (keep - kv_len + torch.tensor(counts, device="cuda")).to(i32)
    assert n_use.tolist() == [3, 1, 1, 0, 4] and count.tolist() == [2, 0, 1, 0, 4]
    g = torch.Generator().manual_seed(44)
    q, k, v = (torch.randn(n, 1, 128, generator=g) * s for s in (0.1, 0.1, 1.0))
    decay, beta = -0.1 * torch.rand(n, 1, generator=g), torch.rand(n, 1, generator=g)
    states = torch.randn(b, 1, 128, 128, generator=g)
    d = [dev(t) for t in (states, q, k, v, decay, beta)]
    own = torch.arange(b, dtype=i32, device="cuda")
    ls.ls_gdn_decode(ls.gdn_decode_desc(*d[1:4], d[0], b, max(counts)), *d, q_start, own, own, None, pws, n_use=n_use)
    ls.ls_pages_advance(book, None, None, None, pws, keep=keep)
    ls.ls_read_device_status(pws)
    for i in range(b):
        used = int(n_use[i])
        assert int(kv_len[i]) == 5 + used
        at = slice(m["q_start"][i], m["q_start"][i] + used)
        _, want, _, mag = ref.state_step(states[i], q[at], k[at], v[at], decay[at], beta[at])
        assert ((d[0][i].double().cpu() - want).abs() <= 28 * used * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("behind", [0, 600])
def test_nothing_to_draw_in_the_last_segments(cuda_device, dtype, behind):
    """The rejected draft alone behind all other tokens, in the last segment or with masked ones behind it, and a random
    number of 1, which asks for the last token: the last that is left comes out."""
    n = 64
    m = make([2] * n, 8191, dtype, False, seed=47)
    m["u"][:] = 1.0
    m["u_next"][:] = 1.0
    for b in range(n):
        r, d = m["q_start"][b], 8180 - behind - b
        m["wide"][r] = -math.inf
        m["wide"][r, d] = -7.0 - 0.13 * b
        m["wide"][r, 4000:4011] = torch.linspace(0, 1, 11).to(dtype)
        m["tokens"][r + 1] = d
    got = run(m)
    assert got[0].tolist() == [1] * n
    assert got[1][::2].tolist() == [4010] * n
