"""Verification of drafted tokens and the draw of the next one against their float64 definition.

Decisions.  p comes from float32 sums: the exponentials of at most 16 KB a block, 32 of them in a row in a
thread, 8 joins, then the row's pieces joined: under 100 roundings of 2^-24 with ex2's 2 ulp, and its own
argument's 2^-24 |s (z - max)|, up to 20 where p matters.  So an acceptance is the definition's unless it is
within 2^-16 of its border (relative).  The draw's weights are good to 2^-31 each, its sums exact: unless
within 2^-30 of the whole of a border, the token is the definition's.  `near` is in units of these: below
2^-16 for the first, and the second counts 2^10 times (2^-20 then).  Nothing is compared there.

logp is log of the row's sum (100 roundings) and s (z - max), each of its two roundings 2^-24 of it."""
import math

import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from oracle import drafts as ref

pytestmark = pytest.mark.gpu
LOW = {torch.float32: torch.finfo(torch.float32).min, torch.bfloat16: torch.finfo(torch.bfloat16).min}


def make(counts, vocab, dtype, probs=True, scale=1.0, pad=0, spread=2.5, seed=0, device="cpu"):
    g = torch.Generator(device=device).manual_seed(seed)
    n, b = sum(counts), len(counts)
    wide = torch.randn(n, vocab + pad, generator=g, device=device).mul_(spread).to(dtype)
    m = dict(wide=wide, vocab=vocab, scale=scale, counts=counts, u=torch.rand(n, generator=g, device=device),
             u_next=torch.rand(b, generator=g, device=device), tokens=torch.randint(0, vocab, (n,), generator=g, device=device),
             kv_len=torch.randint(100, 200, (b,), generator=g, device=device))
    q = torch.softmax((wide[:, :vocab].float() + 0.7 * torch.randn(n, vocab, generator=g, device=device)) * scale, 1)
    if n > 1:
        m["tokens"][1:] = torch.multinomial(q[:-1], 1, generator=g)[:, 0] if probs else q[:-1].argmax(1)
    m["probs"] = torch.cat([q, q[:, :pad]], 1) if probs else None
    m["q_start"] = [sum(counts[:i]) for i in range(b + 1)]
    return m


def run(m, max_q=None, logp=True, q_start=None, status=0, graph=False):
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    logits = c(m["wide"])[:, :m["vocab"]]
    probs = None if m["probs"] is None else c(m["probs"])[:, :m["vocab"]]
    b, n = len(m["counts"]), len(m["tokens"])
    desc = ls.verify_desc(logits, b, max_q or max(m["counts"] + [1]) if n else 0, draft_probs=probs, logit_scale=m["scale"])
    ws = torch.full((ls.ls_draft_verify_workspace_size(desc),), 255, dtype=torch.uint8, device="cuda")
    ls.ls_clear_device_status(ws)
    i64 = torch.int64
    count = torch.full((b,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((n,), -9, dtype=i64, device="cuda")
    lp = torch.full((n,), -9.0, device="cuda") if logp else None
    keep = torch.full((b,), -9, dtype=i64, device="cuda")
    args = (c(m["tokens"]), torch.tensor(q_start or m["q_start"], dtype=torch.int32, device="cuda"), c(m["u"]), c(m["u_next"]))
    kv = c(m["kv_len"])
    call = lambda: ls.ls_draft_verify(desc, logits, *args, count, out, lp, ws, draft_probs=probs, kv_len=kv, keep=keep)  # noqa: E731
    if graph:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            call()
        gr.replay()
    else:
        call()
    try:
        ls.ls_read_device_status(ws)
        got = 0
    except ls.LsError as e:
        got = e.status
    assert got == status
    return count.cpu(), out.cpu(), None if lp is None else lp.cpu(), keep.cpu()


def check(m, got, skip=()):
    count, out, lp, keep = got
    probs = None if m["probs"] is None else m["probs"][:, :m["vocab"]]
    want = ref.verify(m["wide"][:, :m["vocab"]], probs, m["tokens"], m["q_start"], m["u"], m["u_next"], m["scale"])
    left_out = 0
    for b, (toks, logp, near) in enumerate(want):
        if b in skip:
            continue
        first, n = m["q_start"][b], m["counts"][b]
        if near < 2.0 ** -16:
            left_out += 1
            continue
        real = len(toks) - (None in toks)
        assert int(count[b]) == real, (b, near)
        assert int(keep[b]) == int(m["kv_len"][b]) - n + len(toks)
        assert out[first:first + n].tolist() == [-1 if t is None else t for t in toks] + [-1] * (n - len(toks)), (b, near)
        if lp is not None:
            z = m["wide"][first:first + n, :m["vocab"]].double() * m["scale"]
            for i, (t, x) in enumerate(zip(toks, logp)):
                top = float(z[i].max())
                bound = 2.0 ** -24 * (128 + 4 * abs(float(z[i][t]) - top)) if t is not None else 0.0
                assert abs(float(lp[first + i]) - x) <= bound
            assert (lp[first + len(toks):first + n] == 0).all()
    assert left_out <= max(1, len(want) // 50)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("probs", [True, False])
@pytest.mark.parametrize("counts,vocab,scale,pad", [
    ([1], 1, 1.0, 0), ([2, 1], 5, 1.0, 0), ([3, 0, 4, 1], 127, 0.7, 3), ([5, 5, 0, 2, 1, 6], 8191, 1.25, 0),
    ([9, 17, 8, 1], 300, 1.0, 5), ([4] * 12, 8200, 1.0, 8), ([2, 3], 65536, 1.0, 1), ([3, 3], 50003, 2.0, 0)])
def test_drafts_and_draws(cuda_device, dtype, probs, counts, vocab, scale, pad):
    m = make(counts, vocab, dtype, probs, scale, pad, seed=vocab + len(counts))
    got = run(m)
    check(m, got)
    again = run(m, logp=False)
    assert all(torch.equal(a, b) for a, b in zip(got[:2], again[:2]))


@pytest.mark.parametrize("dtype,probs,spread", [(torch.bfloat16, True, 2.5), (torch.float32, True, 0.01), (torch.bfloat16, False, 1.0)])
def test_many_draws_from_a_large_vocabulary(cuda_device, dtype, probs, spread):
    """Where a float32 running sum would give a neighbour of the token one time in a hundred."""
    m = make([2] * 150 if probs else [1] * 300, 100003, dtype, probs, spread=spread, seed=5, device="cuda")
    got = run(m)
    check(m, got)


def test_random_numbers_at_their_ends(cuda_device):
    for u in (0.0, 1.0 - 2.0 ** -24):
        m = make([3] * 8, 1000, torch.float32, seed=6)
        m["u"][:] = u
        m["u_next"][:] = u
        check(m, run(m))
    m = make([1] * 4, 1000, torch.float32, probs=False, seed=7)
    m["u_next"][:] = torch.tensor([1.0, 2.0, -1.0, math.nan])
    count, out, _, _ = run(m)                          # outside [0, 1): the last and the first token
    assert count.tolist() == [1] * 4 and out.tolist() == [999, 999, 0, 0]


def test_equal_probabilities_are_always_accepted(cuda_device):
    """Drafts from the target itself: p / q is 1 but for rounding."""
    m = make([8] * 6, 4001, torch.float32, seed=8)
    m["probs"] = torch.softmax(m["wide"].double(), 1).float()
    m["u"].clamp_(max=0.999)
    count, out, _, _ = run(m)
    assert count.tolist() == [8] * 6
    for b in range(6):
        assert out[8 * b:8 * b + 7].tolist() == m["tokens"][8 * b + 1:8 * b + 8].tolist()


def test_nothing_left_after_a_rejection(cuda_device):
    """q >= p everywhere (it need not sum to 1): the draw is from p."""
    m = make([2] * 5, 600, torch.float32, seed=9)
    m["probs"] = torch.softmax(m["wide"].double(), 1).float() * 1.5
    m["u"][:] = 0.9
    got = run(m)
    check(m, got)
    assert got[0].tolist() == [1] * 5


def test_probabilities_that_are_none(cuda_device):
    """Rows of q with zeros, ones, infinities, NaN and negative numbers in places: what is not above 0 counts as 0."""
    m = make([2] * 6, 900, torch.float32, seed=10)
    m["u"][:] = 0.999999
    for b, x in enumerate((0.0, 1.0, math.inf, math.nan, -1.0, 3.0)):
        r = m["q_start"][b]
        m["probs"][r, 100:500] = x
        m["probs"][r, int(m["tokens"][r + 1])] = 1.0   # rejected
    count, out, _, _ = run(m)
    assert count.tolist() == [1] * 6
    probs = m["probs"].clone()
    probs[probs.isnan() | (probs < 0)] = 0.0
    probs[probs.isinf()] = 3.0
    check(dict(m, probs=probs), run(dict(m, probs=probs)))
    assert torch.equal(out, run(dict(m, probs=probs))[1])


@pytest.mark.parametrize("q", [0.0, -1.0, -math.inf, math.nan])
def test_a_draft_whose_probability_is_none(cuda_device, q):
    """It counts as 0: the draft is taken where the target gives it anything, and not where it is masked."""
    m = make([2] * 4, 900, torch.float32, seed=11)
    m["u"][:] = 0.5
    for b in range(4):
        r = m["q_start"][b]
        m["probs"][r, int(m["tokens"][r + 1])] = q
        if b == 1:
            m["wide"][r, int(m["tokens"][r + 1])] = -math.inf
    got = run(m)
    assert got[0].tolist() == [2, 1, 2, 2]
    check(dict(m, probs=torch.where(m["probs"] > 0, m["probs"], 0.0)), got)


@pytest.mark.parametrize("max_q", [1, 4096])
def test_a_call_behind_one_whose_sequences_are_all_left_out(cuda_device, max_q):
    """The second call's pairs are its own, though the first draws from none of the many rows it reads."""
    big = torch.zeros(4096, 50000, dtype=torch.bfloat16, device="cuda")
    n, b = big.shape[0], 2 if max_q > 1 else 4096
    z = lambda k, dt: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    starts = z(b + 1, i32)
    starts[0], starts[1:] = -1, n                      # below 0 for the first, none for the others
    desc = ls.verify_desc(big, b, max_q)
    m = make([2] * 8 if max_q > 1 else [1] * 8, 8191, torch.float32, probs=False, seed=12)
    small = m["wide"].cuda()
    sdesc = ls.verify_desc(small, 8, max(m["counts"]))
    ws = z(max(ls.ls_draft_verify_workspace_size(desc), ls.ls_draft_verify_workspace_size(sdesc)), torch.uint8)
    k = small.shape[0]
    count, out, lp = z(8, i32), z(k, i64), z(k, f32)
    args = m["tokens"].cuda(), torch.tensor(m["q_start"], dtype=i32, device="cuda"), m["u"].cuda(), m["u_next"].cuda()
    first = z(n, i64), starts, z(n, f32), z(b, f32), z(b, i32), z(n, i64), z(n, f32)
    for _ in range(3):
        ls.ls_draft_verify(desc, big, *first, ws)
        ls.ls_draft_verify(sdesc, small, *args, count, out, lp, ws)
        got = count.cpu(), out.cpu(), lp.cpu(), m["kv_len"] - torch.tensor(m["counts"]) + count.cpu()
        check(m, got)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_tokens(cuda_device, dtype):
    m = make([3, 3, 2, 1], 777, dtype, seed=11)
    m["wide"][0, 5:] = -math.inf                       # five tokens are left
    m["wide"][3, :770] = LOW[dtype]
    m["wide"][6] = LOW[dtype]                          # all alike
    m["wide"][8, ::2] = -math.inf
    got = run(m)
    check(m, got)
    m["tokens"][1] = 700                               # a draft that the mask forbids
    m["u"][0] = 0.0
    got = run(m)
    check(m, got)
    assert got[0][0] == 1 and got[1][0] < 5


def test_rows_without_a_distribution(cuda_device):
    for value in (-math.inf, math.nan, math.inf):
        m = make([3, 1, 2], 4099, torch.bfloat16, seed=12)
        m["u"][:] = 0.0                                # every draft passes
        m["wide"][2] = value if value == -math.inf else m["wide"][2]
        m["wide"][2, 4098] = value
        m["wide"][3, 0] = value                        # with -infinity an ordinary masked token
        got = run(m, status=5)
        check(m, got)
        assert got[0].tolist()[0] == 2 and got[1][2] == -1 and got[3][0] == m["kv_len"][0]


def test_drafts_outside_the_vocabulary(cuda_device):
    for probs in (True, False):
        m = make([3, 3], 512, torch.float32, probs, seed=13)
        m["u"][:] = 0.0
        m["tokens"][2], m["tokens"][4] = 512, -1
        got = run(m, status=5)
        check(m, got)
        assert got[0].tolist() == [2, 1]


def test_sequences_that_are_left_out(cuda_device):
    m = make([2, 2, 2], 100, torch.float32, seed=14)
    for q_start, out_rows in (([0, 2, 4, 9], range(4, 6)), ([0, 4, 4, 6], range(0, 4)), ([0, 2, 1, 3], range(0, 0))):
        count, out, lp, keep = run(m, max_q=2, q_start=q_start, status=5)
        for b in range(3):
            n = q_start[b + 1] - q_start[b]
            if n < 0 or n > 2 or q_start[b + 1] > 6:
                assert count[b] == 0 and keep[b] == m["kv_len"][b]
        for r in out_rows:
            assert out[r] == -9 and lp[r] == -9
    # rows behind the last sequence stay
    count, out, lp, keep = run(m, q_start=[0, 2, 4, 4])
    assert out[4:].tolist() == [-9, -9] and lp[4:].tolist() == [-9, -9] and count[2] == 0
    m = make([0, 0], 100, torch.float32, seed=15)
    assert run(m)[0].tolist() == [0, 0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_far_apart_and_oddly_placed(cuda_device, dtype):
    """Element offsets past 2^31, and a first element at every place within 16 bytes."""
    v, stride = 3001, 1_200_000_001
    m = make([2, 1], v, dtype, False, seed=19)
    big = torch.empty(2 * stride + v + 16, dtype=dtype, device="cuda")
    want = run(m)
    check(m, want)
    for off in range(16 // dtype.itemsize):
        logits = big[off:].as_strided((3, v), (stride, 1))
        logits.copy_(m["wide"])
        desc = ls.verify_desc(logits, 2, 2)
        ws = torch.zeros(ls.ls_draft_verify_workspace_size(desc), dtype=torch.uint8, device="cuda")
        count, out = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int64, device="cuda")
        ls.ls_draft_verify(desc, logits, m["tokens"].cuda(), torch.tensor([0, 2, 3], dtype=torch.int32, device="cuda"), m["u"].cuda(),
                           m["u_next"].cuda(), count, out, None, ws)
        ls.ls_read_device_status(ws)
        assert torch.equal(count.cpu(), want[0]) and torch.equal(out.cpu(), want[1])


def test_scales_at_their_ends(cuda_device):
    """A very small scale makes all tokens alike, a very large one leaves the largest; logits far from zero."""
    m = make([1] * 6, 5003, torch.float32, False, seed=20)
    for scale in (2.0 ** -100, 2.0 ** 100):
        got = run(dict(m, scale=scale))
        if scale > 1:
            assert got[1].tolist() == m["wide"].argmax(1).tolist()
        else:
            assert all(abs(t - float(u) * 5003) <= 1 for t, u in zip(got[1].tolist(), m["u_next"]))
    masked = dict(m, scale=2.0 ** -100, wide=m["wide"].clone())
    masked["wide"][:, 10:] = -math.inf
    assert all(abs(t - float(u) * 10) <= 1 for t, u in zip(run(masked)[1].tolist(), m["u_next"]))
    far = dict(m, wide=(m["wide"] * 4).round() / 4 + 2.0 ** 20)   # the maximum's product leaves the grid of the draw
    check(far, run(far))
    near = dict(m, wide=(m["wide"] * 4).round() / 4)              # the same distribution near zero
    assert torch.equal(run(far)[1], run(near)[1])


def test_tokens_come_out_as_from_the_target(cuda_device):
    """The first token's distribution over 60,000 sequences: each count within 6 standard deviations."""
    n, g = 60000, torch.Generator().manual_seed(16)
    row, other = torch.randn(11, generator=g) * 1.5, torch.randn(11, generator=g)
    q = torch.softmax(other, 0)
    m = make([2] * n, 11, torch.float32, seed=17)
    m["wide"][:] = row
    m["probs"][:] = q
    m["tokens"] = torch.multinomial(q, 2 * n, replacement=True, generator=g)
    count, out, lp, _ = run(m)
    p = torch.softmax(row.double(), 0)
    seen = torch.bincount(out[::2], minlength=11).double()
    assert ((seen - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt()).all()
    accepted = float((count == 2).double().mean())
    rate = float(torch.minimum(p, q.double()).sum())
    assert abs(accepted - rate) <= 6 * math.sqrt(rate * (1 - rate) / n)


def test_graph(cuda_device):
    m = make([4, 1, 0, 3], 5000, torch.bfloat16, seed=18)
    assert all(torch.equal(a, b) for a, b in zip(run(m), run(m, graph=True)))
