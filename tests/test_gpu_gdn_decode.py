"""The recurrent step of the gated-DeltaNet state against its float64 definition.

Bounds, in roundings of u = 2^-24, with M the same recurrence over absolute values (every difference a
sum).  A token's update of S: the row product (16 FMAs of a lane, 3 sums over lanes) 19, exp(g) 4 (CUDA
gives expf within 2 ulp), a u, v - a u, b w and the last FMA 4: at most 27 of b |k| (|v| + M |k|), and 5 of
a M, so that n tokens put S off by at most 28 n u M, and o, through 19 more, by (28 n + 20) u M_o.  An
output in bf16 adds half a step."""
import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from oracle import drafts as ref

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


def make(counts, heads, key_heads, dtype, pad=0, n_states=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    n, b = sum(counts), len(counts)
    wide = torch.randn(n, (2 * key_heads + heads) * 128 + pad, generator=g)
    wide[:, :2 * key_heads * 128] *= 128 ** -0.5
    wide = wide.to(dtype)
    m = dict(q=wide[:, :key_heads * 128].unflatten(1, (key_heads, 128)),
             k=wide[:, key_heads * 128:2 * key_heads * 128].unflatten(1, (key_heads, 128)),
             v=wide[:, 2 * key_heads * 128:(2 * key_heads + heads) * 128].unflatten(1, (heads, 128)),
             g=torch.log(0.85 + 0.15 * torch.rand(n, heads, generator=g)),
             beta=0.05 + 0.9 * torch.rand(n, heads, generator=g),
             states=torch.randn(n_states or 2 * b, heads, 128, 128, generator=g) * 0.1,
             q_start=torch.tensor([sum(counts[:i]) for i in range(b + 1)], dtype=torch.int32))
    m["wide"] = wide
    return m


def on_gpu(m):
    """The tensors on the device, q, k and v as slices of one tensor."""
    wide = m["wide"].cuda()
    out = {n: t.cuda() for n, t in m.items()}
    at = 0
    for name in ("q", "k", "v"):
        size = m[name].shape[1] * 128
        out[name] = wide[:, at:at + size].unflatten(1, (m[name].shape[1], 128))
        at += size
    return out


def run(m, state_in, state_out, n_use=None, with_o=True, max_q=None, ws=None, stream=None):
    d = on_gpu(m)
    b = len(m["q_start"]) - 1
    counts = (m["q_start"][1:] - m["q_start"][:-1]).tolist()
    desc = ls.gdn_decode_desc(d["q"], d["k"], d["v"], d["states"], b, max_q or max(counts))
    o = torch.full(m["v"].shape, 7.0, dtype=m["v"].dtype, device="cuda") if with_o else None
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ls.ls_gdn_decode(desc, d["states"], d["q"], d["k"], d["v"], d["g"], d["beta"], d["q_start"], t(state_in),
                     t(state_out), o, ws, n_use=t(n_use), stream=stream)
    torch.cuda.synchronize()
    return (o.cpu() if with_o else None), d["states"].cpu()


def check(m, o, states, state_in, state_out, n_use=None):
    start = m["q_start"].tolist()
    want = m["states"].double()
    for b in range(len(start) - 1):
        n = start[b + 1] - start[b] if n_use is None else n_use[b]
        rows = slice(start[b], start[b] + n)
        s0 = m["states"][state_in[b]] if state_in[b] >= 0 else torch.zeros_like(m["states"][0])
        ob, sb, om, sm = ref.state_step(s0, m["q"][rows], m["k"][rows], m["v"][rows], m["g"][rows], m["beta"][rows])
        if o is not None:
            half = torch.finfo(o.dtype).eps / 2 if o.dtype != torch.float32 else 0.0
            bound = (28 * n + 20) * EPS * om
            assert ((o[rows].double() - ob).abs() <= bound + half * (ob.abs() + bound)).all()
            assert (o[start[b] + n:start[b + 1]] == 7).all()  # rows that are not used stay
        if state_out is not None and state_out[b] >= 0:
            err = (states[state_out[b]].double() - sb).abs()
            assert (err <= 28 * n * EPS * sm).all(), float((err / sm).max())
            want[state_out[b]] = states[state_out[b]].double()
    assert torch.equal(want, states.double())  # no other slot changed


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("counts,heads,key_heads,pad", [
    ([1], 1, 1, 0), ([1, 1, 1], 4, 2, 8), ([1, 0, 5, 2], 6, 2, 128), ([8, 9, 0, 1, 17], 2, 1, 16), ([33], 3, 3, 0)])
def test_steps(cuda_device, dtype, counts, heads, key_heads, pad):
    m = make(counts, heads, key_heads, dtype, pad, seed=len(counts))
    b = len(counts)
    ins, outs = list(range(b)), list(range(2 * b - 1, b - 1, -1))
    o, states = run(m, ins, outs)
    check(m, o, states, ins, outs)
    o2, states2 = run(m, ins, ins)                     # in place: the same numbers
    assert torch.equal(o, o2) and all(torch.equal(states[outs[i]], states2[i]) for i in range(b))
    o3, states3 = run(m, ins, None)                    # a state that stays
    assert torch.equal(o, o3) and torch.equal(states3, m["states"])
    _, states4 = run(m, ins, outs, with_o=False)
    assert torch.equal(states, states4)


def test_accepted_tokens_move_the_state_on(cuda_device):
    counts, use = [4, 6, 1, 3], [2, 6, 0, 1]
    m = make(counts, 4, 4, torch.float32, seed=5)
    ins, outs = [0, 1, 2, 3], [0, 5, 6, -1]
    o, states = run(m, ins, outs, n_use=use)
    check(m, o, states, ins, outs, use)


def test_fork_from_one_state_and_from_zeros(cuda_device):
    m = make([1, 1, 0, 2], 2, 2, torch.bfloat16, seed=6, n_states=9)
    ins, outs = [8, 8, 8, -1], [0, 1, 2, 3]
    o, states = run(m, ins, outs)
    check(m, o, states, ins, outs)
    assert torch.equal(states[2], m["states"][8])      # no token: a copy


def test_no_tokens_at_all(cuda_device):
    """Sequences without a token move their states only; nothing else is read."""
    states = torch.randn(6, 3, 128, 128, device="cuda")
    want = states.clone()
    e = torch.empty((0, 3, 128), device="cuda")
    z = torch.empty((0, 3), device="cuda")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    desc = ls.gdn_decode_desc(e, e, e, states, 3, 0)
    ls.ls_gdn_decode(desc, states, e, e, e, z, z, ints(0, 0, 0, 0), ints(0, 1, -1), ints(4, -1, 5), e)
    want[4], want[5] = want[0], 0
    assert torch.equal(states, want)


def test_states_far_into_a_pool(cuda_device):
    """Element offsets past 2^31: slots of 64 heads, 1 M elements each."""
    n = 2100
    m = make([1, 2], 64, 32, torch.bfloat16, seed=12, n_states=2)
    d = on_gpu(m)
    states = torch.empty((n, 64, 128, 128), device="cuda")
    states[n - 1], states[0] = d["states"][0], d["states"][1]
    desc = ls.gdn_decode_desc(d["q"], d["k"], d["v"], states, 2, 2)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    o = torch.empty(m["v"].shape, dtype=torch.bfloat16, device="cuda")
    ls.ls_gdn_decode(desc, states, d["q"], d["k"], d["v"], d["g"], d["beta"], d["q_start"], ints(n - 1, 0), ints(n - 2, n - 1 - 1024), o)
    want_o, want = run(dict(m, states=torch.cat([m["states"], torch.zeros_like(m["states"])])), [0, 1], [2, 3])
    assert torch.equal(o.cpu(), want_o)
    assert torch.equal(states[n - 2].cpu(), want[2]) and torch.equal(states[n - 1 - 1024].cpu(), want[3])


def test_step_by_step_is_one_call(cuda_device):
    """Tokens one call at a time give what one call gives, bit for bit."""
    m = make([5, 5], 2, 1, torch.float32, seed=7)
    o, states = run(m, [0, 1], [0, 1])
    cur = m["states"]
    for t in range(5):
        part = {n: x[[t, 5 + t]] if n in ("g", "beta", "wide") else x for n, x in m.items()}
        part |= {n: m[n][[t, 5 + t]] for n in ("q", "k", "v")}
        part |= dict(states=cur, q_start=torch.tensor([0, 1, 2], dtype=torch.int32))
        ot, cur = run(part, [0, 1], [0, 1])
        assert torch.equal(ot, o[[t, 5 + t]])
    assert torch.equal(cur[:2], states[:2])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_sequences_are_those_of_a_few(cuda_device, dtype):
    """Far more units of work than the device holds at once, of all lengths, some of them none, two such calls
    side by side: each sequence's bits are those it has in a call of ten."""
    b, heads = 90, 16
    g = torch.Generator().manual_seed(21)
    counts = torch.randint(0, 8, (b,), generator=g).tolist()
    m = make(counts, heads, 8, dtype, n_states=2 * b, seed=22)
    d = on_gpu(m)
    n = sum(counts)
    ins, outs = torch.arange(b, dtype=torch.int32), torch.arange(b, 2 * b, dtype=torch.int32)
    ins[5], outs[7:9], ins[11] = -1, -1, 10000        # from zeros, not kept, left out
    args, ins, outs = (d["q"], d["k"], d["v"], d["g"], d["beta"]), ins.cuda(), outs.cuda()

    def call(first, end, states, o, stream=None):
        at = d["q_start"][first:end + 1]
        desc = ls.gdn_decode_desc(d["q"], d["k"], d["v"], states, end - first, 7 if end - first == b else n)
        ls.ls_gdn_decode(desc, states, *args, at, ins[first:end], outs[first:end], o, stream=stream)

    def fresh():
        return d["states"].clone(), torch.full(m["v"].shape, 7.0, dtype=dtype, device="cuda")

    few, many, other = fresh(), fresh(), fresh()
    for first in range(0, b, 10):
        call(first, first + 10, *few)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for s, (states, o) in zip(streams, (many, other)):
        for _ in range(3):
            call(0, b, states, o, stream=s)
    torch.cuda.synchronize()
    for states, o in (many, other):
        assert torch.equal(o, few[1]) and torch.equal(states, few[0])


def test_agrees_with_the_replay(cuda_device):
    """A response replayed from the captured state is the same tokens stepped from it."""
    m = make([20], 3, 3, torch.float32, seed=8)
    o, states = run(m, [0], [1])
    d = on_gpu(m)
    ro, rs = torch.empty(20, 3, 128, device="cuda"), torch.empty(1, 3, 128, 128, device="cuda")
    ls.ls_gdn_replay_fwd(d["states"][0], d["q"].contiguous(), d["k"].contiguous(), d["v"].contiguous(), d["g"], d["beta"], ro, rs)
    assert (ro.cpu() - o).abs().max() <= 1e-5 * o.abs().max()
    assert (rs[0].cpu() - states[1]).abs().max() <= 1e-5 * states[1].abs().max()


def test_sequences_out_of_range_are_left_out(cuda_device):
    m = make([2, 2, 2, 2], 2, 2, torch.float32, seed=9)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for ins, outs, use, max_q in (([0, 99, -2, 3], [4, 5, 6, 7], None, None), ([0, 1, 2, 3], [4, 5, 6, 7], [2, 3, -1, 2], None)):
        o, states = run(m, ins, outs, use, ws=ws)
        with pytest.raises(ls.LsError) as e:
            ls.ls_read_device_status(ws)
        assert e.value.status == 5
        assert (o[2:6] == 7).all() and torch.equal(states[5:7], m["states"][5:7])
        part = dict(m, q_start=torch.tensor([0, 2], dtype=torch.int32))
        check(part, o[:2], torch.cat([m["states"][:4], states[4:5], m["states"][5:]]), [0], [4])
    # a slot past the pool is not written, the tokens' results are
    o, states = run(m, [0, 1, 2, 3], [99, 5, 6, 7], ws=ws)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    check(m, o, states, [0, 1, 2, 3], [-1, 5, 6, 7])
    # a range of tokens past the end, and a sequence longer than max_q
    bad = dict(m, q_start=torch.tensor([0, 2, 4, 6, 9], dtype=torch.int32))
    o, states = run(bad, [0, 1, 2, 3], [4, 5, 6, 7], max_q=2, ws=ws)
    with pytest.raises(ls.LsError):
        ls.ls_read_device_status(ws)
    assert (o[6:] == 7).all() and torch.equal(states[7], m["states"][7])


def test_decay_of_zero_and_values_that_are_not_finite(cuda_device):
    m = make([2, 2], 2, 2, torch.float32, seed=10)
    m["g"][0] = -float("inf")                          # forgets everything before
    m["v"][2, 0, 5] = float("nan")                     # one row of one head of the second sequence
    o, states = run(m, [0, 1], [2, 3])
    clean = dict(m, states=m["states"].clone())
    clean["states"][0] = 0
    o2, states2 = run(clean, [0, 1], [2, 3])
    assert torch.equal(o[:2], o2[:2]) and torch.equal(states[2], states2[2])
    bad = o[2:].isnan()
    assert bad[:, 0, 5].all() and bad.sum() == 2 and states[3].isnan().sum() == 128


def test_graph_and_stream(cuda_device):
    m = make([1, 3], 2, 2, torch.bfloat16, seed=11)
    want, _ = run(m, [0, 1], None)
    d = on_gpu(m)
    desc = ls.gdn_decode_desc(d["q"], d["k"], d["v"], d["states"], 2, 3)
    o = torch.zeros(m["v"].shape, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            ls.ls_gdn_decode(desc, d["states"], d["q"], d["k"], d["v"], d["g"], d["beta"], d["q_start"], slots, None, o)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o.cpu(), want)
