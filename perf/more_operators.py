"""The operators of a rollout with drafted tokens, as cases that can be measured.

Three operators stand next to the cache, the cached attention and the scoring:

* the pages of a paged cache: sequences advance (drop rejected tokens, take pages
  for new ones, copy a page that they share before writing into it), fork a
  prompt, and the pool is compacted;
* verification of drafted tokens against the target's logits, from given random
  numbers, with the draw of the next token;
* the recurrent step of the gated-DeltaNet state for one or a few tokens of each
  sequence.

`own = False` computes them with elementary torch operations; `own = True` makes
the calls a user makes of the library.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A group of eight decodes one token each over large pages (latency).
        dict(name="step_group", op="step", batch=8, page=256, per_seq=64, spare=448, q_min=1, q_max=1, drop=0, mix=1),
        # A rollout server's step: sequences of all lengths drop rejected drafts and take slots for the next ones, small pages.
        dict(name="step_drafts", op="step", batch=384, page=16, per_seq=512, spare=32771, q_min=0, q_max=6, drop=5, mix=2),
        # Sixteen members fork a long prompt that ends inside a page, and take their first token's slot.
        dict(name="fork_group", op="fork", batch=16, prompt=100003, page=256, fmt="e4m3", hkv=4, d=256, spare=77, mix=3),
        # The same in bf16 with small pages and many members, a short prompt.
        dict(name="fork_many", op="fork", batch=200, prompt=1717, page=64, fmt="bf16", hkv=8, d=128, spare=301, mix=4),
        # Half of the sequences have ended: the others' pages move to the front of the pool.
        dict(name="compact_pool", op="compact", batch=24, page=256, per_seq=128, pages=3001, fmt="e4m3", hkv=4, d=256, mix=5),
        # A few sequences' drafts against a small float32 vocabulary (latency), drafts looked up rather than drawn.
        dict(name="verify_lookup", op="verify", batch=5, q_min=1, q_max=6, vocab=8191, dtype="f32", probs=False, scale=1.0, pad=0, mix=6),
        # A server's step: up to four drafts a sequence, drawn from a small model, one sequence idle.
        dict(name="verify_server", op="verify", batch=64, q_min=0, q_max=5, vocab=128000, dtype="bf16", probs=True, scale=1.0, pad=0, mix=7),
        # One token drawn for each of many sequences, an odd vocabulary, a sampling temperature.
        dict(name="draw_one", op="verify", batch=256, q_min=1, q_max=1, vocab=50003, dtype="bf16", probs=False, scale=1.25, pad=0, mix=8),
        # One sequence's token through a recurrent layer (latency).
        dict(name="state_one", op="state", batch=1, q_min=1, q_max=1, heads=32, key_heads=16, dtype="bf16", pad=128, mode="step", mix=9),
        # A server's step of one token each: every state is read and written.
        dict(name="state_step", op="state", batch=96, q_min=1, q_max=1, heads=32, key_heads=16, dtype="bf16", pad=128, mode="step", mix=10),
        # Drafted tokens run ahead of the state, which stays.
        dict(name="state_drafts", op="state", batch=64, q_min=1, q_max=6, heads=32, key_heads=32, dtype="f32", pad=0, mode="look", mix=11),
        # The accepted ones among them move the state on.
        dict(name="state_commit", op="state", batch=64, q_min=1, q_max=6, heads=32, key_heads=32, dtype="f32", pad=0, mode="commit", mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "fork", "compact", "verify", "verify", "state", "state"])
    case = dict(op=op, mix=rng.randrange(10**6))
    if op == "step":
        q_hi = rng.choice([1, 1, rng.randint(2, 8), _log_int(rng, 9, 512)])
        page = rng.choice([16, 48, 64, 128, 256])
        batch = _log_int(rng, 1, 512)
        return case | dict(batch=batch, page=page, per_seq=_log_int(rng, 4, max(8, 131072 // batch)) + -(-q_hi // page),
                           spare=batch * (1 + -(-q_hi // page)) + _log_int(rng, 8, 40000), q_min=rng.choice([0, 1, q_hi]), q_max=q_hi,
                           drop=rng.choice([0, rng.randint(1, 7)]))
    if op in ("fork", "compact"):
        fmt = rng.choice(["e4m3", "e4m3", "bf16", "f32"])
        hkv, d = rng.choice([(4, 256), (4, 256), (8, 128), (1, 64), (3, 128)])
        page = rng.choice([16, 48, 64, 128, 256])
        size = 2 * hkv * d * page * dict(e4m3=1, bf16=2, f32=4)[fmt]
        batch = _log_int(rng, 2, 128)
        case |= dict(batch=batch, page=page, fmt=fmt, hkv=hkv, d=d)
        most = 1500 * 2**20 // size  # pages of a pool
        if op == "fork":
            spare = 2 * batch + rng.randint(1, 400)
            return case | dict(prompt=_log_int(rng, 1, page * min(most - min(spare, most - 1), 1024)), spare=spare)
        pages = _log_int(rng, 8, min(most, 20000))
        return case | dict(pages=pages, per_seq=max(1, 2 * pages // (3 * batch)) + rng.randint(0, 3))
    if op == "verify":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        vocab = _log_int(rng, 500, 160000)
        q_hi = rng.choice([1, rng.randint(2, 9)])
        most = 64 * 5 * 128000 // (vocab * q_hi * (1 if dtype == "bf16" else 2))
        return case | dict(batch=_log_int(rng, 1, max(1, min(256, most))), q_min=rng.choice([0, 1, q_hi]), q_max=q_hi, vocab=vocab, dtype=dtype,
                           probs=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 0.7, 1.4]), pad=rng.choice([0, 0, 5, 64]))
    heads, key_heads = rng.choice([(32, 16), (32, 32), (16, 16), (48, 16), (4, 2)])
    mode = rng.choice(["step", "look", "commit"])
    q_hi = 1 if mode == "step" else rng.randint(2, 16)
    return case | dict(batch=_log_int(rng, 1, 96 * 32 // heads // (1 if q_hi < 9 else 2)), q_min=rng.choice([0, 1]), q_max=q_hi, heads=heads, key_heads=key_heads,
                       dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 8, 128]), mode=mode)


def _counts(case):
    """Tokens of each sequence in this step: both ends of the range occur where there are two sequences."""
    rng = random.Random(case["mix"])
    n = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    n[0] = case["q_max"]
    if len(n) > 1:
        n[-1] = case["q_min"]
    return n


def _lengths(case):
    """Tokens in the cache of each sequence before a step or a compaction."""
    rng = random.Random(case["mix"] + 1)
    room = case["per_seq"] * case["page"] - (case["q_max"] if case["op"] == "step" else 0)
    n = [rng.randint(min(room, case.get("drop", 0)), room) for _ in range(case["batch"])]
    if case["op"] == "compact":  # every second sequence has ended
        n = [0 if b % 2 else max(1, m) for b, m in enumerate(n)]
        while sum(-(-m // case["page"]) for m in n) > case["pages"]:
            n = [m // 2 for m in n]
    return n


def _row_bytes(case):
    return 2 * case["hkv"] * (case["d"] * dict(e4m3=1, bf16=2, f32=4)[case["fmt"]] + (1 if case["fmt"] == "e4m3" else 0))


def work(case):
    if case["op"] == "step":
        pages = sum(-(-n // case["page"]) for n in _lengths(case)) + case["spare"]
        return dict(bytes=4 * pages + 28 * case["batch"] + 8 * sum(_counts(case)), flops=pages)
    if case["op"] == "fork":
        pages = -(-case["prompt"] // case["page"])
        rows = case["prompt"] % case["page"]
        return dict(bytes=(1 + case["batch"]) * rows * _row_bytes(case) + 4 * pages * (2 + case["batch"]) + 40 * case["batch"], flops=pages * case["batch"])
    if case["op"] == "compact":
        live = sum(-(-n // case["page"]) for n in _lengths(case))
        moved = live * (case["pages"] - live) // case["pages"]  # live pages lie anywhere in the pool
        return dict(bytes=2 * moved * case["page"] * _row_bytes(case) + 8 * case["pages"] + 8 * live, flops=case["pages"])
    counts = _counts(case)
    n = sum(counts)
    if case["op"] == "verify":
        rows = n * case["vocab"] * (2 if case["dtype"] == "bf16" else 4)
        more = 4 * (n + case["vocab"] * sum(c > 1 for c in counts)) if case["probs"] else 0
        return dict(bytes=rows + more + 24 * n + 32 * case["batch"], flops=3 * n * case["vocab"])
    wide = 2 if case["dtype"] == "bf16" else 4
    tokens = n * (case["heads"] * (128 * wide * (2 if case["mode"] != "commit" else 1) + 8) + case["key_heads"] * 256 * wide)
    # a state is copied on where its sequence has no token, but not read for nothing
    states = (sum(c > 0 for c in counts) if case["mode"] == "look" else 2 * case["batch"]) * case["heads"] * 65536
    return dict(bytes=states + tokens, flops=7 * 128 * 128 * case["heads"] * n)


# ---------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _starts(n, dev):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)


def _pools(case, pages, g):
    shape = (pages, case["hkv"], case["page"], case["d"])
    pools, exps = [], [None, None]
    for i in range(2):
        if case["fmt"] == "e4m3":
            codes = torch.randint(0, 0x78, shape, generator=g, device=g.device, dtype=torch.uint8)
            pools.append(codes.view(torch.float8_e4m3fn))
            exps[i] = torch.randint(-9, -5, shape[:3], generator=g, device=g.device, dtype=torch.int8)
        else:
            pools.append(torch.randn(shape, generator=g, device=g.device, dtype=_TYPES[case["fmt"]]))
    return pools, exps


def _book(lengths, per_seq, pages, g):
    """(page table, lengths, references): each sequence's pages anywhere in the pool."""
    dev = g.device
    table = torch.zeros((len(lengths), per_seq), dtype=torch.int32, device=dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    at = 0
    for b, n in enumerate(lengths):
        table[b, :n] = order[at:at + n]
        at += n
    refs[order[:at].long()] = 1
    return table, refs


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case, kept={})  # kept: what the library's user makes once: descriptors and workspaces
    page = case.get("page", 0)
    if case["op"] == "step":
        lengths, counts = _lengths(case), _counts(case)
        used = [-(-n // page) for n in lengths]
        s["table"], s["refs"] = _book(used, case["per_seq"], sum(used) + case["spare"], g)
        s["kv_len"] = torch.tensor(lengths, dtype=torch.int64, device=dev)
        drop = torch.randint(0, case["drop"] + 1, (case["batch"],), generator=g, device=dev)
        s["keep"] = s["kv_len"] - torch.minimum(drop, s["kv_len"])
        s["q_start"] = _starts(counts, dev)
        s["slots"] = torch.empty(sum(counts), dtype=torch.int64, device=dev)
        s["copies"] = torch.empty((case["batch"], 3), dtype=torch.int32, device=dev)
        s["seqs"] = None
    elif case["op"] == "fork":
        # row 0 holds the prompt; the others hold what the group before this one left
        n = -(-case["prompt"] // page)
        b = case["batch"]
        last = [random.Random(case["mix"] + i).randint(0, min(n, case["spare"] // b - 1)) for i in range(b)]
        s["table"], s["refs"] = _book([n] + last, n + 1, n + case["spare"], g)
        s["kv_len"] = torch.tensor([case["prompt"]] + [m * page for m in last], dtype=torch.int64, device=dev)
        s["src"] = torch.zeros(b, dtype=torch.int32, device=dev)
        s["seqs"] = torch.arange(1, b + 1, dtype=torch.int32, device=dev)
        s["keep"] = None
        s["q_start"] = torch.arange(b + 1, dtype=torch.int32, device=dev)
        s["slots"] = torch.empty(b, dtype=torch.int64, device=dev)
        s["copies"] = torch.empty((b, 3), dtype=torch.int32, device=dev)
        s["pools"], s["exps"] = _pools(case, n + case["spare"], g)
    elif case["op"] == "compact":
        lengths = _lengths(case)
        s["table"], s["refs"] = _book([-(-n // page) for n in lengths], case["per_seq"], case["pages"], g)
        s["kv_len"] = torch.tensor(lengths, dtype=torch.int64, device=dev)
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["copies"] = torch.empty((case["pages"] // 2, 3), dtype=torch.int32, device=dev)
        s["pools"], s["exps"] = _pools(case, case["pages"], g)
    elif case["op"] == "verify":
        counts, v = _counts(case), case["vocab"]
        n, dt = sum(counts), _TYPES[case["dtype"]]
        wide = torch.randn((n, v + case["pad"]), generator=g, device=dev, dtype=torch.float32).mul_(2.5)
        s["logits"] = wide.to(dt)[:, :v]
        s["q_start"] = _starts(counts, dev)
        s["kv_len"] = torch.randint(16, 32768, (case["batch"],), generator=g, device=dev)
        s["u"] = torch.rand(n, generator=g, device=dev)
        s["u_new"] = torch.rand(case["batch"], generator=g, device=dev)
        s["tokens"] = torch.randint(0, v, (n,), generator=g, device=dev)
        # drafts come from a smaller model: its logits are the target's with noise
        draft = s["logits"].float().add_(torch.randn((n, v), generator=g, device=dev, dtype=torch.float32), alpha=0.7)
        q = torch.softmax(draft.mul_(case["scale"]), 1)
        if n > 1:  # token r + 1 is drawn after row r
            pick = torch.multinomial(q[:-1], 1, generator=g)[:, 0] if case["probs"] else q[:-1].argmax(1)
            s["tokens"][1:] = pick
        s["probs"] = q if case["probs"] else None
        s["count"] = torch.empty(case["batch"], dtype=torch.int32, device=dev)
        s["out"] = torch.empty(n, dtype=torch.int64, device=dev)
        s["logp"] = torch.empty(n, device=dev)
        s["keep"] = torch.empty(case["batch"], dtype=torch.int64, device=dev)
        s["max_q"] = max(counts)
    else:
        counts = _counts(case)
        n, h, hk, b = sum(counts), case["heads"], case["key_heads"], case["batch"]
        dt = _TYPES[case["dtype"]]
        # rows of a projection that holds q, k, v and a gate; q and k of unit length
        wide = torch.randn((n, (2 * hk + h) * 128 + case["pad"]), generator=g, device=dev)
        qk = wide[:, :2 * hk * 128].unflatten(1, (2 * hk, 128))
        qk /= qk.norm(dim=2, keepdim=True)
        qk[:, :hk] *= 128 ** -0.5
        wide = wide.to(dt)
        s["q"], s["k"] = (wide[:, i * hk * 128:(i + 1) * hk * 128].unflatten(1, (hk, 128)) for i in range(2))
        s["v"] = wide[:, 2 * hk * 128:(2 * hk + h) * 128].unflatten(1, (h, 128))
        s["g"] = torch.log(0.85 + 0.15 * torch.rand((n, h), generator=g, device=dev))
        s["beta"] = 0.05 + 0.9 * torch.rand((n, h), generator=g, device=dev)
        # a step goes on from a slot to another one, so that a sequence can go back
        write = case["mode"] != "look"
        s["states"] = torch.randn(((2 if write else 1) * b, h, 128, 128), generator=g, device=dev) * 0.1
        order = torch.randperm(len(s["states"]), generator=g, device=dev).to(torch.int32)
        s["state_in"], s["state_out"] = order[:b].contiguous(), order[b:].contiguous() if write else None
        s["q_start"] = _starts(counts, dev)
        s["n_use"] = None
        if case["mode"] == "commit":
            n_tok = s["q_start"][1:] - s["q_start"][:-1]
            s["n_use"] = torch.minimum(n_tok, torch.randint(1, case["q_max"] + 1, (b,), generator=g, device=dev)).to(torch.int32)
        s["o"] = torch.empty((n, h, 128), device=dev, dtype=dt) if case["mode"] != "commit" else None
        s["max_q"] = max(counts)
    return s


# ---------------------------------------------------------------- plain forms
def _per(n, page):
    return (n + page - 1) // page


def _advance_plain(s):
    page, refs = s["case"]["page"], s["refs"]
    pages = refs.shape[0]
    seqs = slice(None) if s["seqs"] is None else s["seqs"].long()
    rows, old = s["table"][seqs].long(), s["kv_len"][seqs]
    keep = old if s["keep"] is None else s["keep"]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    new = keep + n
    have, want = _per(keep, page), _per(new, page)
    at = torch.arange(rows.shape[1], device=rows.device)
    gone = (at >= have[:, None]) & (at < _per(old, page)[:, None])
    refs.scatter_add_(0, torch.where(gone, rows, 0).flatten(), -gone.flatten().int())
    last = rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    shared = (keep % page != 0) & (n > 0) & (refs[last] > 1)
    first = have - shared.long()                    # new entries of the table begin here
    need = want - first
    upto = need.cumsum(0)
    free = refs == 0
    rank = free.cumsum(0) - 1
    ids = torch.zeros(pages + 1, dtype=torch.int64, device=rows.device)
    ids.scatter_(0, torch.where(free, rank, pages), torch.arange(pages, device=rows.device))
    served = (need == 0) | (upto <= free.sum())
    begin = upto - need
    take = (at >= first[:, None]) & (at < want[:, None]) & served[:, None]
    got = ids[(begin[:, None] + at - first[:, None]).clamp(0, pages)]
    moved = shared & served
    refs.scatter_add_(0, torch.where(moved, last, 0), -moved.int())
    refs.scatter_add_(0, torch.where(take, got, 0).flatten(), take.flatten().int())
    rows = torch.where(take, got, rows)
    s["table"][seqs] = rows.int()
    s["kv_len"][seqs] = torch.where(served, new, keep)
    copy = torch.stack([last, ids[begin.clamp(0, pages)], keep % page], 1)
    s["copies"].copy_(torch.where(moved[:, None], copy, -1))
    t = torch.arange(s["slots"].shape[0], device=rows.device)
    b = (t[:, None] >= s["q_start"][None, 1:]).sum(1)
    pos = keep[b] + t - s["q_start"][b]
    slot = rows[b, (pos // page).clamp(max=rows.shape[1] - 1)] * page + pos % page
    s["slots"].copy_(torch.where(served[b], slot, -1))
    return [s["slots"], s["table"], s["kv_len"], s["refs"], s["copies"]]


def _copy_plain(s):
    c = s["copies"][s["copies"][:, 1] >= 0].long()
    pools = s["pools"] + [e for e in s["exps"] if e is not None]
    at = torch.arange(s["case"]["page"], device=c.device)
    rows = at < c[:, 2, None]
    for p in pools:
        x = p.view(torch.uint8) if p.dtype == torch.float8_e4m3fn else p
        x[c[:, 1]] = torch.where(rows[:, None, :, None] if x.dim() == 4 else rows[:, None, :], x[c[:, 0]], x[c[:, 1]])
    return pools


def _fork_plain(s):
    page, refs, table = s["case"]["page"], s["refs"], s["table"]
    src, dst = s["src"].long(), s["seqs"].long()
    at = torch.arange(table.shape[1], device=table.device)
    rows, old = table[src].long(), table[dst].long()
    gone = at < _per(s["kv_len"][dst], page)[:, None]
    refs.scatter_add_(0, torch.where(gone, old, 0).flatten(), -gone.flatten().int())
    held = at < _per(s["kv_len"][src], page)[:, None]
    refs.scatter_add_(0, torch.where(held, rows, 0).flatten(), held.flatten().int())
    table[dst] = torch.where(held, rows, old).int()
    s["kv_len"][dst] = s["kv_len"][src]
    return _advance_plain(s) + _copy_plain(s)


def _compact_plain(s):
    page, refs, table = s["case"]["page"], s["refs"], s["table"].long()
    pages, cap = refs.shape[0], s["copies"].shape[0]
    at = torch.arange(pages, device=refs.device)
    live = refs > 0
    n = live.sum()
    high, low = live & (at >= n), ~live & (at < n)
    # the k-th of the high ones goes to the k-th of the low ones
    to = torch.zeros(pages + 1, dtype=torch.int64, device=refs.device).scatter_(0, torch.where(low, low.cumsum(0) - 1, pages), at)
    frm = torch.zeros_like(to).scatter_(0, torch.where(high, high.cumsum(0) - 1, pages), at)
    goes = torch.where(high, to[high.cumsum(0) - 1], at)
    comes = torch.where(low, frm[low.cumsum(0) - 1], at)
    s["refs_out"].copy_(torch.where(at < n, refs[comes], 0))
    used = torch.arange(table.shape[1], device=refs.device) < _per(s["kv_len"], page)[:, None]
    s["table_out"].copy_(torch.where(used, goes[table], table))
    moves = torch.stack([frm[:cap], to[:cap], torch.full_like(at[:cap], page)], 1)
    s["copies"].copy_(torch.where((at[:cap] < high.sum())[:, None], moves, -1))
    return [s["table_out"], s["refs_out"], s["copies"]] + _copy_plain(s)


def _verify_plain(s):
    case, v = s["case"], s["case"]["vocab"]
    start, tokens = s["q_start"].long(), s["tokens"]
    n, b = tokens.shape[0], case["batch"]
    scale = case["scale"]
    x = s["logits"].float() * scale
    top = x.amax(1, keepdim=True)
    lse = ((x - top).exp().sum(1, keepdim=True).log() + top)[:, 0]
    r = torch.arange(n, device=x.device)
    seq = (r[:, None] >= start[None, 1:]).sum(1)
    drafted = r + 1 < start[seq + 1]
    nxt = torch.where(drafted, tokens[(r + 1).clamp(max=n - 1)], 0)
    p = (x[r, nxt] - lse).double().exp()
    q = s["probs"][r, nxt].double() if s["probs"] is not None else torch.ones_like(p)
    fails = drafted & ~(s["u"].double() * q < p)
    # drafts before the first that fails
    place = r - start[seq]
    count = start[1:] - start[:-1]
    stop = (count - 1).scatter_reduce(0, seq, torch.where(fails, place, n), "amin")
    some = count > 0
    row = torch.where(some, start[:-1] + stop, 0)
    rejected = some & (stop < count - 1)
    # the new token of each sequence: its row again in 64 bits
    z = s["logits"][row].double() * scale
    w = (z - z.amax(1, keepdim=True)).exp()
    w = w / w.sum(1, keepdim=True)
    if s["probs"] is not None:
        taken = s["probs"][row].double()
    else:
        taken = torch.zeros_like(w).scatter_(1, nxt[row][:, None], 1.0)
    rest = torch.where(rejected[:, None], (w - taken).clamp(min=0), w)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
    upto = rest.cumsum(1)
    new = (upto <= s["u_new"].double()[:, None] * upto[:, -1:]).sum(1).clamp(max=v - 1)
    s["count"].copy_(torch.where(some, stop + 1, 0))
    s["keep"].copy_(torch.where(some, s["kv_len"] - count + stop + 1, s["kv_len"]))
    emitted = torch.where(place < stop[seq], nxt, new[seq])
    held = place <= stop[seq]
    s["logp"].copy_(torch.where(held, x[r, emitted] - lse, 0.0))
    s["out"].copy_(torch.where(held, emitted, -1))
    return [s["count"], s["out"], s["logp"], s["keep"]]


def _state_plain(s):
    """All tokens of a sequence at once: with c the running sum of g and e_t = b_t (v_t - exp(g_t) S_{t-1} k_t), the e solve
    (I + N) E = b (V - exp(c) K S_0^T), N_ts = b_t exp(c_t - c_s) k_t.k_s for s < t, and S_t = exp(c_t) S_0 + sum exp(c_t - c_s) e_s k_s^T."""
    case = s["case"]
    start, m = s["q_start"].long(), s["max_q"]
    count = start[1:] - start[:-1]
    if s["n_use"] is not None:
        count = torch.minimum(count, s["n_use"])
    i = torch.arange(m, device=start.device)
    there = i < count[:, None]
    row = torch.where(there, start[:-1, None] + i, 0)
    each = case["heads"] // case["key_heads"]
    q, k, v = (s[name].float()[row].transpose(1, 2) for name in ("q", "k", "v"))   # [b, heads, m, 128]
    q, k = q.repeat_interleave(each, 1), k.repeat_interleave(each, 1)
    c = torch.where(there[..., None], s["g"][row], 0.0).cumsum(1).transpose(1, 2)  # [b, heads, m]
    beta = torch.where(there[..., None], s["beta"][row], 0.0).transpose(1, 2)
    s0 = s["states"][s["state_in"].long()]
    decay = (c[..., :, None] - c[..., None, :]).tril().exp().tril()
    nil = ((k @ k.transpose(-1, -2)) * decay).tril(-1) * beta[..., None]
    gamma = c.exp()[..., None]
    e = beta[..., None] * (v - gamma * (k @ s0.transpose(-1, -2)))
    two = nil @ nil
    four = two @ two
    e = e + four @ (four @ e)                       # (I + N)^-1 = (I - N)(I + N^2)(I + N^4)(I + N^8) for up to 16 tokens
    e = e + four @ e
    e = e + two @ e
    e = e - nil @ e
    out = []
    if s["o"] is not None:
        o = gamma * (q @ s0.transpose(-1, -2)) + ((q @ k.transpose(-1, -2)) * decay) @ e
        s["o"].copy_(o.transpose(1, 2)[there].to(s["o"].dtype))
        out.append(s["o"])
    if s["state_out"] is not None:
        some = count > 0
        new = gamma[:, :, -1:] * s0 + (e * decay[:, :, -1, :, None]).transpose(-1, -2) @ k
        s["states"][s["state_out"].long()] = torch.where(some[:, None, None, None], new, s0)
        out.append(s["states"])
    return out


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    from long_context_grpo_replay_gb300 import binding as ls
    case, kept = s["case"], s["kept"]
    if case["op"] in ("step", "fork", "compact"):
        if not kept:
            kept["book"] = ls.page_book(s["refs"], s["table"], s["kv_len"], case["page"])
            kept["ws"] = torch.zeros(ls.ls_pages_workspace_size(kept["book"]), dtype=torch.uint8, device=s["refs"].device)
            if "pools" in s:
                kept["cache"] = ls.kv_cache_from(s["pools"][0], s["pools"][1], s["exps"][0], s["exps"][1])
                kept["pools"] = s["pools"] + [e for e in s["exps"] if e is not None]
        if case["op"] == "compact":
            ls.ls_pages_compact(kept["book"], s["table_out"], s["refs_out"], s["copies"], kept["ws"])
            ls.ls_cache_copy_pages(kept["cache"], s["copies"], kept["ws"])
            return [s["table_out"], s["refs_out"], s["copies"]] + kept["pools"]
        if case["op"] == "fork":
            ls.ls_pages_fork(kept["book"], s["src"], s["seqs"], kept["ws"])
        ls.ls_pages_advance(kept["book"], s["q_start"], s["slots"], s["copies"], kept["ws"], seqs=s["seqs"], keep=s["keep"])
        out = [s["slots"], s["table"], s["kv_len"], s["refs"], s["copies"]]
        if case["op"] == "fork":
            ls.ls_cache_copy_pages(kept["cache"], s["copies"], kept["ws"])
            out += kept["pools"]
        return out
    if case["op"] == "verify":
        if not kept:
            kept["desc"] = ls.verify_desc(s["logits"], case["batch"], s["max_q"], draft_probs=s["probs"], logit_scale=case["scale"])
            kept["ws"] = torch.zeros(ls.ls_draft_verify_workspace_size(kept["desc"]), dtype=torch.uint8, device=s["logits"].device)
        ls.ls_draft_verify(kept["desc"], s["logits"], s["tokens"], s["q_start"], s["u"], s["u_new"], s["count"], s["out"], s["logp"], kept["ws"],
                           draft_probs=s["probs"], kv_len=s["kv_len"], keep=s["keep"])
        return [s["count"], s["out"], s["logp"], s["keep"]]
    if not kept:
        kept["desc"] = ls.gdn_decode_desc(s["q"], s["k"], s["v"], s["states"], case["batch"], s["max_q"])
        kept["ws"] = torch.zeros(256, dtype=torch.uint8, device=s["q"].device)
    ls.ls_gdn_decode(kept["desc"], s["states"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["q_start"], s["state_in"], s["state_out"], s["o"],
                     kept["ws"], n_use=s["n_use"])
    return [t for t in (s["o"], s["states"] if s["state_out"] is not None else None) if t is not None]


def run(state):
    if own:
        return _run_own(state)
    return {"step": _advance_plain, "fork": _fork_plain, "compact": _compact_plain, "verify": _verify_plain, "state": _state_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    if case["op"] in ("step", "fork", "compact"):
        return None  # whole numbers, and rows that are copied
    s = prepare(case, seed)
    start = s["q_start"].tolist()
    if case["op"] == "verify":
        dev = s["logits"].device
        count = torch.zeros(case["batch"], dtype=torch.int32, device=dev)
        out = torch.full((start[-1],), -1, dtype=torch.int64, device=dev)
        logp = torch.zeros(start[-1], dtype=torch.float64, device=dev)
        keep = s["kv_len"].clone()
        for b in range(case["batch"]):
            rows = range(start[b], start[b + 1])
            for r in rows:
                lp = torch.log_softmax(s["logits"][r].double() * case["scale"], 0)
                p = lp.exp()
                count[b] += 1
                if r + 1 < start[b + 1]:
                    x = int(s["tokens"][r + 1])
                    q = s["probs"][r].double() if case["probs"] else torch.nn.functional.one_hot(s["tokens"][r + 1], case["vocab"]).double()
                    if float(s["u"][r]) * float(q[x]) < float(p[x]):
                        out[r], logp[r] = x, lp[x]
                        continue
                    rest = torch.relu(p - q)
                    p = rest if float(rest.sum()) > 0 else p
                edge = torch.cumsum(p, 0)
                x = min(int(torch.searchsorted(edge, edge[-1:] * float(s["u_new"][b]), right=True)), case["vocab"] - 1)
                out[r], logp[r] = x, lp[x]
                break
            if rows:
                keep[b] += count[b] - len(rows)
        return [count, out, logp, keep]
    each = case["heads"] // case["key_heads"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    q, k = q.repeat_interleave(each, 1), k.repeat_interleave(each, 1)
    o = None if s["o"] is None else torch.zeros(s["o"].shape, dtype=torch.float64, device=q.device)
    states = s["states"].double() if s["state_out"] is not None else None
    ins = s["state_in"].tolist()
    outs = s["state_out"].tolist() if s["state_out"] is not None else None
    use = s["n_use"].tolist() if s["n_use"] is not None else [a - b for a, b in zip(start[1:], start)]
    for b in range(case["batch"]):
        state = s["states"][ins[b]].double()
        for t in range(start[b], start[b] + use[b]):
            state = state * s["g"][t].double().exp()[:, None, None]
            err = (v[t] - torch.einsum("hvk,hk->hv", state, k[t])) * s["beta"][t].double()[:, None]
            state = state + torch.einsum("hv,hk->hvk", err, k[t])
            if o is not None:
                o[t] = torch.einsum("hvk,hk->hv", state, q[t])
        if states is not None:
            states[outs[b]] = state
    return [t for t in (o, states) if t is not None]
