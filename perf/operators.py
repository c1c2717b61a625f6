"""The rollout and scoring operators of the GRPO loop, as cases that can be measured.

Three operators stand next to the response replay:

* the quantised K/V cache: token rows are written into page slots as e4m3 codes
  with one power-of-two scale per row and KV head, and read back by slot;
* cached attention: a chunk of new tokens per sequence (one token when decoding)
  over that sequence's pages, in e4m3, bf16 or float32;
* vocabulary log-probabilities: log softmax(scale * h W^T)[target] over a large
  vocabulary in pieces, and its gradients for h and W.

`own = False` computes them with elementary torch operations in 32 bits;
`own = True` makes the calls a user makes of the library.
"""
import math
import random

import torch

own = False

IGNORE = -100  # target of a row that takes no part (a prompt or padding token)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One decoding step of 64 sequences: each sequence's new token row is written (latency).
        dict(name="write_step", op="write", tokens=64, hkv=4, d=256, page=256, pages=64, src="bf16", pad=0),
        # The capture of a long prompt into scattered pages, from a fused QKV projection's rows.
        dict(name="write_prompt", op="write", tokens=131075, hkv=4, d=256, page=256, pages=1024, src="bf16", pad=6144),
        # Part of a captured prompt read back for a replay that wants bf16 pages.
        dict(name="read_chunk", op="read", tokens=60001, hkv=4, d=256, page=256, pages=512, dst="bf16"),
        # A rollout server's decoding step: 32 sequences of very different lengths, one of them empty.
        dict(name="decode_ragged", op="attn", fmt="e4m3", hkv=4, gq=6, d=256, page=256, batch=32, q_min=1, q_max=1,
             kv_min=0, kv_max=16384, mix=1, causal=True),
        # One sequence far into a long context, one token.
        dict(name="decode_long", op="attn", fmt="e4m3", hkv=4, gq=6, d=256, page=256, batch=1, q_min=1, q_max=1,
             kv_min=1000003, kv_max=1000003, mix=2, causal=True),
        # The eight members of a group decode together over the prompt that they share (their own tokens are merged after).
        dict(name="shared_prefix", op="attn", fmt="e4m3", hkv=4, gq=6, d=256, page=256, batch=1, q_min=8, q_max=8,
             kv_min=262144, kv_max=262144, mix=3, causal=False),
        # A chunk of a long prompt's prefill over the cache that holds the chunks before it.
        dict(name="prefill_chunk", op="attn", fmt="e4m3", hkv=4, gq=6, d=256, page=256, batch=1, q_min=2048, q_max=2048,
             kv_min=32768, kv_max=32768, mix=4, causal=True),
        # Drafted tokens checked against a bf16 cache in small pages, other head sizes.
        dict(name="verify_bf16", op="attn", fmt="bf16", hkv=8, gq=4, d=128, page=16, batch=8, q_min=1, q_max=5,
             kv_min=5, kv_max=8192, mix=5, causal=True),
        # The small float32 configuration: latency, ragged chunks, sequences shorter than a page.
        dict(name="tiny_f32", op="attn", fmt="f32", hkv=1, gq=4, d=64, page=16, batch=4, q_min=0, q_max=64,
             kv_min=1, kv_max=1088, mix=6, causal=True),
        # Scoring the old policy's responses: no gradient, two members of 4096 tokens.
        dict(name="score", op="logprob", grad=False, dtype="bf16", rows=8192, hidden=4096, vocab=128000, scale=1.0),
        # A training step on one member's response, vocabulary of an odd size, a sampling temperature.
        dict(name="step", op="logprob", grad=True, dtype="bf16", rows=4096, hidden=4096, vocab=50003, scale=0.8),
        # A few float32 rows with gradients.
        dict(name="step_f32", op="logprob", grad=True, dtype="f32", rows=37, hidden=1000, vocab=8191, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn", "logprob", "logprob"])
    if op in ("write", "read"):
        hkv, d = rng.choice([(4, 256), (4, 256), (8, 128), (1, 64), (3, 128)])
        page = rng.choice([16, 48, 64, 128, 256])
        tokens = _log_int(rng, 1, 131075 * 1024 // max(1024, hkv * d))
        pages = -(-tokens // page) + rng.randint(0, 1 + tokens // page)
        case = dict(op=op, tokens=tokens, hkv=hkv, d=d, page=page, pages=pages)
        return case | (dict(src=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 8, 1024])) if op == "write"
                       else dict(dst=rng.choice(["bf16", "bf16", "f32"])))
    if op == "attn":
        if rng.random() < 0.15:
            fmt, hkv, gq, d = "f32", rng.choice([1, 2]), rng.choice([1, 4]), 64
            batch, q_hi, kv_hi = rng.randint(1, 4), rng.choice([1, 64]), _log_int(rng, 16, 1088)
        else:
            fmt = rng.choice(["e4m3", "e4m3", "bf16"])
            hkv, gq, d = rng.choice([(4, 6, 256), (4, 6, 256), (8, 4, 128), (2, 8, 64), (3, 1, 128), (1, 12, 256)])
            kind = rng.choice(["decode", "verify", "chunk"])
            batch = 1 if kind == "chunk" and rng.random() < 0.5 else _log_int(rng, 1, 48 if kind == "decode" else 8)
            q_hi = 1 if kind == "decode" else rng.randint(2, 8) if kind == "verify" else _log_int(rng, 9, 2048)
            # a drawn cache holds at most the elements of 1,000,003 tokens of 4 x 256; a chunk's scores at most 2048 x 32768 x 24
            most = 1000003 * 1024 // (batch * hkv * d)
            most = min(most, 2048 * 32768 * 24 // (batch * q_hi * hkv * gq), 1000003)
            kv_hi = _log_int(rng, 16, max(16, most))
        return dict(op="attn", fmt=fmt, hkv=hkv, gq=gq, d=d, page=rng.choice([16, 48, 64, 128, 256]), batch=batch,
                    q_min=q_hi if batch == 1 else rng.choice([0, 1, q_hi]), q_max=q_hi, kv_min=kv_hi if batch == 1 else rng.randint(0, kv_hi),
                    kv_max=kv_hi, mix=rng.randrange(10**6), causal=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    grad = rng.random() < 0.6
    hidden = 8 * _log_int(rng, 8, 640 if dtype == "bf16" else 256)
    vocab = _log_int(rng, 1000, 160000)
    most = (2.0e12 if grad else 4.0e12) / (2.0 * hidden * vocab) * (1.0 if dtype == "bf16" else 0.05)
    return dict(op="logprob", grad=grad, dtype=dtype, rows=_log_int(rng, 1, max(1, min(8192, int(most)))), hidden=hidden, vocab=vocab,
                scale=rng.choice([1.0, 1.0, 0.7, 1.4]))


def _lengths(case):
    """(query lengths, cache lengths) of an attention case: both ends of each range occur where there are two sequences."""
    rng = random.Random(case["mix"])
    n = case["batch"]
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(n)]
    kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(n)]
    q[0], kv[0] = case["q_max"], case["kv_max"]
    if n > 1:
        q[-1], kv[-1] = case["q_min"], case["kv_min"]
    return q, kv


def work(case):
    if case["op"] in ("write", "read"):
        rows = case["tokens"] * case["hkv"]
        wide = 2 if (case.get("src") or case.get("dst")) == "bf16" else 4
        return dict(bytes=2 * rows * (case["d"] * (wide + 1) + 1) + 8 * case["tokens"], flops=2 * rows * case["d"])
    if case["op"] == "attn":
        q, kv = _lengths(case)
        hq = case["hkv"] * case["gq"]
        row = {"e4m3": case["d"] + 1, "bf16": 2 * case["d"], "f32": 4 * case["d"]}[case["fmt"]]
        wide = 4 if case["fmt"] == "f32" else 2
        keys = pairs = 0
        for n, m in zip(q, kv):
            keys += m if n else 0
            first = max(0, n - m) if case["causal"] else 0  # rows before the first position see no key
            rows = n - first
            pairs += (rows * m - rows * (rows - 1) // 2) if case["causal"] else n * m
        return dict(bytes=2 * keys * case["hkv"] * row + sum(q) * hq * (2 * case["d"] * wide + 4), flops=4 * case["d"] * hq * pairs)
    n, d, v = case["rows"], case["hidden"], case["vocab"]
    wide = 2 if case["dtype"] == "bf16" else 4
    return dict(bytes=(n * d + v * d) * wide * (2 if case["grad"] else 1) + 20 * n, flops=(6 if case["grad"] else 2) * n * d * v)


# ---------------------------------------------------------------- inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _quantise(x):
    """e4m3 codes of x's rows (the last axis) and their scales' exponents: the least e with max|x| <= 448 * 2^e."""
    x = x.float()
    m, p = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, p - 8, p - 9).clamp(-126, 127)
    e = torch.where(m == 0, 0, e)
    code = (x * torch.exp2(-e.float())[..., None]).to(torch.float8_e4m3fn)
    return code, e.to(torch.int8)


def _pools(case, g, fill):
    """A cache's two pools [pages, hkv, page, d] (and the exponents of an e4m3 one), NaN in every slot unless `fill`."""
    dev = g.device
    shape = (case["pages"], case["hkv"], case["page"], case["d"])
    fmt = case.get("fmt", "e4m3")
    pools = []
    for _ in range(2):
        if not fill:
            pools.append(torch.full(shape, math.nan, device=dev, dtype=torch.bfloat16).to(_TYPES[fmt]))
        else:
            # per-head factors, and rows of different sizes as trained keys and values have
            x = torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16 if fmt != "f32" else torch.float32)
            x *= 0.5 + 1.5 * torch.rand((1, case["hkv"], 1, 1), generator=g, device=dev, dtype=x.dtype)
            x *= 0.75 + 0.5 * torch.rand((case["pages"], 1, case["page"], 1), generator=g, device=dev, dtype=x.dtype)
            pools.append(x)
    if fmt != "e4m3":
        return pools, [None, None]
    if not fill:
        return pools, [torch.zeros(shape[:3], device=dev, dtype=torch.int8) for _ in range(2)]
    pairs = [_quantise(x) for x in pools]
    return [p[0] for p in pairs], [p[1] for p in pairs]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    if case["op"] in ("write", "read"):
        n, hkv, d = case["tokens"], case["hkv"], case["d"]
        s["pools"], s["exps"] = _pools(case, g, case["op"] == "read")
        # whole pages in an order of their own, as a page table gives them
        order = torch.randperm(case["pages"], generator=g, device=dev)
        at = torch.arange(n, device=dev)
        s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
        if case["op"] == "write":
            # rows of a projection that holds more than this layer's K or V
            wide = torch.randn((n, 2 * hkv * d + case["pad"]), generator=g, device=dev, dtype=_TYPES[case["src"]])
            wide *= 0.25 + 2 * torch.rand((n, 1), generator=g, device=dev, dtype=wide.dtype)
            s["k"], s["v"] = (wide[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
        else:
            s["k"], s["v"] = (torch.empty((n, hkv, d), device=dev, dtype=_TYPES[case["dst"]]) for _ in range(2))
    elif case["op"] == "attn":
        q, kv = _lengths(case)
        hq, page = case["hkv"] * case["gq"], case["page"]
        each = max(1, -(-max(kv) // page))
        used = [-(-m // page) for m in kv]
        case = case | dict(pages=sum(used) + 3)
        s["pools"], s["exps"] = _pools(case, g, True)
        order = torch.randperm(case["pages"], generator=g, device=dev).to(torch.int32)
        table = torch.zeros((case["batch"], each), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(used):
            table[b, :n] = order[at:at + n]
            if kv[b] % page:  # rows past the end of a sequence hold anything
                last = order[at + n - 1].long()
                for p in s["pools"]:
                    p.view(torch.uint8)[last, :, kv[b] % page:] = 0x7F  # NaN in e4m3, large in the others
            at += n
        s["table"] = table
        s["q_start"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device=dev)
        s["kv_len"] = torch.tensor(kv, dtype=torch.int64, device=dev)
        wide = torch.float32 if case["fmt"] == "f32" else torch.bfloat16
        s["q"] = torch.randn((sum(q), hq, case["d"]), generator=g, device=dev, dtype=wide)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((sum(q), hq), device=dev)
        s["scale"] = case["d"] ** -0.5
        s["max_q"], s["max_kv"] = max(q), max(kv)
    else:
        n, d, v = case["rows"], case["hidden"], case["vocab"]
        dt = _TYPES[case["dtype"]]
        s["h"] = torch.randn((n, d), generator=g, device=dev, dtype=dt)
        s["w"] = torch.randn((v, d), generator=g, device=dev, dtype=dt) * (2.0 / math.sqrt(d))
        s["targets"] = torch.randint(0, v, (n,), generator=g, device=dev)
        s["targets"][torch.rand(n, generator=g, device=dev) < 0.1] = IGNORE
        s["dlogp"] = torch.randn(n, generator=g, device=dev) / n  # advantage over response length
        s["logp"], s["lse"] = torch.empty(n, device=dev), torch.empty(n, device=dev)
        if case["grad"]:
            s["dh"], s["dw"] = torch.empty_like(s["h"]), torch.empty_like(s["w"])
    s["kept"] = {}  # what the library's user allocates once: a descriptor and a workspace
    return s


# ---------------------------------------------------------------- plain forms
def _store(x, pool, exps, at):
    code, e = _quantise(x)
    pool.view(torch.uint8)[at] = code.view(torch.uint8)
    exps[at] = e


def _load(pool, exps, at):
    """The values of a pool's pages or rows in 32 bits."""
    if exps is None:
        return pool[at].float()
    return pool.view(torch.uint8)[at].view(pool.dtype).float() * torch.exp2(exps[at].float())[..., None]


def _write_plain(s):
    page = s["pools"][0].shape[2]
    at = s["slots"] // page, slice(None), s["slots"] % page
    _store(s["k"], s["pools"][0], s["exps"][0], at)
    _store(s["v"], s["pools"][1], s["exps"][1], at)
    return [s["pools"][0], s["exps"][0], s["pools"][1], s["exps"][1]]


def _read_plain(s):
    page = s["pools"][0].shape[2]
    at = s["slots"] // page, slice(None), s["slots"] % page
    return [_load(s["pools"][i], s["exps"][i], at).to(s["k"].dtype) for i in range(2)]


def _keys(pool, exps, table, valid):
    """[batch, hkv, length, d] of the sequences' pages, zero where `valid` is false."""
    b, length = valid.shape
    x = _load(pool, exps, table).transpose(1, 2).reshape(b, pool.shape[1], length, pool.shape[3])
    return torch.where(valid[:, None, :, None], x, 0.0)


def _attn_plain(s):
    case = s["case"]
    b, hkv, gq, d, page = case["batch"], case["hkv"], case["gq"], case["d"], case["page"]
    mq = s["max_q"]
    table = s["table"].long()
    length = table.shape[1] * page
    at = torch.arange(length, device=table.device)
    valid = at < s["kv_len"][:, None]                                    # [b, length]
    k, v = (_keys(s["pools"][i], s["exps"][i], table, valid) for i in range(2))
    n = s["q_start"][1:] - s["q_start"][:-1]
    i = torch.arange(mq, device=table.device)
    there = i < n[:, None]                                               # [b, mq]
    row = torch.where(there, s["q_start"][:-1, None] + i, 0).long()
    q = s["q"].float()[row].reshape(b, mq, hkv, gq, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, gq * mq, d)
    x = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(b, hkv, gq, mq, length)
    see = valid[:, None, :]
    if case["causal"]:
        see = see & (at <= (s["kv_len"][:, None] - n[:, None] + i)[:, :, None])
    x.masked_fill_(~see[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(b, hkv, gq * mq, length) @ v).view(b, hkv, gq, mq, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (total.log() + top)[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hkv * gq, d)[there]
    lse = lse.permute(0, 3, 1, 2).reshape(b, mq, hkv * gq)[there]
    return [o.to(s["q"].dtype), lse]


def _logprob_plain(s):
    case = s["case"]
    h, w = s["h"].float(), s["w"].float()
    x = (h @ w.T).mul_(case["scale"])
    top = x.amax(-1, keepdim=True)
    on = s["targets"] != IGNORE
    t = torch.where(on, s["targets"], 0)
    hit = x.gather(1, t[:, None])[:, 0]
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (total.log() + top)[:, 0]
    logp = torch.where(on, hit - lse, 0.0)
    if not case["grad"]:
        return [logp, lse]
    # d logp_target / d x_j = [j = target] - p_j
    c = torch.where(on, s["dlogp"], 0.0) * case["scale"]
    x.mul_(-c[:, None] / total)
    x.scatter_add_(1, t[:, None], c[:, None])
    return [logp, lse, (x @ w).to(s["h"].dtype), (x.T @ h).to(s["w"].dtype)]


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    from long_context_grpo_replay_gb300 import binding as ls
    case, kept = s["case"], s["kept"]
    if case["op"] in ("write", "read"):
        if not kept:
            kept["cache"] = ls.kv_cache_from(s["pools"][0], s["pools"][1], s["exps"][0], s["exps"][1])
        if case["op"] == "read":
            ls.ls_cache_read(kept["cache"], s["slots"], s["k"], s["v"])
            return [s["k"], s["v"]]
        ls.ls_cache_write(kept["cache"], s["k"], s["v"], s["slots"])
        return [s["pools"][0], s["exps"][0], s["pools"][1], s["exps"][1]]
    if case["op"] == "attn":
        if not kept:
            kept["cache"] = ls.kv_cache_from(s["pools"][0], s["pools"][1], s["exps"][0], s["exps"][1])
            kept["desc"] = ls.cached_attn_desc(s["q"], s["o"], case["batch"], s["max_q"], s["max_kv"], causal=case["causal"],
                                               softmax_scale=s["scale"])
            kept["ws"] = torch.zeros(ls.ls_cached_attn_workspace_size(kept["desc"], kept["cache"]), dtype=torch.uint8, device=s["q"].device)
        ls.ls_cached_attn(kept["desc"], kept["cache"], s["q"], s["q_start"], s["kv_len"], s["table"], s["o"], s["lse"], kept["ws"])
        return [s["o"], s["lse"]]
    if not kept:
        kept["desc"] = ls.vocab_desc(s["h"], s["w"], logit_scale=case["scale"], ignore_index=IGNORE)
        kept["ws"] = torch.zeros(ls.ls_vocab_logprob_workspace_size(kept["desc"], case["grad"]), dtype=torch.uint8, device=s["h"].device)
    ls.ls_vocab_logprob_fwd(kept["desc"], s["h"], s["w"], s["targets"], s["logp"], s["lse"], kept["ws"])
    if not case["grad"]:
        return [s["logp"], s["lse"]]
    ls.ls_vocab_logprob_bwd(kept["desc"], s["h"], s["w"], s["targets"], s["lse"], s["dlogp"], s["dh"], s["dw"], kept["ws"])
    return [s["logp"], s["lse"], s["dh"], s["dw"]]


def run(state):
    if own:
        return _run_own(state)
    return {"write": _write_plain, "read": _read_plain, "attn": _attn_plain, "logprob": _logprob_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    if case["op"] == "write":
        return None  # codes and exponents are compared as the whole values that they are
    s = prepare(case, seed)
    if case["op"] == "read":
        page, at = case["page"], s["slots"].long()
        out = []
        for pool, exps in zip(s["pools"], s["exps"]):
            rows = pool.double().transpose(1, 2).flatten(0, 1)[at]
            out.append(torch.ldexp(rows, exps.transpose(1, 2).flatten(0, 1)[at].int()[..., None]))
        return out
    if case["op"] == "attn":
        lens_q, lens_kv = _lengths(case)
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["q"].device)
        first = 0
        for b, (n, m) in enumerate(zip(lens_q, lens_kv)):
            for head in range(case["hkv"] * case["gq"] if n and m else 0):
                side = []
                for pool, exps in zip(s["pools"], s["exps"]):
                    ids = s["table"][b, :-(-m // case["page"])].long()
                    x = pool[:, head // case["gq"]][ids] if exps is None else pool.view(torch.uint8)[:, head // case["gq"]][ids].view(pool.dtype)
                    x = x.double().flatten(0, 1)[:m]
                    if exps is not None:
                        x = torch.ldexp(x, exps[:, head // case["gq"]][ids].flatten()[:m, None].int())
                    side.append(x)
                score = torch.einsum("id,jd->ij", s["q"][first:first + n, head].double(), side[0]) * s["scale"]
                if case["causal"]:
                    late = torch.arange(m, device=score.device)[None] > torch.arange(m - n, m, device=score.device)[:, None]
                    score = score.masked_fill(late, -math.inf)
                each = torch.logsumexp(score, 1)
                some = each > -math.inf
                lse[first:first + n, head] = each
                p = torch.exp(score[some] - each[some][:, None])
                o[first:first + n, head][some] = p @ side[1]
            first += n
        return [o, lse]
    h, w = s["h"].double(), s["w"].double()
    if case["rows"] * case["hidden"] * case["vocab"] * (3 if case["grad"] else 1) > 6e12:
        return None
    log_p = torch.log_softmax(torch.einsum("nd,vd->nv", h, w) * case["scale"], 1)
    lse = torch.logsumexp(torch.einsum("nd,d->n", h, w[0])[:, None] * case["scale"] - log_p[:, :1], 1)
    on = (s["targets"] != IGNORE).double()
    t = s["targets"].clamp(min=0)[:, None]
    logp = log_p.gather(1, t)[:, 0] * on
    if not case["grad"]:
        return [logp, lse]
    slope = torch.zeros_like(log_p).scatter_(1, t, 1.0).sub_(log_p.exp()).mul_((s["dlogp"].double() * on * case["scale"])[:, None])
    return [logp, lse, torch.einsum("nv,vd->nd", slope, w), torch.einsum("nv,nd->vd", slope, h)]
