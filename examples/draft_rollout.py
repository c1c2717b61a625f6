"""A rollout of a two-layer toy model (one attention layer, one recurrent layer) with drafted tokens, on the library's calls:

  capture   the prompt's K/V rows go into pages that the book gives out (ls_pages_advance, ls_cache_write), its
            recurrent state into a slot (ls_gdn_decode)
  fork      the group's members name the prompt's pages (ls_pages_fork); their first step reads its state
  step      drafts are looked up in the member's own history; slots for them (ls_pages_advance, with a copy of a page
            that others name, ls_cache_copy_pages), their rows (ls_cache_write), attention over the member's pages
            (ls_cached_attn), the recurrent layer ahead of its state (ls_gdn_decode), and what the target says of
            them (ls_draft_verify); the accepted ones move the state on, the others' pages are dropped
  end       the members' pages go back, the pool is compacted (ls_pages_release, ls_pages_compact)

The tokens that come out are distributed as if the target alone had drawn them one by one.

Run: python examples/draft_rollout.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import long_context_grpo_replay_gb300.binding as ls  # noqa: E402

HQ, HKV, D, PAGE = 12, 2, 128, 32   # attention layer
H, HK, DS = 4, 2, 128               # recurrent layer
I32, I64, BF16 = torch.int32, torch.int64, torch.bfloat16


class Model:
    """Random weights: embedding, both layers' projections, output matrix."""

    def __init__(self, hidden, vocab, dev, g):
        rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=dev) * scale).to(BF16)  # noqa: E731
        self.embed = rand(vocab, hidden)
        self.w_qkv = rand(hidden, (HQ + 2 * HKV) * D, scale=hidden ** -0.5)
        self.w_o = rand(HQ * D, hidden, scale=(HQ * D) ** -0.5)
        self.w_state = rand(hidden, (2 * HK + H) * DS, scale=hidden ** -0.5)
        self.w_gate = rand(hidden, 2 * H, scale=hidden ** -0.5)
        self.w_so = rand(H * DS, hidden, scale=(H * DS) ** -0.5)
        self.w_out = rand(vocab, hidden, scale=3 * hidden ** -0.5)

    def attention_inputs(self, x):
        return (x @ self.w_qkv).unflatten(1, (HQ + 2 * HKV, D)).split([HQ, HKV, HKV], 1)

    def state_inputs(self, x):
        rows = (x @ self.w_state).float().unflatten(1, (2 * HK + H, DS))
        qk = torch.nn.functional.normalize(rows[:, :2 * HK], dim=2)
        rows = torch.cat([qk[:, :HK] * DS ** -0.5, qk[:, HK:], rows[:, 2 * HK:]], 1).to(BF16)
        gate = (x @ self.w_gate).float()
        decay, beta = torch.nn.functional.logsigmoid(gate[:, :H] + 4).contiguous(), torch.sigmoid(gate[:, H:]).contiguous()
        return rows[:, :HK], rows[:, HK:2 * HK], rows[:, 2 * HK:], decay, beta

    def logits(self, x):
        return torch.nn.functional.normalize(x.float(), dim=1).mul(x.shape[1] ** 0.5).to(BF16) @ self.w_out.T


class Server:
    """The pool of pages and of states: sequence 0 is the prompt, 1 .. the members; the last state is the prompt's."""

    def __init__(self, model, members, most, dev):
        self.model, self.members, self.dev = model, members, dev
        per_seq = -(-most // PAGE)
        pages = per_seq * (members + 2)
        self.pools = [torch.zeros((pages, HKV, PAGE, D), dtype=torch.float8_e4m3fn, device=dev) for _ in range(2)]
        self.exps = [torch.zeros((pages, HKV, PAGE), dtype=torch.int8, device=dev) for _ in range(2)]
        self.cache = ls.kv_cache_from(*self.pools, *self.exps)
        self.refs = torch.zeros(pages, dtype=I32, device=dev)
        self.table = torch.zeros((members + 1, per_seq), dtype=I32, device=dev)
        self.kv_len = torch.zeros(members + 1, dtype=I64, device=dev)
        self.book = ls.page_book(self.refs, self.table, self.kv_len, PAGE)
        self.ws = torch.zeros(ls.ls_pages_workspace_size(self.book), dtype=torch.uint8, device=dev)
        self.states = torch.zeros((members + 1, H, DS, DS), device=dev)
        self.most = most
        self.state_in = self.ints([members] * members)  # the members' first step reads the prompt's
        self.own = self.ints(range(members))
        self.seqs = self.ints(range(1, members + 1))

    def ints(self, x):
        return torch.tensor(list(x), dtype=I32, device=self.dev)

    def grow(self, seqs, counts, keep=None):
        q_start = self.ints([sum(counts[:i]) for i in range(len(counts) + 1)])
        slots = torch.empty(sum(counts), dtype=I64, device=self.dev)
        copies = torch.empty((len(counts), 3), dtype=I32, device=self.dev)
        ls.ls_pages_advance(self.book, q_start, slots, copies, self.ws, seqs=seqs, keep=keep)
        ls.ls_cache_copy_pages(self.cache, copies, self.ws)  # a cache of each layer, in a model of more
        return q_start, slots

    def capture(self, prompt):
        x = self.model.embed[prompt]
        _, k, v = self.model.attention_inputs(x)
        q_start, slots = self.grow(self.ints([0]), [len(prompt)])
        ls.ls_cache_write(self.cache, k, v, slots, self.ws)
        q, k, v, decay, beta = self.model.state_inputs(x)
        desc = ls.gdn_decode_desc(q, k, v, self.states, 1, len(prompt))
        ls.ls_gdn_decode(desc, self.states, q, k, v, decay, beta, q_start, self.ints([-1]), self.ints([self.members]), ws=self.ws)
        ls.ls_pages_fork(self.book, self.ints([0] * self.members), self.seqs, self.ws)

    def step(self, rows, keep):
        """Logits after each of the members' tokens `rows`; `commit(n)` lets the first n[m] of them count."""
        counts = [len(r) for r in rows]
        tokens = torch.tensor([t for r in rows for t in r], dtype=I64, device=self.dev)
        q_start, slots = self.grow(self.seqs, counts, keep)
        n, max_q = len(tokens), max(counts)
        x = self.model.embed[tokens]
        q, k, v = self.model.attention_inputs(x)
        ls.ls_cache_write(self.cache, k, v, slots, self.ws)
        o, lse = torch.empty((n, HQ, D), dtype=BF16, device=self.dev), torch.empty((n, HQ), device=self.dev)
        q = q.contiguous()
        attn = ls.cached_attn_desc(q, o, self.members, max_q, self.most)
        ws = torch.zeros(ls.ls_cached_attn_workspace_size(attn, self.cache), dtype=torch.uint8, device=self.dev)
        ls.ls_cached_attn(attn, self.cache, q, q_start, self.kv_len[1:], self.table[1:], o, lse, ws)
        ls.ls_read_device_status(ws)
        x = x + o.flatten(1) @ self.model.w_o
        q, k, v, decay, beta = self.model.state_inputs(x)
        desc = ls.gdn_decode_desc(q, k, v, self.states, self.members, max_q)
        so = torch.empty((n, H, DS), dtype=BF16, device=self.dev)
        ls.ls_gdn_decode(desc, self.states, q, k, v, decay, beta, q_start, self.state_in, None, so, self.ws)
        before = self.state_in

        def commit(n_use):
            ls.ls_gdn_decode(desc, self.states, q, k, v, decay, beta, q_start, before, self.own, None, self.ws, n_use=n_use)
            self.state_in = self.own

        return self.model.logits(x + so.flatten(1) @ self.model.w_so), tokens, q_start, commit


def look_up(history, most):
    """Drafts: what followed the last token's latest earlier occurrence."""
    for i in range(len(history) - 2, -1, -1):
        if history[i] == history[-1]:
            return history[i + 1:i + 1 + most]
    return []


def main(prompt_len=200, members=4, new_tokens=24, drafts=3, hidden=256, vocab=97, seed=0, verbose=True):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    model = Model(hidden, vocab, dev, g)
    prompt = torch.randint(0, vocab, (prompt_len,), generator=g, device=dev)
    server = Server(model, members, prompt_len + new_tokens + drafts, dev)
    server.capture(prompt[:-1])  # its last token is the members' first query
    history = [prompt.tolist() for _ in range(members)]
    logps = [[] for _ in range(members)]
    keep, steps, offered, taken = None, 0, 0, 0
    while True:
        left = [new_tokens - (len(h) - prompt_len) for h in history]
        if max(left) <= 0:
            break
        # a member's last token and its drafts; no row once it is done
        rows = [[h[-1]] + look_up(h, min(drafts, n - 1)) if n > 0 else [] for h, n in zip(history, left)]
        logits, tokens, q_start, commit = server.step(rows, keep)
        n = len(tokens)
        desc = ls.verify_desc(logits, members, max(len(r) for r in rows))
        ws = torch.zeros(ls.ls_draft_verify_workspace_size(desc), dtype=torch.uint8, device=dev)
        u, u_next = torch.rand(n, generator=g, device=dev), torch.rand(members, generator=g, device=dev)
        count = torch.empty(members, dtype=I32, device=dev)
        out, logp = torch.empty(n, dtype=I64, device=dev), torch.empty(n, device=dev)
        keep = torch.empty(members, dtype=I64, device=dev)
        ls.ls_draft_verify(desc, logits, tokens, q_start, u, u_next, count, out, logp, ws, kv_len=server.kv_len[1:], keep=keep)
        ls.ls_read_device_status(ws)
        commit(count)  # the next step's advance drops the others' pages
        at, out, logp = 0, out.tolist(), logp.tolist()
        for m, (r, c) in enumerate(zip(rows, count.tolist())):
            history[m] += out[at:at + c]
            logps[m] += logp[at:at + c]
            offered += max(0, len(r) - 1)
            taken += max(0, c - 1)
            at += len(r)
        steps += 1
    ls.ls_read_device_status(server.ws)
    in_use = int((server.refs > 0).sum())
    ls.ls_pages_release(server.book, server.ws, server.seqs)
    copies = torch.empty((len(server.refs) // 2, 3), dtype=I32, device=dev)
    ls.ls_pages_compact(server.book, server.table, server.refs, copies, server.ws)
    ls.ls_cache_copy_pages(server.cache, copies, server.ws)
    ls.ls_read_device_status(server.ws)
    if verbose:
        print(f"{members} members x {new_tokens} tokens after a prompt of {prompt_len}: {steps} steps, "
              f"{taken} of {offered} drafts accepted, {in_use} pages in use before the members' went back")
    return dict(model=model, prompt=prompt, tokens=[h[prompt_len:] for h in history], logps=logps, steps=steps, taken=taken,
                offered=offered, server=server)


if __name__ == "__main__":
    main()
