"""One GRPO step of a one-layer toy model on the library's calls, in the order a trainer makes them:

  capture   the prompt's K/V rows go into e4m3 pages (ls_cache_write) and into the bf16 pages of the replay
  rollout   the group's members decode together: their tokens attend over the shared prompt as one sequence
            (ls_cached_attn, float32 parts), each over its own pages as sequences of their own, merged by ls_lse_merge
  scoring   log-probabilities of the sampled tokens, without logits (ls_vocab_logprob_fwd)
  update    advantages from the group's rewards, gradients of the hidden states and of the output matrix
            (ls_vocab_logprob_bwd), then each member's replay backward through its attention (ls_replay_fwd / _bwd)

Run: python examples/grpo_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import long_context_grpo_replay_gb300.binding as ls  # noqa: E402

HQ, HKV, D, PAGE = 24, 4, 256, 256


def workspace(nbytes, dev):
    return torch.zeros(nbytes, dtype=torch.uint8, device=dev)


def e4m3_cache(pages, dev):
    shape = (pages, HKV, PAGE, D)
    k, v = (torch.zeros(shape, dtype=torch.float8_e4m3fn, device=dev) for _ in range(2))
    k_exp, v_exp = (torch.zeros(shape[:3], dtype=torch.int8, device=dev) for _ in range(2))
    return ls.kv_cache_from(k, v, k_exp, v_exp), (k, v, k_exp, v_exp)  # the cache holds addresses only


class Attention:
    """ls_cached_attn with its descriptor and workspace, float32 results for merging."""

    def __init__(self, cache, batch, tokens, max_kv, causal, dev):
        self.cache = cache
        self.q = torch.empty((tokens, HQ, D), dtype=torch.bfloat16, device=dev)
        self.o = torch.empty((tokens, HQ, D), device=dev)
        self.lse = torch.empty((tokens, HQ), device=dev)
        self.desc = ls.cached_attn_desc(self.q, self.o, batch, tokens // batch, max_kv, causal)
        self.ws = workspace(ls.ls_cached_attn_workspace_size(self.desc, cache), dev)
        self.q_start = torch.arange(0, tokens + 1, tokens // batch, dtype=torch.int32, device=dev)

    def __call__(self, q, kv_len, table):
        ls.ls_cached_attn(self.desc, self.cache, q, self.q_start, kv_len, table, self.o, self.lse, self.ws)
        return self.o, self.lse


def main(prompt_len=5000, members=4, steps=12, hidden=512, vocab=4001, seed=0, verbose=True):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device=dev) * scale).to(torch.bfloat16)  # noqa: E731
    embed, w_out = rand(vocab, hidden), rand(vocab, hidden, scale=2 * hidden ** -0.5)
    w_qkv = rand(hidden, (HQ + 2 * HKV) * D, scale=hidden ** -0.5)
    w_o = rand(HQ * D, hidden, scale=(HQ * D) ** -0.5)

    # ---- capture
    k, v = rand(prompt_len, HKV, D), rand(prompt_len, HKV, D)
    n_pages = -(-prompt_len // PAGE)
    order = torch.randperm(n_pages, generator=g, device=dev)
    at = torch.arange(prompt_len, device=dev)
    prompt_cache, keep_prompt = e4m3_cache(n_pages, dev)
    ls.ls_cache_write(prompt_cache, k, v, order[at // PAGE] * PAGE + at % PAGE)
    replay_desc = ls.desc_for(HQ, HKV, D, PAGE, torch.bfloat16)
    pools = [torch.empty((n_pages, HKV, PAGE, D), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    table = order.to(torch.int32)
    ls.ls_kv_page_write(replay_desc, *pools, table, 0, k, v)

    # ---- rollout: one page per member for its own tokens
    own_cache, keep_own = e4m3_cache(members, dev)
    shared = Attention(prompt_cache, 1, members, prompt_len, False, dev)
    own = Attention(own_cache, members, members, steps, True, dev)
    prompt_kv = torch.tensor([prompt_len], device=dev)
    own_table = torch.arange(members, dtype=torch.int32, device=dev)[:, None]
    first_slot = torch.arange(members, device=dev) * PAGE
    tokens = torch.zeros(members, dtype=torch.int64, device=dev)
    o = torch.empty((members, HQ, D), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((members, HQ), device=dev)
    qkv_all, o_all, h_all, sampled = [], [], [], []
    for step in range(steps):
        qkv = (embed[tokens] @ w_qkv).unflatten(1, (HQ + 2 * HKV, D))
        q, kn, vn = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
        ls.ls_cache_write(own_cache, kn, vn, first_slot + step)  # the rows as they lie in the projection
        q = q.contiguous()
        parts = [shared(q, prompt_kv, table[None]), own(q, torch.full((members,), step + 1, device=dev), own_table)]
        ls.ls_lse_merge(torch.stack([p[0] for p in parts]).view(2, -1, D), torch.stack([p[1] for p in parts]).view(2, -1),
                        o.view(-1, D), lse.view(-1))
        h = o.flatten(1) @ w_o
        p = torch.softmax((h @ w_out.T).float(), 1)
        tokens = torch.multinomial(p, 1, generator=g)[:, 0]
        qkv_all.append(qkv.clone()), o_all.append(o.clone()), h_all.append(h), sampled.append(tokens)
    for a in (shared, own):
        ls.ls_read_device_status(a.ws)

    # ---- scoring: all members' tokens at once
    h = torch.stack(h_all, 1).flatten(0, 1).contiguous()           # [members * steps, hidden]
    targets = torch.stack(sampled, 1).flatten().contiguous()
    desc = ls.vocab_desc(h, w_out)
    ws = workspace(ls.ls_vocab_logprob_workspace_size(desc, True), dev)
    logp, row_lse = torch.empty(len(h), device=dev), torch.empty(len(h), device=dev)
    ls.ls_vocab_logprob_fwd(desc, h, w_out, targets, logp, row_lse, ws)

    # ---- update: one reward per member, group-relative advantages, d(-sum adv * logp / steps)
    reward = (torch.stack(sampled, 1) % 7 == 0).float().mean(1)
    adv = (reward - reward.mean()) / (reward.std() + 1e-6)
    d_logp = (-adv / steps).repeat_interleave(steps).contiguous()
    dh, dw = torch.empty_like(h), torch.empty_like(w_out)
    ls.ls_vocab_logprob_bwd(desc, h, w_out, targets, row_lse, d_logp, dh, dw, ws)
    ls.ls_read_device_status(ws)

    # each member's attention again, in bf16 over the captured prompt, and its gradients
    prompt = ls.prompt_from(*pools, table, prompt_len)
    rws = workspace(ls.ls_replay_workspace_size(replay_desc, prompt, steps), dev)
    group = []
    for m in range(members):
        x = torch.stack([s[m] for s in qkv_all])
        mem = dict(q=x[:, :HQ].contiguous(), k=x[:, HQ:HQ + HKV].contiguous(), v=x[:, HQ + HKV:].contiguous())
        mem["d_o"] = (dh.unflatten(0, (members, steps))[m] @ w_o.T).unflatten(1, (HQ, D)).contiguous()
        mem |= {n: torch.empty_like(mem[s]) for n, s in (("o", "q"), ("dq", "q"), ("dk", "k"), ("dv", "v"))}
        mem |= {n: torch.empty((steps, HQ), device=dev) for n in ("lse", "delta")}
        group.append(mem)
    ls.ls_replay_group(replay_desc, prompt, group, rws)
    ls.ls_read_device_status(rws)
    torch.cuda.synchronize()

    decoded = torch.stack(o_all, 1).float()                        # [members, steps, HQ, D], from the e4m3 caches
    replayed = torch.stack([m["o"] for m in group]).float()
    off = float((decoded - replayed).norm() / replayed.norm())
    if verbose:
        print(f"{members} members x {steps} tokens over a shared prompt of {prompt_len}")
        print(f"mean log-probability {float(logp.mean()):.3f}, rewards {[round(float(r), 3) for r in reward]}")
        print(f"|dh| {float(dh.float().norm()):.3e}, |dw| {float(dw.float().norm()):.3e}, "
              f"|dq| {float(torch.stack([m['dq'] for m in group]).float().norm()):.3e}")
        print(f"decoded attention (e4m3 caches) against its bf16 replay: {off:.4f}")
    return dict(h=h, w=w_out, targets=targets, logp=logp, d_logp=d_logp, dh=dh, dw=dw, off=off, group=group)


if __name__ == "__main__":
    main()
