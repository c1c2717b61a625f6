"""Float64 definitions of the operators of a rollout with drafted tokens, written from
their formulas (torch on the CPU; no code shared with the CUDA path): the recurrent step
of the gated-DeltaNet state, the book of a cache's pages and the verification of drafts."""
from __future__ import annotations

import torch

F64 = torch.float64


def state_step(state, q, k, v, g, beta):
    """Tokens [n] of one sequence through state [H, dv, dk]: (o [n, H, dv], the state after them, and the
    magnitudes their error bounds are made of: the same recurrence over absolute values, where every
    difference is a sum)."""
    n, h, dv = v.shape
    each = h // q.shape[1]
    s = state.to(F64)
    mag = s.abs()
    o, om = torch.zeros((n, h, dv), dtype=F64), torch.zeros((n, h, dv), dtype=F64)
    for t in range(n):
        kt, qt = (x[t].to(F64).repeat_interleave(each, 0) for x in (k, q))
        a, b = g[t].to(F64).exp()[:, None, None], beta[t].to(F64)[:, None, None]
        s, mag = a * s, a * mag
        s = s + b * (v[t].to(F64)[..., None] - (s @ kt[..., None])) * kt[:, None, :]
        mag = mag + b * (v[t].to(F64).abs()[..., None] + mag @ kt.abs()[..., None]) * kt.abs()[:, None, :]
        o[t] = (s @ qt[..., None])[..., 0]
        om[t] = (mag @ qt.abs()[..., None])[..., 0]
    return o, s, om, mag


class Book:
    """Pages of a pool, one step at a time: refs, table (a list of page ids per sequence) and lengths."""

    def __init__(self, pool, page, n_seqs, pages_per_seq):
        self.page, self.per_seq = page, pages_per_seq
        self.refs = [0] * pool
        self.table = [[] for _ in range(n_seqs)]
        self.len = [0] * n_seqs

    def _cut(self, s, n):
        keep = -(-n // self.page)
        for p in self.table[s][keep:]:
            self.refs[p] -= 1
        self.table[s] = self.table[s][:keep]
        self.len[s] = n

    def advance(self, seqs, keep, grow):
        """(slots, copies, whether all could grow)."""
        for s, k in zip(seqs, keep):
            self._cut(s, k)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        shared = [self.len[s] % self.page != 0 and n > 0 and self.refs[self.table[s][-1]] > 1 for s, n in zip(seqs, grow)]
        slots, copies, asked, fine = [], [], 0, True
        for s, n, own in zip(seqs, grow, shared):
            have, want = len(self.table[s]), -(-(self.len[s] + n) // self.page)
            row_ends = want > self.per_seq
            need = 0 if row_ends else want - have + own
            asked += need
            if row_ends or (need and asked > len(free)):
                slots += [-1] * n
                copies.append((-1, -1, -1))
                fine = False
                continue
            take = free[asked - need:asked]
            for p in take:
                self.refs[p] = 1
            if own:
                last = self.table[s].pop()
                self.refs[last] -= 1
                copies.append((last, take[0], self.len[s] % self.page))
            else:
                copies.append((-1, -1, -1))
            self.table[s] += take
            slots += [self.table[s][i // self.page] * self.page + i % self.page for i in range(self.len[s], self.len[s] + n)]
            self.len[s] += n
        return slots, copies, fine

    def fork(self, src, dst, lens):
        for s, d, n in zip(src, dst, lens):
            self._cut(d, 0)
            self.table[d] = self.table[s][:-(-n // self.page)]
            for p in self.table[d]:
                self.refs[p] += 1
            self.len[d] = n

    def compact(self):
        """The moves (from, to)."""
        live = [p for p, r in enumerate(self.refs) if r > 0]
        low = [p for p in range(len(live)) if self.refs[p] == 0]
        moves = list(zip([p for p in live if p >= len(live)], low))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return moves


def verify(logits, probs, tokens, q_start, u, u_next, scale):
    """Per sequence (emitted tokens, their log-probabilities, how near the nearest decision was to its border:
    of an acceptance relative to p, of the draw relative to all weights).  logits, probs in any type on any
    device; a sequence whose row has no distribution ends with the token None.  What a rejection leaves is taken for
    nothing, and the draw is from p, where it sums to 2^-30 or less."""
    out = []
    for b in range(len(q_start) - 1):
        toks, logp, near = [], [], float("inf")
        for r in range(q_start[b], q_start[b + 1]):
            x = logits[r].to(F64) * scale
            x = x - x.max()          # before the logarithm: 64 bits lose log(n) beside a row of the type's lowest value
            lse = torch.logsumexp(x, 0)
            p = torch.exp(x - lse)
            valid = bool(torch.isfinite(lse))
            if r + 1 < q_start[b + 1]:
                d = int(tokens[r + 1])
                inside = 0 <= d < len(x)
                q = probs[r].to(F64) if probs is not None else torch.zeros_like(p)
                if probs is None and inside:
                    q[d] = 1.0
                if inside and valid:
                    side = float(u[r]) * float(q[d]), float(p[d])
                    near = min(near, abs(side[0] - side[1]) / max(*side, 1e-300))
                    if side[0] < side[1]:
                        toks.append(d), logp.append(float(x[d] - lse))
                        continue
                rest = (p - q).clamp(min=0)
                if float(rest.sum()) > 2.0 ** -30:
                    w = rest
                else:
                    w = p
            else:
                w = p
            if not valid:
                toks.append(None), logp.append(0.0)
                break
            upto = torch.cumsum(w, 0)
            edge = float(u_next[b]) * float(upto[-1])
            t = min(int((upto <= edge).sum()), len(x) - 1)
            near = min(near, float((upto - edge).abs().min() / upto[-1]) * 2 ** 10 if len(x) > 1 else 1.0)
            toks.append(t), logp.append(float(x[t] - lse))
            break
        out.append((toks, logp, near))
    return out
