"""A book's own lengths as the list of lengths that a call keeps, on one block and on eight."""
import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from test_gpu_pages import I32, I64, Device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool,n_seqs", [(200, 6), (140000, 500)])
def test_lengths_of_the_book_as_what_is_kept(cuda_device, pool, n_seqs):
    d = Device(pool, 4, n_seqs, 12)
    grow = [(7 * i) % 11 for i in range(n_seqs)]
    d.advance(None, None, grow)
    more = [i % 4 for i in range(n_seqs)]
    q_start = d.t([sum(more[:i]) for i in range(n_seqs + 1)])
    slots, copies = torch.full((sum(more),), -5, dtype=I64, device="cuda"), torch.full((n_seqs, 3), -5, dtype=I32, device="cuda")
    ls.ls_pages_advance(d.book, q_start, slots, copies, d.ws, keep=d.kv_len)
    want = d.ref.advance(range(n_seqs), grow, more)
    assert slots.tolist() == want[0] and [tuple(r) for r in copies.tolist()] == want[1]
    d.same()
    half = n_seqs // 2
    src, dst = list(range(half)), list(range(half, 2 * half))
    ls.ls_pages_fork(d.book, d.t(src), d.t(dst), d.ws, lens=d.kv_len[:half])
    d.ref.fork(src, dst, [d.ref.len[s] for s in src])
    d.same()
    ls.ls_pages_compact(d.book, d.table, d.refs, torch.empty((pool // 2, 3), dtype=I32, device="cuda"), d.ws)
    d.ref.compact()
    d.same()
