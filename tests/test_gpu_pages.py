"""Pages of a cache against a book kept in plain Python, and copies of their rows bit for bit."""
import random

import pytest
import torch

import long_context_grpo_replay_gb300.binding as ls
from oracle import drafts as ref

pytestmark = pytest.mark.gpu
I32, I64 = torch.int32, torch.int64


class Device:
    """A book on the device beside the plain one."""

    def __init__(self, pool, page, n_seqs, per_seq):
        self.ref = ref.Book(pool, page, n_seqs, per_seq)
        self.refs = torch.zeros(pool, dtype=I32, device="cuda")
        self.table = torch.full((n_seqs, per_seq), -77, dtype=I32, device="cuda")
        self.kv_len = torch.zeros(n_seqs, dtype=I64, device="cuda")
        self.book = ls.page_book(self.refs, self.table, self.kv_len, page)
        self.ws = torch.full((ls.ls_pages_workspace_size(self.book),), 255, dtype=torch.uint8, device="cuda")
        ls.ls_clear_device_status(self.ws)

    def t(self, x, dtype=I32):
        return None if x is None else torch.tensor(x, dtype=dtype, device="cuda")

    def advance(self, seqs, keep, grow, full=False, **kw):
        n = len(grow)
        q_start = self.t([sum(grow[:i]) for i in range(n + 1)])
        slots = torch.full((sum(grow),), -5, dtype=I64, device="cuda")
        copies = torch.full((n, 3), -5, dtype=I32, device="cuda")
        ls.ls_pages_advance(self.book, q_start, slots, copies, self.ws, seqs=self.t(seqs), keep=self.t(keep, I64), **kw)
        who = list(range(n)) if seqs is None else seqs
        want = self.ref.advance(who, [self.ref.len[s] for s in who] if keep is None else keep, grow)
        assert slots.tolist() == want[0] and [tuple(r) for r in copies.tolist()] == want[1]
        assert want[2] != full
        self.same(7 if full else 0)
        return want

    def fork(self, src, dst, lens=None):
        ls.ls_pages_fork(self.book, self.t(src), self.t(dst), self.ws, lens=self.t(lens, I64))
        self.ref.fork(src, dst, [self.ref.len[s] for s in src] if lens is None else lens)
        self.same()

    def status(self):
        try:
            ls.ls_read_device_status(self.ws)
        except ls.LsError as e:
            return e.status
        return 0

    def same(self, status=0):
        assert self.status() == status
        assert self.kv_len.tolist() == self.ref.len
        assert self.refs.tolist() == self.ref.refs
        for row, want in zip(self.table.tolist(), self.ref.table):
            assert row[:len(want)] == want


@pytest.mark.parametrize("pool,page,n_seqs,per_seq,steps", [
    (40, 4, 5, 12, 60), (5000, 16, 70, 100, 60), (9001, 1, 33, 300, 60), (300, 256, 3, 100, 60),
    (20011, 2, 2500, 6, 25),      # more sequences than a block keeps to itself
    (270007, 3, 40, 5000, 25)])   # more pages than the warps keep a bit for
def test_a_rollout_at_random(cuda_device, pool, page, n_seqs, per_seq, steps):
    """Growth, truncation, forks, release and compaction in a random order, on both sizes of the kernels."""
    rng = random.Random(pool)
    d = Device(pool, page, n_seqs, per_seq)
    for step in range(steps):
        kind = rng.choice(["advance", "advance", "advance", "fork", "release", "compact"])
        seqs = rng.sample(range(n_seqs), rng.randint(1, n_seqs))
        if kind == "advance":
            keep = [rng.choice([n, n, max(0, n - rng.randint(0, 3 * page)), 0]) for n in (d.ref.len[s] for s in seqs)]
            grow = [rng.choice([0, 1, rng.randint(0, 2 * page), rng.randint(0, 3 * page)]) for _ in seqs]
            room = d.ref.refs.count(0) // 2
            while sum(-(-g // page) + 2 for g in grow) > room and any(grow):
                grow = [g // 2 for g in grow]
            grow = [min(g, per_seq * page - k) for g, k in zip(grow, keep)]
            if not any(d.ref.refs.count(0) < 2 * len(seqs) for _ in (0,)):
                d.advance(seqs, keep, grow)
        elif kind == "fork" and len(seqs) > 1:
            cut = rng.randint(1, len(seqs) - 1)
            src = [rng.choice(seqs[:cut]) for _ in seqs[cut:]]
            lens = [rng.choice([d.ref.len[s], rng.randint(0, d.ref.len[s])]) for s in src]
            d.fork(src, seqs[cut:], lens if rng.random() < 0.5 else None)
        elif kind == "release":
            seqs = seqs[:max(1, len(seqs) // 3)]
            ls.ls_pages_release(d.book, d.ws, d.t(seqs))
            for s in seqs:
                d.ref._cut(s, 0)
            d.same()
        elif kind == "compact":
            copies = torch.full((pool // 2, 3), -5, dtype=I32, device="cuda")
            inside = rng.random() < 0.5
            table, refs = (d.table, d.refs) if inside else (torch.empty_like(d.table), torch.empty_like(d.refs))
            ls.ls_pages_compact(d.book, table, refs, copies, d.ws)
            moves = d.ref.compact()
            assert copies.tolist() == [[a, b, page] for a, b in moves] + [[-1] * 3] * (pool // 2 - len(moves))
            d.table.copy_(table), d.refs.copy_(refs)
            d.same()
    ls.ls_pages_release(d.book, d.ws)
    assert d.status() == 0 and d.refs.sum() == 0 and d.kv_len.sum() == 0


def test_all_sequences_in_order(cuda_device):
    d = Device(64, 8, 6, 9)
    d.advance(None, None, [3, 0, 8, 9, 1, 17])
    d.advance(None, [2, 0, 8, 0, 1, 11], [1, 1, 1, 0, 7, 3])
    ls.ls_pages_advance(d.book, None, None, None, d.ws, keep=d.t([0, 1, 0, 0, 8, 2], I64))
    d.ref.advance(range(6), [0, 1, 0, 0, 8, 2], [0] * 6)
    d.same()


def test_group_forks_a_prompt_and_writes_into_its_last_page(cuda_device):
    d = Device(40, 8, 5, 6)
    d.advance([0], None, [21])
    d.fork([0] * 4, [1, 2, 3, 4])
    assert d.refs.tolist()[:3] == [5, 5, 5]
    d.advance([1, 2, 3], None, [1, 4, 2])               # copies: others still name the page
    d.advance([4], None, [1])                           # the prompt's own and this one are left
    d.advance([0], None, [1])                           # alone now: no copy
    assert d.refs.tolist()[:3] == [5, 5, 1]
    d.fork([1], [2], [16])                              # whole pages only: nothing to copy later
    assert d.advance([2], None, [1])[1] == [(-1, -1, -1)]
    d.advance([3], [9], [1])                            # back into a page of the prompt: a copy of one row
    assert d.refs.tolist()[1] == 4


def test_pages_run_out(cuda_device):
    d = Device(6, 4, 5, 4)
    d.advance([0, 1], None, [8, 4])
    # 3 pages are left: the second list entry does not fit, later ones only without pages
    d.advance([2, 3, 4, 0], None, [8, 9, 1, 0], full=True)
    d.advance([1, 2], [3, 8], [1, 0])
    d.advance([1], None, [4])
    d.advance([1], None, [13], full=True)               # 21 tokens: the table's row ends at 16
    d.advance([0, 3, 4], [0, 0, 0], [0, 4, 1])  # what is dropped in a call serves in it


def test_lists_that_are_not_valid_change_nothing(cuda_device):
    d = Device(40, 4, 6, 8)
    d.advance([0, 1, 2], None, [5, 9, 1])
    before = [t.clone() for t in (d.refs, d.table, d.kv_len)]

    def refused(seqs, keep, q_start, total):
        slots, copies = torch.zeros(total, dtype=I64, device="cuda"), torch.zeros((len(q_start) - 1, 3), dtype=I32, device="cuda")
        ls.ls_pages_advance(d.book, d.t(q_start), slots, copies, d.ws, seqs=d.t(seqs), keep=d.t(keep, I64))
        assert d.status() == 5
        assert (slots == -1).all() and (copies == -1).all()
        assert all(torch.equal(a, b) for a, b in zip(before, (d.refs, d.table, d.kv_len)))

    refused([0, 6], None, [0, 1, 2], 2)                 # out of range
    refused([0, -1], None, [0, 1, 2], 2)
    refused([1, 0, 1], None, [0, 1, 2, 3], 3)           # named twice
    refused([0, 1], [6, 9], [0, 1, 2], 2)               # keeps more than it has
    refused([0, 1], [-1, 9], [0, 1, 2], 2)
    refused([0, 1], None, [0, 2, 1], 2)                 # does not rise
    refused([0, 1], None, [1, 1, 2], 2)                 # does not begin at 0
    refused([0, 1], None, [0, 1, 2], 3)                 # does not end at total_q
    refused([0, 1], None, [0, 1, 4], 3)
    for src, dst, lens in (([0, 0], [3, 3], None), ([0], [0], None), ([0, 3], [3, 4], None), ([0], [6], None), ([-1], [2], None),
                           ([0], [3], [6]), ([0], [3], [-1])):
        ls.ls_pages_fork(d.book, d.t(src), d.t(dst), d.ws, lens=d.t(lens, I64))
        assert d.status() == 5
        assert all(torch.equal(a, b) for a, b in zip(before, (d.refs, d.table, d.kv_len)))
    ls.ls_pages_release(d.book, d.ws, d.t([1, 1]))
    assert d.status() == 5 and torch.equal(before[0], d.refs)
    d.kv_len[5] = 33                                    # a length past its row
    for call in (lambda: ls.ls_pages_release(d.book, d.ws), lambda: ls.ls_pages_fork(d.book, d.t([5]), d.t([4]), d.ws)):
        call()
        assert d.status() == 5 and torch.equal(before[0], d.refs)


def test_page_ids_outside_the_pool(cuda_device):
    d = Device(20, 4, 4, 6)
    d.advance([0, 1], None, [10, 6])
    d.table[0, 1] = 20
    d.table[1, 1] = -3
    ls.ls_pages_fork(d.book, d.t([0]), d.t([2]), d.ws)
    assert d.status() == 5 and d.refs.tolist()[:5] == [2, 1, 2, 1, 1]
    # sequence 1 ends in a page that is none: it does not grow
    slots, copies = torch.zeros(2, dtype=I64, device="cuda"), torch.zeros((1, 3), dtype=I32, device="cuda")
    ls.ls_pages_advance(d.book, d.t([0, 2]), slots, copies, d.ws, seqs=d.t([1]))
    assert d.status() == 5 and slots.tolist() == [-1, -1] and d.kv_len[1] == 6
    copies = torch.zeros((10, 3), dtype=I32, device="cuda")
    ls.ls_pages_compact(d.book, d.table, d.refs, copies, d.ws)
    assert d.status() == 5 and d.table[0, 1] == 20
    ls.ls_pages_release(d.book, d.ws)
    assert d.status() == 5 and d.refs.tolist()[:5] == [0, 1, 0, 0, 1]
    ls.ls_clear_device_status(d.ws)
    d.table[:] = 1
    d.refs[:] = 0
    d.kv_len[:] = 4                                     # entries that no reference counts
    ls.ls_pages_release(d.book, d.ws)
    assert d.status() == 5 and (d.refs == 0).all()


def pools(pages, hkv, page, dim, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    raw = [torch.randint(0, 256, (pages, hkv, page, dim * dtype.itemsize), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2)]
    exps = [torch.randint(-128, 128, (pages, hkv, page), generator=g, dtype=torch.int8, device="cuda") for _ in range(2)]
    cache = ls.kv_cache_from(raw[0].view(dtype), raw[1].view(dtype), *(exps if dtype == torch.float8_e4m3fn else (None, None)))
    return cache, raw, exps


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("hkv,page,dim", [(1, 16, 64), (3, 7, 128), (2, 1, 256), (4, 256, 256), (1, 1100, 64)])
def test_copies_are_bit_for_bit(cuda_device, dtype, hkv, page, dim):
    cache, raw, exps = pools(9, hkv, page, dim, dtype)
    copies = [(0, 5, page), (0, 6, 1), (2, 7, page // 2), (3, 8, 0), (-1, 4, page), (1, -1, page), (1, 1, page), (3, 3, 1)]
    want = [t.clone() for t in raw + (exps if dtype == torch.float8_e4m3fn else [])]
    for a, b, n in copies:
        for w in want:
            if a >= 0 and b >= 0:
                w[b, :, :n] = w[a, :, :n]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ls.ls_cache_copy_pages(cache, torch.tensor(copies, dtype=I32, device="cuda"), ws)
    ls.ls_read_device_status(ws)
    assert all(torch.equal(a, b) for a, b in zip(want, raw + exps))
    for bad in ((9, 4, 1), (0, 9, 1), (0, 4, page + 1), (0, 4, -1)):
        ls.ls_cache_copy_pages(cache, torch.tensor([bad], dtype=I32, device="cuda"), ws)
        with pytest.raises(ls.LsError):
            ls.ls_read_device_status(ws)
    assert all(torch.equal(a, b) for a, b in zip(want, raw + exps))
    ls.ls_cache_copy_pages(cache, torch.zeros((0, 3), dtype=I32, device="cuda"))


def test_more_entries_than_one_row_of_blocks(cuda_device):
    cache, raw, exps = pools(4, 1, 1, 64, torch.float8_e4m3fn)
    copies = torch.full((70000, 3), -1, dtype=I32, device="cuda")
    copies[69999] = torch.tensor([2, 3, 1])
    copies[65535] = torch.tensor([0, 1, 1])
    ls.ls_cache_copy_pages(cache, copies)
    for t in raw + exps:
        assert torch.equal(t[3], t[2]) and torch.equal(t[1], t[0])


def test_graph_of_a_fork_with_its_copies(cuda_device):
    """Fork, advance and copy captured together on a side stream, each starting under the one before it; replays begin
    by taking back what the replay before gave."""
    d = Device(60, 8, 5, 6)
    d.advance([0], None, [21])
    cache, raw, exps = pools(60, 2, 8, 64, torch.float8_e4m3fn)
    src, dst, q_start = d.t([0] * 4), d.t([1, 2, 3, 4]), d.t([0, 1, 3, 4, 9])
    slots, copies = torch.zeros(9, dtype=I64, device="cuda"), torch.zeros((4, 3), dtype=I32, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        ls.ls_pages_fork(d.book, src, dst, d.ws)
        ls.ls_pages_advance(d.book, q_start, slots, copies, d.ws, seqs=dst)
        ls.ls_cache_copy_pages(cache, copies, d.ws)
    for _ in range(4):
        graph.replay()
        d.ref.fork([0] * 4, [1, 2, 3, 4], [21] * 4)
        want = d.ref.advance([1, 2, 3, 4], [21] * 4, [1, 2, 1, 5])
        torch.cuda.synchronize()
        assert slots.tolist() == want[0] and [tuple(r) for r in copies.tolist()] == want[1]
        d.same()
        for a, b, n in want[1]:
            assert all(torch.equal(t[a, :, :n], t[b, :, :n]) for t in raw + exps)


def test_pages_far_into_a_pool(cuda_device):
    """Byte offsets past 2^32."""
    pages = 40000
    shape = (pages, 2, 256, 256)                        # 5.2 GB a pool
    k = torch.empty(shape, dtype=torch.uint8, device="cuda")
    v = torch.empty(shape, dtype=torch.uint8, device="cuda")
    exps = [torch.zeros(shape[:3], dtype=torch.int8, device="cuda") for _ in range(2)]
    for i, t in enumerate((k, v)):
        t[5] = torch.randint(0, 256, shape[1:], dtype=torch.uint8, device="cuda")
        t[pages - 1] = 17 + i
    cache = ls.kv_cache_from(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), *exps)
    ls.ls_cache_copy_pages(cache, torch.tensor([[5, pages - 2, 256], [pages - 1, 6, 100]], dtype=I32, device="cuda"))
    for i, t in enumerate((k, v)):
        assert torch.equal(t[pages - 2], t[5]) and (t[6, :, :100] == 17 + i).all() and (t[pages - 1] == 17 + i).all()


def test_graph_of_a_step(cuda_device):
    """A captured advance replayed: each replay drops what the one before took."""
    d = Device(100, 4, 3, 20)
    d.advance([0, 1, 2], None, [9, 3, 4])
    q_start, keep = d.t([0, 2, 5, 6]), d.t([8, 3, 4], I64)
    slots, copies = torch.zeros(6, dtype=I64, device="cuda"), torch.zeros((3, 3), dtype=I32, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        ls.ls_pages_advance(d.book, q_start, slots, copies, d.ws, keep=keep)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = d.ref.advance(range(3), [8, 3, 4], [2, 3, 1])
        assert slots.tolist() == want[0]
        d.same()
