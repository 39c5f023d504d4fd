"""Forking, freeing and compacting page-table rows against a plain Python form
(everything is compared exactly), and the operators together as a server uses
them: prompt, fork, shared decode, eviction, compaction, free."""
import numpy as np
import pytest
import torch

from operator_helpers import assert_within, prefix_reference, prompt_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Book:
    """Host mirror of a pool and its tables."""

    def __init__(self, seed, layers, pages, hkv, d, dtype, rows, max_pages):
        self.rng = np.random.default_rng(seed)
        pool = self.rng.standard_normal((layers, pages, hkv, 2, 16, d)).astype(np.float32)
        self.dpool = torch.from_numpy(pool).to(DT[dtype]).to(DEV)
        self.pool = self.dpool.float().cpu().numpy()
        self.table = np.full((rows, max_pages), -7, dtype=np.int32)
        self.counts = [0] * rows
        self.refs = np.zeros(pages, dtype=np.int32)
        self.mask = np.zeros(pages, dtype=np.int32)
        self.pos = np.full((pages, 16), -1, dtype=np.int32)
        self.free = list(self.rng.permutation(pages))

    def fill(self, row, pages, drop=0.0, last=16):
        for j in range(pages):
            p = self.free.pop()
            self.table[row, j] = p
            self.refs[p] = 1
            n = last if j == pages - 1 else 16
            live = (np.arange(16) < n) & (self.rng.random(16) >= drop)
            self.mask[p] = int((live << np.arange(16)).sum())
            self.pos[p] = np.where(live, 16 * j + np.arange(16), -1)
        self.counts[row] = pages

    def upload(self):
        self.dtable, self.drefs, self.dmask, self.dpos = (torch.from_numpy(x.copy()).to(DEV) for x in
                                                          (self.table, self.refs, self.mask, self.pos))

    def same(self, positions=True):
        torch.cuda.synchronize()
        assert np.array_equal(self.dtable.cpu().numpy(), self.table)
        assert np.array_equal(self.drefs.cpu().numpy(), self.refs)
        assert np.array_equal(self.dmask.cpu().numpy(), self.mask)
        if positions:
            assert np.array_equal(self.dpos.cpu().numpy(), self.pos)
        assert np.array_equal(self.dpool.float().cpu().numpy(), self.pool)

    # plain forms
    def fork(self, parents, children, share):
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        need = 0
        for a in parents:
            n = self.counts[a]
            need += (int(n > 0 and self.mask[self.table[a, n - 1]] != 0xFFFF) if share else n)
        if need > len(free):
            return need - len(free)
        masks = self.mask.copy()
        for a, c in zip(parents, children):
            n = self.counts[a]
            for j in range(n):
                p = self.table[a, j]
                if share and not (j == n - 1 and masks[p] != 0xFFFF):
                    self.refs[p] += 1
                    self.table[c, j] = p
                    continue
                new = free.pop(0)
                self.table[c, j] = new
                self.refs[new] = 1
                self.mask[new] = self.mask[p]
                self.pos[new] = self.pos[p]
                self.pool[:, new] = self.pool[:, p]
            self.counts[c] = n
        return 0

    def free_rows(self, seqs):
        for s in seqs:
            for j in range(self.counts[s]):
                p = self.table[s, j]
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    self.mask[p] = 0
                self.table[s, j] = -1
            self.counts[s] = 0

    def compact(self):
        new = []
        for r, n in enumerate(self.counts):
            ids = [int(p) for p in self.table[r, :n]]
            mine = [p for p in ids if self.refs[p] == 1]
            tokens = sum(bin(self.mask[p]).count("1") for p in mine)
            keep = -(-tokens // 16)
            front, tail = mine[:keep], mine[keep:]
            holes = [(p, s) for p in front for s in range(16) if not (self.mask[p] >> s) & 1]
            movers = [(p, s) for p in tail for s in range(16) if (self.mask[p] >> s) & 1]
            for (p, s), (a, b) in zip(holes, movers):
                self.pool[:, p, :, :, s] = self.pool[:, a, :, :, b]
                self.mask[p] |= 1 << s
                self.pos[p, s] = self.pos[a, b]
            for p in tail:
                self.mask[p] = self.refs[p] = 0
                self.pos[p] = -1
            left = [p for p in ids if p not in tail]
            self.table[r, :n] = left + [-1] * (n - len(left))
            self.counts[r] = len(left)
            new.append(len(left))
        return new


@pytest.mark.parametrize("dtype,layers,hkv,d", [("bf16", 3, 2, 128), ("f32", 1, 1, 64), ("bf16", 2, 5, 64)])
@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("last", [1, 15, 16])
def test_fork_and_free(dtype, layers, hkv, d, share, last):
    from tiered_kv_cache_split_gb300 import fork_sequences, free_sequences
    b = Book(last, layers, 90, hkv, d, dtype, 9, 12)
    b.fill(0, 7, last=last)
    b.fill(4, 1, drop=0.4)
    b.fill(5, 12, drop=0.1, last=last)
    b.upload()
    parents, children = [0, 0, 4, 5, 7], [1, 2, 3, 6, 8]         # row 7 is empty: its child is too
    counts = list(b.counts)
    st = fork_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, parents, children, share=share, positions=b.dpos)
    assert b.fork(parents, children, share) == 0
    b.same()
    assert st.item() == 0
    st = free_sequences(b.dtable, b.counts, b.drefs, b.dmask, [0, 3, 8, 6])
    b.free_rows([0, 3, 8, 6])
    b.same()
    assert st.item() == 0
    # the ids just freed are the ones a next fork takes
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [1, 5], [0, 6], share=share, positions=b.dpos)
    assert b.fork([1, 5], [0, 6], share) == st.item() == 0
    b.same()


@pytest.mark.parametrize("share", [True, False])
def test_a_fork_that_lacks_pages_changes_nothing(share):
    from tiered_kv_cache_split_gb300 import fork_sequences
    b = Book(1, 2, 10, 1, 64, "bf16", 4, 8)
    b.fill(0, 8, last=3)
    b.upload()
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0, 0, 0], [1, 2, 3], share=share, positions=b.dpos)
    assert st.item() == (1 if share else 22) == b.fork([0, 0, 0], [1, 2, 3], share)
    b.same()


@pytest.mark.parametrize("bad", [-1, 40, 2 ** 31 - 1, "free"])
def test_rows_that_list_pages_not_held(bad):
    from tiered_kv_cache_split_gb300 import compact_sequences, fork_sequences, free_sequences
    b = Book(2, 1, 40, 1, 64, "f32", 4, 8)
    b.fill(0, 6, drop=0.5)
    b.fill(1, 5, drop=0.5)
    b.table[0, 3] = b.free[0] if bad == "free" else bad
    b.upload()
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0, 1], [2, 3], positions=b.dpos)
    b.same()
    assert st.item() == -1
    b2 = b.counts[0]
    b.counts[0] = 0
    new = b.compact()
    b.counts[0] = b2
    got = compact_sequences(b.dpool, b.dtable, [6, 5, 0, 0], b.drefs, b.dmask, positions=b.dpos)
    assert got.tolist() == [-1] + new[1:]
    b.same()
    st = free_sequences(b.dtable, b.counts, b.drefs, b.dmask, [0])
    held = [p for p in b.table[0, :6] if 0 <= p < 40 and b.refs[p] > 0]
    b.refs[held] = 0
    b.mask[held] = 0
    b.table[0, :6] = -1
    b.same()
    assert st.item() == -1


@pytest.mark.parametrize("pages", [5000, 16384 + 77, 40000])
def test_the_lowest_free_ids_are_found_in_large_pools(pages):
    from tiered_kv_cache_split_gb300 import fork_sequences
    b = Book(3, 1, pages, 1, 64, "bf16", 3, 64)
    b.fill(0, 40, last=5)
    b.refs[:] = 1                              # all held elsewhere, but for a few free ids
    free = np.sort(b.rng.choice(pages, 41, replace=False))
    free = np.array([p for p in free if p not in set(b.table[0, :40])])
    b.refs[free] = 0
    b.upload()
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0], [2], share=True, positions=b.dpos)
    assert b.fork([0], [2], True) == st.item() == 0
    b.same()
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0], [1], share=False, positions=b.dpos)
    assert b.fork([0], [1], False) == st.item()
    b.same()


@pytest.mark.parametrize("dtype,layers,hkv,d", [("bf16", 3, 2, 128), ("f32", 1, 1, 64), ("f32", 2, 3, 128)])
@pytest.mark.parametrize("drop", [0.0, 0.05, 0.5, 0.95, 1.0])
def test_compact(dtype, layers, hkv, d, drop):
    from tiered_kv_cache_split_gb300 import compact_sequences
    b = Book(int(drop * 100), layers, 160, hkv, d, dtype, 6, 70)
    for r, n in enumerate([1, 70, 17, 0, 33, 2]):
        b.fill(r, n, drop=drop, last=1 + (7 * r) % 16)
    b.upload()
    counts = list(b.counts)
    got = compact_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, positions=b.dpos)
    assert got.tolist() == b.compact()
    b.same()
    again = compact_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, positions=b.dpos)   # nothing left to move
    assert again.tolist() == b.counts
    b.same()


def test_compact_leaves_shared_pages_and_works_without_counts_or_positions():
    from tiered_kv_cache_split_gb300 import compact_sequences, fork_sequences
    b = Book(6, 2, 80, 2, 64, "bf16", 3, 20)
    b.fill(0, 12, drop=0.3, last=9)
    b.upload()
    assert fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0], [1], positions=b.dpos).item() == b.fork([0], [1], True)
    b.fill(2, 15, drop=0.6)
    for p in range(3):                          # row 1 goes on alone, with pages that lose tokens
        new = b.free.pop()
        while b.refs[new]:
            new = b.free.pop()
        b.table[1, 12 + p] = new
        b.refs[new], b.mask[new] = 1, [0x00F0, 0x8001, 0x0003][p]
        b.pos[new] = np.where((b.mask[new] >> np.arange(16)) & 1, 192 + 16 * p + np.arange(16), -1)
    b.counts[1] = 15
    b.upload()
    counts = list(b.counts)
    got = compact_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, positions=b.dpos)
    assert got.tolist() == b.compact()
    b.same()
    c = Book(7, 2, 40, 2, 64, "bf16", 1, 20)
    c.fill(0, 20, drop=0.4)
    c.upload()
    got = compact_sequences(c.dpool, c.dtable, [20], None, c.dmask)
    assert got.tolist() == c.compact()
    c.drefs = torch.from_numpy(c.refs).to(DEV)
    c.same(positions=False)


def test_the_longest_row():
    """16384 pages: every thread of the plan holds its most pages."""
    from tiered_kv_cache_split_gb300 import compact_sequences
    b = Book(8, 1, 16384 + 3, 1, 64, "bf16", 2, 16384)
    b.fill(0, 16384, drop=0.5)
    b.fill(1, 2, drop=0.5)
    b.upload()
    counts = list(b.counts)
    got = compact_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, positions=b.dpos)
    assert got.tolist() == b.compact()
    b.same()


def test_captured_fork_and_free_replay():
    from tiered_kv_cache_split_gb300 import fork_sequences, free_sequences
    b = Book(9, 2, 60, 2, 64, "bf16", 4, 8)
    b.fill(0, 8, last=7)
    b.upload()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0, 0], [1, 3], positions=b.dpos)
        two = free_sequences(b.dtable, [8, 8, 0, 8], b.drefs, b.dmask, [1])
    for _ in range(2):                          # the second time row 3's pages are listed again
        graph.replay()
    torch.cuda.synchronize()
    assert one.item() == two.item() == 0
    b.fork([0, 0], [1, 3], True)
    b.free_rows([1])
    b.counts[3] = 0                             # the replay overwrites row 3: its copied page stays held
    b.fork([0, 0], [1, 3], True)
    b.free_rows([1])
    b.same()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prompt_its_chains_an_eviction_and_their_end(dtype):
    """One prompt attended, stored, forked into three chains that decode over the
    shared pages, lose half of their own tokens, are compacted and freed."""
    from tiered_kv_cache_split_gb300 import (compact_sequences, fork_sequences, free_sequences, paged_attention,
                                             prompt_attention, shared_prefix_attention)
    hq, hkv, d, n, dt = 8, 2, 64, 150, DT[dtype]
    gen = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(n, h, d, generator=gen).to(dt).to(DEV) for h in (hq, hkv, hkv))
    out = prompt_attention(q, k, v, [n])
    want, bound = prompt_reference(q, k, v, [n], [n])
    assert_within(out, want, bound, "prompt")
    b = Book(4, 1, 80, hkv, d, dtype, 4, 20)
    b.fill(0, 10, last=6)
    for j in range(10):
        rows = min(16, n - 16 * j)
        for x, t in enumerate((k, v)):
            b.dpool[0, b.table[0, j], :, x, :rows] = t[16 * j:16 * j + rows].transpose(0, 1)
    b.pool = b.dpool.float().cpu().numpy()
    b.upload()
    fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, [0, 0, 0], [1, 2, 3], positions=b.dpos)
    b.fork([0, 0, 0], [1, 2, 3], True)
    b.same()
    # each chain appends its own tokens: the rest of its copied page, then new pages
    for r, more in ((1, 40), (2, 3), (3, 90)):
        at = n
        while at < n + more:
            j, s = at // 16, at % 16
            if s == 0:
                p = int(np.nonzero(b.refs == 0)[0][0])
                b.table[r, j], b.refs[p], b.counts[r] = p, 1, j + 1
            p = b.table[r, j]
            b.mask[p] |= 1 << s
            b.pos[p, s] = at
            new = torch.randn(2, hkv, d, generator=gen).to(dt)
            b.dpool[0, p, :, :, s] = new.transpose(0, 1).to(DEV)
            at += 1
    b.pool = b.dpool.float().cpu().numpy()
    b.upload()
    live = [1, 2, 3]
    dq = torch.randn(3, hq, d, generator=gen).to(dt).to(DEV)
    counts = [b.counts[r] for r in live]
    alpha = torch.zeros(3, hkv, 20 * 16, device=DEV)
    got = shared_prefix_attention(dq, b.dpool[0], b.dtable[1:].contiguous(), b.dmask, counts, 9, alpha_sum=alpha)
    want, bound, aw, ab = prefix_reference(dq, b.dpool[0], b.table[1:], b.mask, counts, 9)
    assert_within(got, want, bound, "decode")
    assert_within(alpha, aw, ab + 1e-9, "alpha")
    # the chains' own tokens with the least weight leave, the rest is compacted
    w = alpha.sum(1).cpu().numpy()
    for i, r in enumerate(live):
        own = [(w[i, 16 * j + s], j, s) for j in range(9, b.counts[r]) for s in range(16) if (b.mask[b.table[r, j]] >> s) & 1]
        for _, j, s in sorted(own)[:len(own) // 2]:
            b.mask[b.table[r, j]] &= ~(1 << s)
            b.pos[b.table[r, j], s] = -1
    b.upload()
    before = shared_prefix_attention(dq, b.dpool[0], b.dtable[1:].contiguous(), b.dmask, counts, 9)
    want, bound, _, _ = prefix_reference(dq, b.dpool[0], b.table[1:], b.mask, counts, 9)
    assert_within(before, want, bound, "after the eviction")
    new = compact_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, positions=b.dpos).tolist()
    assert new == b.compact()
    b.same()
    counts = new[1:]
    table = b.dtable[1:].contiguous()
    after = shared_prefix_attention(dq, b.dpool[0], table, b.dmask, counts, 9)
    assert_within(after, want, bound, "after the compaction")          # the same tokens, in other slots
    plain = paged_attention(dq, b.dpool[0], torch.where(table < 0, 0, table), b.dmask, counts)
    assert_within(plain, want, 2 * bound, "paged")
    assert free_sequences(b.dtable, b.counts, b.drefs, b.dmask, [0, 1, 2, 3]).item() == 0
    torch.cuda.synchronize()
    assert (b.drefs == 0).all() and (b.dmask == 0).all()
