"""Shared-prefix decode attention against a float64 form of its definition, and
against the paged attention it extends (bounds: operator_helpers)."""
import numpy as np
import pytest
import torch

from operator_helpers import assert_within, f64, prefix_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, dtype, hq, hkv, d, shared, own, holes=True):
    """Pools whose empty slots hold NaN; shared and own are pages."""
    rng = np.random.default_rng(seed)
    B, pages = len(own), shared + sum(own) + 3
    pool = rng.standard_normal((pages, hkv, 2, 16, d)).astype(np.float32)
    pool[:, :, 0] *= rng.lognormal(0, 0.6, (pages, hkv, 16, 1)).astype(np.float32)
    ids = rng.permutation(pages)
    counts = [shared + n for n in own]
    table = np.full((B, max(counts + [1])), 10 ** 6, dtype=np.int32)    # entries past a row's count are never read
    table[:, :shared] = ids[:shared]
    at = shared
    for b, n in enumerate(own):
        table[b, shared:shared + n] = ids[at:at + n]
        at += n
    masks = np.full(pages, 0xFFFF, dtype=np.int64)
    if holes:
        for p in rng.choice(pages, size=max(1, pages // 3), replace=False):
            masks[p] = int(rng.integers(0, 0xFFFF))
    pool[~((masks[:, None] >> np.arange(16)) & 1).astype(bool).reshape(pages, 1, 1, 16).repeat(hkv, 1).repeat(2, 2)] = np.nan
    q = rng.standard_normal((B, hq, d)).astype(np.float32)
    dev = lambda x, t: torch.from_numpy(x).to(t).to(DEV)   # noqa: E731
    return dev(q, DT[dtype]), dev(pool, DT[dtype]), dev(table, torch.int32), dev(masks.astype(np.int32), torch.int32), counts, table, masks


def check(dtype, hq, hkv, d, shared, own, seed=0, holes=True, alpha=True):
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make(seed, dtype, hq, hkv, d, shared, own, holes)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    a = torch.full((len(own), hkv, table.shape[1] * 16), 0.25, device=DEV) if alpha else None
    out = shared_prefix_attention(q, pool, table, mask, counts, shared, alpha_sum=a, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    want, bound, aw, ab = prefix_reference(q, pool, tb, mk, counts, shared)
    assert_within(out, want, bound, "out")
    if alpha:
        assert_within(a, aw + 0.25, ab + 2.0 ** -24 * 2.5, "alpha")     # 0.25 + alpha is rounded once more
        assert (a[:, :, :shared * 16] == 0.25).all()
        for b, n in enumerate(counts):
            assert (a[b, :, n * 16:] == 0.25).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (28, 4, 128)])
@pytest.mark.parametrize("shared,own", [(0, [1]), (0, [5, 1, 17]), (1, [0]), (8, [0, 0]), (7, [1, 9, 0, 8]), (40, [3] * 5),
                                        (129, [1, 2, 30, 7, 8, 9, 16, 17]), (0, [0, 2])])
def test_lengths(dtype, hq, hkv, d, shared, own):
    check(dtype, hq, hkv, d, shared, own, seed=shared)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,batch", [(1, 1, 128, 3), (6, 6, 64, 40), (6, 2, 128, 64), (64, 1, 64, 5), (5, 1, 128, 26),
                                            (16, 8, 64, 64), (12, 3, 128, 33)])
def test_head_layouts_and_batches(dtype, hq, hkv, d, batch):
    """Rows (batch x group) below, at and over one and two row tiles."""
    check(dtype, hq, hkv, d, 20, [(5 * b) % 11 for b in range(batch)], seed=batch)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_without_alpha_and_without_holes(dtype):
    check(dtype, 8, 2, 128, 300, [4, 40, 9], holes=False, alpha=False)


def test_all_slots_empty_gives_zero():
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, _, _ = make(3, "bf16", 8, 2, 64, 4, [2, 0])
    mask.zero_()
    a = torch.zeros(2, 2, table.shape[1] * 16, device=DEV)
    out = shared_prefix_attention(q, pool, table, mask, counts, 4, alpha_sum=a)
    assert (out == 0).all() and (a == 0).all()


def test_a_page_id_outside_the_pool_reads_as_an_empty_page():
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    for dtype in ("bf16", "f32"):
        q, pool, table, mask, counts, tb, mk = make(4, dtype, 8, 2, 64, 6, [9, 12], holes=False)
        without = shared_prefix_attention(q, pool, table, mask, counts, 6)
        for bad in (-1, pool.shape[0], 2 ** 31 - 1, -2 ** 31):
            t2 = table.clone()
            t2[0, 7], t2[0, 3], t2[1, 3] = bad, bad, bad
            m2 = mk.copy()
            tb2 = tb.copy()
            m2[[tb[0, 7], tb[0, 3]]] = 0
            got = shared_prefix_attention(q, pool, t2, mask, counts, 6)
            want, bound, _, _ = prefix_reference(q, pool, tb2, m2, counts, 6)
            assert_within(got, want, bound, f"id {bad}")
        assert not torch.equal(without, got)


@pytest.mark.parametrize("dtype,g", [("bf16", 7), ("f32", 4)])
def test_agrees_with_paged_attention_on_the_same_table(dtype, g):
    """Both are within their bound of the definition, so within twice it of each other."""
    from tiered_kv_cache_split_gb300 import paged_attention, shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make(5, dtype, 2 * g, 2, 128, 33, [5, 60, 1], holes=False)
    table = torch.where(table < pool.shape[0], table, 0)
    a, b = (torch.zeros(3, 2, table.shape[1] * 16, device=DEV) for _ in range(2))
    got = shared_prefix_attention(q, pool, table, mask, counts, 33, alpha_sum=a)
    other = paged_attention(q, pool, table, mask, counts, alpha_sum=b)
    _, bound, _, ab = prefix_reference(q, pool, tb, mk, counts, 33)
    assert_within(got, f64(other), 2 * bound)
    assert_within(a[:, :, 33 * 16:], f64(b)[:, :, 33 * 16:], 2 * ab[:, :, 33 * 16:] + 1e-9)


def test_two_streams_and_a_captured_graph():
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    x = make(6, "bf16", 28, 4, 128, 50, [3, 20, 9])[:5]
    y = make(7, "bf16", 28, 4, 128, 50, [3, 20, 9])[:5]
    one, two = shared_prefix_attention(*x, 50), shared_prefix_attention(*y, 50)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(shared_prefix_attention(*x, 50, stream=s), shared_prefix_attention(*y, 50, stream=t)) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, one) and torch.equal(b, two) for a, b in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = shared_prefix_attention(*x, 50)
    x[0].copy_(y[0]), x[1].copy_(y[1]), x[2].copy_(y[2]), x[3].copy_(y[3])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, two)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_past_32_bits(dtype):
    """A pool of more than 2^32 bytes (2^31 elements in bf16) whose last pages are used."""
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make(8, dtype, 8, 4, 128, 9, [4, 20, 1])
    want, bound, aw, ab = prefix_reference(q, pool, tb, mk, counts, 9)
    n = pool.shape[0]
    record = pool[0].numel() * pool.element_size()
    pages = (9 << 29) // record
    big = torch.empty((pages, *pool.shape[1:]), dtype=pool.dtype, device=DEV)
    big[pages - n:] = pool
    bmask = torch.zeros(pages, dtype=torch.int32, device=DEV)
    bmask[pages - n:] = mask
    alpha = torch.zeros(3, 4, table.shape[1] * 16, device=DEV)
    out = shared_prefix_attention(q, big, torch.where(table < n, table + (pages - n), table), bmask, counts, 9, alpha_sum=alpha)
    assert_within(out, want, bound, "out")
    assert_within(alpha, aw, ab, "alpha")


def test_a_wait_that_runs_out_is_reported_and_the_device_goes_on():
    from tiered_kv_cache_split_gb300 import _lib as L, shared_prefix_attention
    x = make(9, "bf16", 8, 2, 64, 40, [3, 9])[:5]
    good = shared_prefix_attention(*x, 40)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    L.check(L.load().tkv_test_stall_next_tiles(5_000_000))
    shared_prefix_attention(*x, 40, status=status)
    torch.cuda.synchronize()
    assert status.item() == 1
    assert torch.equal(shared_prefix_attention(*x, 40), good)


@pytest.mark.parametrize("hq,hkv,d,shared,own", [(28, 4, 128, 1200, [3, 90, 0, 17, 1] * 6), (32, 32, 128, 600, [40, 200] * 4), (16, 2, 64, 2000, [50] * 20)])
def test_long_units_repeated_over_a_scratch_of_nan(hq, hkv, d, shared, own):
    """Many long key ranges at once, whose copies land in any order, with holes all over."""
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make(3, "bf16", hq, hkv, d, shared, own)
    scratch = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = None
    for _ in range(60):
        out = shared_prefix_attention(q, pool, table, mask, counts, shared, scratch=scratch.fill_(255), status=status)
        if first is None:
            first = out
            want, bound, _, _ = prefix_reference(q, pool, tb, mk, counts, shared)
            assert_within(out, want, bound, "out")
        assert status.item() == 0 and torch.equal(out, first)
