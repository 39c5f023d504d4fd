"""Edges of the prompt, shared-prefix and page operators: buffers of exactly the
stated size, calls beside work on another stream. Bounds are those of
operator_helpers."""
import ctypes

import numpy as np
import pytest
import torch

from operator_helpers import assert_within, attend, f64, prefix_reference, prompt_reference
from test_gpu_pages import Book
from test_gpu_prompt_attention import make as make_prompt
from test_gpu_shared_prefix import make as make_prefix

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 1 << 20


class Guarded:
    """`size` bytes of NaN between two guards."""

    def __init__(self, size):
        self.all = torch.full((size + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=DEV)
        self.mid = self.all[GUARD:GUARD + size].fill_(255)

    def intact(self):
        return bool((self.all[:GUARD] == 0xA5).all() and (self.all[GUARD + self.mid.numel():] == 0xA5).all())


def size_of(call, *args):
    from tiered_kv_cache_split_gb300 import _lib as L
    n = ctypes.c_size_t()
    L.check(getattr(L.load(), call + "_scratch_size")(*args, ctypes.byref(n)))
    return n.value


def ints(v):
    return (ctypes.c_int32 * len(v))(*v)


def code(dtype):
    from tiered_kv_cache_split_gb300 import _lib as L
    return L.DTYPE_BF16 if dtype == "bf16" else L.DTYPE_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,shared,own", [(28, 4, 128, 16, [0] * 31), (28, 4, 128, 256, [0] * 64), (8, 2, 64, 8, [0, 0]),
                                                 (1, 1, 128, 1, [0]), (8, 2, 64, 20, [0, 3, 0]), (32, 32, 128, 40, [1, 9]),
                                                 (6, 2, 64, 0, [2, 0, 5])])
@pytest.mark.parametrize("alpha", [True, False])
def test_a_decode_stays_inside_a_scratch_of_the_stated_size(dtype, hq, hkv, d, shared, own, alpha):
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make_prefix(shared, dtype, hq, hkv, d, shared, own)
    width = table.shape[1]
    a = torch.zeros(len(own), hkv, width * 16, device=DEV) if alpha else None
    s = Guarded(size_of("tkv_shared_prefix_attention", len(own), hq, hkv, d, code(dtype), ints(counts), width, shared, int(alpha)))
    out = shared_prefix_attention(q, pool, table, mask, counts, shared, alpha_sum=a, scratch=s.mid)
    assert s.intact()
    want, bound, aw, ab = prefix_reference(q, pool, tb, mk, counts, shared)
    assert_within(out, want, bound, "out")
    if alpha:
        assert_within(a, aw, ab, "alpha")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,q_lens,k_lens", [(8, 2, 128, [20], [3000]), (28, 4, 128, [1, 300, 0, 7], [5000, 300, 4, 900]),
                                                    (6, 2, 64, [20], [970]), (4, 4, 64, [500], [2000])])
def test_a_prompt_stays_inside_a_scratch_of_the_stated_size(dtype, hq, hkv, d, q_lens, k_lens):
    from tiered_kv_cache_split_gb300 import prompt_attention
    x = make_prompt(1, dtype, hq, hkv, d, q_lens, k_lens)
    need = size_of("tkv_prompt_attention", len(q_lens), ints(q_lens), ints(k_lens), hq, hkv, d, code(dtype))
    assert need > 0
    s = Guarded(need)
    out = prompt_attention(*x, q_lens, k_lens, scratch=s.mid)
    assert s.intact()
    assert_within(out, *prompt_reference(*x, q_lens, k_lens))


@pytest.mark.parametrize("share", [True, False])
def test_fork_and_compact_stay_inside_a_scratch_of_the_stated_size(share):
    from tiered_kv_cache_split_gb300 import compact_sequences, fork_sequences
    b = Book(1, 2, 400, 2, 64, "bf16", 12, 40)
    b.fill(0, 37, last=5)
    b.fill(1, 3, drop=0.5)
    b.upload()
    parents, children = [0, 1, 0, 1, 0, 0], [2, 3, 5, 7, 11, 4]
    s = Guarded(size_of("tkv_fork_sequences", 12, 40, ints(b.counts), 6, ints(parents), ints(children), int(share)))
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, parents, children, share=share, positions=b.dpos, scratch=s.mid)
    assert b.fork(parents, children, share) == st.item() == 0 and s.intact()
    b.same()
    for r in (6, 8):                            # empty pages ahead of as many full ones: the most moves
        b.free = [p for p in range(400) if b.refs[p] == 0]
        b.fill(r, 40)
        for p in b.table[r, 0:20]:
            b.mask[p], b.pos[p] = 0, -1
    b.upload()
    counts = list(b.counts)
    s = Guarded(size_of("tkv_compact_sequences", 12, 40, ints(counts)))
    got = compact_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, positions=b.dpos, scratch=s.mid)
    assert got.tolist() == b.compact() and s.intact()
    b.same()


class Behind:
    """Blocks of the current stream's memory, given back while copies out of
    them wait behind a long kernel there."""

    def __init__(self, sizes):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        blocks = [torch.full((n,), 77, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        self.copies = [torch.zeros_like(x) for x in blocks]
        torch.cuda.synchronize()
        torch.cuda._sleep(200_000_000)          # about 0.1 s
        for x, y in zip(blocks, self.copies):
            y.copy_(x)

    def check(self):
        torch.cuda.synchronize()
        assert all(bool((y == 77).all()) for y in self.copies)


def test_calls_on_another_stream_beside_work_that_still_uses_freed_blocks():
    from tiered_kv_cache_split_gb300 import (compact_sequences, fork_sequences, free_sequences, prompt_attention,
                                             shared_prefix_attention)
    side = torch.cuda.Stream()
    q_lens, k_lens = [40, 300], [3000, 300]
    x = make_prompt(2, "bf16", 8, 2, 128, q_lens, k_lens)
    need = size_of("tkv_prompt_attention", 2, ints(q_lens), ints(k_lens), 8, 2, 128, code("bf16"))
    good = prompt_attention(*x, q_lens, k_lens)
    b = Behind([need, good.numel() * 2])
    got = prompt_attention(*x, q_lens, k_lens, stream=side)
    b.check()
    assert torch.equal(got, good)

    q, pool, table, mask, counts = make_prefix(3, "bf16", 28, 4, 128, 40, [9, 0, 30])[:5]
    need = size_of("tkv_shared_prefix_attention", 3, 28, 4, 128, code("bf16"), ints(counts), table.shape[1], 40, 0)
    good = shared_prefix_attention(q, pool, table, mask, counts, 40)
    b = Behind([need, good.numel() * 2])
    got = shared_prefix_attention(q, pool, table, mask, counts, 40, stream=side)
    b.check()
    assert torch.equal(got, good)

    k = Book(3, 1, 300, 2, 64, "bf16", 4, 60)
    k.fill(0, 60, drop=0.5)
    k.upload()
    old = list(k.counts)
    b = Behind([size_of("tkv_fork_sequences", 4, 60, ints(old), 2, ints([0, 0]), ints([1, 2]), 0), 4])
    st = fork_sequences(k.dpool, k.dtable, old, k.drefs, k.dmask, [0, 0], [1, 2], share=False, positions=k.dpos, stream=side)
    b.check()
    assert k.fork([0, 0], [1, 2], False) == st.item() == 0
    k.same()
    counts = list(k.counts)
    b = Behind([size_of("tkv_compact_sequences", 4, 60, ints(counts)), 16])
    new = compact_sequences(k.dpool, k.dtable, counts, k.drefs, k.dmask, positions=k.dpos, stream=side)
    b.check()
    assert new.tolist() == k.compact()
    k.same()
    b = Behind([4])
    st = free_sequences(k.dtable, k.counts, k.drefs, k.dmask, [1, 2], stream=side)
    b.check()
    k.free_rows([1, 2])
    k.same()
    assert st.item() == 0


def test_the_other_stateless_calls_on_another_stream_beside_work_that_still_uses_freed_blocks():
    from tiered_kv_cache_split_gb300 import classify, paged_attention, quantize_rows
    side = torch.cuda.Stream()
    q, pool, table, mask, counts = make_prefix(5, "bf16", 28, 4, 128, 40, [9, 2, 30])[:5]
    table = torch.where(table < pool.shape[0], table, 0)
    need = size_of("tkv_paged_attention", 3, 28, 4, 128, table.shape[1])
    good = paged_attention(q, pool, table, mask, counts)
    b = Behind([need, good.numel() * 2])
    got = paged_attention(q, pool, table, mask, counts, stream=side)
    b.check()
    assert torch.equal(got, good)

    x = torch.randn(3000, 512, device=DEV)
    good = quantize_rows(x)
    b = Behind([3000 * 512, 3000 * 4])
    got = quantize_rows(x, stream=side)
    b.check()
    assert all(torch.equal(m, n) for m, n in zip(got, good))

    scores = torch.rand(3, 4000, dtype=torch.float64, device=DEV)
    tiers = torch.zeros(3, 4000, dtype=torch.uint8, device=DEV)
    params = [[4000, 100, 500, 900, 800]] * 3
    good = classify(scores, tiers, params, 4, 128)
    b = Behind([size_of("tkv_classify", 3, ctypes.c_int64(4000)), 12000])
    got = classify(scores, tiers, params, 4, 128, stream=side)
    b.check()
    assert torch.equal(got, good)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k_len,key", [(970, 955), (970, 951), (970, 965), (1000, 990), (1025, 1010), (1025, 1022)])
def test_an_infinite_value_at_the_end_of_a_short_piece_behind_cached_keys(dtype, k_len, key):
    """20 rows behind cached keys, whose keys are split: the infinity reaches the
    rows that see its key as what it is, whichever part of the last key block it
    is in and whether or not a row sees the part behind it."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    q, k, v = make_prompt(4, dtype, 6, 2, 64, [20], [k_len])
    want, bound = prompt_reference(q, k, v, [20], [k_len])
    v[key, 0, 3], v[key, 1, 9], v[key, 1, 10] = float("inf"), float("-inf"), float("nan")
    got = prompt_attention(q, k, v, [20], [k_len]).float().cpu().numpy().astype(np.float64)
    row = key - (k_len - 20)                    # the first row that sees it
    assert (got[row:, :3, 3] == np.inf).all() and (got[row:, 3:, 9] == -np.inf).all() and np.isnan(got[row:, 3:, 10]).all()
    got[row:, :3, 3], got[row:, 3:, 9:11] = want[row:, :3, 3], want[row:, 3:, 9:11]
    assert_within(torch.from_numpy(got), want, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alpha_of_a_row_whose_prefix_has_nothing_but_nan_keys(dtype):
    """The row's weights are all NaN, as its output is; the other KV head's are not."""
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make_prefix(6, dtype, 8, 2, 64, 33, [40, 2], holes=False)
    pool[table[0, :33].long(), 0, 0] = float("nan")
    alpha = torch.zeros(2, 2, table.shape[1] * 16, device=DEV)
    out = shared_prefix_attention(q, pool, table, mask, counts, 33, alpha_sum=alpha)
    assert out[:, :4].isnan().all() and not out[:, 4:].isnan().any()
    for b, n in enumerate(counts):
        assert alpha[b, 0, 33 * 16:n * 16].isnan().all()
    pool[table[0, :33].long(), 0, 0] = 0
    want, bound, aw, ab = prefix_reference(q, pool, tb, mk, counts, 33)
    assert_within(out[:, 4:], want[:, 4:], bound[:, 4:], "out")
    assert_within(alpha[:, 1], aw[:, 1], ab[:, 1], "alpha")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_slots_get_no_alpha_from_a_row_of_nan(dtype):
    """A later token in that slot would start from it."""
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make_prefix(7, dtype, 8, 2, 64, 5, [40, 3])
    page = next(p for p in tb[0, 5:counts[0]] if mk[p])
    pool[page, 0, 0, int(mk[page]).bit_length() - 1] = float("nan")
    alpha = torch.full((2, 2, table.shape[1] * 16), 0.5, device=DEV)
    shared_prefix_attention(q, pool, table, mask, counts, 5, alpha_sum=alpha)
    ids = tb[0, 5:counts[0]]
    live = torch.from_numpy(((mk[ids][:, None] >> np.arange(16)) & 1).astype(bool).reshape(-1)).to(DEV)
    own = alpha[0, 0, 5 * 16:counts[0] * 16]
    assert own[live].isnan().all() and (own[~live] == 0.5).all()
    assert not alpha[0, 1].isnan().any() and not alpha[1].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e33, 1e36, 1e-33])
def test_values_of_any_size_behind_logits_that_rise(dtype, scale):
    """The first keys have logit 0 and later ones up to 13 (19 in base 2): results
    that fit the type are found whatever the size of V."""
    from tiered_kv_cache_split_gb300 import prompt_attention, shared_prefix_attention
    d, n = 64, 700
    q, k, v = make_prompt(5, dtype, 4, 2, d, [200], [n])
    level = torch.zeros(n, device=DEV)
    level[64:], level[300:] = 6.0, 13.0
    q[:] = 0.01 * q
    q[..., 0], k[..., 0] = 1.0, level[:, None].to(k.dtype) * d ** 0.5
    v = (v.float() * scale).to(v.dtype)
    out = prompt_attention(q, k, v, [200], [n])
    want, bound = prompt_reference(q, k, v, [200], [n])
    assert_within(out, want, bound, "prompt")
    pages = 43
    pool = torch.zeros(pages, 2, 2, 16, d, dtype=q.dtype, device=DEV)
    for x, t in enumerate((k, v)):
        pool[:, :, x] = t[:pages * 16].view(pages, 16, 2, d).transpose(1, 2)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).repeat(3, 1)
    mask = torch.full((pages,), 0xFFFF, dtype=torch.int32, device=DEV)
    alpha = torch.zeros(3, 2, pages * 16, device=DEV)
    rows = q[:3].contiguous()
    out = shared_prefix_attention(rows, pool, table, mask, [pages, 20, 35], 20, alpha_sum=alpha)
    want, bound, aw, ab = prefix_reference(rows, pool, table.cpu().numpy(), mask.cpu().numpy(), [pages, 20, 35], 20)
    assert_within(out, want, bound, "prefix")
    assert_within(alpha, aw, ab, "alpha")


@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_sums_over_two_million_keys(spread):
    """Enough rows that none needs its keys split for speed. V is constant along
    the keys, so that the result is V and every sum's error has the same sign."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    n, hkv, d, rows = 1 << 21, 8, 64, 76 * 256
    q = torch.randn(rows, hkv, d, dtype=torch.bfloat16, device=DEV)
    k = torch.randn(n, hkv, d, dtype=torch.bfloat16, device=DEV) * spread
    col = torch.linspace(0.5, 2.0, d, device=DEV).to(torch.bfloat16)
    v = col.expand(n, hkv, d).contiguous()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = prompt_attention(q, k, v, [rows], [n], status=status)
    err = (out.float() / col.float() - 1).abs().max().item()
    assert status.item() == 0
    # Half a step of the output, 2^-8. At most 2^18 keys meet in one fp32 sum of the tensor core, at least 8
    # to an addition, each off by a step of the sum so far at most, 2^-23 of it: 2^15 2^-23 = 2^-8.
    # The sum of weights takes 64 to an addition, rounded to nearest: 2^12 2^-24. Joining eight parts: 2^-20.
    assert err <= 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11


@pytest.mark.parametrize("dtype,q_lens,k_lens", [("bf16", [300, 5100, 1], [300, (1 << 18) + 5100, 900]),
                                                 ("bf16", [2500, 6, 4000], [(1 << 18) + 3000, 6, (1 << 18) + 4001]),
                                                 ("f32", [2500, 40], [(1 << 18) + 700, 40])])
def test_a_long_sequence_that_takes_turns_over_the_scratch(dtype, q_lens, k_lens):
    """More rows than four waves of tiles over more than 2^18 keys, other
    sequences beside it; rows at the ends of the turns and a few between them."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    hq, d = 64, 64
    x = make_prompt(9, dtype, hq, 1, d, q_lens, k_lens)
    s = Guarded(size_of("tkv_prompt_attention", len(q_lens), ints(q_lens), ints(k_lens), hq, 1, d, code(dtype)))
    out = torch.full_like(x[0], float("nan"))
    prompt_attention(*x, q_lens, k_lens, scratch=s.mid, out=out)
    assert s.intact() and not out.isnan().any()
    turn = (4 * 152 * 256 if dtype == "bf16" else 4 * 304 * 64) // hq // sum(n > 1 << 18 for n in k_lens)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        rows = sorted({i for i in (0, 1, turn - 1, turn, turn + 1, 2 * turn - 1, 2 * turn, nq // 2, nq - 1) if i < nq})
        k, v = f64(x[1][k0:k0 + nk, 0]), f64(x[2][k0:k0 + nk, 0])
        seen = np.arange(nk)[None] <= np.array(rows)[:, None] + nk - nq
        for h in (0, 41):
            at = torch.tensor(rows, device=DEV) + q0
            want, bound, _ = attend(f64(x[0][at, h]), k, v, seen, DT[dtype])
            assert_within(out[at, h], want, bound, f"{nq} of {nk}, head {h}")
        q0, k0 = q0 + nq, k0 + nk


def stalled(call, *args, **kw):
    from tiered_kv_cache_split_gb300 import _lib as L
    L.check(L.load().tkv_test_stall_next_tiles(5_000_000))
    return call(*args, **kw)


def test_a_wait_that_runs_out_is_raised_later_where_the_caller_gave_no_status():
    from tiered_kv_cache_split_gb300 import TkvError, _lib as L, attention_synchronize, prompt_attention, shared_prefix_attention
    x = make_prompt(6, "bf16", 8, 2, 128, [400], [400])
    y = make_prefix(9, "bf16", 8, 2, 64, 40, [3, 9])[:5]
    good_x, good_y = prompt_attention(*x, [400]), shared_prefix_attention(*y, 40)
    attention_synchronize()
    for again, same, args, good in ((prompt_attention, prompt_attention, (*x, [400]), good_x),
                                    (shared_prefix_attention, prompt_attention, (*x, [400]), good_x),
                                    (prompt_attention, shared_prefix_attention, (*y, 40), good_y)):
        stalled(same, *args)
        torch.cuda.synchronize()
        with pytest.raises(TkvError, match="gave up") as err:
            again(*((*x, [400]) if again is prompt_attention else (*y, 40)))
        assert err.value.status == L.ERR_TIMEOUT
        assert torch.equal(same(*args), good)   # raised once
        stalled(same, *args)
        with pytest.raises(TkvError, match="gave up"):
            attention_synchronize()
        attention_synchronize()
        assert torch.equal(same(*args), good)
    # a caller's word keeps the library's clean
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    stalled(prompt_attention, *x, [400], status=status)
    attention_synchronize()
    assert status.item() == 1
    # the wait of a captured call
    stalled_graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(stalled_graph):
        stalled(prompt_attention, *x, [400])
    attention_synchronize()
    stalled_graph.replay()
    with pytest.raises(TkvError, match="gave up"):
        attention_synchronize()
    # a call on another stream
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stalled(shared_prefix_attention, *y, 40, stream=side)
    with pytest.raises(TkvError, match="gave up"):
        attention_synchronize(side)
    assert torch.equal(prompt_attention(*x, [400]), good_x)


FIRST_CALL = """
import torch, sys
from tiered_kv_cache_split_gb300 import attention_synchronize, prompt_attention
gen = torch.Generator().manual_seed(0)
q, k, v = (torch.randn(300, h, 64, generator=gen).to(torch.bfloat16).cuda() for h in (4, 2, 2))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = prompt_attention(q, k, v, [300])
graph.replay()
attention_synchronize()
assert torch.equal(out, prompt_attention(q, k, v, [300]))
print("fine")
"""


def test_the_first_call_of_a_process_may_be_a_captured_one():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_by_token_over_a_compaction(dtype):
    """alpha goes by slot and stays behind when tokens move: added to the tokens'
    scores by positions ahead of the eviction, and started again from zeros, the
    sums are those of the tokens."""
    from tiered_kv_cache_split_gb300 import compact_sequences, shared_prefix_attention
    hq, hkv, d, tokens = 8, 2, 64, 16 * 30
    b = Book(11, 1, 120, hkv, d, dtype, 3, 32)
    for r, n in enumerate((30, 3, 17)):
        b.fill(r, n, drop=0.1, last=5)
    b.upload()
    gen = torch.Generator().manual_seed(2)
    scores = torch.zeros(3, tokens, device=DEV)
    want, tolerance = np.zeros((3, tokens)), np.zeros((3, tokens))
    for step in range(3):
        q = torch.randn(3, hq, d, generator=gen).to(DT[dtype]).to(DEV)
        alpha = torch.zeros(3, hkv, 32 * 16, device=DEV)
        shared_prefix_attention(q, b.dpool[0], b.dtable, b.dmask, b.counts, 0, alpha_sum=alpha)
        at = b.dpos[b.dtable.clamp(min=0).long()].clamp(min=0).flatten(1).long()
        scores.scatter_add_(1, at, alpha.sum(1))
        _, _, aw, ab = prefix_reference(q, b.dpool[0], b.table, b.mask, b.counts)
        for r, n in enumerate(b.counts):
            for j in range(n):
                for s in range(16):
                    if (b.mask[b.table[r, j]] >> s) & 1:
                        t = b.pos[b.table[r, j], s]
                        want[r, t] += aw[r, :, 16 * j + s].sum()
                        tolerance[r, t] += ab[r, :, 16 * j + s].sum()
        for p in range(120):                                 # half of the tokens leave, the rest moves up
            for s in range(16):
                if (b.mask[p] >> s) & 1 and b.rng.random() < 0.5:
                    b.mask[p] &= ~(1 << s)
                    b.pos[p, s] = -1
        b.upload()
        new = compact_sequences(b.dpool, b.dtable, list(b.counts), b.drefs, b.dmask, positions=b.dpos)
        assert new.tolist() == b.compact()
        b.same()
    # the sum over heads and steps is rounded a few times more, in fp32
    assert_within(scores, want, tolerance + 8 * 2.0 ** -24 * want + 1e-30, "scores")


def test_a_stalled_round_is_one_round():
    """The hook stalls the first launch of a call that takes several; the others
    wait for nothing."""
    import time

    from tiered_kv_cache_split_gb300 import prompt_attention
    x = make_prompt(9, "bf16", 64, 1, 64, [5100], [(1 << 18) + 5100])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = prompt_attention(*x, [5100], [(1 << 18) + 5100])
    torch.cuda.synchronize()
    t = time.monotonic()
    stalled(prompt_attention, *x, [5100], [(1 << 18) + 5100], status=status)
    torch.cuda.synchronize()
    assert status.item() == 1 and time.monotonic() - t < 1.5       # a wait of the default length takes 2 s
    assert torch.equal(prompt_attention(*x, [5100], [(1 << 18) + 5100]), good)


@pytest.mark.parametrize("dtype,layers,hkv,d", [("bf16", 2, 4, 128), ("f32", 1, 2, 64)])
@pytest.mark.parametrize("chains", [5, 31, 63])
def test_compaction_of_many_chains_behind_a_shared_prefix(dtype, layers, hkv, d, chains):
    """Rows that share their first pages and lost tokens everywhere: the shared
    pages stay, with their holes; the end of a chain makes pages of the last row
    that lists them its own."""
    from tiered_kv_cache_split_gb300 import compact_sequences, fork_sequences, free_sequences
    b = Book(chains, layers, 8 + chains * 9, hkv, d, dtype, chains + 1, 24)
    b.fill(0, 8, drop=0.2, last=7)
    b.upload()
    forks = [0] * chains, list(range(1, chains + 1))
    st = fork_sequences(b.dpool, b.dtable, b.counts, b.drefs, b.dmask, *forks, positions=b.dpos)
    assert b.fork(*forks, True) == st.item() == 0
    b.same()
    for r in range(1, chains + 1):                       # each goes on by up to seven pages of its own
        b.free = [p for p in range(len(b.refs)) if b.refs[p] == 0]
        n, more = b.counts[r], r % 8
        before = b.table[r, :n].copy()
        b.fill(r, more, drop=0.1 * (r % 10), last=1 + r % 16)
        b.table[r, n:n + more] = b.table[r, :more].copy()
        b.table[r, :n] = before
        b.counts[r] = n + more
    b.upload()
    for round in range(2):
        counts = list(b.counts)
        got = compact_sequences(b.dpool, b.dtable, counts, b.drefs, b.dmask, positions=b.dpos)
        assert got.tolist() == b.compact()
        b.same()
        gone = list(range(0, chains)) if round == 0 else [chains]     # all but one end
        st = free_sequences(b.dtable, b.counts, b.drefs, b.dmask, gone)
        b.free_rows(gone)
        b.same()
        assert st.item() == 0
    assert not b.refs.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(64, 1, 64), (28, 4, 128), (3, 3, 64)])
def test_sums_that_are_large_already_are_rounded_once(dtype, hq, hkv, d):
    """However many heads share a KV head."""
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    q, pool, table, mask, counts, tb, mk = make_prefix(8, dtype, hq, hkv, d, 20, [38, 0, 9, 55])
    alpha = torch.full((4, hkv, table.shape[1] * 16), 4096.0, device=DEV)
    shared_prefix_attention(q, pool, table, mask, counts, 20, alpha_sum=alpha)
    _, _, aw, ab = prefix_reference(q, pool, tb, mk, counts, 20)
    assert_within(alpha, 4096 + aw, ab + (4096 + aw) * 2.0 ** -24, "alpha")
