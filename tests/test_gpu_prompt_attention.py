"""Prompt attention against a float64 form of its definition (every bound is
derived in operator_helpers.attend), and how calls share the device."""
import numpy as np
import pytest
import torch

from operator_helpers import assert_within, f64, prompt_reference

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, dtype, hq, hkv, d, q_lens, k_lens, spread=0.5):
    gen = torch.Generator().manual_seed(seed)
    tq, tk = sum(q_lens), sum(k_lens)
    q = torch.randn(tq, hq, d, generator=gen)
    k = torch.randn(tk, hkv, d, generator=gen) * torch.exp(spread * torch.randn(tk, hkv, 1, generator=gen))
    v = torch.randn(tk, hkv, d, generator=gen)
    return tuple(x.to(DT[dtype]).to(DEV) for x in (q, k, v))


def check(q, k, v, q_lens, k_lens, **kw):
    from tiered_kv_cache_split_gb300 import prompt_attention
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = prompt_attention(q, k, v, q_lens, k_lens, status=status, **kw)
    want, bound = prompt_reference(q, k, v, q_lens, k_lens)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert_within(out, want, bound, f"{q_lens} {k_lens}")
    return out


LENS = [([1], [1]), ([1], [300]), ([5], [5]), ([63, 64, 65], [63, 64, 65]), ([127], [127]), ([128], [128]), ([129], [129]),
        ([256], [256]), ([257], [257]), ([300, 1, 0, 17], [300, 1, 0, 17]), ([40, 0, 130, 1], [555, 70, 131, 129]),
        ([16], [2500]), ([0, 0, 3], [9, 0, 3])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (7, 1, 128)])
@pytest.mark.parametrize("lens", range(len(LENS)))
def test_lengths(dtype, hq, hkv, d, lens):
    q_lens, k_lens = LENS[lens]
    check(*make(lens, dtype, hq, hkv, d, q_lens, k_lens), q_lens, k_lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (6, 6, 64), (6, 2, 128), (5, 1, 64), (64, 1, 64), (28, 4, 128), (16, 8, 128)])
def test_head_layouts(dtype, hq, hkv, d):
    q_lens = [70, 3, 150]
    check(*make(hq, dtype, hq, hkv, d, q_lens, [90, 3, 150]), q_lens, [90, 3, 150])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_enough_units_to_fill_the_device(dtype):
    """64 sequences: units write the output themselves, none is split."""
    q_lens = [(37 * i) % 190 for i in range(64)]
    k_lens = [n + (i % 5) * 40 for i, n in enumerate(q_lens)]
    check(*make(5, dtype, 16, 8, 64, q_lens, k_lens), q_lens, k_lens)


def test_a_long_row_of_units_per_sequence():
    q_lens = k_lens = [1500, 700]
    check(*make(6, "bf16", 8, 2, 128, q_lens, k_lens), q_lens, k_lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_key_takes_all_the_weight(dtype):
    """Logits in the hundreds, rising along the keys: the running maximum moves in every block."""
    q, k, v = make(7, dtype, 4, 2, 64, [400], [400])
    k = (k.float() * torch.linspace(0.1, 12.0, 400, device=DEV)[:, None, None]).to(q.dtype)
    check(q, k, v, [400], [400])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_views_of_one_projection_and_a_strided_output(dtype):
    hq, hkv, d, n = 8, 2, 128, 200
    gen = torch.Generator().manual_seed(1)
    qkv = torch.randn(n, hq + 2 * hkv + 1, d, generator=gen).to(DT[dtype]).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:hq + 2 * hkv]
    wide = torch.full((n, hq + 3, d), 7.0, dtype=DT[dtype], device=DEV)
    out = check(q, k, v, [150, 50], [150, 50], out=wide[:, 1:hq + 1])
    assert out.data_ptr() == wide[:, 1].data_ptr()
    assert (wide[:, 0] == 7).all() and (wide[:, hq + 1:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [([100, 60], [100, 60]), ([700, 60, 33], [700, 300, 33]), ([9, 4], [1000, 4])])
def test_non_finite_values_reach_the_rows_that_see_them_only(dtype, lens):
    """NaN and infinities in K and V of one sequence, at a key its later rows
    see: other sequences and earlier rows keep their values."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    q_lens, k_lens = lens
    q, k, v = make(8, dtype, 6, 2, 64, q_lens, k_lens)
    clean, bound = prompt_reference(q, k, v, q_lens, k_lens)
    at = k_lens[0] - q_lens[0] // 2            # a key of sequence 0 that half of its rows see
    row = at - (k_lens[0] - q_lens[0])         # the first row that sees it
    v2, k2 = v.clone(), k.clone()
    v2[at, 0, 3], v2[at, 0, 5], v2[at, 1, 7] = float("nan"), float("inf"), float("-inf")
    got = f64(prompt_attention(q, k, v2, q_lens, k_lens))
    assert_within(torch.from_numpy(got[:row]), clean[:row], bound[:row], "earlier rows")
    assert_within(torch.from_numpy(got[q_lens[0]:]), clean[q_lens[0]:], bound[q_lens[0]:], "other sequences")
    mine = got[row:q_lens[0]]
    assert np.isnan(mine[:, :3, 3]).all() and (mine[:, :3, 5] == np.inf).all() and (mine[:, 3:, 7] == -np.inf).all()
    mine = mine.copy()
    mine[:, :3, 3], mine[:, :3, 5], mine[:, 3:, 7] = (clean[row:q_lens[0], :3, 3], clean[row:q_lens[0], :3, 5],
                                                      clean[row:q_lens[0], 3:, 7])
    assert_within(torch.from_numpy(mine), clean[row:q_lens[0]], bound[row:q_lens[0]], "other columns")
    k2[at, 0, 0] = float("nan")
    got = f64(prompt_attention(q, k2, v, q_lens, k_lens))
    assert_within(torch.from_numpy(got[:row]), clean[:row], bound[:row], "earlier rows, K")
    assert_within(torch.from_numpy(got[q_lens[0]:]), clean[q_lens[0]:], bound[q_lens[0]:], "other sequences, K")
    assert np.isnan(got[row:q_lens[0], :3]).all() and not np.isnan(got[:, 3:]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_the_last_sequence_stay(dtype):
    from tiered_kv_cache_split_gb300 import prompt_attention
    q, k, v = make(9, dtype, 4, 2, 64, [33, 95], [33, 95])
    back = torch.full((200, 4, 64), 3.0, dtype=q.dtype, device=DEV)
    prompt_attention(q, k, v, [33, 95], out=back[:128])
    assert (back[128:] == 3).all()


def test_repeats_are_bitwise_equal_and_two_streams_do_not_mix():
    from tiered_kv_cache_split_gb300 import prompt_attention
    a = make(10, "bf16", 8, 2, 128, [20], [3000])
    b = make(11, "bf16", 8, 2, 128, [20], [3000])
    one, two = prompt_attention(*a, [20], [3000]), prompt_attention(*b, [20], [3000])
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((prompt_attention(*a, [20], [3000], stream=s), prompt_attention(*b, [20], [3000], stream=t)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, one) and torch.equal(y, two)


@pytest.mark.parametrize("q_lens,k_lens", [([20], [2000]), ([300, 200], [300, 200])])
def test_captured_and_replayed_on_new_inputs(q_lens, k_lens):
    from tiered_kv_cache_split_gb300 import prompt_attention
    q, k, v = make(12, "bf16", 8, 2, 64, q_lens, k_lens)
    prompt_attention(q, k, v, q_lens, k_lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = prompt_attention(q, k, v, q_lens, k_lens)
    q2, k2, v2 = make(13, "bf16", 8, 2, 64, q_lens, k_lens)
    q.copy_(q2), k.copy_(k2), v.copy_(v2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, prompt_attention(q2, k2, v2, q_lens, k_lens))


def test_an_output_aligned_to_16_bytes_only():
    from tiered_kv_cache_split_gb300 import prompt_attention
    q_lens = [150, 40]
    for dtype in ("bf16", "f32"):
        q, k, v = make(14, dtype, 6, 2, 128, q_lens, q_lens)
        unit = 16 // q.element_size()
        buf = torch.full((190 * 6 * 128 + 64,), 5.0, dtype=q.dtype, device=DEV)
        out = buf[unit:unit + 190 * 6 * 128].view(190, 6, 128)
        check(q, k, v, q_lens, q_lens, out=out)
        assert (buf[:unit] == 5).all() and (buf[unit + 190 * 6 * 128:] == 5).all()


def test_no_query_at_all():
    from tiered_kv_cache_split_gb300 import prompt_attention
    q, k, v = make(15, "bf16", 4, 2, 64, [0, 0], [5, 0])
    assert prompt_attention(q, k, v, [0, 0], [5, 0]).shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """Token strides that put the last keys and rows more than 2^32 bytes in."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    n, d = 300, 64
    q, k, v = make(16, dtype, 2, 1, d, [n], [n])
    stride = (1 << 33) // q.element_size() // n // 8 * 8
    wide = torch.empty(n * stride, dtype=q.dtype, device=DEV)
    far = lambda h: wide.as_strided((n, h, d), (stride, d, 1))   # noqa: E731
    want, bound = prompt_reference(q, k, v, [n], [n])
    far(1).copy_(k)
    assert_within(prompt_attention(q, far(1), v, [n]), want, bound, "k")
    far(1).copy_(v)
    assert_within(prompt_attention(q, k, far(1), [n]), want, bound, "v")
    far(2).copy_(q)
    assert_within(prompt_attention(far(2), k, v, [n]), want, bound, "q")
    assert_within(prompt_attention(q, k, v, [n], out=far(2)), want, bound, "out")


def test_one_scratch_for_calls_in_turn():
    """A caller's scratch, just large enough, used by different calls one after the other."""
    import ctypes
    from tiered_kv_cache_split_gb300 import _lib as L, prompt_attention
    shapes = [([20], [3000]), ([3, 40], [900, 2000])]
    most = 0
    for ql, kl in shapes:
        need = ctypes.c_size_t()
        a, b = (ctypes.c_int32 * len(ql))(*ql), (ctypes.c_int32 * len(kl))(*kl)
        L.check(L.load().tkv_prompt_attention_scratch_size(len(ql), a, b, 8, 2, 128, L.DTYPE_BF16, ctypes.byref(need)))
        most = max(most, need.value)
    scratch = torch.full((most,), 255, dtype=torch.uint8, device=DEV)      # NaN wherever it is read as float
    for _ in range(2):
        for i, (ql, kl) in enumerate(shapes):
            check(*make(20 + i, "bf16", 8, 2, 128, ql, kl), ql, kl, scratch=scratch)
    with pytest.raises(L.TkvError, match="too small"):
        prompt_attention(*make(20, "bf16", 8, 2, 128, *shapes[0]), *shapes[0], scratch=scratch[:1024])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(7, 1, 128), (8, 2, 64), (4, 4, 128)])
def test_prompts_beside_decoding_sequences(dtype, hq, hkv, d):
    """Sequences whose keys are split, ones whose units write the output and
    ones of few rows in one call; the scratch starts as NaN, the output too."""
    q_lens = [400, 1, 0, 90, 260, 1, 17]
    k_lens = [n + c for n, c in zip(q_lens, [0, 9000, 5, 6000, 100, 0, 4000])]
    x = make(23, dtype, hq, hkv, d, q_lens, k_lens)
    scratch = torch.full((64 << 20,), 255, dtype=torch.uint8, device=DEV)
    out = torch.full((sum(q_lens) + 3, hq, d), float("nan"), dtype=x[0].dtype, device=DEV)
    check(*x, q_lens, k_lens, scratch=scratch, out=out[:-3])
    assert out[-3:].isnan().all()


@pytest.mark.parametrize("hq,hkv,d", [(32, 32, 128), (16, 4, 128), (32, 8, 64)])
def test_long_units_repeated_over_a_scratch_of_nan(hq, hkv, d):
    """Many long key ranges at once, whose copies land in any order: every call
    finishes every range (a partial that stayed unwritten would read as NaN)."""
    from tiered_kv_cache_split_gb300 import prompt_attention
    q_lens = [43, 51, 318, 2, 8, 5, 10, 44, 5, 32, 35, 2]
    k_lens = [n + c for n, c in zip(q_lens, [7271, 2, 1793, 0, 2771, 5922, 0, 3, 12, 290, 0, 0])]
    x = make(19, "bf16", hq, hkv, d, q_lens, k_lens)
    scratch = torch.empty(256 << 20, dtype=torch.uint8, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = check(*x, q_lens, k_lens, scratch=scratch.fill_(255))
    for _ in range(60):
        assert torch.equal(prompt_attention(*x, q_lens, k_lens, scratch=scratch.fill_(255), status=status), first)
        assert status.item() == 0


def test_a_wait_that_runs_out_is_reported_and_the_device_goes_on():
    from tiered_kv_cache_split_gb300 import _lib as L, prompt_attention
    q, k, v = make(17, "bf16", 8, 2, 128, [400], [400])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    L.check(L.load().tkv_test_stall_next_tiles(5_000_000))
    prompt_attention(q, k, v, [400], status=status)
    torch.cuda.synchronize()
    assert status.item() == 1
    check(q, k, v, [400], [400])
