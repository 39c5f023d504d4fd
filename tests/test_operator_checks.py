"""Refusals of the prompt, shared-prefix and page operators: every check comes
before any device work, so all of it runs without a CUDA device."""
import ctypes
import os

import pytest
import torch

from tiered_kv_cache_split_gb300 import _lib as L

I = 1 << 20          # a 256-byte aligned address that is never read
STRIDE = 1024        # elements between tokens


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from tiered_kv_cache_split_gb300 import build
        build.build()
    return L.load()


def ints(*v):
    return (ctypes.c_int32 * max(len(v), 1))(*v)


def refused(lib, status, want, *words):
    assert status == want
    msg = lib.tkv_last_error(None).decode()
    for w in words:
        assert w in msg, msg


def prompt(lib, batch=2, ql=(5, 7), kl=(5, 9), hq=8, hkv=2, d=64, dt=L.DTYPE_BF16, q=I, sq=STRIDE, k=I, sk=STRIDE, v=I, sv=STRIDE,
           out=I, so=STRIDE, scratch=None, nbytes=0, status=None):
    a, b = (ints(*ql) if ql is not None else None), (ints(*kl) if kl is not None else None)
    return lib.tkv_prompt_attention(batch, a, b, hq, hkv, d, dt, q, sq, k, sk, v, sv, out, so, scratch, nbytes, status, None)


@pytest.mark.parametrize("bad,words", [
    (dict(batch=0), ("batch",)), (dict(batch=65), ("batch",)), (dict(ql=None), ("null",)), (dict(kl=None), ("null",)),
    (dict(ql=(5, -1)), ("sequence 1",)), (dict(kl=(4, 9)), ("sequence 0",)), (dict(hq=7), ("n_q_heads",)), (dict(hkv=0), ("n_q_heads",)),
    (dict(hq=0), ("n_q_heads",)), (dict(hq=130, hkv=2), ("n_q_heads",)), (dict(d=96), ("head_dim",)), (dict(dt=2), ("kv_dtype",)),
    (dict(q=None), ("null",)), (dict(k=None), ("null",)), (dict(v=None), ("null",)), (dict(out=None), ("null",)),
    (dict(q=I + 8), ("aligned",)), (dict(v=I + 2), ("aligned",)), (dict(out=I + 4), ("aligned",)),
    (dict(sq=504), ("strides",)), (dict(sk=120), ("strides",)), (dict(sv=1025), ("strides",)), (dict(so=-1024), ("strides",)),
    (dict(sk=1 << 37), ("strides",)),
    (dict(batch=2, ql=(1, 1), kl=(1 << 26, (1 << 26) + 1)), ("sequence 1", "2^26")),
    (dict(batch=64, ql=(1,) * 64, kl=(1 << 26,) * 64), ("2^31",)),
    (dict(batch=9, ql=(1 << 26,) * 9, kl=(1 << 26,) * 9), ("2^31",)),
])
def test_prompt_refusals(lib, bad, words):
    refused(lib, prompt(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_prompt_scratch(lib):
    n = ctypes.c_size_t(7)
    size = lib.tkv_prompt_attention_scratch_size
    assert size(1, ints(16), ints(20000), 32, 8, 128, L.DTYPE_BF16, ctypes.byref(n)) == L.OK and n.value > 0
    refused(lib, prompt(lib, 1, (16,), (20000,), 32, 8, 128, sq=4096, so=4096), L.ERR_INVALID_ARG, "null scratch")
    refused(lib, prompt(lib, 1, (16,), (20000,), 32, 8, 128, sq=4096, so=4096, scratch=I, nbytes=n.value - 1), L.ERR_CAPACITY, "too small")
    refused(lib, prompt(lib, 1, (16,), (20000,), 32, 8, 128, sq=4096, so=4096, scratch=I + 16, nbytes=n.value), L.ERR_INVALID_ARG, "256")
    assert size(1, ints(8192), ints(8192), 32, 8, 128, L.DTYPE_BF16, ctypes.byref(n)) == L.OK and n.value == 0
    assert size(1, ints(1), ints(1), 32, 8, 128, L.DTYPE_BF16, None) == L.ERR_INVALID_ARG
    # no query: nothing to do, nothing read
    assert prompt(lib, 2, (0, 0), (3, 0), q=None, k=None, v=None, out=None) == L.OK


def prefix(lib, batch=2, hq=8, hkv=2, d=64, dt=L.DTYPE_BF16, q=I, pool=I, pages=100, table=I, mask=I, counts=(5, 9), width=12, shared=4,
           out=I, alpha=None, scratch=I, nbytes=1 << 40, status=None):
    c = ints(*counts) if counts is not None else None
    return lib.tkv_shared_prefix_attention(batch, hq, hkv, d, dt, q, pool, pages, table, mask, c, width, shared, out, alpha, scratch,
                                           nbytes, status, None)


@pytest.mark.parametrize("bad,words", [
    (dict(batch=0), ("batch",)), (dict(batch=65), ("batch",)), (dict(hq=9), ("n_q_heads",)), (dict(d=80), ("head_dim",)),
    (dict(dt=-1), ("kv_dtype",)), (dict(counts=None), ("null",)), (dict(counts=(3, 9)), ("page_counts[0]",)),
    (dict(counts=(5, 13)), ("page_counts[1]",)), (dict(shared=-1), ("shared_pages",)), (dict(shared=13), ("shared_pages",)),
    (dict(width=0), ("max_pages",)), (dict(width=16385), ("max_pages",)), (dict(pages=0), ("pool_pages",)),
    (dict(pages=(1 << 29) + 1), ("pool_pages",)), (dict(q=None), ("null",)), (dict(pool=None), ("null",)), (dict(table=None), ("null",)),
    (dict(mask=None), ("null",)), (dict(out=None), ("null",)), (dict(q=I + 8), ("aligned",)), (dict(alpha=I + 4), ("aligned",)),
    (dict(scratch=None), ("scratch",)), (dict(scratch=I + 64), ("256",)),
])
def test_prefix_refusals(lib, bad, words):
    refused(lib, prefix(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_prefix_scratch(lib):
    n = ctypes.c_size_t()
    args = (2, 8, 2, 64, L.DTYPE_BF16, ints(5, 9), 12, 4)
    assert lib.tkv_shared_prefix_attention_scratch_size(*args, 0, ctypes.byref(n)) == L.OK
    small = n.value
    assert lib.tkv_shared_prefix_attention_scratch_size(*args, 1, ctypes.byref(n)) == L.OK and n.value > small > 0
    refused(lib, prefix(lib, nbytes=small - 1), L.ERR_CAPACITY, "too small")
    refused(lib, prefix(lib, alpha=I, nbytes=small), L.ERR_CAPACITY, "too small")
    assert lib.tkv_shared_prefix_attention_scratch_size(*args, 0, None) == L.ERR_INVALID_ARG


def fork(lib, pool=I, layers=2, pages=50, hkv=2, d=64, dt=L.DTYPE_F32, table=I, rows=4, width=8, counts=(5, 0, 0, 8), refs=I, mask=I,
         n=2, parents=(0, 3), children=(1, 2), share=1, scratch=I, nbytes=1 << 40, status=I):
    p, c, k = (ints(*x) if x is not None else None for x in (parents, children, counts))
    return lib.tkv_fork_sequences(pool, layers, pages, hkv, d, dt, table, rows, width, k, refs, mask, None, n, p, c, share, scratch,
                                  nbytes, status, None)


@pytest.mark.parametrize("bad,words", [
    (dict(pool=None), ("null",)), (dict(pool=I + 8), ("aligned",)), (dict(layers=0), ("pool shape",)), (dict(pages=0), ("pool shape",)),
    (dict(pages=(1 << 27) + 1), ("pool shape",)), (dict(hkv=0), ("pool shape",)), (dict(d=32), ("head_dim",)), (dict(dt=5), ("kv_dtype",)),
    (dict(table=None), ("null",)), (dict(refs=None), ("null",)), (dict(mask=None), ("null",)), (dict(status=None), ("null",)),
    (dict(counts=None), ("null",)), (dict(counts=(5, 0, 0, 9)), ("page_counts[3]",)), (dict(counts=(-1, 0, 0, 8)), ("page_counts[0]",)),
    (dict(rows=0), ("rows",)), (dict(width=20000), ("max_pages",)), (dict(n=0), ("forks",)), (dict(n=65), ("forks",)),
    (dict(parents=None), ("null",)), (dict(children=None), ("null",)), (dict(parents=(0, 4)), ("fork 1",)),
    (dict(children=(-1, 2)), ("fork 0",)), (dict(children=(1, 1)), ("twice",)), (dict(children=(1, 0)), ("holds pages",)),
    (dict(parents=(0, 1), children=(1, 2)), ("a parent too",)), (dict(counts=(5, 1, 0, 8)), ("holds pages",)),
    (dict(scratch=None), ("scratch",)), (dict(scratch=I + 8), ("256",)),
])
def test_fork_refusals(lib, bad, words):
    refused(lib, fork(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_fork_and_compact_scratch(lib):
    n = ctypes.c_size_t()
    assert lib.tkv_fork_sequences_scratch_size(4, 8, ints(5, 0, 0, 8), 2, ints(0, 3), ints(1, 2), 0, ctypes.byref(n)) == L.OK and n.value > 0
    refused(lib, fork(lib, share=0, nbytes=n.value - 1), L.ERR_CAPACITY, "too small")
    assert lib.tkv_fork_sequences_scratch_size(4, 8, ints(5, 0, 0, 8), 2, ints(0, 3), ints(1, 2), 0, None) == L.ERR_INVALID_ARG
    assert lib.tkv_compact_sequences_scratch_size(2, 8, ints(5, 8), ctypes.byref(n)) == L.OK and n.value >= 2 * 13 * 8 * 4
    refused(lib, compact(lib, nbytes=n.value - 1), L.ERR_CAPACITY, "too small")


def free(lib, table=I, rows=4, width=8, counts=(5, 0, 0, 8), pages=50, refs=I, mask=I, n=2, seqs=(0, 3), status=I):
    return lib.tkv_free_sequences(table, rows, width, ints(*counts), pages, refs, mask, n, ints(*seqs) if seqs else None, status, None)


@pytest.mark.parametrize("bad,words", [
    (dict(table=None), ("null",)), (dict(refs=None), ("null",)), (dict(mask=None), ("null",)), (dict(status=None), ("null",)),
    (dict(seqs=None), ("null",)), (dict(seqs=(0, 4)), ("sequence 1",)), (dict(seqs=(3, 3)), ("twice",)), (dict(n=0), ("1 to 64",)),
    (dict(n=65), ("1 to 64",)), (dict(pages=0), ("pool shape",)), (dict(counts=(9, 0, 0, 0)), ("page_counts[0]",)),
])
def test_free_refusals(lib, bad, words):
    refused(lib, free(lib, **bad), L.ERR_INVALID_ARG, *words)


def compact(lib, pool=I, layers=1, pages=50, hkv=2, d=64, dt=L.DTYPE_F32, table=I, rows=2, width=8, counts=(5, 8), refs=I, mask=I,
            new=I, scratch=I, nbytes=1 << 40):
    return lib.tkv_compact_sequences(pool, layers, pages, hkv, d, dt, table, rows, width, ints(*counts), refs, mask, None, new, scratch,
                                     nbytes, None)


@pytest.mark.parametrize("bad,words", [
    (dict(pool=None), ("null",)), (dict(pool=I + 4), ("aligned",)), (dict(table=None), ("null",)), (dict(mask=None), ("null",)),
    (dict(new=None), ("null",)), (dict(counts=(5, 9)), ("page_counts[1]",)), (dict(rows=65, counts=(0,) * 65), ("1 to 64",)),
    (dict(d=100), ("head_dim",)), (dict(scratch=None), ("scratch",)), (dict(scratch=I + 32), ("256",)),
])
def test_compact_refusals(lib, bad, words):
    refused(lib, compact(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_stall_hook_limits(lib):
    for bad in (0, 999_999, 2_000_000_001):
        refused(lib, lib.tkv_test_stall_next_tiles(bad), L.ERR_INVALID_ARG, "1 ms")


def test_python_checks_name_the_argument():
    import tiered_kv_cache_split_gb300 as t
    q, k = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64)
    for args, word in (((q[..., ::2], k[..., ::2], k[..., ::2], [6]), "contiguous"), ((q, k.double(), k, [6]), "k:"),
                       ((q, k, k[:5], [6]), "v:"), ((q, k, k, [5]), "q_lens"), ((q, k, k, [6], [5]), "k_lens"),
                       ((q, k, k, [6], [3, 3]), "k_lens"), ((q.half(), k.half(), k.half(), [6]), "q:"),
                       ((q.transpose(0, 1), k, k, [4]), "heads"), ((q, k, k, [6]), "CUDA")):
        with pytest.raises(ValueError, match=word):
            t.prompt_attention(*args)
    pool, table, mask = torch.zeros(9, 2, 2, 16, 64), torch.zeros(3, 4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    qd = torch.zeros(3, 4, 64)
    for args, word in (((qd, pool[:, :, :1], table, mask, [1] * 3, 0), "pool"), ((qd, pool, table.long(), mask, [1] * 3, 0), "page_table"),
                       ((qd, pool, table, mask[:8], [1] * 3, 0), "slot_mask"), ((qd, pool, table, mask, [1] * 2, 0), "page_counts"),
                       ((qd, pool, table[:2], mask, [1] * 3, 0), "page_table"), ((qd.bfloat16(), pool, table, mask, [1] * 3, 0), "pool"),
                       ((qd, pool, table, mask, [1] * 3, 0), "CUDA")):
        with pytest.raises(ValueError, match=word):
            t.shared_prefix_attention(*args)
    refs = torch.zeros(9, dtype=torch.int32)
    for args, word in (((pool[0], table, [1] * 3, refs, mask, [0], [1]), "pool"), ((pool, table, [1] * 3, refs[:4], mask, [0], [1]), "page_refs"),
                       ((pool, table, [1] * 3, refs, mask, [0, 0], [1]), "children"), ((pool, table, [1], refs, mask, [0], [1]), "page_counts"),
                       ((pool, table, [1] * 3, refs, mask, [0], [1]), "CUDA")):
        with pytest.raises(ValueError, match=word):
            t.fork_sequences(*args)
    with pytest.raises(ValueError, match="page_refs"):
        t.free_sequences(table, [1] * 3, None, mask, [0])
    with pytest.raises(ValueError, match="contiguous"):
        t.compact_sequences(pool, table.t(), [1] * 4, refs, mask)
