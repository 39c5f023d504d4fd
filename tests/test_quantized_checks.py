"""Refusals of the rotary and 8-bit cache operators: every check comes before
any device work, so all of it runs without a CUDA device."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from quantized_helpers import INV_2PI
from tiered_kv_cache_split_gb300 import _lib as L

I = 1 << 20          # a 256-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from tiered_kv_cache_split_gb300 import build
        build.build()
    return L.load()


def ints(v):
    return None if v is None else (ctypes.c_int32 * max(len(v), 1))(*v)


def refused(lib, status, want, *words):
    assert status == want
    msg = lib.tkv_last_error(None).decode()
    for w in words:
        assert w in msg, msg


def rotate(lib, n=5, hq=8, hk=2, d=64, r=64, dt=L.DTYPE_BF16, il=0, inv=0, scale=1.0, steps=I, pos=I, bits=64, q=I, sq=640, k=I, sk=640,
           qo=2 * I, so=512, ko=3 * I, to=128):
    return lib.tkv_rotate(n, hq, hk, d, r, dt, il, inv, scale, steps, pos, bits, q, sq, k, sk, qo, so, ko, to, None)


@pytest.mark.parametrize("bad,words", [
    (dict(n=-1), ("n_tokens",)), (dict(n=1 << 31), ("n_tokens",)), (dict(hq=-1), ("heads",)), (dict(hq=0, hk=0), ("heads",)),
    (dict(hk=65536), ("heads",)), (dict(d=1), ("head_dim",)), (dict(d=514), ("head_dim",)), (dict(r=0), ("rotary_dim",)),
    (dict(r=66), ("rotary_dim",)), (dict(r=63), ("rotary_dim",)), (dict(dt=2), ("dtype",)), (dict(bits=16), ("position_bits",)),
    (dict(scale=math.inf), ("scale",)), (dict(scale=math.nan), ("scale",)), (dict(steps=None), ("null",)), (dict(pos=None), ("null",)),
    (dict(q=None), ("null",)), (dict(k=None), ("null",)), (dict(qo=None), ("null",)), (dict(ko=None), ("null",)),
    (dict(steps=I + 4), ("aligned",)), (dict(pos=I + 4), ("aligned",)), (dict(q=I + 1), ("aligned",)), (dict(dt=0, ko=I + 2), ("aligned",)),
    (dict(sq=511), ("strides",)), (dict(sk=127), ("strides",)), (dict(so=500), ("strides",)), (dict(to=-128), ("strides",)),
    (dict(sq=1 << 36), ("strides",)), (dict(qo=I), ("in place",)), (dict(ko=I), ("in place",)),
    (dict(ko=2 * I), ("the same",)), (dict(so=640, qo=I, to=640, ko=I), ("the same",)),
])
def test_rotate_refusals(lib, bad, words):
    refused(lib, rotate(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_rotate_of_nothing(lib):
    assert rotate(lib, n=0, steps=None, pos=None, q=None, k=None, qo=None, ko=None) == L.OK


def test_rotary_steps(lib):
    freq = [1.0, 0.5, 1e-4, 1e-300, 0.0, -0.25, 3.5, 2.0 ** 32, -1e-18, 6.283185307179586, 12345.678]
    n = len(freq)
    got = (ctypes.c_uint64 * n)()
    assert lib.tkv_rotary_steps(n, (ctypes.c_double * n)(*freq), got) == L.OK
    from fractions import Fraction
    for f, g in zip(freq, got):
        want = (Fraction(f) * INV_2PI * (1 << 64)) % (1 << 64)
        off = (g - want) % (1 << 64)
        # turns are a sum of two doubles: off by 2^-106 of their size, 2^-64 in the last place, and the rounding of f * lo
        assert min(off, (1 << 64) - off) <= 2 + abs(f) * 2.0 ** -45, f
    for bad in (math.nan, math.inf, 1e10, -1e10):
        refused(lib, lib.tkv_rotary_steps(1, (ctypes.c_double * 1)(bad), got), L.ERR_INVALID_ARG, "inv_freq[0]")
    for n in (0, 257, -1):
        refused(lib, lib.tkv_rotary_steps(n, (ctypes.c_double * 300)(), (ctypes.c_uint64 * 300)()), L.ERR_INVALID_ARG, "n must")
    assert lib.tkv_rotary_steps(1, None, got) == L.ERR_INVALID_ARG and lib.tkv_rotary_steps(1, (ctypes.c_double * 1)(), None) == L.ERR_INVALID_ARG


def append(lib, rows=2, lens=(5, 16), new=(3, 1), hkv=2, d=64, dt=L.DTYPE_BF16, k=I, sk=128, v=I, sv=128, pool=I, scales=I, pages=50, table=I,
           width=8, mask=I, refs=None, status=None):
    return lib.tkv_append_quantized(rows, ints(lens), ints(new), hkv, d, dt, k, sk, v, sv, pool, scales, pages, table, width, mask, refs, status,
                                    None)


POOL_REFUSALS = [
    (dict(rows=0), ("rows",)), (dict(rows=65), ("rows",)), (dict(hkv=0), ("pool_pages",)), (dict(hkv=65536), ("pool_pages",)),
    (dict(pages=0), ("pool_pages",)), (dict(pages=(1 << 28) + 1), ("pool_pages",)), (dict(d=96), ("head_dim",)), (dict(dt=2), ("dtype",)),
    (dict(width=0), ("max_pages",)), (dict(width=16385), ("max_pages",)), (dict(lens=None), ("null",)), (dict(pool=None), ("null",)),
    (dict(scales=None), ("null",)), (dict(table=None), ("null",)), (dict(k=None), ("null",)), (dict(v=None), ("null",)),
    (dict(pool=I + 8), ("aligned",)), (dict(scales=I + 4), ("aligned",)), (dict(k=I + 8), ("aligned",)), (dict(v=I + 2), ("aligned",)),
    (dict(sk=120), ("strides",)), (dict(sv=132), ("strides",)), (dict(sk=1 << 37), ("strides",)),
]


@pytest.mark.parametrize("bad,words", POOL_REFUSALS + [
    (dict(new=None), ("null",)), (dict(lens=(-1, 16)), ("row 0",)), (dict(new=(3, -1)), ("row 1",)), (dict(lens=(126, 16)), ("row 0", "max_pages")),
    (dict(lens=(5, 2 ** 31 - 1)), ("row 1",)), (dict(new=(3, 113)), ("row 1", "max_pages")),
])
def test_append_refusals(lib, bad, words):
    refused(lib, append(lib, **bad), L.ERR_INVALID_ARG, *words)


def read(lib, rows=2, first=(0, 3), lens=(5, 16), hkv=2, d=64, dt=L.DTYPE_BF16, pool=I, scales=I, pages=50, table=I, width=8, mask=None, k=I,
         sk=128, v=I, sv=128):
    return lib.tkv_read_quantized(rows, ints(first), ints(lens), hkv, d, dt, pool, scales, pages, table, width, mask, k, sk, v, sv, None)


@pytest.mark.parametrize("bad,words", POOL_REFUSALS + [
    (dict(first=None), ("null",)), (dict(first=(-1, 3)), ("row 0",)), (dict(first=(0, 17)), ("row 1",)), (dict(lens=(129, 16)), ("row 0", "max_pages")), (dict(lens=(5, 2 ** 31 - 1)), ("row 1", "max_pages")),
])
def test_read_refusals(lib, bad, words):
    refused(lib, read(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_nothing_to_write_or_read(lib):
    assert append(lib, new=(0, 0), k=None, v=None) == L.OK
    assert read(lib, first=(5, 16), k=None, v=None) == L.OK


def attend(lib, batch=2, hq=8, hkv=2, d=64, dt=L.DTYPE_BF16, q=I, pool=I, scales=I, pages=50, table=I, mask=I, counts=(5, 8), width=8, out=I,
           alpha=None, scratch=I, nbytes=1 << 40):
    return lib.tkv_quantized_attention(batch, hq, hkv, d, dt, q, pool, scales, pages, table, mask, ints(counts), width, out, alpha, scratch,
                                       nbytes, None)


@pytest.mark.parametrize("bad,words", [
    (dict(batch=0), ("batch",)), (dict(batch=65), ("batch",)), (dict(hq=9), ("n_q_heads",)), (dict(hq=130), ("n_q_heads",)),
    (dict(hkv=0), ("n_q_heads",)), (dict(d=80), ("head_dim",)), (dict(dt=-1), ("dtype",)), (dict(counts=None), ("null",)),
    (dict(counts=(5, 9)), ("page_counts[1]",)), (dict(counts=(-1, 8)), ("page_counts[0]",)), (dict(width=0), ("max_pages",)),
    (dict(width=16385), ("max_pages",)), (dict(pages=0), ("pool_pages",)), (dict(pages=(1 << 28) + 1), ("pool_pages",)),
    (dict(q=None), ("null",)), (dict(pool=None), ("null",)), (dict(scales=None), ("null",)), (dict(table=None), ("null",)),
    (dict(mask=None), ("null",)), (dict(out=None), ("null",)), (dict(q=I + 8), ("aligned",)), (dict(out=I + 8), ("aligned",)),
    (dict(pool=I + 8), ("aligned",)), (dict(scales=I + 4), ("aligned",)), (dict(alpha=I + 4), ("aligned",)),
    (dict(batch=64, hq=4096, hkv=4096, counts=(16384,) * 64, width=16384), ("2^30",)),
])
def test_attention_refusals(lib, bad, words):
    refused(lib, attend(lib, **bad), L.ERR_INVALID_ARG, *words)


def test_attention_scratch(lib):
    n = ctypes.c_size_t()
    args = (2, 32, 8, 128, L.DTYPE_BF16, ints((5, 8000)), 8000)
    big = dict(hq=32, hkv=8, d=128, counts=(5, 8000), width=8000, alpha=I)
    assert lib.tkv_quantized_attention_scratch_size(*args, 1, ctypes.byref(n)) == L.OK and n.value > 0
    refused(lib, attend(lib, **big, scratch=None), L.ERR_INVALID_ARG, "null scratch")
    refused(lib, attend(lib, **big, nbytes=n.value - 1), L.ERR_CAPACITY, "too small")
    refused(lib, attend(lib, **big, scratch=I + 128), L.ERR_INVALID_ARG, "256")
    assert lib.tkv_quantized_attention_scratch_size(*args, 1, None) == L.ERR_INVALID_ARG


def test_rotary_table_checks():
    import tiered_kv_cache_split_gb300 as t
    for kw, word in ((dict(rotary_dim=63), "rotary_dim"), (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=514), "rotary_dim"),
                     (dict(rotary_dim=8, base=0.0), "base"), (dict(rotary_dim=8, factor=-1.0), "factor"),
                     (dict(rotary_dim=8, factor=math.nan), "factor"), (dict(rotary_dim=8, trained=0), "trained"),
                     (dict(rotary_dim=8, trained=10, low=2, high=2), "high"), (dict(rotary_dim=8, scale=math.inf), "scale"),
                     (dict(rotary_dim=8, inv_freq=[1.0] * 3), "inv_freq")):
        with pytest.raises(ValueError, match=word):
            t.rotary_table(device="cpu", **kw)
    with pytest.raises(t.TkvError, match="inv_freq"):
        t.rotary_table(2, inv_freq=[math.nan], device="cpu")
    tab = t.rotary_table(64, factor=8.0, trained=2048, device="cpu")
    f = 10000.0 ** (-np.arange(32) / 32)
    g = np.clip((2048 * f / (2 * np.pi) - 1) / 31, 0, 1)
    assert np.allclose(tab.inv_freq, f * (g + (1 - g) / 8), rtol=1e-14) and tab.rotary_dim == 64 and tab.steps.shape == (32,)
    assert np.allclose(t.rotary_table(64, factor=8.0, device="cpu").inv_freq, f / 8, rtol=1e-14)


def test_python_checks_name_the_argument():
    import tiered_kv_cache_split_gb300 as t
    tab = t.rotary_table(64, device="cpu")
    q, k, pos = torch.zeros(6, 4, 64), torch.zeros(6, 2, 64), torch.zeros(6, dtype=torch.int64)
    for args, kw, word in (((q[..., ::2], k, pos, tab), {}, "contiguous"), ((q, k.double(), pos, tab), {}, "k:"), ((q.half(), None, pos, tab), {}, "q:"),
                           ((q, k[:5], pos, tab), {}, "k:"), ((q, k[..., :32], pos, tab), {}, "k:"), ((q, k, pos[:5], tab), {}, "positions"),
                           ((q, k, pos.float(), tab), {}, "positions"), ((q, k, pos, None), {}, "table"), ((q, k, pos, tab), {}, "CUDA"),
                           ((torch.zeros(6, 4, 64).requires_grad_(), k, pos, tab), {}, "backward")):
        with pytest.raises(ValueError, match=word):
            t.rotate(*args, **kw)
    pool, scales = torch.zeros(9, 2, 2, 16, 64, dtype=torch.int8), torch.zeros(9, 2, 2)
    table, mask = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(9, dtype=torch.int32)
    x = torch.zeros(6, 2, 64)
    ok = (x, x, pool, scales, table, mask, [0, 1, 2], [3, 3, 0])
    for i, bad, word in ((0, x.half(), "v:"), (0, x[:5], "v:"), (1, x[..., :32], "k|v:"), (2, pool.float(), "pool"), (2, pool[:, :, :1], "pool"),
                         (3, scales[:8], "scales"), (3, scales.double(), "scales"), (3, scales.clone().requires_grad_(), "scales.*backward"), (3, None, "scales"), (4, table.long(), "page_table"), (4, table[:2], "page_table"),
                         (5, mask[:8], "slot_mask"), (6, [0, 1], "new_lens"), (7, [3, 3, 1], "new_lens"), (7, [3, 3], "new_lens"), (0, x[:, :1], "k:|v:")):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError, match=word):
            t.append_quantized(*args)
    with pytest.raises(ValueError, match="page_refs"):
        t.append_quantized(*ok, page_refs=mask[:3])
    with pytest.raises(ValueError, match="CUDA"):
        t.append_quantized(*ok)
    for args, kw, word in (((pool, scales, table, mask, [1, 2]), {}, "page_table"), ((pool, scales, table, mask, [1, 2, 3]), dict(first=[0]), "first"),
                           ((pool, scales, table, mask, [1, 2, 3]), {}, "CUDA")):
        with pytest.raises(ValueError, match=word):
            t.read_quantized(*args, **kw)
    qd = torch.zeros(3, 4, 64)
    for args, kw, word in (((qd.half(), pool, scales, table, mask, [1] * 3), {}, "q:"), ((qd[:2], pool, scales, table, mask, [1] * 2), {}, "page_table"),
                           ((torch.zeros(3, 4, 128), pool, scales, table, mask, [1] * 3), {}, "d must"),
                           ((qd, pool, scales, table, None, [1] * 3), {}, "slot_mask"), ((qd, pool, scales, table, mask, [1] * 2), {}, "page_counts"),
                           ((qd, pool, scales, table, mask, [1] * 3), dict(alpha_sum=torch.zeros(3, 2, 63)), "alpha_sum"),
                           ((qd, pool, scales, table, mask, [1] * 3), {}, "CUDA")):
        with pytest.raises(ValueError, match=word):
            t.quantized_attention(*args, **kw)
