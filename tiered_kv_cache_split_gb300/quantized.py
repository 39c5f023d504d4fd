"""Rotary positions and a paged cache held in 8 bits.

Argument marshalling only, with the checks, streams and errors of operators.py;
include/tkv.h states each operator. Small calls are bound by this file: a call
first asks whether all its arguments are as they should be, and only where they
are not goes through the checks that name the one that is not.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib as L
from .operators import _DTYPES, _I32, _MASK, _On, _at, _dense, _ints, _no_gradient, _tokens

_I8, _F32 = (torch.int8,), (torch.float32,)
# Up to here (8 CTAs of a cluster with 24 pages each) a call is tried without scratch first. Where it needs
# none that saves 2 us of 11; where it does after all (more than 16 query heads per KV head, fp32 8; many rows
# whose logits leave shared memory) the attempt costs 1.5 to 2.5 us of 22.
_SHORT_PAGES = 192


def _like(on, x):
    """A dense tensor like x, from the memory of the call's stream."""
    return torch.empty_like(x) if on.given is None else on.empty(x.shape, x.dtype)


class RotaryTable:
    """The frequencies of rotate, made once by rotary_table: steps, int64
    [rotary_dim / 2] on the device (turns per position in 2^-64 turns),
    inv_freq (host floats, radians per position), scale and the pairs' layout."""

    __slots__ = ("steps", "inv_freq", "rotary_dim", "scale", "interleaved")

    def __init__(self, steps, inv_freq, scale, interleaved):
        self.steps, self.inv_freq, self.scale, self.interleaved = steps, inv_freq, scale, interleaved
        self.rotary_dim = 2 * len(inv_freq)


def rotary_table(rotary_dim, base=10000.0, factor=1.0, trained=None, low=1.0, high=32.0, scale=1.0, interleaved=False,
                 inv_freq=None, device="cuda"):
    """Frequencies base^(-2 i / rotary_dim) for pairs i of a head's first
    rotary_dim elements, scaled for contexts longer than a model was trained on:

    trained None: every frequency is divided by `factor` (positions interpolated);
    trained given (tokens): by parts. A pair that turns n times over them keeps
      its frequency where n >= high, has it divided where n <= low, and lies
      linearly between by n in between (Peng et al. 2023, who also set
      scale = 0.1 ln(factor) + 1).
    scale multiplies the rotated elements. interleaved: pairs are elements (2 i,
    2 i + 1), else (i, i + rotary_dim / 2). inv_freq: host numbers in place of
    base, factor and trained.
    """
    if not isinstance(rotary_dim, int) or rotary_dim < 2 or rotary_dim % 2 or rotary_dim > 512:
        raise ValueError("rotary_dim: even, 2 to 512")
    if not math.isfinite(scale):
        raise ValueError("scale: must be finite")
    if inv_freq is None:
        if not (base > 0 and math.isfinite(base)):
            raise ValueError("base: must be positive and finite")
        if not (factor > 0 and math.isfinite(factor)):
            raise ValueError("factor: must be positive and finite")
        inv_freq = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
        if trained is None:
            inv_freq = [f / factor for f in inv_freq]
        else:
            if not trained > 0:
                raise ValueError("trained: must be positive")
            if not high > low:
                raise ValueError("high: must be above low")
            keep = [min(max((trained * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in inv_freq]
            inv_freq = [f * (g + (1.0 - g) / factor) for f, g in zip(inv_freq, keep)]
    else:
        inv_freq = [float(f) for f in inv_freq]
        if len(inv_freq) != rotary_dim // 2:
            raise ValueError("inv_freq: one entry per pair")
    n = len(inv_freq)
    steps = torch.empty(n, dtype=torch.int64)
    L.check(L.load().tkv_rotary_steps(n, (ctypes.c_double * n)(*inv_freq), steps.data_ptr()))
    return RotaryTable(steps.to(device), tuple(inv_freq), float(scale), bool(interleaved))


def rotate(q, k, positions, table, inverse=False, out=None, stream=None):
    """Rotary positions of queries and keys (see tkv_rotate).

    q [tokens, Hq, d], k [tokens, Hkv, d] or None, in float32 or bfloat16, their
    tokens possibly strided, as views of a fused projection are; positions int32
    or int64 [tokens] on their device; table of rotary_table on it. inverse turns
    by the opposite angles; the table's scale multiplies then too, so that there
    and back gives the input times scale^2. out: (q_out, k_out) or None; a tensor of
    it may be the input itself (in place) and overlaps no other way. Returns
    (q_out, k_out).
    """
    lib = L.load()
    n, hq, d, sq = _tokens(q, "q")
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError("q: float32 or bfloat16")
    hk = sk = 0
    if k is not None:
        nk, hk, dk, sk = _tokens(k, "k", q)
        if nk != n or dk != d:
            raise ValueError("k: tokens and d must be those of q")
        _no_gradient("q, k", q, k)
    else:
        _no_gradient("q", q)
    if not isinstance(table, RotaryTable):
        raise ValueError("table: of rotary_table")
    dev = q.get_device()
    pp = _dense(positions, "positions", (torch.int64, torch.int32), dev, (n,))
    ps = _dense(table.steps, "table", (torch.int64,), dev)
    with _On(dev, stream) as on:
        if out is None:
            qo, so = _like(on, q), hq * d
            ko, to = (None, 0) if k is None else (_like(on, k), hk * d)
        else:
            if not isinstance(out, (tuple, list)) or len(out) != 2 or (out[1] is None) != (k is None):
                raise ValueError("out: (q_out, k_out)")
            qo, ko = out
            no, ho, do, so = _tokens(qo, "out", q)
            if no != n or ho != hq or do != d:
                raise ValueError("out: shape must be that of q")
            to = 0
            if k is not None:
                no, ho, do, to = _tokens(ko, "out", q)
                if no != n or ho != hk or do != d:
                    raise ValueError("out: shape must be that of k")
        st = lib.tkv_rotate(n, hq, hk, d, table.rotary_dim, dt, table.interleaved, bool(inverse), table.scale, ps, pp,
                            64 if positions.dtype is torch.int64 else 32, q.data_ptr(), sq, k.data_ptr() if hk else None, sk,
                            qo.data_ptr(), so, ko.data_ptr() if hk else None, to, on.raw)
        if st:
            L.check(st)
    return qo, ko


def _blocks(pool, scales, page_table, slot_mask, rows):
    """(device, pages, Hkv, d, and the addresses) of an 8-bit pool and its rows."""
    try:
        pages, hkv, two, page, d = pool.shape
        n, max_pages = page_table.shape
        dev = pool.get_device()
        if (two == 2 and page == 16 and n == rows and pool.dtype is torch.int8 and scales.dtype is torch.float32
                and page_table.dtype is torch.int32 and scales.shape == (pages, hkv, 2) and pool.is_contiguous()
                and scales.is_contiguous() and page_table.is_contiguous() and scales.get_device() == dev
                and page_table.get_device() == dev and not scales.requires_grad):
            if slot_mask is None:
                return dev, pages, hkv, d, pool.data_ptr(), scales.data_ptr(), page_table.data_ptr(), None, max_pages
            if (slot_mask.dtype in _MASK and slot_mask.shape == (pages,) and slot_mask.is_contiguous()
                    and slot_mask.get_device() == dev):
                return (dev, pages, hkv, d, pool.data_ptr(), scales.data_ptr(), page_table.data_ptr(), slot_mask.data_ptr(),
                        max_pages)
    except (AttributeError, ValueError):
        pass
    if not isinstance(pool, torch.Tensor) or pool.dim() != 5:
        raise ValueError("pool: must be int8 [pages, Hkv, 2, 16, d]")
    dev = pool.get_device()
    pages, hkv, _, _, d = pool.shape
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != rows:
        raise ValueError("page_table: must be [rows, max_pages]")
    if isinstance(scales, torch.Tensor):
        _no_gradient("scales", scales)
    return (dev, pages, hkv, d, _dense(pool, "pool", _I8, dev, (pages, hkv, 2, 16, d)),
            _dense(scales, "scales", _F32, dev, (pages, hkv, 2)), _dense(page_table, "page_table", _I32, dev),
            None if slot_mask is None else _dense(slot_mask, "slot_mask", _MASK, dev, (pages,)), page_table.shape[1])


def _pair(k, v):
    """(tokens, heads, d, token strides, dtype) of keys and values of one shape and kind."""
    try:
        n, h, d = k.shape
        if k.dtype is v.dtype and v.shape == k.shape and k.get_device() == v.get_device():
            (sk, a, b), (sv, e, f) = k.stride(), v.stride()
            if n > 1 and b == f == 1 and a == e == d and k.dtype in _DTYPES:
                return n, h, d, sk, sv, _DTYPES[k.dtype]
    except (AttributeError, ValueError):
        pass
    n, h, d, sk = _tokens(k, "k")
    tv, hv, dv, sv = _tokens(v, "v", k)
    if k.dtype not in _DTYPES:
        raise ValueError("k: float32 or bfloat16")
    if tv != n or hv != h or dv != d:
        raise ValueError("v: shape must be that of k")
    return n, h, d, sk, sv, _DTYPES[k.dtype]


def append_quantized(k, v, pool, scales, page_table, slot_mask, lens, new_lens, page_refs=None, status=None, stream=None):
    """Quantises new tokens into the pages their rows list (see
    tkv_append_quantized).

    k, v [sum new_lens, Hkv, d] float32 or bfloat16, packed in row order, tokens
    possibly strided; pool int8 [pages, Hkv, 2, 16, d]; scales float32 [pages,
    Hkv, 2]; page_table int32 [rows, max_pages]; slot_mask int32/uint32 [pages]
    or None; lens, new_lens host ints [rows]: tokens a row holds and gets (lens
    stays the caller's to update). page_refs int32 [pages] or None: pages that
    several rows list are not written. status int32 [1] becomes -1 if a listed
    page was outside the pool or not the row's alone; its tokens are not written.
    """
    lib = L.load()
    tk, hk, dk, sk, sv, dt = _pair(k, v)
    _no_gradient("k, v", k, v)
    a = _ints(lens, None, "lens")
    rows = len(a)
    b = _ints(new_lens, rows, "new_lens")
    dev, pages, hkv, d, pp, ps, pt, pm, max_pages = _blocks(pool, scales, page_table, slot_mask, rows)
    if k.get_device() != dev:
        raise ValueError("k: on another device")
    if hk != hkv or dk != d:
        raise ValueError("k: heads and d must be those of pool")
    if sum(b) != tk:
        raise ValueError("new_lens: must add up to the tokens of k")
    pr = None if page_refs is None else _dense(page_refs, "page_refs", _I32, dev, (pages,))
    with _On(dev, stream) as on:
        st = lib.tkv_append_quantized(rows, _at(a), _at(b), hkv, d, dt, k.data_ptr(), sk, v.data_ptr(), sv, pp, ps, pages, pt,
                                      max_pages, pm, pr,
                                      None if status is None else _dense(status, "status", _I32, dev, (1,)), on.raw)
        if st:
            L.check(st)


def read_quantized(pool, scales, page_table, slot_mask, lens, first=None, dtype=torch.bfloat16, out=None, stream=None):
    """Slots first .. lens - 1 (host ints [rows]; first defaults to 0) of each
    row as packed keys and values [sum (lens - first), Hkv, d] (see
    tkv_read_quantized); slots without their mask bit (slot_mask None: none) read
    as zeros. out: (k, v), tokens possibly strided, their dtype then counts.
    Returns (k, v).
    """
    lib = L.load()
    b = _ints(lens, None, "lens")
    rows = len(b)
    a = _ints([0] * rows if first is None else first, rows, "first")
    dev, pages, hkv, d, pp, ps, pt, pm, max_pages = _blocks(pool, scales, page_table, slot_mask, rows)
    n = sum(b) - sum(a)
    with _On(dev, stream) as on:
        if out is None:
            if n < 0:
                raise ValueError("first: must not pass lens")
            if dtype not in _DTYPES:
                raise ValueError("dtype: float32 or bfloat16")
            k = on.empty((n, hkv, d), dtype)
            v = _like(on, k)
            sk = sv = hkv * d
        else:
            if not isinstance(out, (tuple, list)) or len(out) != 2:
                raise ValueError("out: (k, v)")
            k, v = out
            tk, hk, dk, sk = _tokens(k, "out")
            tv, hv, dv, sv = _tokens(v, "out", k)
            if k.get_device() != dev:
                raise ValueError("out: on another device")
            if (tk, hk, dk) != (n, hkv, d) or (tv, hv, dv) != (n, hkv, d):
                raise ValueError(f"out: shapes must be {[n, hkv, d]}")
            dtype = k.dtype
            if dtype not in _DTYPES:
                raise ValueError("out: float32 or bfloat16")
        st = lib.tkv_read_quantized(rows, _at(a), _at(b), hkv, d, _DTYPES[dtype], pp, ps, pages, pt, max_pages, pm,
                                    k.data_ptr(), sk, v.data_ptr(), sv, on.raw)
        if st:
            L.check(st)
    return k, v


def quantized_attention(q, pool, scales, page_table, slot_mask, page_counts, out=None, alpha_sum=None, scratch=None,
                        stream=None):
    """Decode attention over an 8-bit pool (see tkv_quantized_attention):
    paged_attention with scales beside the codes.

    q [B, Hq, d] float32 or bfloat16; pool int8 [pages, Hkv, 2, 16, d]; scales
    float32 [pages, Hkv, 2]; page_table int32 [B, max_pages]; slot_mask
    int32/uint32 [pages]; page_counts host ints [B]; alpha_sum float32 [B, Hkv,
    max_pages * 16] or None (accumulated into).
    """
    lib = L.load()
    dt = _DTYPES.get(q.dtype) if isinstance(q, torch.Tensor) else None
    if dt is None or q.dim() != 3:
        raise ValueError("q: float32 or bfloat16 [B, Hq, d]")
    _no_gradient("q", q)
    batch, hq, d = q.shape
    dev, pages, hkv, dp, pp, ps, pt, pm, max_pages = _blocks(pool, scales, page_table, slot_mask, batch)
    pq = _dense(q, "q", (q.dtype,), dev)
    if dp != d:
        raise ValueError("q: d must be that of pool")
    if pm is None:
        raise ValueError("slot_mask: int32 or uint32 [pages]")
    pa = None if alpha_sum is None else _dense(alpha_sum, "alpha_sum", _F32, dev, (batch, hkv, max_pages * 16))
    counts = _ints(page_counts, batch, "page_counts")
    with _On(dev, stream) as on:
        if out is None:
            out = _like(on, q)
            po = out.data_ptr()
        else:
            po = _dense(out, "out", (q.dtype,), dev, (batch, hq, d))
        c = _at(counts)
        if scratch is None and max(counts, default=0) <= _SHORT_PAGES:
            st = lib.tkv_quantized_attention(batch, hq, hkv, d, dt, pq, pp, ps, pages, pt, pm, c, max_pages, po, pa, None, 0, on.raw)
            if st == L.OK:
                return out
            if st != L.ERR_INVALID_ARG:
                L.check(st)
        need = ctypes.c_size_t()
        st = lib.tkv_quantized_attention_scratch_size(batch, hq, hkv, d, dt, c, max_pages, pa is not None, ctypes.byref(need))
        if st:
            L.check(st)
        keep, scratch, nbytes = on.scratch(scratch, need.value)
        st = lib.tkv_quantized_attention(batch, hq, hkv, d, dt, pq, pp, ps, pages, pt, pm, c, max_pages, po, pa, scratch, nbytes,
                                         on.raw)
        if st:
            L.check(st)
    return out
