"""Prompt attention, shared-prefix decode attention and the page operators.

Argument marshalling only, as in cache.py: torch owns the buffers, the CUDA
kernels of libtkv.so do the work (include/tkv.h states each operator). Every
tensor of a call lies on one CUDA device, which need not be the current one;
a call on a stream other than the current one keeps the buffers it made alive
for that stream. ValueError names an argument of the wrong type, shape, layout
or device; the library's own checks raise TkvError.
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _ints(values, n, name):
    """(C int32 array, entries) of host integers."""
    if isinstance(values, torch.Tensor):
        _need(values.device.type == "cpu", f"{name}: host integers")
        values = values.tolist()
    try:
        values = array("i", values)
    except (TypeError, OverflowError) as e:
        raise ValueError(f"{name}: host integers of 32 bits ({e})") from None
    k = len(values)
    if n is not None and k != n:
        raise ValueError(f"{name}: one entry per sequence")
    return (ctypes.c_int32 * k).from_buffer(values) if k else None, k


def _dense(t, name, dtypes, device, shape=None):
    """The address of a contiguous tensor of the given kind."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{name}: wrong dtype")
    if t.device != device:
        raise ValueError(f"{name}: on another device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape must be {list(shape)}")
    return t.data_ptr()


def _tokens(t, name, like=None):
    """(pointer, token stride) of [tokens, heads, d] whose tokens are dense."""
    _need(isinstance(t, torch.Tensor) and t.dim() == 3, f"{name}: must be [tokens, heads, d]")
    _need(like is None or (t.dtype == like.dtype and t.device == like.device and t.shape[2] == like.shape[2]),
          f"{name}: dtype, device and d must be those of q")
    n, h, d = t.shape
    st = t.stride()
    _need((st[2] == 1 or d == 1) and (st[1] == d or h == 1), f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (st[0] if n > 1 else h * d)


class _On:
    """The call's device made current if it is not, and its stream."""

    __slots__ = ("device", "guard", "given", "raw")

    def __init__(self, device, stream):
        _need(device.type == "cuda", "the tensors must be on a CUDA device")
        self.device, self.given, self.guard = device, stream, None
        if torch.cuda.current_device() != device.index:
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        self.raw = torch.cuda.current_stream(self.device).cuda_stream
        if self.given is not None:
            _need(self.given.device == self.device, "stream: of another device")
            if self.given.cuda_stream == self.raw:
                self.given = None
            else:
                self.raw = self.given.cuda_stream
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc) if self.guard is not None else None

    def empty(self, shape, dtype):
        """A buffer made for this call."""
        t = torch.empty(shape, dtype=dtype, device=self.device)
        if self.given is not None:
            t.record_stream(self.given)
        return t

    def scratch(self, given, need):
        if given is None:
            return self.empty(need, torch.uint8) if need else None
        _need(isinstance(given, torch.Tensor) and given.is_contiguous() and given.device == self.device,
              "scratch: a contiguous tensor on the call's device")
        return given


def _bytes(t):
    return (t.data_ptr(), t.numel() * t.element_size()) if t is not None else (None, 0)


def _status(status, device):
    return None if status is None else _dense(status, "status", (torch.int32,), device, (1,))


def prompt_attention(q, k, v, q_lens, k_lens=None, out=None, scratch=None, status=None, stream=None):
    """Causal attention over packed prompts (see tkv_prompt_attention).

    q [sum q_len, Hq, d]; k, v [sum k_len, Hkv, d]; q_lens, k_lens host ints
    per sequence (k_lens defaults to q_lens; the keys ahead of a sequence's
    queries are an already cached part). The tokens of q, k, v and out may be
    strided, as views of a fused projection are.
    """
    lib = L.load()
    pq, sq = _tokens(q, "q")
    pk, sk = _tokens(k, "k", q)
    pv, sv = _tokens(v, "v", q)
    _need(q.dtype in _DTYPES, "q: float32 or bfloat16")
    _need(k.shape == v.shape, "v: shape must be that of k")
    ql, batch = _ints(q_lens, None, "q_lens")
    kl, _ = (ql, batch) if k_lens is None else _ints(k_lens, batch, "k_lens")
    _need(sum(ql or ()) == q.shape[0], "q_lens: must add up to the tokens of q")
    _need(sum(kl or ()) == k.shape[0], "k_lens: must add up to the tokens of k")
    hq, hkv, d, dt = q.shape[1], k.shape[1], q.shape[2], _DTYPES[q.dtype]
    with _On(q.device, stream) as on:
        need = ctypes.c_size_t()
        L.check(lib.tkv_prompt_attention_scratch_size(batch, ql, kl, hq, hkv, d, dt, ctypes.byref(need)))
        if out is None:
            out = on.empty(q.shape, q.dtype)
        po, so = _tokens(out, "out", q)
        _need(out.shape == q.shape, "out: shape must be that of q")
        scratch = on.scratch(scratch, need.value)
        L.check(lib.tkv_prompt_attention(batch, ql, kl, hq, hkv, d, dt, pq, sq, pk, sk, pv, sv, po, so,
                                         *_bytes(scratch), _status(status, q.device), on.raw))
    return out


def shared_prefix_attention(q, pool, page_table, slot_mask, page_counts, shared_pages, out=None, alpha_sum=None,
                            scratch=None, status=None, stream=None):
    """Decode attention of sequences whose first `shared_pages` pages are the
    same: paged_attention with the prefix read once for the batch (see
    tkv_shared_prefix_attention).

    q [B, Hq, d]; pool [pages, Hkv, 2, 16, d]; page_table int32 [B, max_pages];
    slot_mask int32/uint32 [pages]; page_counts host ints [B], the prefix among
    them; alpha_sum float32 [B, Hkv, max_pages * 16] or None (accumulated into
    behind the prefix).
    """
    lib = L.load()
    dev = q.device
    _need(q.dim() == 3 and q.dtype in _DTYPES, "q: float32 or bfloat16 [B, Hq, d]")
    batch, hq, d = q.shape
    pq = _dense(q, "q", (q.dtype,), dev)
    _need(pool.dim() == 5, "pool: must be [pages, Hkv, 2, 16, d]")
    pages, hkv = pool.shape[:2]
    pp = _dense(pool, "pool", (q.dtype,), dev, (pages, hkv, 2, 16, d))
    _need(page_table.dim() == 2 and page_table.shape[0] == batch, "page_table: must be [B, max_pages]")
    pt = _dense(page_table, "page_table", (torch.int32,), dev)
    pm = _dense(slot_mask, "slot_mask", (torch.int32, torch.uint32), dev, (pages,))
    max_pages, dt = page_table.shape[1], _DTYPES[q.dtype]
    counts, _ = _ints(page_counts, batch, "page_counts")
    pa = None
    if alpha_sum is not None:
        pa = _dense(alpha_sum, "alpha_sum", (torch.float32,), dev, (batch, hkv, max_pages * 16))
    with _On(dev, stream) as on:
        need = ctypes.c_size_t()
        L.check(lib.tkv_shared_prefix_attention_scratch_size(batch, hq, hkv, d, dt, counts, max_pages, shared_pages,
                                                             pa is not None, ctypes.byref(need)))
        if out is None:
            out = on.empty(q.shape, q.dtype)
        po = _dense(out, "out", (q.dtype,), dev, q.shape)
        scratch = on.scratch(scratch, need.value)
        L.check(lib.tkv_shared_prefix_attention(batch, hq, hkv, d, dt, pq, pp, pages, pt, pm, counts, max_pages,
                                                shared_pages, po, pa, *_bytes(scratch), _status(status, dev),
                                                on.raw))
    return out


def _pool(pool):
    """(pointer, layers, pages, Hkv, d, dtype) of [layers, pages, Hkv, 2, 16, d], or of one layer of it."""
    _need(isinstance(pool, torch.Tensor) and pool.dim() in (5, 6) and tuple(pool.shape[-3:-1]) == (2, 16),
          "pool: must be [layers, pages, Hkv, 2, 16, d] or one layer of it")
    _need(pool.dtype in _DTYPES, "pool: float32 or bfloat16")
    _need(pool.is_contiguous(), "pool: not contiguous")
    shape = pool.shape if pool.dim() == 6 else (1, *pool.shape)
    return pool.data_ptr(), shape[0], shape[1], shape[2], shape[5], _DTYPES[pool.dtype]


def _book(page_table, page_refs, slot_mask, device, pages):
    _need(isinstance(page_table, torch.Tensor) and page_table.dim() == 2, "page_table: must be [rows, max_pages]")
    return (_dense(page_table, "page_table", (torch.int32,), device),
            None if page_refs is None else _dense(page_refs, "page_refs", (torch.int32,), device, (pages,)),
            _dense(slot_mask, "slot_mask", (torch.int32, torch.uint32), device, (pages,)))


def _positions(positions, device, pages):
    return None if positions is None else _dense(positions, "positions", (torch.int32,), device, (pages, 16))


def fork_sequences(pool, page_table, page_counts, page_refs, slot_mask, parents, children, share=True,
                   positions=None, scratch=None, stream=None):
    """Forks rows `parents` of the page table into the empty rows `children`
    (see tkv_fork_sequences): full pages are shared by count and an unfilled
    last page copied (share), or every page copied. Returns the device status
    int32 [1]: 0, the pages lacking (nothing changed), or -1 (a parent lists a
    page that is not held; nothing changed). The children's counts are their
    parents'; page_counts (host ints [rows]) stays the caller's to update.
    """
    lib = L.load()
    pp, layers, pages, hkv, d, dt = _pool(pool)
    pt, pr, pm = _book(page_table, page_refs, slot_mask, pool.device, pages)
    rows, max_pages = page_table.shape
    counts, _ = _ints(page_counts, rows, "page_counts")
    par, n = _ints(parents, None, "parents")
    chi, _ = _ints(children, n, "children")
    pos = _positions(positions, pool.device, pages)
    with _On(pool.device, stream) as on:
        need = ctypes.c_size_t()
        L.check(lib.tkv_fork_sequences_scratch_size(rows, max_pages, counts, n, par, chi, bool(share), ctypes.byref(need)))
        scratch = on.scratch(scratch, need.value)
        status = on.empty(1, torch.int32)
        L.check(lib.tkv_fork_sequences(pp, layers, pages, hkv, d, dt, pt, rows, max_pages, counts, pr, pm, pos, n, par,
                                       chi, bool(share), *_bytes(scratch), status.data_ptr(), on.raw))
    return status


def free_sequences(page_table, page_counts, page_refs, slot_mask, seqs, stream=None):
    """Frees rows `seqs` of the page table (see tkv_free_sequences): pages no
    row lists any more become free. Returns the device status int32 [1]: 0, or
    -1 if a row listed a page that was not held.
    """
    lib = L.load()
    dev = page_table.device
    _need(page_refs is not None and page_refs.dim() == 1, "page_refs: must be [pages]")
    pages = page_refs.shape[0]
    pt, pr, pm = _book(page_table, page_refs, slot_mask, dev, pages)
    rows, max_pages = page_table.shape
    counts, _ = _ints(page_counts, rows, "page_counts")
    seq, n = _ints(seqs, None, "seqs")
    with _On(dev, stream) as on:
        status = on.empty(1, torch.int32)
        L.check(lib.tkv_free_sequences(pt, rows, max_pages, counts, pages, pr, pm, n, seq, status.data_ptr(),
                                       on.raw))
    return status


def compact_sequences(pool, page_table, page_counts, page_refs, slot_mask, positions=None, scratch=None, stream=None):
    """Moves the tokens of every row of the page table into its first pages and
    frees the emptied ones (see tkv_compact_sequences). page_refs None: no page
    is shared. Returns the new page counts, device int32 [rows] (-1: that row
    lists a page that is not held and was not changed).
    """
    lib = L.load()
    pp, layers, pages, hkv, d, dt = _pool(pool)
    pt, pr, pm = _book(page_table, page_refs, slot_mask, pool.device, pages)
    rows, max_pages = page_table.shape
    counts, _ = _ints(page_counts, rows, "page_counts")
    pos = _positions(positions, pool.device, pages)
    with _On(pool.device, stream) as on:
        need = ctypes.c_size_t()
        L.check(lib.tkv_compact_sequences_scratch_size(rows, max_pages, counts, ctypes.byref(need)))
        scratch = on.scratch(scratch, need.value)
        new = on.empty(rows, torch.int32)
        L.check(lib.tkv_compact_sequences(pp, layers, pages, hkv, d, dt, pt, rows, max_pages, counts, pr, pm, pos,
                                          new.data_ptr(), *_bytes(scratch), on.raw))
    return new
