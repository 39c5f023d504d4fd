"""Prompt attention, shared-prefix decode attention and the page operators.

Argument marshalling only, as in cache.py: torch owns the buffers, the CUDA
kernels of libtkv.so do the work (include/tkv.h states each operator). Every
tensor of a call lies on one CUDA device, which need not be the current one;
a call on a stream other than the current one takes the buffers it makes from
that stream's memory; the caller has other streams wait for it before they use
the result. ValueError names an argument of the wrong type, shape, layout
or device, or one that asks for a gradient; the library's own checks raise
TkvError.
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from . import _lib as L

_DTYPES = {torch.float32: L.DTYPE_F32, torch.bfloat16: L.DTYPE_BF16}
_I32 = (torch.int32,)
_MASK = (torch.int32, torch.uint32)
# The small calls are bound by this file, so it stays flat: cheap checks first,
# names and messages only on the way out.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _ints(values, n, name):
    """Host integers as an array of C ints."""
    if isinstance(values, torch.Tensor):
        if values.device.type != "cpu":
            raise ValueError(f"{name}: host integers")
        values = values.tolist()
    try:
        values = array("i", values)
    except (TypeError, OverflowError) as e:
        raise ValueError(f"{name}: host integers of 32 bits ({e})") from None
    if n is not None and len(values) != n:
        raise ValueError(f"{name}: one entry per sequence")
    return values


def _at(ints):
    return ints.buffer_info()[0]


def _dense(t, name, dtypes, device, shape=None):
    """The address of a contiguous tensor of the given kind on a device, by its index."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{name}: wrong dtype")
    if t.get_device() != device:
        raise ValueError(f"{name}: on another device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape must be {list(shape)}")
    return t.data_ptr()


def _tokens(t, name, like=None):
    """(tokens, heads, d, token stride) of [tokens, heads, d] whose tokens are dense."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name}: must be [tokens, heads, d]")
    if like is not None and (t.dtype is not like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name}: dtype and device must be those of q")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 and d != 1) or (s1 != d and h != 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return n, h, d, (s0 if n > 1 else h * d)


def _no_gradient(names, *tensors):
    for t in tensors:
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{names}: the operator has no backward pass; call it under torch.no_grad() or detach them")


class _On:
    """The call's device made current if it is not, its stream, and buffers made
    for the call."""

    __slots__ = ("device", "guard", "given", "raw")

    def __init__(self, device, stream):
        if device < 0:
            raise ValueError("the tensors must be on a CUDA device")
        self.device = device
        self.guard = None if _current_device() == device else torch.cuda.device(device)
        self.given = None
        self.raw = _raw_stream(device)
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                raise ValueError("stream: a torch.cuda.Stream")
            if stream.device_index != device:
                raise ValueError("stream: of another device")
            if stream.cuda_stream != self.raw:
                self.given, self.raw = stream, stream.cuda_stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)

    def empty(self, shape, dtype, returned=True):
        """A buffer from the memory of the stream that uses it: a block of the
        current stream's may still be in use by work queued there. A returned
        one may be dropped with work on the current stream outstanding."""
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.given):
            t = torch.empty(shape, dtype=dtype, device=self.device)
        if returned:
            t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def scratch(self, given, need):
        """(tensor, address, bytes)"""
        if given is None:
            if need == 0:
                return None, None, 0
            given = self.empty(need, torch.uint8, returned=False)
            return given, given.data_ptr(), need
        if not isinstance(given, torch.Tensor) or not given.is_contiguous() or given.get_device() != self.device:
            raise ValueError("scratch: a contiguous tensor on the call's device")
        return given, given.data_ptr(), given.numel() * given.element_size()


def prompt_attention(q, k, v, q_lens, k_lens=None, out=None, scratch=None, status=None, stream=None):
    """Causal attention over packed prompts (see tkv_prompt_attention).

    q [sum q_len, Hq, d]; k, v [sum k_len, Hkv, d]; q_lens, k_lens host ints
    per sequence (k_lens defaults to q_lens; the keys ahead of a sequence's
    queries are an already cached part). The tokens of q, k, v and out may be
    strided, as views of a fused projection are.
    status: int32 [1] that becomes 1 if a bounded device wait gave up (rows of
    out are not valid then); without one, the next attention call on the device
    raises TkvError, and so does attention_synchronize.
    """
    lib = L.load()
    tq, hq, d, sq = _tokens(q, "q")
    tk, hkv, dk, sk = _tokens(k, "k", q)
    tv, hv, dv, sv = _tokens(v, "v", q)
    _no_gradient("q, k, v", q, k, v)
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError("q: float32 or bfloat16")
    if dk != d:
        raise ValueError("k: d must be that of q")
    if tv != tk or hv != hkv or dv != d:
        raise ValueError("v: shape must be that of k")
    ql = _ints(q_lens, None, "q_lens")
    batch = len(ql)
    kl = ql if k_lens is None else _ints(k_lens, batch, "k_lens")
    if sum(ql) != tq:
        raise ValueError("q_lens: must add up to the tokens of q")
    if sum(kl) != tk:
        raise ValueError("k_lens: must add up to the tokens of k")
    dev = q.get_device()
    with _On(dev, stream) as on:
        if out is None:
            out, so = on.empty((tq, hq, d), q.dtype), hq * d
        else:
            to, ho, do, so = _tokens(out, "out", q)
            if to != tq or ho != hq or do != d:
                raise ValueError("out: shape must be that of q")
        a, b, need = _at(ql), _at(kl), ctypes.c_size_t()
        st = lib.tkv_prompt_attention_scratch_size(batch, a, b, hq, hkv, d, dt, ctypes.byref(need))
        if st:
            L.check(st)
        keep, scratch, nbytes = on.scratch(scratch, need.value)
        st = lib.tkv_prompt_attention(batch, a, b, hq, hkv, d, dt, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv,
                                      out.data_ptr(), so, scratch, nbytes,
                                      None if status is None else _dense(status, "status", _I32, dev, (1,)), on.raw)
        if st:
            L.check(st)
    return out


def shared_prefix_attention(q, pool, page_table, slot_mask, page_counts, shared_pages, out=None, alpha_sum=None,
                            scratch=None, status=None, stream=None):
    """Decode attention of sequences whose first `shared_pages` pages are the
    same: paged_attention with the prefix read once for the batch (see
    tkv_shared_prefix_attention).

    q [B, Hq, d]; pool [pages, Hkv, 2, 16, d]; page_table int32 [B, max_pages];
    slot_mask int32/uint32 [pages]; page_counts host ints [B], the prefix among
    them; alpha_sum float32 [B, Hkv, max_pages * 16] or None (accumulated into
    behind the prefix); status as for prompt_attention.
    """
    lib = L.load()
    dt = _DTYPES.get(q.dtype) if isinstance(q, torch.Tensor) else None
    if dt is None or q.dim() != 3:
        raise ValueError("q: float32 or bfloat16 [B, Hq, d]")
    if not isinstance(pool, torch.Tensor) or pool.dim() != 5:
        raise ValueError("pool: must be [pages, Hkv, 2, 16, d]")
    _no_gradient("q, pool", q, pool)
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != q.shape[0]:
        raise ValueError("page_table: must be [B, max_pages]")
    dev, dtypes = q.get_device(), (q.dtype,)
    batch, hq, d = q.shape
    pages, hkv = pool.shape[:2]
    max_pages = page_table.shape[1]
    pq = _dense(q, "q", dtypes, dev)
    pp = _dense(pool, "pool", dtypes, dev, (pages, hkv, 2, 16, d))
    pt = _dense(page_table, "page_table", _I32, dev)
    pm = _dense(slot_mask, "slot_mask", _MASK, dev, (pages,))
    pa = None if alpha_sum is None else _dense(alpha_sum, "alpha_sum", (torch.float32,), dev, (batch, hkv, max_pages * 16))
    counts = _ints(page_counts, batch, "page_counts")
    shared_pages = _ints([shared_pages], 1, "shared_pages")[0]
    with _On(dev, stream) as on:
        if out is None:
            out = on.empty((batch, hq, d), q.dtype)
            po = out.data_ptr()
        else:
            po = _dense(out, "out", dtypes, dev, (batch, hq, d))
        c, need = _at(counts), ctypes.c_size_t()
        st = lib.tkv_shared_prefix_attention_scratch_size(batch, hq, hkv, d, dt, c, max_pages, shared_pages, pa is not None,
                                                          ctypes.byref(need))
        if st:
            L.check(st)
        keep, scratch, nbytes = on.scratch(scratch, need.value)
        st = lib.tkv_shared_prefix_attention(batch, hq, hkv, d, dt, pq, pp, pages, pt, pm, c, max_pages, shared_pages, po, pa,
                                             scratch, nbytes,
                                             None if status is None else _dense(status, "status", _I32, dev, (1,)), on.raw)
        if st:
            L.check(st)
    return out


def attention_synchronize(stream=None):
    """Waits for a stream (the current one); TkvError if a wait of
    prompt_attention or shared_prefix_attention gave up on its device in a call
    without a status of its own (see tkv_attention_synchronize)."""
    if stream is None:
        stream = torch.cuda.current_stream()
    with torch.cuda.device(stream.device_index):
        L.check(L.load().tkv_attention_synchronize(stream.cuda_stream))


def _pool(pool):
    """(address, layers, pages, Hkv, d, dtype) of [layers, pages, Hkv, 2, 16, d], or of one layer of it."""
    shape = tuple(pool.shape) if isinstance(pool, torch.Tensor) else ()
    if len(shape) == 5:
        shape = (1, *shape)
    if len(shape) != 6 or shape[3:5] != (2, 16):
        raise ValueError("pool: must be [layers, pages, Hkv, 2, 16, d] or one layer of it")
    dt = _DTYPES.get(pool.dtype)
    if dt is None:
        raise ValueError("pool: float32 or bfloat16")
    if not pool.is_contiguous():
        raise ValueError("pool: not contiguous")
    return pool.data_ptr(), shape[0], shape[1], shape[2], shape[5], dt


def _book(page_table, page_refs, slot_mask, device, pages):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table: must be [rows, max_pages]")
    return (_dense(page_table, "page_table", _I32, device),
            None if page_refs is None else _dense(page_refs, "page_refs", _I32, device, (pages,)),
            _dense(slot_mask, "slot_mask", _MASK, device, (pages,)))


def fork_sequences(pool, page_table, page_counts, page_refs, slot_mask, parents, children, share=True,
                   positions=None, scratch=None, stream=None):
    """Forks rows `parents` of the page table into the empty rows `children`
    (see tkv_fork_sequences): full pages are shared by count and an unfilled
    last page copied (share), or every page copied. Returns the device status
    int32 [1]: 0, the pages lacking (nothing changed), or -1 (a parent lists a
    page that is not held; nothing changed). If it is 0 the children's counts are
    their parents'; page_counts (host ints [rows]) stays the caller's to update.
    Read it before the children are used: their rows are not forked otherwise.
    """
    lib = L.load()
    pp, layers, pages, hkv, d, dt = _pool(pool)
    dev = pool.get_device()
    pt, pr, pm = _book(page_table, page_refs, slot_mask, dev, pages)
    rows, max_pages = page_table.shape
    counts = _ints(page_counts, rows, "page_counts")
    par = _ints(parents, None, "parents")
    n = len(par)
    chi = _ints(children, n, "children")
    pos = None if positions is None else _dense(positions, "positions", _I32, dev, (pages, 16))
    share = bool(share)
    with _On(dev, stream) as on:
        c, a, b, need = _at(counts), _at(par), _at(chi), ctypes.c_size_t()
        st = lib.tkv_fork_sequences_scratch_size(rows, max_pages, c, n, a, b, share, ctypes.byref(need))
        if st:
            L.check(st)
        keep, scratch, nbytes = on.scratch(scratch, need.value)
        status = on.empty(1, torch.int32)
        st = lib.tkv_fork_sequences(pp, layers, pages, hkv, d, dt, pt, rows, max_pages, c, pr, pm, pos, n, a, b, share,
                                    scratch, nbytes, status.data_ptr(), on.raw)
        if st:
            L.check(st)
    return status


def free_sequences(page_table, page_counts, page_refs, slot_mask, seqs, stream=None):
    """Frees rows `seqs` of the page table (see tkv_free_sequences): pages no
    row lists any more become free. Returns the device status int32 [1]: 0, or
    -1 if a row listed a page that was not held (its other pages are freed).
    """
    lib = L.load()
    if not isinstance(page_table, torch.Tensor):
        raise ValueError("page_table: must be [rows, max_pages]")
    dev = page_table.get_device()
    if not isinstance(page_refs, torch.Tensor) or page_refs.dim() != 1:
        raise ValueError("page_refs: must be [pages]")
    pages = page_refs.shape[0]
    pt, pr, pm = _book(page_table, page_refs, slot_mask, dev, pages)
    rows, max_pages = page_table.shape
    counts = _ints(page_counts, rows, "page_counts")
    seq = _ints(seqs, None, "seqs")
    with _On(dev, stream) as on:
        status = on.empty(1, torch.int32)
        st = lib.tkv_free_sequences(pt, rows, max_pages, _at(counts), pages, pr, pm, len(seq), _at(seq), status.data_ptr(),
                                    on.raw)
        if st:
            L.check(st)
    return status


def compact_sequences(pool, page_table, page_counts, page_refs, slot_mask, positions=None, scratch=None, stream=None):
    """Moves the tokens of every row of the page table into its first pages and
    frees the emptied ones (see tkv_compact_sequences). page_refs None: no page
    is shared. Returns the new page counts, device int32 [rows] (-1: that row
    lists a page that is not held and was not changed). alpha_sum of earlier
    attention calls does not move with the tokens: add it to their scores, by
    positions, before slots are emptied, and start the next one from zeros.
    """
    lib = L.load()
    pp, layers, pages, hkv, d, dt = _pool(pool)
    dev = pool.get_device()
    pt, pr, pm = _book(page_table, page_refs, slot_mask, dev, pages)
    rows, max_pages = page_table.shape
    counts = _ints(page_counts, rows, "page_counts")
    pos = None if positions is None else _dense(positions, "positions", _I32, dev, (pages, 16))
    with _On(dev, stream) as on:
        c, need = _at(counts), ctypes.c_size_t()
        st = lib.tkv_compact_sequences_scratch_size(rows, max_pages, c, ctypes.byref(need))
        if st:
            L.check(st)
        keep, scratch, nbytes = on.scratch(scratch, need.value)
        new = on.empty(rows, torch.int32)
        st = lib.tkv_compact_sequences(pp, layers, pages, hkv, d, dt, pt, rows, max_pages, c, pr, pm, pos, new.data_ptr(),
                                       scratch, nbytes, on.raw)
        if st:
            L.check(st)
    return new
