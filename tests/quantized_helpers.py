"""Plain forms of the rotary and 8-bit cache operators, and the error bounds
their tests use. Nothing here is shared with the library."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

from operator_helpers import HALF, f64

PAGE = 16
E32 = 2.0 ** -24                      # half a step of fp32, relative
# 1 / 2 pi to 256 bits
INV_2PI = Fraction(0x28be60db9391054a7f09d5f47d4d377036d8a5664f10e4107f9458eaf7aef158, 1 << 256)


def rotate_reference(x, positions, inv_freq, scale, interleaved, inverse, dtype, steps=None):
    """(y, bound) float64 of [tokens, heads, d]; angles in exact arithmetic, from the
    frequencies or, where given, the steps (turns per position in 2^-64 turns) they are held as.

    A step is off by at most 2^-64 turns, which is |pos| 2^-64 turns of angle: for
    positions of up to 2^33, 2^-28.3, well below a sine's own error, and more than
    the bound for positions beyond; so tests of those give the steps.

    The bound: sine and cosine are off by 2^-27 half turns of the angle (2^-25.3)
    and a step of fp32 (2^-24), each product and the scale by e, their sum by e:
    (|a| + |b|) |scale| (2^-23 + 5 e) with the above, and u |y| for the output's rounding.
    """
    x = f64(x)
    n, r = x.shape[0], 2 * len(inv_freq)
    t = np.empty((n, r // 2))
    for j, f in enumerate(inv_freq):
        turns = Fraction(f) * INV_2PI if steps is None else Fraction(steps[j], 1 << 64)
        for i, pos in enumerate(positions):
            part = (turns * int(pos)) % 1
            t[i, j] = float(part if part < Fraction(1, 2) else part - 1) * 2 * math.pi
    if inverse:
        t = -t
    c, s = np.cos(t)[:, None] * scale, np.sin(t)[:, None] * scale
    y, bound = x.copy(), np.zeros_like(x)
    ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    slack = (np.abs(a) + np.abs(b)) * abs(scale) * (2.0 ** -23 + 5 * E32)
    for at in (ia, ib):
        bound[..., at] = slack * (1 + HALF[dtype]) + HALF[dtype] * np.abs(y[..., at]) + 1e-38
    return y, bound


class Cache:
    """Rows of tokens in 8-bit blocks, as the operators define them, in NumPy fp32."""

    def __init__(self, pages, hkv, d, codes=None, scales=None, mask=None):
        self.codes = np.zeros((pages, hkv, 2, PAGE, d), np.int8) if codes is None else codes.copy()
        self.scales = np.zeros((pages, hkv, 2), np.float32) if scales is None else scales.copy()
        self.mask = np.zeros(pages, np.int64) if mask is None else mask.astype(np.int64)

    def append(self, k, v, table, lens, new):
        """k, v float32 [tokens, hkv, d]."""
        pages, t0 = self.codes.shape[0], 0
        with np.errstate(all="ignore"):
            for b, (n0, n) in enumerate(zip(lens, new)):
                for p in range(n0 // PAGE, -(-(n0 + n) // PAGE)):
                    lo, hi = max(n0 - p * PAGE, 0), min(n0 + n - p * PAGE, PAGE)
                    page = table[b][p]
                    if not 0 <= page < pages or lo >= hi:
                        continue
                    at = t0 + p * PAGE + lo - n0
                    for j, x in enumerate((k, v)):
                        for h in range(x.shape[1]):
                            self._block(page, h, j, lo, hi, x[at:at + hi - lo, h])
                    bits = (1 << hi) - (1 << lo)
                    self.mask[page] = bits | (self.mask[page] if lo else 0)
                t0 += n

    def _block(self, page, h, j, lo, hi, x):
        codes = self.codes[page, h, j]
        old = self.scales[page, h, j] if lo else np.float32(0)
        top = np.abs(x).max()                                    # a NaN wins
        mine = top / np.float32(127)
        scale = mine if mine > old or np.isnan(mine) else old
        if not np.isfinite(scale):
            codes[lo:hi] = 0
            self.scales[page, h, j] = np.nan
            return
        self.scales[page, h, j] = scale
        codes[lo:hi] = np.clip(np.rint(x / scale), -127, 127) if scale > 0 else 0
        if lo and scale > old:
            codes[:lo] = np.rint(codes[:lo].astype(np.float32) * (old / scale))

    def read(self, table, first, lens, mask=True):
        """(k, v) float32."""
        pages, (_, hkv, _, _, d), out = self.codes.shape[0], self.codes.shape, [[], []]
        for b, (lo, hi) in enumerate(zip(first, lens)):
            for s in range(lo, hi):
                page = table[b][s // PAGE]
                live = 0 <= page < pages and (not mask or self.mask[page] >> (s % PAGE) & 1)
                for j in range(2):
                    out[j].append(self.codes[page, :, j, s % PAGE].astype(np.float32) * self.scales[page, :, j, None]
                                  if live else np.zeros((hkv, d), np.float32))
        return tuple(np.stack(x) if x else np.zeros((0, hkv, d), np.float32) for x in out)


def attend_reference(q, codes, scales, table, masks, counts):
    """(out, bound, alpha [B, Hkv, width * 16], its bound) float64.

    With u half a step of the output type, A = sum_j p_j |v_j|, m keys, e = 2^-23
    (a tensor core may cut where a sum is rounded), t = 2^-11 (weights in fp16) for
    bf16 and 2^-21 for fp32 (two fp16 parts, the second to 2^-11 of a first rounded
    to 2^-11, both sums):
      output rounding         u |o|
      weights                 t A, and 2^-36 max|v| for each weight below fp16's range
      queries in fp16 parts   each element off by 2^-24 max|q| (bf16), 2^-22 max|q| (fp32)
      logits                  D = (d + 4) e max_j sum|q k| / sqrt(d) + that of the queries
      exponents               X = e (1.45 max|l| + max|log2 scale of V| + 32): logit, the power of two of
                              V's scale and the reference are added in base 2 in fp32
      weights of those        2 (D + X) A
      sums of m terms         2 m e A
    """
    dtype = q.dtype
    u, e = HALF[dtype], 2.0 ** -23
    t, dq = (2.0 ** -11, 2.0 ** -24) if dtype == torch.bfloat16 else (2.0 ** -21, 2.0 ** -22)
    q, codes, scales = f64(q), codes.astype(np.float64), scales.astype(np.float64)
    B, hq, d = q.shape
    pages, hkv = codes.shape[:2]
    g, width = hq // hkv, len(table[0])
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    alpha, ab = np.zeros((B, hkv, width * PAGE)), np.zeros((B, hkv, width * PAGE))
    with np.errstate(all="ignore"):
        for b in range(B):
            at = [(i * PAGE + s, page, s) for i, page in enumerate(table[b][:counts[b]]) if 0 <= page < pages
                  for s in range(PAGE) if masks[page] >> s & 1]
            if not at:
                continue
            slot, page, s = (np.array(x) for x in zip(*at))
            for h in range(hkv):
                k = codes[page, h, 0, s] * scales[page, h, 0, None]
                v = codes[page, h, 1, s] * scales[page, h, 1, None]
                rows = q[b, h * g:(h + 1) * g]
                l = rows @ k.T / math.sqrt(d)
                mag = (np.abs(rows) @ np.abs(k).T).max(1, keepdims=True) / math.sqrt(d)
                qerr = dq * np.abs(rows).max(1, keepdims=True) * np.abs(k).sum(1).max() / math.sqrt(d)
                top = l.max(1, keepdims=True)
                p = np.exp(l - np.where(np.isneginf(top), 0, top))
                z = p.sum(1, keepdims=True)
                p = p / np.where(z == 0, 1, z)
                o, a = p @ v, p @ np.abs(v)
                sv = scales[page, h, 1]
                power = np.abs(np.log2(np.where((sv > 0) & np.isfinite(sv), sv, 1.0))).max()
                delta = (d + 4) * e * mag + qerr + e * (1.45 * mag + power + 32)
                n = len(at)
                out[b, h * g:(h + 1) * g] = o
                bound[b, h * g:(h + 1) * g] = (u * np.abs(o) + (t + 2 * delta + 2 * n * e) * a
                                               + n * 2.0 ** -36 * np.abs(v).max()) * (1 + 2.0 ** -6) + 1e-30
                alpha[b, h, slot] = p.sum(0)
                ab[b, h, slot] = (p * (2 * delta + (n + 16) * e)).sum(0) + 1e-30
    return out, bound, alpha, ab
