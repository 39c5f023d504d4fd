"""Plain float64 forms of the prompt, shared-prefix and page operators, and the
error bounds their tests use. Nothing here is shared with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def attend(q, k, v, seen, dtype):
    """Rows q [n, d] over k, v [m, d] where seen [n, m]; float64 NumPy.

    Returns (o, bound, p). The bound counts, with u = half a step of the dtype
    and e = 2^-24, A = sum_j p_j |v_j| per row:
      output rounding        u |o|
      weights rounded to bf16, w (1 + t) with |t| <= u, in the product with V and in
      their sum (bf16 only): sum t w v - o sum t w, at most u (A + |o|)
      a logit is a d-term fp32 sum: off by D = (d + 2) e max_j sum|q k| / sqrt(d),
      so each weight and the sum of weights by a relative D + 4 e (exp2, its
      argument): 2 (D + 4 e) A, and 2^-20 for arguments up to 16 in base 2
      fp32 sums of m terms   2 m e A
    """
    u, e = HALF[dtype], 2.0 ** -24
    n, d = q.shape
    m = k.shape[0]
    if m == 0:
        return np.zeros((n, v.shape[1] if v.size else d)), np.zeros((n, d)), np.zeros((n, 0))
    k0, v0 = np.where(seen.any(0)[:, None], k, 0.0), np.where(seen.any(0)[:, None], v, 0.0)
    l = q @ k0.T / math.sqrt(d)
    mag = np.abs(q) @ np.abs(k0.T) / math.sqrt(d)
    l = np.where(seen, l, -np.inf)
    top = l.max(1, keepdims=True)
    p = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    p = np.where(seen, p, 0.0)
    z = p.sum(1, keepdims=True)
    p = p / np.where(z > 0, z, 1.0)
    o, a = p @ v0, p @ np.abs(v0)
    mag = np.where(seen, mag, 0.0).max(1, keepdims=True)
    delta = (d + 2) * e * mag + 4 * e + e * mag * 1.5
    bound = u * np.abs(o) + (u * (a + np.abs(o)) if dtype == torch.bfloat16 else 0.0) + (2 * delta + 2 * m * e) * a
    return o, bound * (1 + 2.0 ** -6) + 1e-30, p


def alpha_bound(p, q, k, seen, d):
    """Bound of sum_g p_g: each weight is off by 2 (D + 4 e) relative, its sum over
    m keys by m e, the sum over the heads by a few e."""
    e = 2.0 ** -24
    mag = np.where(seen, np.abs(q) @ np.abs(np.where(seen.any(0)[:, None], k, 0.0).T) / math.sqrt(d), 0.0).max(1, keepdims=True)
    delta = (d + 2) * e * mag + 4 * e + e * mag * 1.5
    return (p * (2 * delta + (p.shape[1] + 16) * e)).sum(0) + 1e-30


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def prompt_reference(q, k, v, q_lens, k_lens):
    """(out, bound) float64 [tokens, Hq, d] of packed causal prompts."""
    dtype = q.dtype
    q, k, v = f64(q), f64(k), f64(v)
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        seen = np.arange(nk)[None] <= np.arange(nq)[:, None] + nk - nq
        for h in range(hq):
            kv = h // (hq // hkv)
            if nq:
                out[q0:q0 + nq, h], bound[q0:q0 + nq, h], _ = attend(q[q0:q0 + nq, h], k[k0:k0 + nk, kv], v[k0:k0 + nk, kv], seen, dtype)
        q0, k0 = q0 + nq, k0 + nk
    return out, bound


def prefix_reference(q, pool, table, masks, counts, first=0):
    """(out, bound, alpha [B, Hkv, max_pages * 16] of pages >= first, its bound)."""
    dtype = q.dtype
    q, pool = f64(q), f64(pool)
    table, masks = np.asarray(table), np.asarray(masks)
    B, hq, d = q.shape
    hkv = pool.shape[1]
    g = hq // hkv
    width = table.shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    alpha, ab = np.zeros((B, hkv, width * 16)), np.zeros((B, hkv, width * 16))
    for b in range(B):
        n = counts[b]
        ids = table[b, :n]
        live = ((masks[ids][:, None] >> np.arange(16)) & 1).astype(bool).reshape(-1)
        for h in range(hkv):
            k = pool[ids, h, 0].reshape(-1, d)
            v = pool[ids, h, 1].reshape(-1, d)
            seen = np.broadcast_to(live, (g, live.size))
            rows = q[b, h * g:(h + 1) * g]
            o, bd, p = attend(rows, k, v, seen, dtype)
            out[b, h * g:(h + 1) * g], bound[b, h * g:(h + 1) * g] = o, bd
            if n:
                alpha[b, h, :n * 16] = p.sum(0)
                ab[b, h, :n * 16] = alpha_bound(p, rows, k, seen, d)
        alpha[b, :, :first * 16] = 0
    return out, bound, alpha, ab


def assert_within(got, want, bound, what=""):
    got = f64(got)
    bad = ~(np.abs(got - want) <= bound)
    if bad.any():
        i = tuple(int(x[0]) for x in np.nonzero(bad))
        ratio = np.nanmax(np.where(bad, np.abs(got - want) / bound, 0))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: {got[i]} vs {want[i]} "
                             f"(bound {bound[i]}); worst {ratio:.3g} times the bound")
