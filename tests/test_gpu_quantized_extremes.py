"""The 8-bit operators where logits, scales and queries are far from one, with
bounds that a wrong weight cannot hide in."""
import math

import numpy as np
import pytest
import torch

import tiered_kv_cache_split_gb300 as t
from operator_helpers import HALF, assert_within
from quantized_helpers import PAGE, Cache, attend_reference

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WEIGHT = {"f32": 2.0 ** -21, "bf16": 2.0 ** -11}     # a weight in two fp16 parts, and in one


class Rows:
    """Sequences of pages of one pool, all in NumPy: codes, scales, masks (10 % of the slots empty, slot 0 never)."""

    def __init__(self, lens, hkv, d, seed):
        rng = np.random.default_rng(seed)
        self.counts = [-(-n // PAGE) for n in lens]
        self.pages = sum(self.counts) + 2
        ids, at = rng.permutation(self.pages), 0
        self.table = np.full((len(lens), max(self.counts)), -1, np.int32)
        self.live = np.zeros((len(lens), self.table.shape[1] * PAGE), bool)
        self.masks = np.zeros(self.pages, np.int32)
        for b, n in enumerate(self.counts):
            self.table[b, :n] = ids[at:at + n]
            at += n
            self.live[b, :lens[b]] = rng.random(lens[b]) >= 0.1
            self.live[b, 0] = lens[b] > 0
            self.masks[self.table[b, :n]] = (self.live[b, :n * PAGE].reshape(n, PAGE) << np.arange(PAGE)).sum(1)
        self.codes = rng.integers(-127, 128, (self.pages, hkv, 2, PAGE, d)).astype(np.int8)
        self.scales = np.ones((self.pages, hkv, 2), np.float32)
        self.rng = rng

    def attend(self, q, alpha=True):
        a = torch.zeros(len(self.counts), self.codes.shape[1], self.table.shape[1] * PAGE).cuda() if alpha else None
        out = t.quantized_attention(q, torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda(),
                                    torch.from_numpy(self.table).cuda(), torch.from_numpy(self.masks).cuda(), self.counts, alpha_sum=a)
        return out, a


SHAPES = [([1], 1, 64), ([40, 7], 2, 128), ([700, 1, 2600], 4, 64), ([1500, 641, 20, 900], 9, 128), ([9000, 33, 4100], 3, 64),
          ([9000, 33, 4100], 9, 128), ([333, 40], 17, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("lens,g,d", SHAPES)
def test_one_key_above_all_at_large_logits(dtype, sign, lens, g, d):
    """Logits of 2^20 to 2^30 of either sign, one key far above the rest: its V is the
    output and its weight one, however coarse the logits are. In clusters, on the line and
    joined by the second launch.

    The gap between the largest logit and the next is a quarter of it, far above its error of some
    2^-20, so the weights are one and zero. The bound: the output's rounding, the
    weight's, and 2^-20 for the exponential, the sum of one and the powers of two."""
    hkv, hq = 2, 2 * g
    c = Rows(lens, hkv, d, seed=g + d)
    c.codes[:, :, 0] = 0
    top = 127 if sign > 0 else -40
    c.codes[:, :, 0, :, 0] = c.rng.integers(-127, -79, c.codes[:, :, 0, :, 0].shape) if sign < 0 else c.rng.integers(-127, 80, c.codes[:, :, 0, :, 0].shape)
    c.scales[:, :, 1] = np.exp2(c.rng.uniform(-9, 9, c.scales[:, :, 1].shape))
    want, wa = np.zeros((len(lens), hq, d)), np.zeros((len(lens), hkv, c.table.shape[1] * PAGE))
    for b in range(len(lens)):
        at = c.rng.choice(np.flatnonzero(c.live[b]))
        page, slot = c.table[b, at // PAGE], at % PAGE
        c.codes[page, :, 0, slot, 0] = top
        v = c.codes[page, :, 1, slot].astype(np.float64) * c.scales[page, :, 1, None]
        want[b], wa[b, :, at] = np.repeat(v, g, 0), g
    size = np.exp2(c.rng.uniform(20, 30, (len(lens), hq))) * math.sqrt(d) / abs(top)
    q = np.zeros((len(lens), hq, d), np.float32)
    q[..., 0] = size
    q = torch.from_numpy(q).to(DT[dtype]).cuda()
    bound = (HALF[DT[dtype]] + WEIGHT[dtype] + 2.0 ** -20) * np.abs(want)
    out, a = c.attend(q)
    assert_within(out, want, bound)
    assert_within(a, wa, wa * 2.0 ** -20, "alpha")
    assert torch.equal(c.attend(q, alpha=False)[0], out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["both", "negative", "apart"])
@pytest.mark.parametrize("lens,g,d", SHAPES)
def test_scales_of_either_sign(dtype, kind, lens, g, d):
    """A row's value is code * scale, whatever the scale's sign, and as read_quantized has it. The reference gets
    the same values from scales above 0 and codes of the other sign."""
    c = Rows(lens, 2, d, seed=7 + g + d)
    size = np.exp(0.5 * c.rng.standard_normal(c.scales.shape)) / 64
    if kind == "apart":                              # V's blocks up to 2^30 from each other
        size[..., 1] = np.exp2(c.rng.uniform(-15, 15, size[..., 1].shape))
    sign = c.rng.choice([-1, 1], c.scales.shape) if kind != "negative" else np.full(c.scales.shape, -1)
    c.scales = (size * sign).astype(np.float32)
    q = torch.from_numpy(c.rng.standard_normal((len(lens), 2 * g, d)).astype(np.float32)).to(DT[dtype]).cuda()
    want, bound, wa, ab = attend_reference(q, c.codes * sign[..., None, None].astype(np.int8), np.abs(c.scales), c.table, c.masks, c.counts)
    out, a = c.attend(q)
    assert_within(out, want, bound)
    assert_within(a, wa, ab, "alpha")
    for b, n in enumerate(lens):
        k, v = t.read_quantized(torch.from_numpy(c.codes).cuda(), torch.from_numpy(c.scales).cuda(), torch.from_numpy(c.table[b:b + 1]).cuda(), None, [n],
                                dtype=torch.float32)
        rows = c.codes[c.table[b, :c.counts[b]]].astype(np.float32) * c.scales[c.table[b, :c.counts[b]], :, :, None, None]
        for x, j in ((k, 0), (v, 1)):
            assert np.array_equal(x.cpu().numpy(), rows[:, :, j].transpose(0, 2, 1, 3).reshape(-1, 2, d)[:n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -70])
def test_append_behind_scales_below_zero(dtype, d, size):
    """A block whose scale a caller made negative keeps its earlier tokens, whether the scale grows or not. The
    twin holds the same values with scales above 0; rounding to even is the same on both sides of 0."""
    hkv, pages, rng = 2, 24, np.random.default_rng(d)
    codes = rng.integers(-127, 128, (pages, hkv, 2, PAGE, d)).astype(np.int8)
    scales = (np.exp(rng.uniform(-3, 3, (pages, hkv, 2))) * size / 64).astype(np.float32)
    sign = rng.choice([-1, 1], scales.shape)
    twin = Cache(pages, hkv, d, codes * sign[..., None, None].astype(np.int8), scales, np.zeros(pages))
    pool, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales * sign.astype(np.float32)).cuda()
    mask, table = torch.zeros(pages, dtype=torch.int32).cuda(), torch.from_numpy(rng.permutation(pages).reshape(12, 2).astype(np.int32)).cuda()
    lens, new = list(range(1, 13)), [1, 20, 3, 5, 1, 12, 9, 1, 2, 21, 1, 4]
    k, v = (torch.from_numpy((rng.standard_normal((sum(new), hkv, d)) * size / 2).astype(np.float32)).to(DT[dtype]).cuda() for _ in range(2))
    t.append_quantized(k, v, pool, s, table, mask, lens, new)
    twin.append(k.float().cpu().numpy(), v.float().cpu().numpy(), table.tolist(), lens, new)
    s = s.cpu().numpy()
    assert np.array_equal(np.abs(s), twin.scales) and (s < 0).any() and (np.abs(s) > scales).any()
    held = np.zeros((pages, PAGE), bool)              # the bytes of other slots stay, whatever becomes of their block's scale
    for b in range(12):
        held[table[b].cpu().numpy()] = (np.arange(2 * PAGE) < lens[b] + new[b]).reshape(2, PAGE)
    got = pool.cpu().numpy() * np.sign(s)[..., None, None].astype(np.int8)
    assert np.array_equal(got.transpose(0, 3, 1, 2, 4)[held], twin.codes.transpose(0, 3, 1, 2, 4)[held])
    assert np.array_equal(mask.cpu().numpy(), twin.mask)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-125, -123, -64, 64, 118, 126])
@pytest.mark.parametrize("lens,g,d", SHAPES[1:4])
def test_queries_and_scales_of_opposite_size(dtype, power, lens, g, d):
    """Queries of 2^power and scales of 2^-power: the logits are ordinary ones."""
    c = Rows(lens, 2, d, seed=11 + g + d)
    c.scales[..., 0] = c.rng.integers(4, 8, c.scales[..., 0].shape) * np.exp2(-8.0 - power)
    c.scales[..., 1] = np.exp(0.5 * c.rng.standard_normal(c.scales[..., 1].shape)) / 64
    q = np.clip(c.rng.standard_normal((len(lens), 2 * g, d)), -1.9, 1.9) * 2.0 ** power
    check(c, torch.from_numpy(q.astype(np.float32)).to(DT[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,g,d", SHAPES[1:4])
def test_the_largest_queries_and_subnormal_scales(dtype, lens, g, d):
    """Scales of 3 to 7 times 2^-137, queries of up to 2^128: logits of up to some 12, all of whose products have one sign."""
    c = Rows(lens, 2, d, seed=13 + g + d)
    c.scales[..., 0] = c.rng.integers(3, 8, c.scales[..., 0].shape) * 2.0 ** -137
    c.scales[..., 1] = 1 / 64
    sign = c.rng.choice([-1, 1], d)
    c.codes[:, :, 0] = c.rng.integers(40, 128, c.codes[:, :, 0].shape) * sign
    q = c.rng.uniform(1.5, 1.99, (len(lens), 2 * g, d)) * 2.0 ** 127 * sign
    check(c, torch.from_numpy(q.astype(np.float32)).to(DT[dtype]).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens,g,d", SHAPES[1:4])
def test_an_infinite_query_element(dtype, lens, g, d):
    """Logits that are all -inf give 0, one of +inf or of inf * 0 gives NaN; other heads get what
    is theirs (not bit for bit what they were: the references of a page's heads are moved together, when one of them
    passes its own, and their powers of two need not be whole)."""
    c = Rows(lens, 2, d, seed=17 + g + d)
    c.scales = (np.exp(0.5 * c.rng.standard_normal(c.scales.shape)) / 64).astype(np.float32)
    c.codes[..., 0] = -np.abs(c.codes[..., 0]) - (c.codes[..., 0] == 0)     # element 0: codes below 0
    c.codes[..., 1] = 0
    q = torch.from_numpy(c.rng.standard_normal((len(lens), 2 * g, d)).astype(np.float32)).to(DT[dtype]).cuda()
    exact, bound, _, _ = attend_reference(q, c.codes, c.scales, c.table, c.masks, c.counts)
    keep = [h for h in range(2 * g) if h != 1]
    for element, value, want in ((0, math.inf, 0.0), (0, -math.inf, math.nan), (1, math.inf, math.nan)):
        p = q.clone()
        p[:, 1, element] = value
        out, a = c.attend(p)
        assert torch.equal(out[:, 1], torch.full_like(out[:, 1], want)) if want == want else torch.isnan(out[:, 1]).all()
        assert_within(out[:, keep], exact[:, keep], bound[:, keep])
        if want == want:
            assert (a[:, 0][torch.from_numpy(c.live).cuda()] >= 0).all() and torch.isfinite(a).all()


def check(c, q):
    want, bound, wa, ab = attend_reference(q, c.codes, c.scales, c.table, c.masks, c.counts)
    out, a = c.attend(q)
    assert_within(out, want, bound)
    assert_within(a, wa, ab, "alpha")
