"""append_quantized and read_quantized against the definition in NumPy fp32:
codes, scales, masks and values bit for bit."""
import math

import numpy as np
import pytest
import torch

import tiered_kv_cache_split_gb300 as t
from quantized_helpers import PAGE, Cache

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


class Pool:
    """A pool of garbage on the device and the same in NumPy."""

    def __init__(self, pages, hkv, d, seed=0):
        rng = np.random.default_rng(seed)
        codes = rng.integers(-127, 128, (pages, hkv, 2, PAGE, d)).astype(np.int8)
        scales = rng.uniform(0.001, 0.02, (pages, hkv, 2)).astype(np.float32)
        self.want = Cache(pages, hkv, d, codes, scales, np.zeros(pages))
        self.pool, self.scales = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
        self.mask = torch.zeros(pages, dtype=torch.int32).cuda()

    def append(self, k, v, table, lens, new, **kw):
        t.append_quantized(k, v, self.pool, self.scales, table, self.mask, lens, new, **kw)
        self.want.append(k.float().cpu().numpy(), v.float().cpu().numpy(), table.tolist(), lens, new)

    def check(self):
        assert np.array_equal(self.scales.cpu().numpy(), self.want.scales, equal_nan=True)
        assert np.array_equal(self.pool.cpu().numpy(), self.want.codes)
        assert np.array_equal(self.mask.cpu().numpy(), self.want.mask)


def rows(pages, n_pages, seed=1):
    """A table of rows that list n_pages[b] pages each, no page twice."""
    ids = np.random.default_rng(seed).permutation(pages)
    table, at = np.full((len(n_pages), max(max(n_pages), 1)), -1, np.int32), 0
    for b, n in enumerate(n_pages):
        table[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(table).cuda()


def data(seed, n, hkv, d, dtype):
    size = torch.exp(rand(seed + 100, n, hkv, 1))
    return (rand(seed, n, hkv, d) * size).to(DT[dtype]).cuda(), (rand(seed + 1, n, hkv, d) * size.flip(0)).to(DT[dtype]).cuda()


LENS = [([0], [1]), ([0], [16]), ([0], [17]), ([15], [1]), ([16], [1]), ([7], [3]), ([5], [40]), ([0, 3, 16, 31, 0, 100], [5, 1, 0, 2, 33, 16]),
        ([0, 0], [0, 1]), ([250] * 3, [1, 1, 1]), ([0], [300])]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hkv,d", [(2, 64), (4, 128), (1, 128), (5, 64)])
@pytest.mark.parametrize("lens,new", LENS)
def test_append_and_read(dtype, hkv, d, lens, new):
    n_pages = [-(-(a + b) // PAGE) for a, b in zip(lens, new)]
    p = Pool(sum(n_pages) + 4, hkv, d)
    table = rows(sum(n_pages) + 4, n_pages)
    k0, v0 = data(2, sum(lens), hkv, d, dtype)
    p.append(k0, v0, table, [0] * len(lens), lens)
    p.check()
    k, v = data(5, sum(new), hkv, d, dtype)
    p.append(k, v, table, lens, new)
    p.check()
    ends = [a + b for a, b in zip(lens, new)]
    for first in ([0] * len(ends), lens, [max(0, n - 1) for n in ends]):
        want = p.want.read(table.tolist(), first, ends)
        for out in (torch.float32, torch.bfloat16):
            gk, gv = t.read_quantized(p.pool, p.scales, table, p.mask, ends, first=first, dtype=out)
            assert torch.equal(gk.cpu(), torch.from_numpy(want[0]).to(out)) and torch.equal(gv.cpu(), torch.from_numpy(want[1]).to(out))
    # a value is off by at most half a step of its block's scale
    gk, _ = t.read_quantized(p.pool, p.scales, table, p.mask, [n if m else 0 for n, m in zip(ends, new)], dtype=torch.float32,
                             first=[min(a, b) if m else 0 for a, b, m in zip(lens, ends, new)])
    err = (gk - k.float()).abs()
    assert (err <= p.scales.max() * (0.5 + 2.0 ** -14)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_token_by_token(dtype, d):
    """Blocks fill a token at a time; scales grow and earlier codes follow."""
    p = Pool(12, 3, d)
    table = rows(12, [4, 4])
    for i in range(50):
        k, v = data(10 + 2 * i, 2, 3, d, dtype)
        grow = 1.15 ** i
        p.append((k * grow).to(k.dtype), v, table, [i, i + 7], [1, 1])
        if i % 7 == 0 or i > 46:
            p.check()
    p.check()


def test_scale_edges():
    """Zeros, the smallest and largest values, ties, and the values next to them."""
    hkv, d = 1, 64
    p = Pool(8, hkv, d)
    table = rows(8, [8])
    k, v = rand(3, 128, hkv, d).cuda(), rand(4, 128, hkv, d).cuda()
    k[:16] = 0.0
    k[16:32] = k[16:32] * 1e-41                       # subnormal values and scales
    k[32:48] = k[32:48].clamp(-1, 1) * 3.4e38
    k[48:64] = 127.0
    k[48:64, 0, :40] = torch.arange(40).cuda() + 0.5  # ties go to the even code
    k[64:80] = 1.4e-45
    v[:16, 0, 1:] = -0.0
    v[16:32] = 1e-38 * v[16:32]
    p.append(k, v, table, [0], [128])
    p.check()
    got, _ = t.read_quantized(p.pool, p.scales, table, p.mask, [128], dtype=torch.float32)
    assert torch.equal(got[:16], torch.zeros_like(got[:16])) and torch.isfinite(got).all()


def test_quotients_next_to_borders():
    """Values a few steps from the middle of two codes, over scales of every size:
    the code is that of the rounded quotient."""
    rng = np.random.default_rng(5)
    pages, hkv, d = 64, 4, 128
    p = Pool(pages, hkv, d)
    table = rows(pages, [pages])
    x = np.empty((2, pages, hkv, PAGE * d), np.float32)
    for block in np.ndindex(x.shape[:3]):
        top = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-70, 100))
        scale = np.float32(top / np.float32(127))
        mid = ((rng.integers(0, 127, PAGE * d) + 0.5) * np.float64(scale)).astype(np.float32)
        near = (mid.view(np.int32) + rng.integers(-3, 4, PAGE * d)).astype(np.int32).view(np.float32)
        x[block] = np.minimum(near, top) * rng.choice([-1, 1], PAGE * d)
        x[block][rng.integers(PAGE * d)] = top
    k, v = (torch.from_numpy(a.reshape(pages, hkv, PAGE, d).transpose(0, 2, 1, 3).reshape(pages * PAGE, hkv, d).copy()).cuda() for a in x)
    p.append(k, v, table, [0], [pages * PAGE])
    p.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_infinity(dtype):
    """They make their block, and no other, read as NaN until it starts anew."""
    hkv, d = 2, 64
    p = Pool(6, hkv, d)
    table = rows(6, [3, 2])
    k, v = data(7, 60, hkv, d, dtype)
    k[3, 1, 5], v[20, 0, 63], k[50, 0, 0] = math.nan, -math.inf, math.inf
    p.append(k, v, table, [0, 0], [35, 25])
    p.check()
    k2, v2 = data(9, 5, hkv, d, dtype)
    p.append(k2, v2, table, [35, 25], [3, 2])
    p.check()
    gk, gv = t.read_quantized(p.pool, p.scales, table, p.mask, [38, 27], dtype=torch.float32)
    bk, bv = torch.isnan(gk).flatten(2).all(2), torch.isnan(gv).all(2)
    want_k, want_v = torch.zeros_like(bk), torch.zeros_like(bv)
    want_k[:16, 1] = True
    want_k[38:54, 0] = True
    want_v[16:32, 0] = True
    assert torch.equal(bk, want_k) and torch.equal(bv, want_v) and torch.equal(torch.isnan(gk).any(2), want_k)
    k3, v3 = data(11, 16, hkv, d, dtype)
    p.append(k3, v3, table, [0, 27], [16, 0])          # the first page starts anew
    p.check()
    assert torch.isfinite(t.read_quantized(p.pool, p.scales, table, p.mask, [16, 0])[0]).all()


def test_strides_streams_and_graphs():
    hkv, d, n = 2, 128, 37
    qkv = rand(5, n, 8 + 2 * hkv, d, dtype=torch.bfloat16).cuda()
    k, v = qkv[:, 8:8 + hkv], qkv[:, 8 + hkv:]
    p, q = Pool(5, hkv, d), Pool(5, hkv, d)
    table = rows(5, [4])
    p.append(k, v, table, [3], [n])
    p.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q.append(k.contiguous(), v.contiguous(), table, [3], [n], stream=side)
    a = t.read_quantized(q.pool, q.scales, table, q.mask, [3 + n], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    q.check()
    b = t.read_quantized(p.pool, p.scales, table, p.mask, [3 + n])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    both = torch.full((3 + n, 2 * hkv + 1, d), 7.0, dtype=torch.bfloat16).cuda()   # strided outputs
    t.read_quantized(p.pool, p.scales, table, p.mask, [3 + n], out=(both[:, :hkv], both[:, hkv:2 * hkv]))
    assert torch.equal(both[:, :hkv], b[0]) and torch.equal(both[:, hkv:2 * hkv], b[1]) and (both[:, -1] == 7).all()
    r = Pool(5, hkv, d)
    out = torch.empty_like(b[0]), torch.empty_like(b[1])
    kc, vc = k.clone(), v.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.append_quantized(kc, vc, r.pool, r.scales, table, r.mask, [3], [n])
        t.read_quantized(r.pool, r.scales, table, r.mask, [3 + n], out=out)
    kc.mul_(0.5)
    graph.replay()
    r.want.append(kc.float().cpu().numpy(), vc.float().cpu().numpy(), table.tolist(), [3], [n])
    r.check()
    want = r.want.read(table.tolist(), [0], [3 + n])
    assert torch.equal(out[0].cpu(), torch.from_numpy(want[0]).bfloat16())


def test_bad_and_shared_pages_are_not_written():
    hkv, d = 2, 64
    p = Pool(6, hkv, d)
    table = torch.tensor([[0, 6, 2], [3, -1, 4]], dtype=torch.int32).cuda()
    k, v = data(3, 80, hkv, d, "f32")
    status = torch.zeros(1, dtype=torch.int32).cuda()
    p.append(k, v, table, [0, 0], [40, 40], status=status)
    p.check()
    assert status.item() == -1
    got, _ = t.read_quantized(p.pool, p.scales, table, p.mask, [40, 40], dtype=torch.float32)
    want = p.want.read(table.tolist(), [0, 0], [40, 40])[0]
    assert torch.equal(got.cpu(), torch.from_numpy(want)) and (got[16:32] == 0).all() and (got[56:72] == 0).all()
    refs = torch.tensor([1, 0, 1, 2, 1, 0], dtype=torch.int32).cuda()
    status.zero_()
    before = p.pool.clone(), p.scales.clone(), p.mask.clone()
    table = torch.tensor([[3, 2], [1, 5]], dtype=torch.int32).cuda()
    t.append_quantized(k[:20], v[:20], p.pool, p.scales, table, p.mask, [5, 0], [15, 5], page_refs=refs, status=status)
    assert status.item() == -1
    same = [0, 1, 3, 4, 5]                            # page 2 alone is a row's own
    for x, y in zip((p.pool, p.scales, p.mask), before):
        assert torch.equal(x[same], y[same])
    assert p.mask[2].item() == (1 << 4) - 1
    status.zero_()
    t.append_quantized(k[:4], v[:4], p.pool, p.scales, table, p.mask, [16, 0], [4, 0], page_refs=refs, status=status)
    assert status.item() == 0


def test_empty_slots_read_as_zeros():
    p = Pool(4, 2, 64)
    table = rows(4, [3])
    k, v = data(3, 48, 2, 64, "bf16")
    p.append(k, v, table, [0], [48])
    p.mask[table[0, 1]] = 0x8001
    p.want.mask[table[0, 1].item()] = 0x8001
    got = t.read_quantized(p.pool, p.scales, table, p.mask, [48], first=[2], dtype=torch.float32)
    want = p.want.read(table.tolist(), [2], [48])
    assert torch.equal(got[0].cpu(), torch.from_numpy(want[0])) and torch.equal(got[1].cpu(), torch.from_numpy(want[1]))
    every = t.read_quantized(p.pool, p.scales, table, None, [48], first=[2], dtype=torch.float32)
    want = p.want.read(table.tolist(), [2], [48], mask=False)
    assert torch.equal(every[0].cpu(), torch.from_numpy(want[0]))
    p.scales[table[0, 1]] = math.nan                  # an empty slot of a bad block is still a zero
    got, _ = t.read_quantized(p.pool, p.scales, table, p.mask, [48], dtype=torch.float32)
    assert torch.isnan(got[16]).all() and (got[17:31] == 0).all() and torch.isnan(got[31]).all()


def test_offsets_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the pool, and packed tokens more than 2^31 bytes apart."""
    hkv, d, pages = 16, 128, 70000                    # 4.6 GB of codes
    pool = torch.zeros((pages, hkv, 2, PAGE, d), dtype=torch.int8, device="cuda")
    scales, mask = torch.zeros((pages, hkv, 2), device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, 40000, 1]], dtype=torch.int32, device="cuda")
    k, v = data(3, 40, hkv, d, "bf16")
    t.append_quantized(k, v, pool, scales, table, mask, [0], [40])
    small = Pool(3, hkv, d)
    near = torch.tensor([[2, 1, 0]], dtype=torch.int32, device="cuda")
    small.append(k, v, near, [0], [40])
    assert torch.equal(pool[[pages - 1, 40000]], small.pool[[2, 1]]) and torch.equal(scales[[pages - 1, 40000]], small.scales[[2, 1]])
    a, b = t.read_quantized(pool, scales, table, mask, [40]), t.read_quantized(small.pool, small.scales, near, small.mask, [40])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    wide = torch.zeros((3, 1 << 29), dtype=torch.bfloat16, device="cuda")[:, :hkv * d].unflatten(1, (hkv, d))
    wide.copy_(k[:3])
    t.append_quantized(wide, v[:3], pool, scales, table, mask, [40], [3])
    small.append(k[:3], v[:3], near, [40], [3])
    assert torch.equal(pool[1][:, :, :11], small.pool[0][:, :, :11]) and (pool[1][:, :, 11:] == 0).all()
