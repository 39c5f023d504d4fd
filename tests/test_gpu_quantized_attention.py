"""quantized_attention against softmax attention in 64 bits over the values the
codes stand for, and the 8-bit operators together."""
import math

import numpy as np
import pytest
import torch

import tiered_kv_cache_split_gb300 as t
from operator_helpers import assert_within, prompt_reference
from quantized_helpers import PAGE, Cache, attend_reference

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


class Case:
    def __init__(self, lens, hq, hkv, d, dtype="bf16", holes=0.1, seed=0, spread=0.5, width=None):
        rng = np.random.default_rng(seed)
        n_pages = [-(-n // PAGE) for n in lens]
        self.pages, self.counts = sum(n_pages) + 3, n_pages
        ids, at = rng.permutation(self.pages), 0
        self.table = np.full((len(lens), width or max(max(n_pages), 1)), -1, np.int32)
        self.masks = rng.integers(0, 1 << 16, self.pages)
        for b, n in enumerate(n_pages):
            self.table[b, :n] = ids[at:at + n]
            at += n
            live = (np.arange(n * PAGE) < lens[b]) & (rng.random(n * PAGE) >= holes)
            self.masks[self.table[b, :n]] = (live.reshape(n, PAGE) << np.arange(PAGE)).sum(1)
        self.codes = rng.integers(-127, 128, (self.pages, hkv, 2, PAGE, d)).astype(np.int8)
        self.scales = (np.exp(spread * rng.standard_normal((self.pages, hkv, 2))) / 64).astype(np.float32)
        self.q = torch.from_numpy(rng.standard_normal((len(lens), hq, d)).astype(np.float32)).to(DT[dtype]).cuda()
        self.d, self.hkv = d, hkv

    def device(self):
        return (torch.from_numpy(self.codes).cuda(), torch.from_numpy(self.scales).cuda(), torch.from_numpy(self.table).cuda(),
                torch.from_numpy(self.masks.astype(np.int32)).cuda(), self.counts)

    def check(self, alpha=True, what="", **kw):
        want, bound, wa, ab = attend_reference(self.q, self.codes, self.scales, self.table, self.masks, self.counts)
        a = torch.full((len(self.counts), self.hkv, self.table.shape[1] * PAGE), 0.25).cuda() if alpha else None
        out = t.quantized_attention(self.q, *self.device(), alpha_sum=a, **kw)
        assert_within(out, want, bound, what)
        if alpha:   # added to what was there: one more rounding of a sum of up to 64.25
            assert_within(a, wa + 0.25, ab + 2.0 ** -24 * (np.abs(wa) + 0.25), what + " alpha")
        return out, a


LENS = [[1], [16], [17], [100], [0, 5], [1, 2, 33, 64, 65, 127, 128, 129, 300], [1000, 3], [5000], [700] * 5]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 64), (28, 4, 128), (4, 4, 128), (3, 1, 64)])
@pytest.mark.parametrize("lens", LENS)
def test_lengths(dtype, hq, hkv, d, lens):
    c = Case(lens, hq, hkv, d, dtype)
    out, _ = c.check()
    assert torch.equal(out, c.check(alpha=False)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 5, 7, 8, 9, 12, 16, 17, 24, 33, 64])
def test_heads_per_kv_head(dtype, d, g):
    Case([333, 40], 2 * g, 2, d, dtype, seed=g).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,g", [(64, 1), (128, 3), (64, 4), (128, 5), (128, 7), (64, 9), (128, 16), (128, 17), (64, 33), (128, 64)])
@pytest.mark.parametrize("lens", [[1500, 641, 20, 900], [9000, 33, 0, 4100]])
def test_heads_of_sequences_that_are_cut(dtype, d, g, lens):
    """In clusters (up to 16 heads), and on the line."""
    Case(lens, 2 * g, 2, d, dtype, seed=100 + g).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,longest", [(1, 200), (1, 1700), (40, 310), (60, 250), (64, 70), (3, 127), (3, 129), (9, 1025)])
def test_clusters_of_every_size(dtype, batch, longest):
    """1 to 8 CTAs a sequence and KV head, some of them without a page."""
    Case([longest * (i + 1) // batch for i in range(batch)], 12, 4, 64, dtype, seed=batch).check()


@pytest.mark.parametrize("dtype,hkv,g,d,batch,n", [("bf16", 32, 1, 128, 2, 16384), ("f32", 32, 2, 64, 2, 16384), ("bf16", 32, 9, 64, 2, 16384),
                                                   ("bf16", 32, 4, 64, 19, 450), ("f32", 4, 7, 128, 19, 4000)])
def test_pieces_longer_than_a_window(dtype, hkv, g, d, batch, n):
    """A CTA's pages come in windows of 384: many pages (listed again and again) of many
    heads give each more than that, on the line and in clusters of 1 and 8. Against the values in
    64 bits, on some of the heads."""
    gen = torch.Generator().manual_seed(1)
    pages, hq = 300, hkv * g
    pool = torch.randint(-127, 128, (pages, hkv, 2, PAGE, d), generator=gen, dtype=torch.int8).cuda()
    scales = (torch.rand(pages, hkv, 2, generator=gen) / 32).cuda()
    mask = torch.randint(0, 1 << 16, (pages,), generator=gen, dtype=torch.int32).cuda()
    table = torch.randint(0, pages, (batch, n), generator=gen, dtype=torch.int32).cuda()
    counts = [n - b * (n // 16 if batch == 2 else 1) for b in range(batch)]
    q = torch.randn(batch, hq, d, generator=gen).to(DT[dtype]).cuda()
    alpha = torch.zeros(batch, hkv, n * PAGE, device="cuda")
    out = t.quantized_attention(q, pool, scales, table, mask, counts, alpha_sum=alpha)
    slots = torch.arange(PAGE, device="cuda")
    for b, c in list(enumerate(counts))[::max(1, batch - 1)]:
        ids = table[b, :c].long()
        live = ((mask[ids][:, None] >> slots) & 1).flatten() != 0
        for h in (0, hkv // 2, hkv - 1):
            kv = pool[ids, h].double() * scales[ids, h].double()[..., None, None]
            k, v = kv[:, 0].reshape(-1, d)[live], kv[:, 1].reshape(-1, d)[live]
            rows = q[b, h * g:(h + 1) * g].double()
            p = torch.softmax(rows @ k.T / math.sqrt(d), 1)
            o, a = p @ v, p @ v.abs()
            m, e = k.shape[0], 2.0 ** -23
            # the bound of attend_reference; scales are below 2^-5 and above 2^-40, logits below 60
            mag = (rows.abs() @ k.abs().T).amax(1, keepdim=True) / math.sqrt(d)
            dq = 2.0 ** -24 if dtype == "bf16" else 2.0 ** -22
            qerr = dq * rows.abs().amax(1, keepdim=True) * k.abs().sum(1).max() / math.sqrt(d)
            delta = (d + 4) * e * mag + qerr + e * (1.45 * mag + 40 + 32)
            u, w = (2.0 ** -8, 2.0 ** -11) if dtype == "bf16" else (2.0 ** -24, 2.0 ** -21)
            bound = (u * o.abs() + (w + 2 * delta + 2 * m * e) * a + m * 2.0 ** -36 * v.abs().max()) * 1.02
            assert ((out[b, h * g:(h + 1) * g].double() - o).abs() <= bound).all()
            got = alpha[b, h, :c * PAGE].double()
            assert ((got[live] - p.sum(0)).abs() <= (p * (2 * delta + (m + 16) * e)).sum(0) + 1e-30).all()
            assert (got[~live] == 0).all() and (alpha[b, h, c * PAGE:] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_that_keep_nothing(dtype):
    """No page, no valid slot, pages outside the pool: output 0, alpha untouched; other rows as they were."""
    c = Case([100, 50, 0, 64, 40], 8, 2, 64, dtype)
    c.masks[c.table[1, :4]] = 0
    c.table[3, :4] = [-5, c.pages, 2 ** 31 - 1, -2 ** 31]
    out, a = c.check()
    assert (out[1:4] == 0).all() and (a[1:4] == 0.25).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pages_outside_the_pool_read_as_empty(dtype):
    c = Case([300, 300], 8, 2, 128, dtype)
    c.table[0, 3], c.table[1, 0], c.table[1, 18] = -1, c.pages, c.pages + 7
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1)])
def test_nan_blocks_reach_the_rows_that_see_them(dtype, hq, hkv):
    c = Case([200, 200, 200, 200], hq, hkv, 64, dtype, holes=0)
    clean, ca = c.check()
    c.scales[c.table[0, 5], 0, 1] = np.nan          # V of head 0
    c.scales[c.table[1, 5], 0, 0] = np.nan          # K of head 0
    c.scales[c.table[2, 2]] = np.nan                # an emptied page
    c.masks[c.table[2, 2]] = 0
    c.scales[c.table[3, 12], :, :] = np.inf         # the last page, 8 of its slots empty
    a = torch.zeros_like(ca)
    out = t.quantized_attention(c.q, *c.device(), alpha_sum=a)
    g = hq // hkv
    assert torch.isnan(out[0, :g]).all() and torch.isnan(out[1, :g]).all()
    assert torch.equal(out[:2, g:], clean[:2, g:])
    assert torch.isfinite(out[2]).all() and torch.isfinite(a[2]).all() and (a[2, :, 32:48] == 0).all()
    assert torch.isnan(out[3]).all() and (a[3, :, 200:] == 0).all()
    assert torch.isfinite(a[0]).all() and torch.isnan(a[1, 0, :200]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_queries_that_are_not_finite_reach_their_row_only(dtype):
    c = Case([150, 90], 14, 2, 64, dtype)
    clean, _ = c.check()
    c.q[0, 3, 7], c.q[1, 0, 0], c.q[1, 13, 5] = math.nan, math.inf, -math.inf
    out = t.quantized_attention(c.q, *c.device())
    bad = torch.zeros(2, 14, dtype=torch.bool)
    bad[0, 3] = bad[1, 0] = bad[1, 13] = True
    assert torch.equal(out.cpu()[~bad], clean.cpu()[~bad])
    assert not torch.isfinite(out.cpu()[0, 3]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["zero_k", "zero_v", "one_hot", "wide_v", "tiny", "huge_v", "tiny_q", "huge_q", "rising"])
def test_scales_far_apart(dtype, kind):
    c = Case([700, 65], 8, 2, 128, dtype, seed=3)
    n = c.counts[0]
    if kind == "zero_k":
        c.scales[:, :, 0] = 0                       # every key counts the same
    elif kind == "zero_v":
        c.scales[::2, :, 1] = 0
    elif kind == "one_hot":
        c.scales[:, :, 0] *= 64                     # logits of hundreds
    elif kind == "wide_v":                          # V's blocks 2^60 apart
        c.scales[c.table[0, :n], :, 1] = np.exp2(np.linspace(-30, 30, n))[:, None]
    elif kind == "tiny":
        c.scales[:] = 1e-40                         # subnormal
    elif kind == "huge_v":
        c.scales[:, :, 1] = 2.0 ** 119
    elif kind == "tiny_q":
        c.q = (c.q.float() * 1e-38).to(c.q.dtype)
    elif kind == "huge_q":
        c.q = (c.q.float() * 2.0 ** 100).to(c.q.dtype)
        c.scales[:, :, 0] *= 2.0 ** -100
    elif kind == "rising":                          # each page's logits above the one before
        c.scales[c.table[0, :n], :, 0] = (np.arange(n) / (16 * n))[:, None]
        c.codes[:, :, 0] = np.abs(c.codes[:, :, 0])
        c.q = c.q.abs()
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_keys_below_one(dtype):
    """One key far above thousands: their sum still counts."""
    c = Case([20000], 4, 1, 64, dtype, holes=0)
    c.codes[:, :, 0] = 0
    c.codes[c.table[0, 600], 0, 0, 3] = 127
    c.scales[:, :, 0] = 0.01
    c.q = torch.ones_like(c.q) * 1.5
    c.codes[:, :, 1] = 100
    c.codes[c.table[0, 600], 0, 1, 3] = -100
    c.check()


def test_the_same_twice_and_scratch_of_anything():
    """Runs repeat bit for bit, whatever the scratch held."""
    for dtype in ("f32", "bf16"):
        c = Case([3000, 1, 777, 0, 4096], 28, 4, 128, dtype)
        first, fa = c.check()
        for fill in (0, 255):
            scratch = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
            out, a = c.check(scratch=scratch)
            assert torch.equal(out, first) and torch.equal(a, fa)


def test_a_row_does_not_depend_on_its_neighbours():
    """A batch gives what its sequences give alone, up to the order of sums."""
    c = Case([2000, 30, 500, 9000], 16, 4, 128, "f32", seed=5)
    want, bound, _, _ = attend_reference(c.q, c.codes, c.scales, c.table, c.masks, c.counts)
    codes, scales, table, masks, counts = c.device()
    for b in range(4):
        alone = t.quantized_attention(c.q[b:b + 1], codes, scales, table[b:b + 1].contiguous(), masks, counts[b:b + 1])
        assert_within(alone, want[b:b + 1], bound[b:b + 1])


def test_streams_graphs_and_outputs():
    c = Case([600, 2000, 31], 28, 4, 128)
    dev = c.device()
    want, wa = c.check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = t.quantized_attention(c.q, *dev, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out, a = torch.empty_like(c.q), torch.zeros_like(wa)
    q = c.q.clone()
    with torch.cuda.graph(graph):
        a.zero_()
        t.quantized_attention(q, *dev, out=out, alpha_sum=a)
    q.copy_(c.q.flip(1))
    graph.replay()
    graph.replay()
    c.q = c.q.flip(1).contiguous()
    want, wa = c.check()
    assert torch.equal(out, want)
    b = torch.zeros_like(a)
    t.quantized_attention(c.q, *dev, alpha_sum=b)
    assert torch.equal(a, b)
    assert torch.equal(t.quantized_attention(c.q, *dev[:3], dev[3].view(torch.uint32), dev[4]), want)


def test_two_calls_at_once():
    c, e = Case([4000, 2500], 32, 8, 128, seed=1), Case([50, 6000], 8, 2, 64, "f32", seed=2)
    cd, ed = c.device(), e.device()
    cw, ew = t.quantized_attention(c.q, *cd), t.quantized_attention(e.q, *ed)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(t.quantized_attention(c.q, *cd, stream=a), t.quantized_attention(e.q, *ed, stream=b)) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, cw) and torch.equal(y, ew) for x, y in outs)


def test_offsets_past_32_bits():
    hkv, d, pages = 16, 128, 70000
    pool = torch.zeros((pages, hkv, 2, PAGE, d), dtype=torch.int8, device="cuda")
    scales, mask = torch.full((pages, hkv, 2), 0.01, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    near = Case([300], 64, hkv, d, seed=4)
    far = torch.from_numpy(pages - 1 - near.table).cuda()
    ids = far[0].long()
    dev = near.device()
    pool[ids], scales[ids], mask[ids] = (x[dev[2][0].long()] for x in (dev[0], dev[1], dev[3]))
    assert torch.equal(t.quantized_attention(near.q, pool, scales, far, mask, near.counts), t.quantized_attention(near.q, *dev))


def test_full_page_table():
    """16384 pages of one sequence, and 64 sequences."""
    c = Case([1 << 18], 8, 1, 64, holes=0.3)
    dev = c.device()
    a = torch.zeros(1, 1, 1 << 18).cuda()
    out = t.quantized_attention(c.q, *dev, alpha_sum=a)
    want, bound, wa, ab = attend_reference(c.q, c.codes, c.scales, c.table, c.masks, c.counts)
    assert_within(out, want, bound)
    assert_within(a, wa, ab)
    Case([(37 * b) % 260 for b in range(64)], 4, 2, 64, width=40).check()


def test_a_prompt_in_two_chunks_then_decoding():
    """The operators together: rotate, append, read the cached part back for the next
    chunk, attend the prompt, then decode token by token over the 8-bit pages."""
    hq, hkv, d, n, half = 8, 2, 64, 150, 70
    gen = torch.Generator().manual_seed(0)
    qkv = torch.randn(2 * n + 12, hq + 2 * hkv, d, generator=gen).bfloat16().cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    tab = t.rotary_table(d, factor=4.0, trained=100)
    lens = [0, 0]
    ends = [n, 61]                                   # two prompts
    pages = 40
    pool, scales = torch.zeros((pages, hkv, 2, PAGE, d), dtype=torch.int8, device="cuda"), torch.zeros((pages, hkv, 2), device="cuda")
    mask = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.randperm(pages, generator=gen)[:32].view(2, 16).to(torch.int32).cuda()
    twin = Cache(pages, hkv, d)
    at = 0
    for new in ([half, 61], [n - half, 0]):
        m = sum(new)
        pos = torch.cat([torch.arange(a, a + b) for a, b in zip(lens, new)]).cuda()
        qr, kr = t.rotate(q[at:at + m], k[at:at + m], pos, tab)
        cached = t.read_quantized(pool, scales, table, mask, lens)
        ck, cv = [], []
        c0 = x0 = 0
        for a, b in zip(lens, new):                  # each row's cached keys ahead of its new ones
            if b:
                ck += [cached[0][c0:c0 + a], kr[x0:x0 + b]]
                cv += [cached[1][c0:c0 + a], v[at:at + m][x0:x0 + b]]
            c0, x0 = c0 + a, x0 + b
        kk, vv = torch.cat(ck), torch.cat(cv)
        ql, kl = zip(*[(b, a + b) for a, b in zip(lens, new) if b])
        o = t.prompt_attention(qr, kk, vv, list(ql), list(kl))
        want, bound = prompt_reference(qr, kk, vv, ql, kl)
        assert_within(o, want, bound)
        t.append_quantized(kr, v[at:at + m], pool, scales, table, mask, lens, new)
        twin.append(kr.float().cpu().numpy(), v[at:at + m].float().cpu().numpy(), table.tolist(), lens, new)
        lens = [a + b for a, b in zip(lens, new)]
        at += m
    assert lens == ends
    alpha = torch.zeros(2, hkv, 16 * PAGE).cuda()
    total = 0.0
    for step in range(20):
        qr, kr = t.rotate(q[at:at + 2], k[at:at + 2], torch.tensor(lens).cuda(), tab)
        t.append_quantized(kr, v[at:at + 2], pool, scales, table, mask, lens, [1, 1])
        twin.append(kr.float().cpu().numpy(), v[at:at + 2].float().cpu().numpy(), table.tolist(), lens, [1, 1])
        lens = [a + 1 for a in lens]
        at += 2
        counts = [-(-a // PAGE) for a in lens]
        o = t.quantized_attention(qr, pool, scales, table, mask, counts, alpha_sum=alpha)
        want, bound, wa, ab = attend_reference(qr, twin.codes, twin.scales, table.tolist(), twin.mask, counts)
        assert_within(o, want, bound)
        total = total + wa
    assert np.array_equal(pool.cpu().numpy(), twin.codes) and np.array_equal(mask.cpu().numpy(), twin.mask)
    # every weight's bound is far below 2^-12 here; 20 sums of up to 20 in fp32
    assert np.abs(alpha.cpu().double().numpy() - total).max() <= 20 * 2.0 ** -12
    # the sums of a row's weights are its heads, every step
    assert np.allclose(alpha.sum((1, 2)).cpu().numpy(), 20 * hq, rtol=1e-5)
