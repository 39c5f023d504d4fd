"""rotate against the rotation in 64 bits with exact angles."""
import math

import numpy as np
import pytest
import torch

import tiered_kv_cache_split_gb300 as t
from operator_helpers import assert_within
from quantized_helpers import rotate_reference

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def check(x, got, pos, table, inverse, what="", steps=None):
    want, bound = rotate_reference(x, pos.tolist(), table.inv_freq, table.scale, table.interleaved, inverse, x.dtype, steps)
    assert_within(got, want, bound, what)
    r = table.rotary_dim
    assert torch.equal(got.cpu()[..., r:], x.cpu()[..., r:])   # what passes, passes unchanged


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,r,interleaved", [(64, 64, False), (64, 64, True), (128, 128, False), (128, 128, True), (128, 64, False),
                                             (128, 32, True), (128, 50, False), (128, 50, True), (64, 2, False), (96, 96, False),
                                             (80, 48, True), (6, 6, False), (33, 10, True), (512, 512, False), (256, 8, True)])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 8, 2), (37, 3, 1), (5, 28, 4)])
def test_layouts(dtype, d, r, interleaved, tokens, hq, hk):
    table = t.rotary_table(r, interleaved=interleaved)
    q, k = rand(1, tokens, hq, d, dtype=DT[dtype]).cuda(), rand(2, tokens, hk, d, dtype=DT[dtype]).cuda()
    pos = torch.randint(0, 5000, (tokens,), generator=torch.Generator().manual_seed(3)).cuda()
    for inverse in (False, True):
        qo, ko = t.rotate(q, k, pos, table, inverse=inverse)
        check(q, qo, pos, table, inverse, "q")
        check(k, ko, pos, table, inverse, "k")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(dtype, interleaved):
    table = t.rotary_table(128, interleaved=interleaved)
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 2 ** 40 + 12345, -2 ** 52 - 7, 2 ** 62 + 3, -2 ** 63, 2 ** 63 - 1])
    q = rand(4, len(pos), 2, 128, dtype=DT[dtype]).cuda()
    qo, none = t.rotate(q, None, pos.cuda(), table)
    assert none is None
    check(q, qo, pos, table, False, steps=table.steps.tolist())   # beyond 2^33 the frequencies' 64 bits count
    check(q[:6], qo[:6], pos[:6], table, False)
    small = pos[:6].to(torch.int32).cuda()
    qs, _ = t.rotate(q[:6], None, small, table)
    assert torch.equal(qs, qo[:6])


@pytest.mark.parametrize("factor,trained,scale", [(4.0, None, 1.0), (32.0, 4096, 0.1 * math.log(32.0) + 1), (0.5, None, -2.0), (8.0, 100, 0.25)])
def test_scaled_for_long_contexts(factor, trained, scale):
    table = t.rotary_table(64, factor=factor, trained=trained, scale=scale)
    f = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    if trained is None:
        want = f / factor
    else:
        g = np.clip((trained * f / (2 * np.pi) - 1) / 31, 0, 1)
        want = g * f + (1 - g) * f / factor
    assert np.allclose(table.inv_freq, want, rtol=1e-14, atol=0)
    q = rand(5, 9, 4, 64).cuda()
    pos = torch.arange(9).cuda() * 20011
    check(q, t.rotate(q, None, pos, table)[0], pos, table, False)


def test_given_frequencies_and_zero():
    table = t.rotary_table(8, inv_freq=[0.0, 1e-30, 3.0e9, -0.25])
    q = rand(6, 7, 2, 8).cuda()
    pos = torch.tensor([0, 5, 2 ** 33, -9, 1, 2, 3]).cuda()
    qo, _ = t.rotate(q, None, pos, table)
    check(q, qo, pos, table, False)
    assert torch.equal(qo[..., [0, 4]], q[..., [0, 4]])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_strides_in_place_and_alignment(dtype, interleaved, shift):
    """Views of a fused projection, in place, and rows off 16-byte boundaries, give what packed rows give."""
    hq, hk, d, n = 6, 2, 64, 11
    flat = rand(7, n * (hq + 2 * hk) * d + 8, dtype=DT[dtype]).cuda()
    qkv = flat[shift:shift + n * (hq + 2 * hk) * d].view(n, hq + 2 * hk, d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    table = t.rotary_table(48, interleaved=interleaved)
    pos = torch.arange(100, 100 + n, dtype=torch.int32).cuda()
    want = t.rotate(q.contiguous(), k.contiguous(), pos, table)
    got = t.rotate(q, k, pos, table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    before, back = v.clone(), flat.clone()
    qo, ko = t.rotate(q, k, pos, table, out=(q, k))
    assert qo is q and ko is k and torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)
    assert torch.equal(flat[:shift], back[:shift]) and torch.equal(flat[shift + n * (hq + 2 * hk) * d:], back[shift + n * (hq + 2 * hk) * d:])


def test_there_and_back():
    table = t.rotary_table(128)
    q = rand(8, 300, 5, 128).cuda()
    pos = torch.randint(0, 1 << 20, (300,), generator=torch.Generator().manual_seed(9)).cuda()
    there, _ = t.rotate(q, None, pos, table)
    back, _ = t.rotate(there, None, pos, table, inverse=True)
    # two rotations, each off by at most (|a| + |b|) (2^-23 + 5 e) + e |y|, and a rotation keeps |a| + |b| within sqrt(2)
    a, b = q[..., :64].abs(), q[..., 64:].abs()
    slack = 3 * (a + b) * (2.0 ** -23 + 6 * 2.0 ** -24)
    assert ((back[..., :64] - q[..., :64]).abs() <= slack).all() and ((back[..., 64:] - q[..., 64:]).abs() <= slack).all()


def test_rotated_products_depend_on_distance():
    """What rotary positions are for: q at i and k at j give a product of i - j alone."""
    table = t.rotary_table(64)
    q, k = rand(10, 1, 1, 64).cuda().expand(4, 1, 64).contiguous(), rand(11, 1, 1, 64).cuda().expand(4, 1, 64).contiguous()
    far = torch.tensor([50, 1050, 100050, 2 ** 40 + 50]).cuda()
    qo, _ = t.rotate(q, None, far, table)
    ko, _ = t.rotate(k, None, far - 50, table)
    dots = (qo.double() * ko.double()).sum((1, 2))
    size = (q.abs().double() * k.abs().double()).sum((1, 2)).max().item() + (q.norm() * k.norm()).item()
    assert (dots - dots[0]).abs().max().item() <= size * 2.0 ** -19


def test_streams_graphs_and_empty():
    table = t.rotary_table(64)
    q, k = rand(12, 33, 8, 64).cuda(), rand(13, 33, 2, 64).cuda()
    pos = torch.arange(33).cuda()
    want = t.rotate(q, k, pos, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = t.rotate(q, k, pos, table, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    outs = (torch.empty_like(q), torch.empty_like(k))
    with torch.cuda.graph(graph):
        t.rotate(q, k, pos, table, out=outs)
    pos.add_(7)
    graph.replay()
    want = t.rotate(q, k, pos, table)
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    qo, ko = t.rotate(q[:0], k[:0], pos[:0], table)
    assert qo.shape == (0, 8, 64) and ko.shape == (0, 2, 64)


def test_nan_and_infinity_stay_in_their_pair():
    table = t.rotary_table(64)
    q = rand(14, 3, 2, 64).cuda()
    clean, _ = t.rotate(q, None, torch.arange(3).cuda() + 5, table)
    q[1, 0, 3], q[2, 1, 40] = math.nan, math.inf
    got, _ = t.rotate(q, None, torch.arange(3).cuda() + 5, table)
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[1, 0, [3, 35]] = True
    want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want) and torch.equal(got[~bad], clean[~bad])


def test_many_tokens():
    """More tokens than CTAs, heads of odd counts."""
    table = t.rotary_table(128)
    q, k = rand(15, 5001, 3, 128, dtype=torch.bfloat16).cuda(), rand(16, 5001, 1, 128, dtype=torch.bfloat16).cuda()
    pos = torch.arange(5001).cuda()
    qo, ko = t.rotate(q, k, pos, table)
    rows = torch.tensor([0, 1, 2431, 2432, 2433, 4863, 4864, 5000])
    check(q[rows.cuda()], qo[rows.cuda()], rows, table, False)
    check(k[rows.cuda()], ko[rows.cuda()], rows, table, False)
    for i in range(0, 5001, 97):
        one, _ = t.rotate(q[i:i + 1], None, pos[i:i + 1], table)
        assert torch.equal(one[0], qo[i])


def test_outputs_are_packed():
    """Whatever the inputs' strides."""
    table = t.rotary_table(64)
    qkv = rand(17, 9, 12, 64).cuda()
    for q, k in ((qkv[:, :8], qkv[:, 8:10]), (qkv[::2, :1], qkv[::2, 8:9]), (qkv[:1, :8], qkv[:1, 9:]), (qkv[:, 3:4], qkv[:, 4:8])):
        qo, ko = t.rotate(q, k, torch.arange(len(q)).cuda(), table)
        assert qo.is_contiguous() and ko.is_contiguous() and qo.shape == q.shape and ko.shape == k.shape
        wq, wk = t.rotate(q.contiguous(), k.contiguous(), torch.arange(len(q)).cuda(), table)
        assert torch.equal(qo, wq) and torch.equal(ko, wk)
