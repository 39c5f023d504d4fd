"""rotate with several tokens per CTA, on vectors and element by element, and turned back with a scale."""
import pytest
import torch

import tiered_kv_cache_split_gb300 as t
from operator_helpers import assert_within
from quantized_helpers import rotate_reference

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,r", [(128, 128), (128, 64), (128, 50), (33, 10), (80, 20)])
@pytest.mark.parametrize("tokens,hq,hk,shift", [(1825, 3, 1, 0), (5001, 2, 1, 0), (1825, 2, 2, 1), (7331, 1, 0, 1)])
def test_many_tokens(dtype, interleaved, d, r, tokens, hq, hk, shift):
    """From 1824 tokens on a CTA has two and more, and the last one may have fewer. shift: rows
    off 16-byte boundaries. Some rows against the rotation in 64 bits and against calls of one token."""
    table = t.rotary_table(r, interleaved=interleaved, factor=4.0, trained=1000, scale=1.25)
    flat = rand(tokens + d + r, tokens * (hq + hk) * d + shift, dtype=DT[dtype]).cuda()
    qk = flat[shift:].view(tokens, hq + hk, d)
    q, k = qk[:, :hq], qk[:, hq:] if hk else None
    pos = torch.randint(-5000, 100000, (tokens,), generator=torch.Generator().manual_seed(d)).cuda()
    at = torch.tensor(sorted({0, 1, 2, 3, 911, 912, 913, 1823, 1824, tokens // 2, tokens - 4, tokens - 3, tokens - 2, tokens - 1})).cuda()
    outs = t.rotate(q, k, pos, table)
    for x, got in zip((q, k), outs):
        if x is None:
            assert got is None
            continue
        want, bound = rotate_reference(x[at], pos[at].tolist(), table.inv_freq, table.scale, interleaved, False, x.dtype)
        assert_within(got[at], want, bound)
        assert torch.equal(got[..., r:], x[..., r:])
        for i in at.tolist():
            one = torch.empty(1 + x[i].numel(), dtype=x.dtype, device="cuda")[shift:shift + x[i].numel()].view(1, *x[i].shape)
            one.copy_(x[i:i + 1])
            assert torch.equal(t.rotate(one, None, pos[i:i + 1], table)[0][0], got[i])
    t.rotate(q, k, pos, table, out=(q, k))            # in place
    assert torch.equal(q, outs[0]) and (k is None or torch.equal(k, outs[1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scale", [1.3, -0.5])
def test_inverse_with_a_scale(dtype, interleaved, scale):
    """inverse turns by the opposite angles and multiplies by the scale again: there and back is scale^2."""
    table = t.rotary_table(64, scale=scale, interleaved=interleaved)
    q, pos = rand(1, 50, 3, 64, dtype=DT[dtype]).cuda(), torch.arange(50).cuda() * 77
    back, _ = t.rotate(q, None, pos, table, inverse=True)
    want, bound = rotate_reference(q, pos.tolist(), table.inv_freq, scale, interleaved, True, q.dtype)
    assert_within(back, want, bound)
    there, _ = t.rotate(q, None, pos, table)
    both, _ = t.rotate(there, None, pos, table, inverse=True)
    want, bound = rotate_reference(there, pos.tolist(), table.inv_freq, scale, interleaved, True, q.dtype)
    assert_within(both, want, bound)
    # |there - exact| <= (|a| + |b|) |scale| (2^-23 + 5 e) + u |y|, and the way back multiplies it by at most |scale| sqrt(2)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    pair = (q.double() ** 2).view(50, 3, 32, 2).sum(-1) if interleaved else q.double()[..., :32] ** 2 + q.double()[..., 32:] ** 2
    size = pair.sqrt().repeat_interleave(2, -1) if interleaved else pair.sqrt().repeat(1, 1, 2)
    slack = size * scale * scale * (3 * 2.0 ** 0.5 * (2.0 ** -23 + 6 * 2.0 ** -24) + 3 * u)
    assert ((both.double() - scale * scale * q.double()).abs() <= slack).all()
