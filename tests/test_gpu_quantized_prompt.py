"""A prompt's next chunk over a pool in 8 bits: several rows read into their places of one buffer."""
import pytest
import torch

import tiered_kv_cache_split_gb300 as t

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_read_into_their_places(dtype):
    """Each row's cached keys directly ahead of its new ones, read there, give prompt_attention what a packed
    read and a copy give."""
    hq, hkv, d, lens, new = 8, 2, 64, [37, 0, 160, 5], [20, 33, 1, 64]
    gen = torch.Generator().manual_seed(3)
    pages = torch.randperm(64, generator=gen).view(4, 16).to(torch.int32).cuda()
    pool, scales = torch.zeros(64, hkv, 2, 16, d, dtype=torch.int8).cuda(), torch.zeros(64, hkv, 2).cuda()
    mask = torch.zeros(64, dtype=torch.int32).cuda()
    old = [torch.randn(sum(lens), hkv, d, generator=gen).to(dtype).cuda() for _ in range(2)]
    t.append_quantized(*old, pool, scales, pages, mask, [0] * 4, lens)
    q = torch.randn(sum(new), hq, d, generator=gen).to(dtype).cuda()
    k, v = (torch.randn(sum(new), hkv, d, generator=gen).to(dtype).cuda() for _ in range(2))
    keys, values = (torch.full((sum(lens) + sum(new), hkv, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    packed = t.read_quantized(pool, scales, pages, mask, lens, dtype=dtype)
    parts = [[], []]
    at = x = c = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        t.read_quantized(pool, scales, pages[b:b + 1], mask, [n], out=(keys[at:at + n], values[at:at + n]))
        keys[at + n:at + n + m], values[at + n:at + n + m] = k[x:x + m], v[x:x + m]
        for part, cached, fresh in zip(parts, packed, (k, v)):
            part += [cached[c:c + n], fresh[x:x + m]]
        at, x, c = at + n + m, x + m, c + n
    assert torch.equal(keys, torch.cat(parts[0])) and torch.equal(values, torch.cat(parts[1]))
    k_lens = [n + m for n, m in zip(lens, new)]
    assert torch.equal(t.prompt_attention(q, keys, values, new, k_lens), t.prompt_attention(q, torch.cat(parts[0]), torch.cat(parts[1]), new, k_lens))
