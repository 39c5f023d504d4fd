"""Cases of the operators around a cache held in 8 bits, with their plain forms.

A case names its operator in "op":
  rotate  rotary positions of q and k
  append  tokens quantised as they are written into pages of 8-bit blocks (and the touched blocks read back)
  read    tokens of 8-bit pages as packed keys and values
  attend  one decode token per sequence over 8-bit pages
A block is the 16 tokens of a page, one KV head, K or V; it has one scale.
"""
import math

import torch

own = False
PAGE = 16


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(text):
    return [int(x) for x in text.split(",")]


BATCH = ("1024,8192,4000,2500,6001,7333,3500,4321,1500,2048,5000,7777,6400,1100,3900,4608,"
         "8001,2222,5555,6789,1234,4096,7000,3333,2999,5821,6150,1777,4850,3600,7900,2400")


def listed():
    return [
        # one decode step of the smallest workload: one launch's latency
        dict(name="rotate_step_f32", op="rotate", dtype="f32", hq=8, hkv=2, d=64, rotary=64, tokens=1, top=512,
             interleaved=False, factor=1.0, trained=0, inverse=False),
        # a prompt's queries and keys, views of one projection, at positions far past the trained length
        dict(name="rotate_prompt", op="rotate", dtype="bf16", hq=32, hkv=8, d=128, rotary=128, tokens=8192, top=131072,
             interleaved=False, factor=32.0, trained=4096, inverse=False),
        # half of each head turned back, in neighbouring pairs
        dict(name="rotate_part_f32", op="rotate", dtype="f32", hq=32, hkv=32, d=128, rotary=64, tokens=1501, top=16384,
             interleaved=True, factor=4.0, trained=0, inverse=True),
        # one new token of each of 32 sequences: most join a block that holds tokens
        dict(name="append_step", op="append", dtype="bf16", hkv=4, d=128, lens=BATCH, new=",".join(["1"] * 32)),
        # prompts that arrive together, some behind what is cached already
        dict(name="append_prompts", op="append", dtype="bf16", hkv=4, d=128, lens="0,0,37,512,1000,0,7,0",
             new="256,37,512,1024,1,700,333,129"),
        # long documents
        dict(name="append_long", op="append", dtype="bf16", hkv=8, d=128, lens="0,15360", new="32768,8191"),
        # a short row of the smallest workload
        dict(name="read_tiny_f32", op="read", dtype="f32", hkv=2, d=64, lens="512", first="0"),
        # the keys ahead of the last chunk of long prompts
        dict(name="read_prompts", op="read", dtype="bf16", hkv=8, d=128, lens="15872,4096,9001,333", first="0,0,1000,5"),
        # two chains of the smallest workload
        dict(name="attend_tiny_f32", op="attend", dtype="f32", hq=8, hkv=2, d=64, lens="512,77", alpha=True),
        # a decode step of the benchmark's batch, with the scores of its tokens
        dict(name="attend_batch", op="attend", dtype="bf16", hq=28, hkv=4, d=128, lens=BATCH, alpha=True),
        # four long contexts
        dict(name="attend_long", op="attend", dtype="bf16", hq=32, hkv=8, d=128, lens="131072,131072,131059,130000", alpha=False),
        # a model without grouped heads
        dict(name="attend_mha", op="attend", dtype="bf16", hq=32, hkv=32, d=128,
             lens="16384,15361,15900,16000,16100,16200,16300,15555", alpha=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(8, 2, 64), (28, 4, 128), (32, 8, 128), (32, 32, 128), (16, 8, 64), (8, 8, 128), (32, 2, 128), (12, 4, 64)]


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "attend", "attend"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    hq, hkv, d = rng.choice(HEADS)
    if op == "rotate":
        scaling = rng.choice(["none", "all", "parts"])
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, rotary=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                    tokens=_log_int(rng, 1, 8192 if dtype == "bf16" else 4096), top=_log_int(rng, 2, 1 << 20),
                    interleaved=rng.random() < 0.5, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]),
                    trained=rng.choice([2048, 8192]) if scaling == "parts" else 0, inverse=rng.random() < 0.25)
    rows = _log_int(rng, 1, 64)
    if op == "attend":
        longest = _log_int(rng, 1, min(131072, (1 << 30) // (rows * hkv * d * 2)))
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, alpha=rng.random() < 0.5,
                    lens=",".join(str(_log_int(rng, 1, longest)) for _ in range(rows)))
    longest = _log_int(rng, 1, min(32768, (1 << 26) // (rows * hkv * d)))
    lens = [_log_int(rng, 1, longest) for _ in range(rows)]
    if op == "read":
        first = [0 if rng.random() < 0.5 else rng.randint(0, n) for n in lens]
        first[0] = 0
        return dict(op=op, dtype=dtype, hkv=hkv, d=d, lens=",".join(map(str, lens)), first=",".join(map(str, first)))
    new = [1] * rows if rng.random() < 0.4 else [_log_int(rng, 1, longest) for _ in range(rows)]
    lens = [0 if rng.random() < 0.3 else n for n in lens]
    return dict(op=op, dtype=dtype, hkv=hkv, d=d, lens=",".join(map(str, lens)), new=",".join(map(str, new)))


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _keys(gen, shape, dtype):
    """Keys whose tokens differ in length (lognormal), so that softmax rows are neither flat nor one-hot."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    w = torch.randn(shape[:-1], generator=gen, device="cuda", dtype=torch.float32).mul_(0.5).exp_()
    return (x * w.unsqueeze(-1)).to(dtype)


def _starts(lens):
    at, out = 0, []
    for n in lens:
        out.append(at)
        at += n
    return out


def _cuda(values):
    return torch.tensor(values, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"rotate": _prepare_rotate, "append": _prepare_append, "read": _prepare_read,
            "attend": _prepare_attend}[case["op"]](case, gen)


def _inverse_frequencies(case):
    """float64 [rotary / 2], by parts where the trained length is given."""
    r = case["rotary"]
    f = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    if not case["trained"]:
        return f / case["factor"]
    keep = ((case["trained"] * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / case["factor"])


def _scale(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["trained"] else 1.0


def _prepare_rotate(case, gen):
    n, hq, hkv, d, dt = case["tokens"], case["hq"], case["hkv"], case["d"], _dt(case)
    qkv = _normal(gen, (n, hq + 2 * hkv, d), dt)                # one projection's output
    if n == 1:
        pos = torch.randint(case["top"], (1,), generator=gen, device="cuda")
    else:  # runs of consecutive positions, as packed prompts and chains have them
        runs = torch.randint(case["top"], (-(-n // 300),), generator=gen, device="cuda")
        pos = (runs.repeat_interleave(300)[:n] + torch.arange(n, device="cuda") % 300) % case["top"]
    s = dict(op="rotate", q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], pos=pos, freq=_inverse_frequencies(case).cuda(),
             scale=_scale(case), interleaved=case["interleaved"], inverse=case["inverse"], r=case["rotary"])
    if own:
        from tiered_kv_cache_split_gb300 import rotary_table
        s["rotary"] = rotary_table(case["rotary"], base=10000.0, factor=case["factor"], trained=case["trained"] or None,
                                   scale=s["scale"], interleaved=case["interleaved"], device="cuda")
    return s


def _blocks(x):
    """Codes and scales of [pages, Hkv, 2, 16, d]: one scale per page, head, K and V."""
    scale = x.abs().amax((3, 4)) / 127.0
    by = torch.where(scale > 0, scale, 1.0)[..., None, None]
    return (x / by).round_().clamp_(-127, 127).to(torch.int8), scale


def _pool(gen, pages, hkv, d, dt):
    """A pool of keys and values as they are after they were quantised, a slice at a time."""
    pool = torch.empty((pages, hkv, 2, PAGE, d), dtype=torch.int8, device="cuda")
    scales = torch.empty((pages, hkv, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (hkv * 2 * PAGE * d))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        x = torch.stack([_keys(gen, (n, hkv, PAGE, d), dt), _normal(gen, (n, hkv, PAGE, d), dt)], 2)
        pool[i:i + n], scales[i:i + n] = _blocks(x.float())
    return pool, scales


def _table(gen, n_pages, pages):
    """Rows that list n_pages[b] pages of the pool each, in random order; -1 behind them."""
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(max(max(n_pages), 1), device="cuda")
    in_row = col < _cuda(n_pages)[:, None]
    at = (_cuda(_starts(n_pages))[:, None] + col).clamp_(max=pages - 1)
    return torch.where(in_row, ids[at], -1), in_row


def _prepare_append(case, gen):
    hkv, d, dt = case["hkv"], case["d"], _dt(case)
    lens, new = _ints(case["lens"]), _ints(case["new"])
    ends = [a + b for a, b in zip(lens, new)]
    n_pages = [-(-n // PAGE) for n in ends]
    pages = sum(n_pages) + 3
    pool, scales = _pool(gen, pages, hkv, d, dt)
    table, in_row = _table(gen, n_pages, pages)
    live = (torch.arange(table.shape[1], device="cuda")[:, None] * PAGE + torch.arange(PAGE, device="cuda")) < _cuda(lens)[:, None, None]
    mask = torch.zeros(pages, dtype=torch.int32, device="cuda")
    mask[table[in_row].long()] = (live.to(torch.int32) << torch.arange(PAGE, device="cuda")).sum(-1).to(torch.int32)[in_row]
    total = sum(new)
    kv = torch.cat([_keys(gen, (total, hkv, d), dt), _normal(gen, (total, hkv, d), dt)], 1)
    first = [n // PAGE * PAGE for n in lens]                    # the first slot of the first block written
    # where each token goes, for the plain form
    row = torch.repeat_interleave(torch.arange(len(new), device="cuda"), _cuda(new))
    slot = _cuda(lens)[row] + torch.arange(total, device="cuda") - _cuda(_starts(new))[row]
    n_touched = [p - f // PAGE for p, f in zip(n_pages, first)]
    block = _cuda(_starts(n_touched))[row] + slot // PAGE - _cuda(first)[row] // PAGE
    trow = torch.repeat_interleave(torch.arange(len(new), device="cuda"), _cuda(n_touched))
    tcol = _cuda(first)[trow] // PAGE + torch.arange(sum(n_touched), device="cuda") - _cuda(_starts(n_touched))[trow]
    held = (_cuda(lens)[trow] - tcol * PAGE).clamp(min=0)       # tokens a touched block holds already
    tslot = tcol[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    return dict(op="append", k=kv[:, :hkv], v=kv[:, hkv:], pool=pool, scales=scales, table=table, mask=mask, lens=lens, new=new,
                ends=ends, first=first, slot=slot % PAGE, block=block, trow=trow, tcol=tcol, held=held,
                back=tslot < _cuda(ends)[trow][:, None])


def _prepare_read(case, gen):
    hkv, d, dt = case["hkv"], case["d"], _dt(case)
    lens, first = _ints(case["lens"]), _ints(case["first"])
    n_pages = [-(-n // PAGE) for n in lens]
    pages = sum(n_pages) + 3
    pool, scales = _pool(gen, pages, hkv, d, dt)
    table, _ = _table(gen, n_pages, pages)
    mask = torch.full((pages,), 0xFFFF, dtype=torch.int32, device="cuda")
    count = [n - f for n, f in zip(lens, first)]
    row = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), _cuda(count))
    at = _cuda(first)[row] + torch.arange(sum(count), device="cuda") - _cuda(_starts(count))[row]
    return dict(op="read", pool=pool, scales=scales, table=table, mask=mask, lens=lens, first=first, dt=dt, row=row, at=at)


def _prepare_attend(case, gen):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dt(case)
    lens = _ints(case["lens"])
    n_pages = [-(-n // PAGE) for n in lens]
    pages = sum(n_pages) + 3
    pool, scales = _pool(gen, pages, hkv, d, dt)
    table, in_row = _table(gen, n_pages, pages)
    # a row ends where the sequence does; 5 % of the slots were evicted
    tok = torch.arange(table.shape[1], device="cuda")[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    live = tok < _cuda(lens)[:, None, None]
    live &= (torch.rand(live.shape, generator=gen, device="cuda") >= 0.05) | (tok == 0)
    mask = torch.zeros(pages, dtype=torch.int32, device="cuda")
    mask[table[in_row].long()] = (live.to(torch.int32) << torch.arange(PAGE, device="cuda")).sum(-1).to(torch.int32)[in_row]
    alpha = torch.zeros((len(lens), hkv, table.shape[1] * PAGE), dtype=torch.float32, device="cuda") if case["alpha"] else None
    return dict(op="attend", q=_normal(gen, (len(lens), hq, d), dt), pool=pool, scales=scales, table=table, mask=mask,
                counts=n_pages, in_row=in_row, alpha=alpha)


def run(state):
    if own:
        return {"rotate": _own_rotate, "append": _own_append, "read": _own_read, "attend": _own_attend}[state["op"]](state)
    return {"rotate": _plain_rotate, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[state["op"]](state)


# ---------------------------------------------------------------- the framework's calls
def _own_rotate(s):
    from tiered_kv_cache_split_gb300 import rotate
    return rotate(s["q"], s["k"], s["pos"], s["rotary"], inverse=s["inverse"])


def _own_append(s):
    from tiered_kv_cache_split_gb300 import append_quantized, read_quantized
    append_quantized(s["k"], s["v"], s["pool"], s["scales"], s["table"], s["mask"], s["lens"], s["new"])
    k, v = read_quantized(s["pool"], s["scales"], s["table"], s["mask"], s["ends"], first=s["first"], dtype=s["k"].dtype)
    return {"k": k, "v": v, "scales": s["scales"], "mask": s["mask"]}


def _own_read(s):
    from tiered_kv_cache_split_gb300 import read_quantized
    return read_quantized(s["pool"], s["scales"], s["table"], s["mask"], s["lens"], first=s["first"], dtype=s["dt"])


def _own_attend(s):
    from tiered_kv_cache_split_gb300 import quantized_attention
    if s["alpha"] is not None:
        s["alpha"].zero_()
    out = quantized_attention(s["q"], s["pool"], s["scales"], s["table"], s["mask"], s["counts"], alpha_sum=s["alpha"])
    return {"out": out, "alpha": s["alpha"]}


# ---------------------------------------------------------------- plain forms
def _plain_rotate(s):
    r = s["r"]
    angle = s["pos"].double()[:, None] * s["freq"]
    if s["inverse"]:
        angle = -angle
    cos, sin = angle.cos().float()[:, None] * s["scale"], angle.sin().float()[:, None] * s["scale"]
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if s["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
        c, e = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack([c, e], -1).flatten(-2) if s["interleaved"] else torch.cat([c, e], -1)
        out.append(torch.cat([turned, y[..., r:]], -1).to(x.dtype))
    return tuple(out)


def _plain_append(s):
    pool, scales, mask = s["pool"], s["scales"], s["mask"]
    x = torch.stack([s["k"].float(), s["v"].float()], 2)                      # [T, Hkv, 2, d]
    ids = s["table"][s["trow"], s["tcol"]].long()                             # the blocks written
    n, hkv = ids.shape[0], x.shape[1]
    top = torch.zeros((n, hkv, 2), device=x.device)
    top.scatter_reduce_(0, s["block"][:, None, None].expand(-1, hkv, 2), x.abs().amax(-1), "amax")
    old = torch.where((s["held"] > 0)[:, None, None], scales[ids], 0.0)
    scale = torch.maximum(old, top / 127.0)
    by = torch.where(scale > 0, scale, 1.0)
    codes = pool[ids].float() * (old / by)[..., None, None]                   # earlier tokens, where the scale grew
    codes = torch.where((scale > old)[..., None, None], codes.round(), pool[ids].float())
    codes.permute(0, 3, 1, 2, 4)[s["block"], s["slot"]] = (x / by[s["block"]][..., None]).round_().clamp_(-127, 127)
    pool[ids] = codes.to(torch.int8)
    scales[ids] = scale
    slots = torch.arange(PAGE, device=x.device)
    bits = ((s["back"] & (slots >= s["held"][:, None])).to(torch.int32) << slots).sum(-1).to(torch.int32)
    mask[ids] = torch.where(s["held"] > 0, mask[ids] | bits, bits)
    back = pool[ids].float() * scales[ids][..., None, None]
    back = back.permute(2, 0, 3, 1, 4)[:, s["back"]].to(s["k"].dtype)
    return {"k": back[0], "v": back[1], "scales": scales, "mask": mask}


def _plain_read(s):
    ids = s["table"][s["row"], s["at"] // PAGE].long()
    kv = s["pool"][ids, :, :, s["at"] % PAGE].float() * s["scales"][ids][..., None]
    return kv[:, :, 0].to(s["dt"]).contiguous(), kv[:, :, 1].to(s["dt"]).contiguous()


def _plain_attend(s):
    q, table = s["q"], s["table"].long().clamp(min=0)
    b, hq, d = q.shape
    hkv = s["pool"].shape[1]
    kv = s["pool"][table].float() * s["scales"][table][..., None, None]       # [b, pages, hkv, 2, 16, d]
    k, v = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, b, hkv, -1, d)
    del kv
    x = torch.matmul(q.float().view(b, hkv, -1, d), k.transpose(2, 3)).mul_(1.0 / math.sqrt(d))
    live = (((s["mask"][table][:, :, None] >> torch.arange(PAGE, device=q.device)) & 1) != 0) & s["in_row"][:, :, None]
    x.masked_fill_(~live.view(b, 1, 1, -1), -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    if s["alpha"] is not None:
        s["alpha"].zero_()
        s["alpha"] += x.sum(2)
    return {"out": torch.matmul(x, v).view(b, hq, d).to(q.dtype), "alpha": s["alpha"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)


def _exact_rotate(case, s):
    """The pairs as complex numbers, multiplied by scale * exp(+-i pos f)."""
    r = case["rotary"]
    turn = torch.polar(torch.full_like(s["freq"], _scale(case)).expand(len(s["pos"]), -1).contiguous(),
                       torch.outer(s["pos"].double(), s["freq"]))
    turn = (turn.conj() if case["inverse"] else turn)[:, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * turn
            y[..., :r] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * turn
            y[..., :r] = torch.cat([z.real, z.imag], -1)
        out.append(y)
    return tuple(out)


def _exact_append(case, s):
    """Row by row and block by block: scales are held in 32 bits, all else in 64."""
    k, v, t0 = s["k"].double(), s["v"].double(), 0
    scales, out = s["scales"].double(), [[], []]
    if len(s["trow"]) > 4096:
        return None
    for b, (n0, n1) in enumerate(zip(s["lens"], s["ends"])):
        for p in range(n0 // PAGE, -(-n1 // PAGE)):
            lo, hi = max(n0, p * PAGE), min(n1, (p + 1) * PAGE)
            held = max(0, n0 - p * PAGE)
            page = int(s["table"][b, p])
            for j, x in enumerate((k, v)):
                new = x[t0 + lo - n0:t0 + hi - n0]                            # [n, hkv, d]
                old = scales[page, :, j].clone() if held else torch.zeros_like(scales[page, :, j])
                now = torch.maximum((new.abs().amax((0, 2)) / 127.0).float().double(), old)
                by = torch.where(now > 0, now, 1.0)[:, None]
                before = s["pool"][page, :, j, :held].double().permute(1, 0, 2)
                ratio = torch.where(now > old, old / by[:, 0], 1.0)[:, None]
                out[j].append(torch.cat([torch.round(before * ratio), torch.round(new / by).clamp(-127, 127)]) * now[:, None])
                scales[page, :, j] = now
        t0 += n1 - n0
    return {"k": torch.cat(out[0]), "v": torch.cat(out[1]), "scales": scales, "mask": None}


def _exact_read(case, s):
    out = [[], []]
    for b, (lo, hi) in enumerate(zip(s["first"], s["lens"])):
        ids = s["table"][b, :-(-hi // PAGE)].long()
        for j in range(2):
            x = s["pool"][ids, :, j].double() * s["scales"][ids, :, j].double()[..., None, None]
            out[j].append(x.permute(0, 2, 1, 3).flatten(0, 1)[lo:hi])
    return torch.cat(out[0]), torch.cat(out[1])


def _exact_attend(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    alpha = torch.zeros_like(s["alpha"], dtype=torch.float64) if s["alpha"] is not None else None
    for b, n in enumerate(s["counts"]):
        ids = s["table"][b, :n].long()
        at = torch.nonzero(((s["mask"][ids][:, None] >> torch.arange(PAGE, device="cuda")) & 1).flatten()).flatten()
        for h in range(hkv):
            kv = s["pool"][ids, h].double() * s["scales"][ids, h].double()[..., None, None]
            k, v = kv[:, 0].reshape(-1, d)[at], kv[:, 1].reshape(-1, d)[at]
            x = s["q"][b].view(hkv, -1, d)[h].double() @ k.T / math.sqrt(d)
            p = torch.exp(x - x.max(dim=1, keepdim=True).values)
            p /= p.sum(dim=1, keepdim=True)
            out[b].view(hkv, -1, d)[h] = p @ v
            if alpha is not None:
                alpha[b, h, at] = p.sum(0)
    return {"out": out, "alpha": alpha}


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotate":
        elements = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 2 * esz * elements + 8 * case["tokens"], "flops": 3 * elements * case["rotary"] // case["d"]}
    row = 2 * case["hkv"] * case["d"]                                         # elements of a token
    lens = _ints(case["lens"])
    if case["op"] == "append":
        new = _ints(case["new"])
        back = sum(a % PAGE + b for a, b in zip(lens, new))                   # tokens of the blocks written
        return {"bytes": row * (esz * sum(new) + back + esz * back) + 8 * case["hkv"] * back // PAGE, "flops": 4 * row * sum(new)}
    if case["op"] == "read":
        n = sum(lens) - sum(_ints(case["first"]))
        return {"bytes": row * (1 + esz) * n + 8 * case["hkv"] * n // PAGE, "flops": row * n}
    tokens = sum(lens)
    return {"bytes": row * tokens + 8 * case["hkv"] * tokens // PAGE + 2 * esz * len(lens) * case["hq"] * case["d"]
            + (8 * case["hkv"] * tokens if case["alpha"] else 0), "flops": 4 * case["d"] * case["hq"] * tokens}
