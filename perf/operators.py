"""Cases of the prompt, shared-prefix and page operators, with their plain forms.

A case names its operator in "op":
  prompt    causal attention over packed prompts (q_lens new tokens each, behind `cached` tokens)
  prefix    one decode token per sequence over a prefix all sequences share plus pages of their own
  fork      children of one sequence: full pages shared (share) or copied, then freed again
  compact   tokens behind evicted slots are moved down and the emptied pages freed
"""
import math

import torch

own = False
PAGE = 16


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _ints(text):
    return [int(x) for x in text.split(",")]


def listed():
    return [
        # the prompt of the smallest workload: one launch's latency
        dict(name="prompt_tiny_f32", op="prompt", dtype="f32", hq=8, hkv=2, d=64, q_lens="32", cached="0"),
        # a batch of prompts of a 28-head model as they arrive together, read from one fused projection
        dict(name="prompt_packed", op="prompt", dtype="bf16", hq=28, hkv=4, d=128,
             q_lens="256,37,512,1024,1,700,333,129", cached="0,0,0,0,0,0,0,0"),
        # one long document
        dict(name="prompt_long", op="prompt", dtype="bf16", hq=32, hkv=8, d=128, q_lens="8192", cached="0"),
        # the last chunk of a 16k prompt with as many KV heads as query heads
        dict(name="prompt_chunk", op="prompt", dtype="bf16", hq=32, hkv=32, d=128, q_lens="512", cached="15872"),
        # two chains of the smallest workload
        dict(name="prefix_tiny_f32", op="prefix", dtype="f32", hq=8, hkv=2, d=64, shared=512, own_lens="64,17", alpha=True),
        # 32 chains of up to 2000 tokens behind one prompt, with the scores of their own tokens
        dict(name="prefix_chains", op="prefix", dtype="bf16", hq=28, hkv=4, d=128, shared=4096,
             own_lens="1,2000,64,127,900,1500,333,15,16,17,1024,48,700,256,1999,800,5,450,1200,90,"
                      "600,31,32,33,1750,220,1000,512,77,1300,8,405", alpha=True),
        # 64 questions about one long document
        dict(name="prefix_document", op="prefix", dtype="bf16", hq=32, hkv=8, d=128, shared=131072,
             own_lens=",".join(str(16 + (37 * b) % 240) for b in range(64)), alpha=False),
        # eight samples of a model without grouped heads
        dict(name="prefix_mha", op="prefix", dtype="bf16", hq=32, hkv=32, d=128, shared=15360,
             own_lens="100,1024,300,1,640,77,512,960", alpha=False),
        # 31 chains forked from a 256-token prompt and its first answer tokens
        dict(name="fork_share", op="fork", dtype="bf16", layers=28, hkv=4, d=128, tokens=265, children=31, share=True),
        # three whole copies of a chain at its 2000-token limit
        dict(name="fork_copy", op="fork", dtype="bf16", layers=28, hkv=4, d=128, tokens=2000, children=3, share=False),
        # one short sequence after an eviction
        dict(name="compact_tiny_f32", op="compact", dtype="f32", layers=1, hkv=2, d=64, lens="512", evict=25),
        # a layer group of a batch after half of its tokens left
        dict(name="compact_batch", op="compact", dtype="bf16", layers=7, hkv=4, d=128,
             lens="1024,8192,4000,2500,6001,7333,3500,4321", evict=50),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(8, 2, 64), (28, 4, 128), (32, 8, 128), (32, 32, 128), (16, 8, 64), (8, 8, 128)]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prefix", "prefix", "fork", "compact"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    hq, hkv, d = rng.choice(HEADS)
    if op == "prompt":
        top = 1024 if dtype == "f32" else 8192
        longest = _log_int(rng, 1, top)
        batch = max(1, min(rng.randint(1, 16), (1 << 31) // (hq * longest * longest * 2)))
        lens = [longest] + [_log_int(rng, 1, longest) for _ in range(batch - 1)]
        rng.shuffle(lens)
        cached = [0] * batch
        if rng.random() < 0.4:
            most = min(16384 if dtype == "bf16" else 2048, (1 << 30) // (batch * hq * longest)) - longest
            cached = [_log_int(rng, 1, most) if most >= 1 and rng.random() < 0.8 else 0 for _ in lens]
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, q_lens=",".join(map(str, lens)),
                    cached=",".join(map(str, cached)))
    if op == "prefix":
        batch = _log_int(rng, 1, 64)
        shared = PAGE * _log_int(rng, 1, 512 if dtype == "f32" else min(8192, (1 << 25) // (hkv * d * 8)))
        longest = _log_int(rng, 1, 2000)
        return dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, shared=shared, alpha=rng.random() < 0.5,
                    own_lens=",".join(str(_log_int(rng, 1, longest)) for _ in range(batch)))
    layers = rng.choice([1, 4, 7, 28])
    record = layers * hkv * 2 * PAGE * d * (4 if dtype == "f32" else 2)
    most = (384 << 20) // record  # pages of the pool
    if op == "fork":
        share = rng.random() < 0.6
        children = _log_int(rng, 1, min(63, most // 2))
        tokens = PAGE * _log_int(rng, 1, max(1, min(256, most // 2 if share else most // (children + 1)))) - rng.randint(0, 15)
        return dict(op=op, dtype=dtype, layers=layers, hkv=hkv, d=d, tokens=tokens, children=children, share=share)
    batch = _log_int(rng, 1, min(32, max(1, most // 8)))
    longest = PAGE * max(1, min(512, most // batch))
    return dict(op=op, dtype=dtype, layers=layers, hkv=hkv, d=d, evict=rng.choice([5, 25, 50, 75]),
                lens=",".join(str(_log_int(rng, 1, longest)) for _ in range(batch)))


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"prompt": _prepare_prompt, "prefix": _prepare_prefix, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, gen)


def _prepare_prompt(case, gen):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dt(case)
    q_lens, cached = _ints(case["q_lens"]), _ints(case["cached"])
    k_lens = [a + b for a, b in zip(q_lens, cached)]
    tq, tk = sum(q_lens), sum(k_lens)
    if any(cached):
        q = _normal(gen, (tq, hq, d), dt)
        k, v = _keys(gen, (tk, hkv, d), dt), _normal(gen, (tk, hkv, d), dt)
    else:  # views of one projection's output
        qkv = torch.cat([_normal(gen, (tq, hq, d), dt), _keys(gen, (tq, hkv, d), dt), _normal(gen, (tq, hkv, d), dt)], 1)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    # where each token sits in a padded batch, for the plain form
    mq, mk = max(q_lens), max(k_lens)
    lq, lk = torch.tensor(q_lens, device="cuda"), torch.tensor(k_lens, device="cuda")
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    at_q = (torch.tensor(_starts(q_lens), device="cuda")[:, None] + iq).clamp_(max=tq - 1)
    at_k = (torch.tensor(_starts(k_lens), device="cuda")[:, None] + ik).clamp_(max=tk - 1)
    seq = torch.repeat_interleave(torch.arange(len(q_lens), device="cuda"), lq)
    back = seq * mq + torch.arange(tq, device="cuda") - torch.tensor(_starts(q_lens), device="cuda")[seq]
    return dict(op="prompt", q=q, k=k, v=v, q_lens=q_lens, k_lens=k_lens, lq=lq, lk=lk, iq=iq, ik=ik,
                at_q=at_q, at_k=at_k, back=back)


def _prepare_prefix(case, gen):
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dt(case)
    own_lens, ns = _ints(case["own_lens"]), case["shared"] // PAGE
    batch = len(own_lens)
    own_pages = [-(-n // PAGE) for n in own_lens]
    counts = [ns + n for n in own_pages]
    pages = ns + sum(own_pages) + 5
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    width = max(counts)
    table = torch.zeros((batch, width), dtype=torch.int32, device="cuda")
    table[:, :ns] = ids[:ns]
    n_own = torch.tensor(own_pages, device="cuda")
    col = torch.arange(width - ns, device="cuda")
    at = ns + torch.tensor(_starts(own_pages), device="cuda")[:, None] + col
    in_row = col < n_own[:, None]
    table[:, ns:][in_row] = ids[at[in_row]]
    # the last page of a sequence ends where the sequence does; 5 % of its own slots were evicted
    slot = torch.arange(PAGE, device="cuda")
    tok = col[:, None] * PAGE + slot
    live = tok < torch.tensor(own_lens, device="cuda")[:, None, None]
    live &= torch.rand(live.shape, generator=gen, device="cuda") >= 0.05
    bits = (live.to(torch.int32) << slot).sum(-1).to(torch.int32)
    mask = torch.full((pages,), 0xFFFF, dtype=torch.int32, device="cuda")
    mask[table[:, ns:][in_row].long()] = bits[in_row]
    pool = torch.stack([_keys(gen, (pages, hkv, PAGE, d), dt), _normal(gen, (pages, hkv, PAGE, d), dt)], 2)
    alpha = torch.zeros((batch, hkv, width * PAGE), dtype=torch.float32, device="cuda") if case["alpha"] else None
    return dict(op="prefix", q=_normal(gen, (batch, hq, d), dt), pool=pool, table=table, mask=mask, counts=counts,
                shared=ns, alpha=alpha, n_pages=torch.tensor(counts, device="cuda"))


def _prepare_fork(case, gen):
    n, c, share = -(-case["tokens"] // PAGE), case["children"], case["share"]
    pages = n + (c if share else c * n) + 9
    pool = _normal(gen, (case["layers"], pages, case["hkv"], 2, PAGE, case["d"]), _dt(case))
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c + 1, n + 4), -1, dtype=torch.int32, device="cuda")
    table[0, :n] = ids[:n]
    mask = torch.zeros(pages, dtype=torch.int32, device="cuda")
    mask[table[0, :n].long()] = 0xFFFF
    mask[table[0, n - 1].long()] = (1 << (case["tokens"] - PAGE * (n - 1))) - 1
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[0, :n].long()] = 1
    return dict(op="fork", pool=pool, table0=table, mask0=mask, refs0=refs, table=table.clone(), mask=mask.clone(),
                refs=refs.clone(), counts=[n] + [0] * c, children=list(range(1, c + 1)), n=n, share=share)


def _prepare_compact(case, gen):
    lens = _ints(case["lens"])
    n = [-(-x // PAGE) for x in lens]
    pages, width = sum(n) + 7, max(n) + 1
    pool = _normal(gen, (case["layers"], pages, case["hkv"], 2, PAGE, case["d"]), _dt(case))
    ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    in_row = col < torch.tensor(n, device="cuda")[:, None]
    at = (torch.tensor(_starts(n), device="cuda")[:, None] + col).clamp_(max=pages - 1)
    table = torch.where(in_row, ids[at], -1)
    tok = col[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    live = tok < torch.tensor(lens, device="cuda")[:, None, None]
    live &= torch.rand(live.shape, generator=gen, device="cuda") * 100 >= case["evict"]
    held = table[in_row].long()
    mask = torch.zeros(pages, dtype=torch.int32, device="cuda")
    mask[held] = (live.to(torch.int32) << torch.arange(PAGE, device="cuda")).sum(-1).to(torch.int32)[in_row]
    pos = torch.full((pages, PAGE), -1, dtype=torch.int32, device="cuda")
    pos[held] = torch.where(live, tok, -1).to(torch.int32)[in_row]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[held] = 1
    return dict(op="compact", pool=pool, table0=table, mask0=mask, refs0=refs, pos0=pos, table=table.clone(),
                mask=mask.clone(), refs=refs.clone(), pos=pos.clone(), counts=n, in_row=in_row)


def run(state):
    if own:
        return {"prompt": _own_prompt, "prefix": _own_prefix, "fork": _own_fork, "compact": _own_compact}[state["op"]](state)
    return {"prompt": _plain_prompt, "prefix": _plain_prefix, "fork": _plain_fork, "compact": _plain_compact}[state["op"]](state)


# ---------------------------------------------------------------- the framework's calls
def _own_prompt(s):
    from tiered_kv_cache_split_gb300 import prompt_attention
    return prompt_attention(s["q"], s["k"], s["v"], s["q_lens"], s["k_lens"])


def _own_prefix(s):
    from tiered_kv_cache_split_gb300 import shared_prefix_attention
    if s["alpha"] is not None:
        s["alpha"].zero_()
    out = shared_prefix_attention(s["q"], s["pool"], s["table"], s["mask"], s["counts"], s["shared"], alpha_sum=s["alpha"])
    return {"out": out, "alpha": s["alpha"]}


def _own_fork(s):
    from tiered_kv_cache_split_gb300 import fork_sequences, free_sequences
    s["table"].copy_(s["table0"]), s["mask"].copy_(s["mask0"]), s["refs"].copy_(s["refs0"])
    lacking = fork_sequences(s["pool"], s["table"], s["counts"], s["refs"], s["mask"], [0] * len(s["children"]),
                             s["children"], share=s["share"])
    forked = s["table"].clone(), s["mask"].clone(), s["refs"].clone()
    bad = free_sequences(s["table"], [s["n"]] * s["table"].shape[0], s["refs"], s["mask"], s["children"])
    return {"pool": s["pool"], "forked": forked, "lacking": lacking, "bad": bad, "table": s["table"], "mask": s["mask"], "refs": s["refs"]}


def _own_compact(s):
    from tiered_kv_cache_split_gb300 import compact_sequences
    s["table"].copy_(s["table0"]), s["mask"].copy_(s["mask0"]), s["refs"].copy_(s["refs0"]), s["pos"].copy_(s["pos0"])
    counts = compact_sequences(s["pool"], s["table"], s["counts"], s["refs"], s["mask"], positions=s["pos"])
    return {"pool": s["pool"], "counts": counts, "table": s["table"], "mask": s["mask"], "refs": s["refs"], "pos": s["pos"]}


# ---------------------------------------------------------------- plain forms
def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    hq, d = q.shape[1:]
    hkv = k.shape[1]
    b, mq = s["at_q"].shape
    qp = q.float()[s["at_q"]].view(b, mq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    kp = k.float()[s["at_k"]].permute(0, 2, 3, 1)
    vp = v.float()[s["at_k"]].permute(0, 2, 1, 3)
    x = torch.matmul(qp, kp).mul_(1.0 / math.sqrt(d)).view(b, hkv, hq // hkv, mq, -1)
    # key j is seen by query i when j <= i + (k_len - q_len) and both exist
    last = torch.minimum(s["iq"] + (s["lk"] - s["lq"])[:, None], s["lk"][:, None] - 1)
    x.masked_fill_((s["ik"] > last[:, :, None])[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, -1, x.shape[-1]), vp).view(b, hkv, hq // hkv, mq, d).div_(z)
    return o.permute(0, 3, 1, 2, 4).reshape(b * mq, hq, d)[s["back"]].to(q.dtype)


def _plain_prefix(s):
    q, pool, table, ns = s["q"], s["pool"], s["table"].long(), s["shared"]
    b, hq, d = q.shape
    hkv = pool.shape[1]
    g = hq // hkv
    qf = q.float().view(b, hkv, g, d)
    first = pool[table[0, :ns]].float()                       # [ns, hkv, 2, 16, d]
    rest = pool[table[:, ns:]].float()                        # [b, pages, hkv, 2, 16, d]
    kp, vp = first.permute(2, 1, 0, 3, 4).reshape(2, hkv, ns * PAGE, d)
    ko, vo = rest.permute(3, 0, 2, 1, 4, 5).reshape(2, b, hkv, -1, d)
    x1 = torch.matmul(qf.permute(1, 0, 2, 3).reshape(hkv, b * g, d), kp.transpose(1, 2))
    x1 = x1.view(hkv, b, g, -1).permute(1, 0, 2, 3)
    x = torch.cat([x1, torch.matmul(qf, ko.transpose(2, 3))], -1).mul_(1.0 / math.sqrt(d))
    bits = (s["mask"][table][:, :, None] >> torch.arange(PAGE, device=q.device)) & 1
    live = (bits != 0) & (torch.arange(table.shape[1], device=q.device) < s["n_pages"][:, None])[:, :, None]
    x.masked_fill_(~live.view(b, 1, 1, -1), -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    x.div_(x.sum(-1, keepdim=True))
    o1 = torch.matmul(x[..., :ns * PAGE].permute(1, 0, 2, 3).reshape(hkv, b * g, -1), vp)
    o = torch.matmul(x[..., ns * PAGE:], vo) + o1.view(hkv, b, g, d).permute(1, 0, 2, 3)
    if s["alpha"] is not None:
        s["alpha"].zero_()
        s["alpha"][:, :, ns * PAGE:] += x[..., ns * PAGE:].sum(2)
    return {"out": o.reshape(b, hq, d).to(q.dtype), "alpha": s["alpha"]}


def _plain_fork(s):
    table, mask, refs, pool, n = s["table"], s["mask"], s["refs"], s["pool"], s["n"]
    table.copy_(s["table0"]), mask.copy_(s["mask0"]), refs.copy_(s["refs0"])
    c = len(s["children"])
    row = table[0, :n].long()
    fresh = (mask[row] != 0xFFFF) & (torch.arange(n, device=row.device) == n - 1) if s["share"] else torch.ones_like(row, dtype=torch.bool)
    want = fresh.expand(c, n)
    rank = want.flatten().long().cumsum(0).view(c, n) - 1
    free = torch.nonzero(refs == 0).flatten()
    lacking = (want.sum() - free.numel()).clamp(min=0).to(torch.int32).view(1)
    rows = torch.where(want, free[rank.clamp(min=0)], row)
    pool[:, rows[want]] = pool[:, row.expand(c, n)[want]]
    mask[rows[want]] = mask[row.expand(c, n)[want]]
    refs.index_add_(0, rows.flatten(), torch.ones(c * n, dtype=torch.int32, device=row.device))
    table[1:, :n] = rows.to(torch.int32)
    forked = table.clone(), mask.clone(), refs.clone()
    refs.index_add_(0, rows.flatten(), torch.full((c * n,), -1, dtype=torch.int32, device=row.device))
    mask[rows.flatten()] = torch.where(refs[rows.flatten()] == 0, 0, mask[rows.flatten()])
    table[1:, :n] = -1
    return {"pool": pool, "forked": forked, "lacking": lacking, "bad": torch.zeros_like(lacking), "table": table, "mask": mask, "refs": refs}


def _plain_compact(s):
    pool, table, mask, refs, pos = s["pool"], s["table"], s["mask"], s["refs"], s["pos"]
    table.copy_(s["table0"]), mask.copy_(s["mask0"]), refs.copy_(s["refs0"]), pos.copy_(s["pos0"])
    b, width = table.shape
    slots = torch.arange(PAGE, device=table.device)
    ids = table.long().clamp(min=0)
    mine = s["in_row"] & (refs[ids] == 1)                         # pages of this sequence alone
    live = (((mask[ids][:, :, None] >> slots) & 1) != 0) & mine[:, :, None]
    keep = (live.sum((1, 2)) + PAGE - 1) // PAGE                  # pages its tokens need
    front = mine & (mine.long().cumsum(1) <= keep[:, None])
    tail = mine & ~front
    hole = (front[:, :, None] & ~live).view(b, -1)
    move = (tail[:, :, None] & live).view(b, -1)
    nth_hole = torch.where(hole, hole.long().cumsum(1) - 1, width * PAGE)
    by_rank = torch.zeros((b, width * PAGE + 1), dtype=torch.long, device=table.device)
    by_rank.scatter_(1, nth_hole, torch.arange(width * PAGE, device=table.device).expand(b, -1))
    row = torch.arange(b, device=table.device)[:, None].expand(b, width * PAGE)
    src = torch.arange(width * PAGE, device=table.device).expand(b, -1)[move]
    dst = by_rank.gather(1, (move.long().cumsum(1) - 1).clamp(min=0))[move]
    r = row[move]
    sp, ss, dp, ds = ids[r, src // PAGE], src % PAGE, ids[r, dst // PAGE], dst % PAGE
    pool[:, dp, :, :, ds] = pool[:, sp, :, :, ss]
    pos[dp, ds] = pos[sp, ss]
    mask.index_add_(0, dp, (1 << ds).to(torch.int32))
    gone = ids[tail]
    mask[gone] = 0
    refs[gone] = 0
    pos[gone] = -1
    stay = s["in_row"] & ~tail
    order = torch.argsort((~stay).long(), dim=1, stable=True)
    counts = stay.sum(1).to(torch.int32)
    table.copy_(torch.where(torch.arange(width, device=table.device) < counts[:, None], table.gather(1, order), -1))
    return {"pool": pool, "counts": counts, "table": table, "mask": mask, "refs": refs, "pos": pos}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "prompt":
        return _exact_prompt(case, prepare(case, seed))
    if case["op"] == "prefix":
        return _exact_prefix(case, prepare(case, seed))
    return None  # pages are moved, not computed


def _softmax64(x):
    e = torch.exp(x - x.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _exact_prompt(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["q_lens"], s["k_lens"]):
        for h in range(hq):
            k = s["k"][k0:k0 + nk, h // (hq // hkv)].double()
            v = s["v"][k0:k0 + nk, h // (hq // hkv)].double()
            for i in range(0, nq, 2048):
                q = s["q"][q0 + i:q0 + min(nq, i + 2048), h].double()
                seen = nk - nq + i + len(q)   # keys the last of these queries sees
                x = q @ k[:seen].T / math.sqrt(d)
                x += torch.full_like(x, -math.inf).triu(nk - nq + i + 1)
                out[q0 + i:q0 + i + len(q), h] = _softmax64(x) @ v[:seen]
        q0, k0 = q0 + nq, k0 + nk
    return out


def _exact_prefix(case, s):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    alpha = torch.zeros_like(s["alpha"], dtype=torch.float64) if s["alpha"] is not None else None
    for b, n in enumerate(s["counts"]):
        ids = s["table"][b, :n].long()
        at = torch.nonzero(((s["mask"][ids][:, None] >> torch.arange(PAGE, device="cuda")) & 1).flatten()).flatten()
        for h in range(hkv):
            kv = s["pool"][ids, h]            # [n, 2, 16, d]
            k, v = kv[:, 0].reshape(-1, d)[at].double(), kv[:, 1].reshape(-1, d)[at].double()
            p = _softmax64(s["q"][b].view(hkv, -1, d)[h].double() @ k.T / math.sqrt(d))
            out[b].view(hkv, -1, d)[h] = p @ v
            if alpha is not None:
                mine = at >= s["shared"] * PAGE
                alpha[b, h, at[mine]] = p.sum(0)[mine]
    return {"out": out, "alpha": alpha}


def work(case):
    esz = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "prompt":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        q_lens, cached = _ints(case["q_lens"]), _ints(case["cached"])
        pairs = sum(n * c + n * (n + 1) // 2 for n, c in zip(q_lens, cached))
        tq, tk = sum(q_lens), sum(q_lens) + sum(cached)
        return {"bytes": esz * d * (2 * tq * hq + 2 * tk * hkv), "flops": 4 * d * hq * pairs}
    if case["op"] == "prefix":
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        lens = _ints(case["own_lens"])
        tokens = case["shared"] + sum(lens)
        return {"bytes": esz * d * (2 * tokens * hkv + 2 * len(lens) * hq) + (8 * hkv * sum(lens) if case["alpha"] else 0),
                "flops": 4 * d * hq * (len(lens) * case["shared"] + sum(lens))}
    record = case["layers"] * case["hkv"] * 2 * PAGE * case["d"] * esz
    if case["op"] == "fork":
        n, c = -(-case["tokens"] // PAGE), case["children"]
        copied = c * n if not case["share"] else c if case["tokens"] % PAGE else 0
        read = min(copied, 1 if case["share"] else n)   # the parent's pages, once
        return {"bytes": record * (copied + read) + 4 * n * (1 + 4 * c), "flops": 0}
    lens, f = _ints(case["lens"]), case["evict"] / 100.0
    pages = sum(-(-n // PAGE) for n in lens)
    return {"bytes": 2 * record // PAGE * f * (1 - f) * sum(lens) + 4 * pages * (4 + PAGE), "flops": 0}
