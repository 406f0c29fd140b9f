"""Cases of the operators around the paged latent cache: batch tables from
request lengths, the gather of cached rows, the products with the kv_b weight
(expanded and absorbed forms) and the prompt attention of the expanded form.

``run`` makes the framework's calls when ``own`` is true, and computes the
same thing with elementary torch operations in 32 bits otherwise; ``exact``
gives the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

NOPE, ROPE, VDIM = 128, 64, 128
SM_SCALE = 1.0 / math.sqrt(NOPE + ROPE)
KV_SCALE = 0.05


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 running requests with 1024 to 4096 tokens each, one new token
        # each: what runs before every step, where only latency counts
        dict(name="batch_decode_step", op="batch", reqs=64, min_new=1, max_new=1, min_ctx=1024,
             max_ctx=4096, page=64, rows=100, pad=0, lens=1),
        # a mixed step of a large server: chunks of prompts and single tokens beside long
        # contexts in small pages, token rows padded for a captured graph
        dict(name="batch_mixed_large", op="batch", reqs=1000, min_new=1, max_new=200, min_ctx=0,
             max_ctx=65536, page=16, rows=1500, pad=777, lens=2),
        # cached prefixes of a few requests, E4M3 cache with the 256-wide latent, odd lengths
        dict(name="gather_e4m3_prefixes", op="gather", seqs=7, min_len=1, max_len=2500, rank=256,
             fmt="e4m3", page=64, lens=3),
        # long cached contexts taken out for the expanded form, bf16 cache
        dict(name="gather_bf16_long", op="gather", seqs=8, min_len=8192, max_len=32768, rank=512,
             fmt="bf16", page=64, lens=4),
        # the absorbed query of a decode step on one shard's heads: 64 requests, 16 heads
        dict(name="absorb_q_decode_shard", op="absorb_q", tokens=64, heads=16, rank=512),
        # values from the latent output of a decode step with all 128 heads
        dict(name="project_v_decode_full", op="project_v", tokens=128, heads=128, rank=512),
        # keys and values of a prompt chunk on one shard's heads
        dict(name="expand_kv_chunk_shard", op="expand_kv", tokens=8192, heads=16, rank=512),
        # keys and values of an odd number of tokens, all heads, 256-wide latent
        dict(name="expand_kv_full_r256", op="expand_kv", tokens=5001, heads=128, rank=256),
        # three short prompts, one of a single token: latency
        dict(name="prefill_short_ragged", op="prefill", seqs=3, min_q=1, max_q=150, min_ctx=0,
             max_ctx=0, heads=16, causal=True, lens=5),
        # one long prompt on one shard's heads
        dict(name="prefill_prompt_shard", op="prefill", seqs=1, min_q=8192, max_q=8192, min_ctx=0,
             max_ctx=0, heads=16, causal=True, lens=6),
        # chunks of prompts behind cached contexts, all heads
        dict(name="prefill_chunks_full", op="prefill", seqs=4, min_q=500, max_q=2048,
             min_ctx=0, max_ctx=8192, heads=128, causal=True, lens=7),
        # a few new tokens each against long contexts in the expanded form (speculated tokens, the
        # end of a prompt): few rows, a long key axis
        dict(name="prefill_few_rows_long", op="prefill", seqs=8, min_q=1, max_q=5, min_ctx=4096,
             max_ctx=32768, heads=16, causal=True, lens=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["batch", "gather", "absorb_q", "project_v", "expand_kv", "prefill",
                     "prefill"])
    lens = rng.randrange(1, 1 << 20)
    if op == "batch":
        mx = _log_int(rng, 1, 4096)
        ctx = _log_int(rng, 1, 65536)
        return dict(op=op, reqs=_log_int(rng, 1, 1000), min_new=rng.choice([0, 1]), max_new=mx,
                    min_ctx=rng.randrange(0, ctx), max_ctx=ctx, page=rng.choice([16, 32, 64, 128]),
                    rows=_log_int(rng, 1000, 1500), pad=rng.choice([0, 1, 500]), lens=lens)
    if op == "gather":
        mx = _log_int(rng, 1, 32768)
        return dict(op=op, seqs=_log_int(rng, 1, 64), min_len=rng.choice([0, 1, max(1, mx // 2)]),
                    max_len=mx, rank=rng.choice([256, 512]),
                    fmt=rng.choice(["bf16", "e4m3", "e5m2"]), page=rng.choice([16, 32, 64, 128, 256]),
                    lens=lens)
    if op in ("absorb_q", "project_v", "expand_kv"):
        return dict(op=op, tokens=_log_int(rng, 1, 8192), heads=rng.choice([1, 7, 16, 32, 64, 128]),
                    rank=rng.choice([256, 512]))
    mq = _log_int(rng, 1, 8192)
    ctx = rng.choice([0, _log_int(rng, 1, 32768)])
    return dict(op=op, seqs=_log_int(rng, 1, 16), min_q=rng.choice([0, 1, max(1, mq // 2)]),
                max_q=mq, min_ctx=rng.randrange(0, ctx + 1), max_ctx=ctx,
                heads=rng.choice([1, 5, 16, 32, 64, 128]), causal=rng.random() < 0.7, lens=lens)


def draw(rng):
    top = [work(c) for c in listed()]
    max_b, max_f = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        c = _draw_once(rng)
        w = work(c)
        empty = w["bytes"] == 0 or (c["op"] == "prefill" and w["flops"] == 0) or (
            c["op"] == "batch" and sum(_batch_lens(c)[0]) == 0)
        if not empty and w["bytes"] <= max_b and w["flops"] <= max_f:
            return c


def _lengths(n, lo, hi, seed):
    r = random.Random(seed)
    return [r.randint(lo, hi) for _ in range(n)]


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _cdiv(a, b):
    return -(-a // b)


def _batch_lens(c):
    new = _lengths(c["reqs"], c["min_new"], c["max_new"], c["lens"])
    ctx = _lengths(c["reqs"], c["min_ctx"], c["max_ctx"], c["lens"] + 1)
    if c["max_new"] > 1:  # every other request decodes one token
        new = [1 if i % 2 else x for i, x in enumerate(new)]
    return new, ctx


def _prefill_lens(c):
    lq = _lengths(c["seqs"], c["min_q"], c["max_q"], c["lens"])
    ctx = _lengths(c["seqs"], c["min_ctx"], c["max_ctx"], c["lens"] + 1)
    return lq, [a + b for a, b in zip(lq, ctx)]


def work(c):
    op = c["op"]
    if op == "batch":
        new, ctx = _batch_lens(c)
        seq = [a + b for a, b in zip(new, ctx)]
        old_pages = sum(_cdiv(x, c["page"]) for x in ctx)
        pages = sum(_cdiv(x, c["page"]) for x in seq)
        tokens = sum(new) + c["pad"]
        # lengths and ids in; old pages read, new ones read from the free list and written to
        # the requests' table, all written to the batch's; lengths, sums, positions, slots out
        b = 12 * c["reqs"] + 4 * pages + 4 * (pages - old_pages) + 4 * pages \
            + 12 * c["reqs"] + 16 * tokens
        return {"bytes": b, "flops": 0}
    if op == "gather":
        t = sum(_lengths(c["seqs"], c["min_len"], c["max_len"], c["lens"]))
        elt = 2 if c["fmt"] == "bf16" else 1
        return {"bytes": t * (c["rank"] + ROPE) * (elt + 2), "flops": 0}
    if op in ("absorb_q", "project_v", "expand_kv"):
        t, h, r = c["tokens"], c["heads"], c["rank"]
        if op == "expand_kv":
            return {"bytes": 2 * (t * r + h * (NOPE + VDIM) * r + t * h * (NOPE + VDIM)),
                    "flops": 2 * t * h * (NOPE + VDIM) * r}
        d = NOPE if op == "absorb_q" else VDIM
        return {"bytes": 2 * (t * h * d + h * d * r + t * h * r), "flops": 2 * t * h * d * r}
    lq, lk = _prefill_lens(c)
    tq, tk, h = sum(lq), sum(lk), c["heads"]
    pairs = 0
    for a, b in zip(lq, lk):
        pairs += a * b - (a * (a - 1) // 2 if c["causal"] else 0)
    return {"bytes": 2 * (tq * h * (NOPE + ROPE) + tk * h * (NOPE + VDIM) + tk * ROPE
                          + tq * h * VDIM) + 4 * tq * h,
            "flops": 2 * (NOPE + ROPE + VDIM) * pairs * h}


# ----------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    out = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        n = min(step, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device="cuda") * scale
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def prepare(case, seed):
    c = dict(case)
    g = _gen(seed)
    s = {"case": c}
    op = c["op"]
    if op == "batch":
        new, ctx = _batch_lens(c)
        bs = c["page"]
        old = [_cdiv(x, bs) for x in ctx]
        pages = [_cdiv(a + b, bs) for a, b in zip(new, ctx)]
        maxb = _cdiv(c["max_ctx"] + c["max_new"], bs)
        num_blocks = sum(pages) + 1000
        ids = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
        rows = torch.randperm(c["rows"], generator=g, device="cuda")[:c["reqs"]].to(torch.int32)
        table = torch.full((c["rows"], maxb), -1, dtype=torch.int32, device="cuda")
        n_old = _i32(old).long()
        at = torch.arange(sum(old), device="cuda")
        row_of = torch.repeat_interleave(torch.arange(len(old), device="cuda"), n_old)
        col = at - (torch.cumsum(n_old, 0) - n_old)[row_of]
        table[rows.long()[row_of], col] = ids[:sum(old)]
        free = ids[sum(old):].contiguous()
        tokens = sum(new) + c["pad"]
        s.update(new=_i32(new), ctx=_i32(ctx), rows=rows, table=table, free=free,
                 count=_i32([free.numel()]), page=bs, num_blocks=num_blocks, tokens=tokens,
                 total=sum(new), maxb=maxb)
        B = c["reqs"]
        s["out"] = dict(
            block_table=torch.full((B, maxb), -1, dtype=torch.int32, device="cuda"),
            seq_lens=torch.empty(B, dtype=torch.int32, device="cuda"),
            cu_seqlens_q=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
            cu_seqlens_k=torch.empty(B + 1, dtype=torch.int32, device="cuda"),
            positions=torch.empty(tokens, dtype=torch.int64, device="cuda"),
            slot_mapping=torch.empty(tokens, dtype=torch.int64, device="cuda"),
            free_count_out=torch.empty(1, dtype=torch.int32, device="cuda"))
    elif op == "gather":
        lens = _lengths(c["seqs"], c["min_len"], c["max_len"], c["lens"])
        bs, d = c["page"], c["rank"] + ROPE
        pages = [_cdiv(x, bs) for x in lens]
        num_blocks = sum(pages) + 17
        maxb = max(1, max(pages))
        perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(c["seqs"], maxb, dtype=torch.int32, device="cuda")
        a = 0
        for b, n in enumerate(pages):
            table[b, :n] = perm[a:a + n]
            a += n
        cache = _normal(g, num_blocks, bs, d)
        if c["fmt"] != "bf16":
            flat = cache.view(-1)
            codes = torch.empty(flat.numel(), dtype=_FP8[c["fmt"]], device="cuda")
            step = 1 << 28
            for a in range(0, flat.numel(), step):
                codes[a:a + step] = (flat[a:a + step].float() / KV_SCALE).to(_FP8[c["fmt"]])
            cache = codes.view(num_blocks, bs, d)
        s.update(cache=cache, table=table, cu=_i32(_cu(lens)), tokens=sum(lens), lens=lens,
                 scale=torch.tensor([KV_SCALE], dtype=torch.float32, device="cuda"),
                 rank=c["rank"], page=bs)
    elif op in ("absorb_q", "project_v", "expand_kv"):
        t, h, r = c["tokens"], c["heads"], c["rank"]
        s["w"] = _normal(g, h * (NOPE + VDIM), r, scale=1.0 / math.sqrt(r))
        if op == "expand_kv":
            s["x"] = _normal(g, t, r)
        elif op == "absorb_q":
            # the nope columns of the projected query [t, h, nope + rope]
            s["x"] = _normal(g, t, h, NOPE + ROPE)[:, :, :NOPE]
        else:
            s["x"] = _normal(g, t, h, r, scale=0.3)
        s["heads"], s["rank"] = h, r
    else:
        lq, lk = _prefill_lens(c)
        tq, tk, h = sum(lq), sum(lk), c["heads"]
        s["q"] = _normal(g, tq, h, NOPE + ROPE)
        kv = _normal(g, tk, h, NOPE + VDIM)  # one buffer, keys and values side by side
        s["k"], s["v"] = kv[:, :, :NOPE], kv[:, :, NOPE:]
        s["k_pe"] = _normal(g, tk, ROPE)
        s["cu_q"], s["cu_k"] = _i32(_cu(lq)), _i32(_cu(lk))
        s["lq"], s["lk"], s["causal"] = lq, lk, c["causal"]
        s["sms"] = torch.cuda.get_device_properties(0).multi_processor_count
    return s


# -------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _own_batch(s):
    import mla_paged_kv_concat_gb300 as mla
    o = s["out"]
    mla.batch_build(s["new"], s["ctx"], s["table"], s["free"], s["count"], s["page"],
                    s["num_blocks"], req_ids=s["rows"], **o)
    return [o["block_table"], s["table"], o["seq_lens"], o["cu_seqlens_q"], o["cu_seqlens_k"],
            o["positions"], o["slot_mapping"], o["free_count_out"]]


def _plain_batch(s):
    o, bs = s["out"], s["page"]
    new, ctx, rows = s["new"].long(), s["ctx"].long(), s["rows"].long()
    B = new.numel()
    dev = new.device
    seq = new + ctx
    old, pages = (ctx + bs - 1) // bs, (seq + bs - 1) // bs
    add = pages - old
    off = torch.cumsum(add, 0) - add
    col = torch.arange(s["maxb"], device=dev)[None, :]
    src = s["count"].long() - 1 - (off[:, None] + col - old[:, None])
    fresh = s["free"][src.clamp(0, max(s["free"].numel() - 1, 0))]
    here = s["table"][rows]
    is_new = (col >= old[:, None]) & (col < pages[:, None])
    here = torch.where(is_new, fresh, here)
    s["table"][rows] = here
    o["block_table"].copy_(torch.where(col < pages[:, None], here, o["block_table"]))
    o["seq_lens"].copy_(seq)
    for name, x in (("cu_seqlens_q", new), ("cu_seqlens_k", seq)):
        o[name][0] = 0
        o[name][1:] = torch.cumsum(x, 0)
    cu = torch.cumsum(new, 0)
    t = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(cu, t, right=True).clamp(max=B - 1)
    pos = ctx[b] + t - (cu - new)[b]
    real = t < cu[-1]
    pos = torch.where(real, pos, torch.zeros_like(pos))
    slot = here[b, pos // bs].long() * bs + pos % bs
    o["positions"].copy_(pos)
    o["slot_mapping"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    o["free_count_out"].copy_(s["count"] - add.sum().to(torch.int32))
    return [o["block_table"], s["table"], o["seq_lens"], o["cu_seqlens_q"], o["cu_seqlens_k"],
            o["positions"], o["slot_mapping"], o["free_count_out"]]


def _own_gather(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.gather_cache(s["cache"], s["table"], s["cu"], s["tokens"],
                            kv_lora_rank=s["rank"],
                            kv_scale=None if s["cache"].dtype == torch.bfloat16 else s["scale"])


def _plain_gather(s):
    bs, r = s["page"], s["rank"]
    t = torch.arange(s["tokens"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = t - cu[b]
    rows = s["cache"].view(-1, r + ROPE)[s["table"][b, pos // bs].long() * bs + pos % bs] \
        if s["cache"].dtype == torch.bfloat16 else \
        s["cache"].view(torch.uint8).view(-1, r + ROPE)[
            s["table"][b, pos // bs].long() * bs + pos % bs].view(s["cache"].dtype)
    if s["cache"].dtype != torch.bfloat16:
        rows = (rows.float() * s["scale"]).to(torch.bfloat16)
    return rows[:, :r].contiguous(), rows[:, r:].contiguous()


def _weights(s, dtype):
    w = s["w"].to(dtype).view(s["heads"], NOPE + VDIM, s["rank"])
    return w[:, :NOPE], w[:, NOPE:]


def _own_expand(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.expand_kv(s["x"], s["w"], s["heads"])


def _plain_expand(s):
    y = (s["x"].float() @ s["w"].float().t()).to(torch.bfloat16)
    y = y.view(-1, s["heads"], NOPE + VDIM)
    return y[:, :, :NOPE], y[:, :, NOPE:]


def _own_absorb(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.absorb_q(s["x"], s["w"])


def _plain_absorb(s):
    wk, _ = _weights(s, torch.float32)
    y = torch.matmul(s["x"].float().transpose(0, 1), wk)  # [h, t, r]
    return y.transpose(0, 1).to(torch.bfloat16).contiguous()


def _own_project(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.project_v(s["x"], s["w"])


def _plain_project(s):
    _, wv = _weights(s, torch.float32)
    y = torch.matmul(s["x"].float().transpose(0, 1), wv.transpose(1, 2))
    return y.transpose(0, 1).to(torch.bfloat16).contiguous()


def _own_prefill(s):
    import mla_paged_kv_concat_gb300 as mla
    tq, h, _ = s["q"].shape
    n = mla.mla_prefill_num_kv_splits(tq, len(s["lq"]), h, max(s["lk"]), s["sms"])
    return mla.prefill(s["q"], s["k"], s["v"], s["k_pe"], s["cu_q"], s["cu_k"], SM_SCALE,
                       causal=s["causal"], num_kv_splits=n)


def _plain_prefill(s):
    tq, h, _ = s["q"].shape
    o = torch.empty(tq, h, VDIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(tq, h, dtype=torch.float32, device="cuda")
    a = b = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        if lq > 0:
            step = max(1, min(h, (1 << 29) // max(1, lq * lk)))
            for h0 in range(0, h, step):
                hh = slice(h0, min(h, h0 + step))
                n = hh.stop - hh.start
                k = torch.cat([s["k"][b:b + lk, hh].float(),
                               s["k_pe"][b:b + lk, None].float().expand(lk, n, ROPE)], 2)
                q = s["q"][a:a + lq, hh].float().transpose(0, 1)
                x = torch.matmul(q, k.permute(1, 2, 0)) * SM_SCALE
                if s["causal"]:
                    i = torch.arange(lq, device="cuda")[:, None]
                    j = torch.arange(lk, device="cuda")[None, :]
                    x = x.masked_fill_(j > i + (lk - lq), -math.inf)
                m = x.amax(-1, keepdim=True) if lk else x.new_full((n, lq, 1), -math.inf)
                m = torch.where(m == -math.inf, torch.zeros_like(m), m)
                p = x.sub_(m).exp_()
                z = p.sum(-1, keepdim=True)
                y = torch.matmul(p, s["v"][b:b + lk, hh].float().transpose(0, 1))
                y = torch.where(z > 0, y / z, torch.zeros_like(y))
                o[a:a + lq, hh] = y.transpose(0, 1).to(torch.bfloat16)
                lse[a:a + lq, hh] = (m + z.log())[..., 0].transpose(0, 1)
        a += lq
        b += lk
    return o, lse


_own = dict(batch=_own_batch, gather=_own_gather, expand_kv=_own_expand, absorb_q=_own_absorb,
            project_v=_own_project, prefill=_own_prefill)
_plain = dict(batch=_plain_batch, gather=_plain_gather, expand_kv=_plain_expand,
              absorb_q=_plain_absorb, project_v=_plain_project, prefill=_plain_prefill)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "batch":
        return _exact_batch(s)
    if op == "gather":
        return _exact_gather(s)
    if op == "prefill":
        return _exact_prefill(s)
    w = s["w"].double().view(s["heads"], NOPE + VDIM, s["rank"])
    x = s["x"].double()
    if op == "expand_kv":
        k = torch.empty(x.shape[0], s["heads"], NOPE, dtype=torch.float64, device="cuda")
        v = torch.empty(x.shape[0], s["heads"], VDIM, dtype=torch.float64, device="cuda")
        for h in range(s["heads"]):
            k[:, h] = x @ w[h, :NOPE].t()
            v[:, h] = x @ w[h, NOPE:].t()
        return k, v
    n = s["rank"] if op == "absorb_q" else VDIM
    y = torch.empty(x.shape[0], s["heads"], n, dtype=torch.float64, device="cuda")
    for h in range(s["heads"]):
        y[:, h] = x[:, h] @ (w[h, :NOPE] if op == "absorb_q" else w[h, NOPE:].t())
    return y


def _exact_batch(s):
    bs = s["page"]
    new, ctx = s["new"].cpu().numpy(), s["ctx"].cpu().numpy()
    rows, free = s["rows"].cpu().numpy(), s["free"].cpu().numpy()
    table = s["table"].cpu().numpy().copy()
    bt = s["out"]["block_table"].cpu().numpy().copy()
    top = int(s["count"].item())
    pos = np.zeros(s["tokens"], np.int64)
    slot = np.full(s["tokens"], -1, np.int64)
    t = 0
    for b in range(len(new)):
        n, c = int(new[b]), int(ctx[b])
        for page in range(_cdiv(c, bs), _cdiv(c + n, bs)):
            top -= 1
            table[rows[b], page] = free[top]
        m = _cdiv(c + n, bs)
        bt[b, :m] = table[rows[b], :m]
        p = np.arange(c, c + n)
        pos[t:t + n] = p
        slot[t:t + n] = bt[b, p // bs].astype(np.int64) * bs + p % bs
        t += n
    return [bt, table, (new + ctx).astype(np.int32), np.asarray(_cu(new.tolist()), np.int32),
            np.asarray(_cu((new + ctx).tolist()), np.int32), pos, slot,
            np.asarray([top], np.int32)]


def _exact_gather(s):
    bs, r = s["page"], s["rank"]
    out = torch.empty(s["tokens"], r + ROPE, dtype=torch.float64, device="cuda")
    t = 0
    for b, n in enumerate(s["lens"]):
        for page in range(_cdiv(n, bs)):
            m = min(bs, n - page * bs)
            blk = s["cache"][int(s["table"][b, page].item())][:m]
            out[t:t + m] = blk.to(torch.float32).double()
            t += m
    if s["cache"].dtype != torch.bfloat16:
        out *= s["scale"].double()
    return out[:, :r].contiguous(), out[:, r:].contiguous()


def _exact_prefill(s):
    tq, h, _ = s["q"].shape
    o = torch.zeros(tq, h, VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full((tq, h), -math.inf, dtype=torch.float64, device="cuda")
    a = b = 0
    for lq, lk in zip(s["lq"], s["lk"]):
        rows = max(1, (1 << 27) // max(1, lk))
        for head in range(h):
            k = s["k"][b:b + lk, head].double()
            kp = s["k_pe"][b:b + lk].double()
            v = s["v"][b:b + lk, head].double()
            for i0 in range(0, lq, rows):
                i1 = min(lq, i0 + rows)
                q = s["q"][a + i0:a + i1, head].double()
                last = min(lk, i1 + lk - lq) if s["causal"] else lk
                if last <= 0:
                    continue
                x = (q[:, :NOPE] @ k[:last].t() + q[:, NOPE:] @ kp[:last].t()) * SM_SCALE
                if s["causal"]:
                    lim = torch.arange(i0, i1, device="cuda")[:, None] + (lk - lq)
                    x[torch.arange(last, device="cuda")[None, :] > lim] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[a + i0:a + i1, head] = z
                p = torch.exp(x - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
                o[a + i0:a + i1, head] = p @ v[:last]
        a += lq
        b += lk
    return o, lse
