"""Cases of the operators for a batch that shares a long prefix, and of the
layer's projections: attention over the paged latent cache with the prefix's
rows read once for all sequences (absorbed form, single tokens), attention of
the expanded form behind a shared prefix (prompts), and the matrix product with
bias, activation and residual in its epilogue.

``run`` makes the framework's calls when ``own`` is true, and computes the
same thing with elementary torch operations in 32 bits otherwise; ``exact``
gives the definition in 64 bits.
"""
import math
import random

import torch

own = False

NOPE, ROPE, VDIM = 128, 64, 128
SM_SCALE = 1.0 / math.sqrt(NOPE + ROPE)
KV_SCALE = 0.05
_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of users behind a short system prompt, a few own tokens each: latency
        dict(name="decode_shared_small", op="decode", groups=1, seqs=4, rows=1, heads=16, rank=512,
             fmt="bf16", page=64, min_prefix=512, max_prefix=512, min_own=1, max_own=64, pad=0,
             lens=1),
        # a decode step of 64 requests on one shard's heads, a long common prompt
        dict(name="decode_shared_shard", op="decode", groups=1, seqs=64, rows=1, heads=16,
             rank=512, fmt="bf16", page=64, min_prefix=8192, max_prefix=8192, min_own=64,
             max_own=1024, pad=0, lens=2),
        # E4M3 cache with the 256-wide latent, odd prefix, graph rows without a request at the end
        dict(name="decode_shared_e4m3_r256", op="decode", groups=2, seqs=45, rows=1, heads=32,
             rank=256, fmt="e4m3", page=64, min_prefix=3001, max_prefix=9001, min_own=1,
             max_own=2000, pad=3, lens=3),
        # two speculated tokens a request, E5M2 cache, small pages
        dict(name="decode_shared_e5m2_rows", op="decode", groups=1, seqs=33, rows=2, heads=16,
             rank=512, fmt="e5m2", page=16, min_prefix=4097, max_prefix=4097, min_own=1,
             max_own=700, pad=0, lens=4),
        # a large server with all 128 heads and three system prompts
        dict(name="decode_shared_full", op="decode", groups=3, seqs=128, rows=1, heads=128,
             rank=512, fmt="bf16", page=64, min_prefix=4096, max_prefix=16384, min_own=0,
             max_own=2048, pad=0, lens=5),
        # three short questions on a document, one shard's heads: latency
        dict(name="prefill_shared_small", op="prefill", groups=1, seqs=3, min_q=1, max_q=40,
             min_ctx=0, max_ctx=0, min_prefix=700, max_prefix=700, heads=16, causal=True, lens=6),
        # many short questions behind a long prompt
        dict(name="prefill_shared_questions", op="prefill", groups=1, seqs=48, min_q=5, max_q=90,
             min_ctx=0, max_ctx=0, min_prefix=8192, max_prefix=8192, heads=16, causal=True,
             lens=7),
        # long prompts and chunks with contexts of their own behind two shared documents, 32 heads
        dict(name="prefill_shared_prompts", op="prefill", groups=2, seqs=8, min_q=500, max_q=1500,
             min_ctx=0, max_ctx=1000, min_prefix=4000, max_prefix=8192, heads=32, causal=True,
             lens=8),
        # the output projection of a decode step on one shard's heads, added to the residual stream
        dict(name="linear_out_decode", op="linear", tokens=64, k=2048, n=5120, bias=False,
             act=None, residual=True),
        # one token through a wide layer: the weight is the work
        dict(name="linear_one_token", op="linear", tokens=1, k=8192, n=7168, bias=True, act=None,
             residual=True),
        # an odd number of tokens through a projection with bias and activation
        dict(name="linear_silu_odd", op="linear", tokens=1001, k=1536, n=6136, bias=True,
             act="silu", residual=False),
        # a prompt chunk's output projection with all 128 heads
        dict(name="linear_out_prompt", op="linear", tokens=8192, k=16384, n=5120, bias=True,
             act=None, residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["decode", "decode", "prefill", "linear"])
    lens = rng.randrange(1, 1 << 20)
    if op == "linear":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), k=8 * _log_int(rng, 8, 2048),
                    n=8 * _log_int(rng, 8, 2048), bias=rng.random() < 0.5,
                    act=rng.choice([None, "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.random() < 0.5)
    groups = rng.choice([1, 1, 2, 3])
    top = _log_int(rng, 16, 32768)
    if op == "decode":
        return dict(op=op, groups=groups, seqs=max(groups, _log_int(rng, 1, 256)),
                    rows=rng.choice([1, 1, 1, 2, 4]), heads=rng.choice([1, 5, 16, 16, 32, 64, 128]),
                    rank=rng.choice([256, 512, 512]), fmt=rng.choice(["bf16", "bf16", "e4m3", "e5m2"]),
                    page=rng.choice([16, 32, 64, 128, 256]),
                    min_prefix=rng.choice([top, max(1, top // 3)]), max_prefix=top,
                    min_own=rng.choice([0, 1]), max_own=_log_int(rng, 1, 4096),
                    pad=rng.choice([0, 0, 1, 5]), lens=lens)
    ctx = rng.choice([0, _log_int(rng, 1, 2048)])
    return dict(op=op, groups=groups, seqs=max(groups, _log_int(rng, 1, 64)),
                min_q=rng.choice([0, 1]), max_q=_log_int(rng, 1, 2048), min_ctx=0, max_ctx=ctx,
                min_prefix=rng.choice([top, max(1, top // 3)]), max_prefix=top,
                heads=rng.choice([1, 5, 16, 32, 64, 128]), causal=rng.random() < 0.8, lens=lens)


def draw(rng):
    top = [work(c) for c in listed()]
    max_b, max_f = max(w["bytes"] for w in top), max(w["flops"] for w in top)
    while True:
        c = _draw_once(rng)
        w = work(c)
        if 0 < w["bytes"] <= max_b and 0 < w["flops"] <= max_f:
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


def _groups(c):
    """First sequence of each group and the end: groups as equal as they can be."""
    return [c["seqs"] * g // c["groups"] for g in range(c["groups"] + 1)]


def _prefixes(c):
    return _lengths(c["groups"], c["min_prefix"], c["max_prefix"], c["lens"] + 2)


def _owns(c):
    return _lengths(c["seqs"], c["min_own"], c["max_own"], c["lens"])


def _prompt_lens(c):
    lq = _lengths(c["seqs"], c["min_q"], c["max_q"], c["lens"])
    ctx = _lengths(c["seqs"], c["min_ctx"], c["max_ctx"], c["lens"] + 1)
    return lq, [a + b for a, b in zip(lq, ctx)]


def work(c):
    if c["op"] == "linear":
        t, k, n = c["tokens"], c["k"], c["n"]
        return {"bytes": 2 * (t * k + n * k + t * n * (2 if c["residual"] else 1)
                              + (n if c["bias"] else 0)),
                "flops": 2 * t * n * k}
    gs, pre, h = _groups(c), _prefixes(c), c["heads"]
    if c["op"] == "decode":
        r, d, own_ = c["rank"], c["rank"] + ROPE, _owns(c)
        elt = 2 if c["fmt"] == "bf16" else 1
        vecs = (c["seqs"] + c["pad"]) * c["rows"] * h
        keys = sum(own_) + sum((gs[g + 1] - gs[g]) * pre[g] for g in range(c["groups"]))
        return {"bytes": vecs * d * 2 + (sum(own_) + sum(pre)) * d * elt + vecs * (2 * r + 4),
                "flops": 2 * (r + d) * c["rows"] * h * keys}
    lq, lk = _prompt_lens(c)
    tq, tk = sum(lq), sum(lk) + sum(pre)
    pairs = sum(sum(lq[gs[g]:gs[g + 1]]) * pre[g] for g in range(c["groups"]))
    for a, b in zip(lq, lk):
        pairs += a * b - (a * (a - 1) // 2 if c["causal"] else 0)
    return {"bytes": 2 * (tq * h * (NOPE + ROPE + VDIM) + tk * (h * (NOPE + VDIM) + ROPE))
            + 4 * tq * h,
            "flops": 2 * (NOPE + ROPE + VDIM) * pairs * h}


# ----------------------------------------------------------------- inputs
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


def _prepare_decode(c, g, s):
    bs, d = c["page"], c["rank"] + ROPE
    gs, pre, own_ = _groups(c), _prefixes(c), _owns(c)
    B, pad = c["seqs"], c["pad"]
    # a group's whole pages of the prefix are the same ones in every table; the page that the
    # prefix ends in is each sequence's own copy, which its own tokens go on in
    shared = [p // bs for p in pre]
    group = [i for i in range(c["groups"]) for _ in range(gs[i + 1] - gs[i])]
    lens = [pre[group[b]] + own_[b] for b in range(B)]
    mine = [_cdiv(lens[b], bs) - shared[group[b]] for b in range(B)]
    num_blocks = sum(shared) + sum(mine) + 17
    maxb = max(1, max(_cdiv(x, bs) for x in lens))
    perm = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(B + pad, maxb, dtype=torch.int32, device="cuda")
    cache = _normal(g, num_blocks, bs, d)
    at = sum(shared)
    first = _cu(shared)
    for b in range(B):
        i, n = group[b], shared[group[b]]
        table[b, :n] = perm[first[i]:first[i] + n]
        table[b, n:n + mine[b]] = perm[at:at + mine[b]]
        tail = pre[i] % bs
        if tail and b > gs[i]:
            cache[perm[at].long(), :tail] = cache[table[gs[i], n].long(), :tail]
        at += mine[b]
    if c["fmt"] != "bf16":
        flat = cache.view(-1)
        codes = torch.empty(flat.numel(), dtype=_FP8[c["fmt"]], device="cuda")
        step = 1 << 28
        for a in range(0, flat.numel(), step):
            codes[a:a + step] = (flat[a:a + step].float() / KV_SCALE).to(_FP8[c["fmt"]])
        cache = codes.view(num_blocks, bs, d)
        s["scale"] = torch.tensor([KV_SCALE], dtype=torch.float32, device="cuda")
    else:
        s["scale"] = None
    ends = gs[:-1] + [B + pad]  # rows without a request belong to the last group
    s.update(cache=cache, table=table, lens=lens + [0] * pad, group_list=gs, pre=pre,
             seq_lens=_i32(lens + [0] * pad), group_seqs=_i32(ends), prefix_lens=_i32(pre),
             q=_normal(g, (B + pad) * c["rows"], c["heads"], d), rank=c["rank"], page=bs,
             rows=c["rows"])


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "linear":
        t, k, n = c["tokens"], c["k"], c["n"]
        s["x"] = _normal(g, t, k)
        s["w"] = _normal(g, n, k, scale=1.0 / math.sqrt(k))
        s["bias"] = _normal(g, n) if c["bias"] else None
        s["residual"] = _normal(g, t, n) if c["residual"] else None
    elif c["op"] == "decode":
        _prepare_decode(c, g, s)
    else:
        gs, pre = _groups(c), _prefixes(c)
        lq, lk = _prompt_lens(c)
        tq, tp, h = sum(lq), sum(pre), c["heads"]
        tk = tp + sum(lk)
        s["q"] = _normal(g, tq, h, NOPE + ROPE)
        kv = _normal(g, tk, h, NOPE + VDIM)  # the prefixes' keys and values, then the sequences'
        s["k"], s["v"] = kv[:, :, :NOPE], kv[:, :, NOPE:]
        s["k_pe"] = _normal(g, tk, ROPE)
        s["cu_q"], s["cu_k"] = _i32(_cu(lq)), _i32([tp + x for x in _cu(lk)])
        s["group_seqs"], s["cu_prefix"] = _i32(gs), _i32(_cu(pre))
        s["lq"], s["lk"], s["pre"], s["group_list"] = lq, lk, pre, gs
        s["causal"] = c["causal"]
        s["sms"] = torch.cuda.get_device_properties(0).multi_processor_count
    return s


# -------------------------------------------------------------------- run
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _own_linear(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.linear(s["x"], s["w"], bias=s["bias"], activation=s["case"]["act"],
                      residual=s["residual"])


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y += s["bias"].float()
    act = s["case"]["act"]
    if act == "relu":
        y = y.clamp_(min=0)
    elif act == "silu":
        y = y / (1 + torch.exp(-y))
    elif act == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif act == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


def _own_decode(s):
    import mla_paged_kv_concat_gb300 as mla
    return mla.decode_shared(s["q"], s["cache"], s["table"], s["seq_lens"], s["group_seqs"],
                             s["prefix_lens"], SM_SCALE, kv_lora_rank=s["rank"],
                             kv_scale=s["scale"])


def _cache_rows(s, row, n, dtype):
    """The first ``n`` cached tokens of table row ``row``."""
    blocks = s["table"][row, :_cdiv(n, s["page"])].long()
    cache = s["cache"]
    if cache.dtype == torch.bfloat16:
        return cache[blocks].reshape(-1, cache.shape[2])[:n].to(dtype)
    x = cache.view(torch.uint8)[blocks].reshape(-1, cache.shape[2])[:n].view(cache.dtype)
    return x.to(torch.float32).to(dtype) * s["scale"].to(dtype)


def _plain_decode(s):
    T, h, _ = s["q"].shape
    r, rows = s["rank"], s["rows"]
    o = torch.zeros(T, h, r, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, h), -math.inf, dtype=torch.float32, device="cuda")
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        k = _cache_rows(s, b, n, torch.float32)
        a = slice(b * rows, (b + 1) * rows)
        x = (s["q"][a].float().view(rows * h, -1) @ k.t()) * SM_SCALE
        m = x.amax(1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(1, keepdim=True)
        o[a] = ((p @ k[:, :r]) / z).view(rows, h, r).to(torch.bfloat16)
        lse[a] = (m + z.log()).view(rows, h)
    return o, lse


def _own_prefill(s):
    import mla_paged_kv_concat_gb300 as mla
    tq, h, _ = s["q"].shape
    n = mla.mla_prefill_shared_num_kv_splits(tq, len(s["lq"]), len(s["pre"]), h, max(s["pre"]),
                                             max(s["lk"]), s["sms"])
    return mla.prefill_shared(s["q"], s["k"], s["v"], s["k_pe"], s["cu_q"], s["cu_k"],
                              s["group_seqs"], s["cu_prefix"], SM_SCALE, causal=s["causal"],
                              num_kv_splits=n)


def _plain_prefill(s):
    tq, h, _ = s["q"].shape
    o = torch.zeros(tq, h, VDIM, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((tq, h), -math.inf, dtype=torch.float32, device="cuda")
    a, b, p0 = 0, sum(s["pre"]), 0
    for g, lp in enumerate(s["pre"]):
        for i in range(s["group_list"][g], s["group_list"][g + 1]):
            lq, lk = s["lq"][i], s["lk"][i]
            if lq > 0:
                n = lp + lk
                step = max(1, min(h, (1 << 29) // max(1, lq * n)))
                keep = None
                if s["causal"]:
                    iq = torch.arange(lq, device="cuda")[:, None]
                    keep = torch.arange(n, device="cuda")[None, :] <= iq + (n - lq)
                for h0 in range(0, h, step):
                    hh = slice(h0, min(h, h0 + step))
                    k = torch.cat([s["k"][p0:p0 + lp, hh], s["k"][b:b + lk, hh]]).float()
                    v = torch.cat([s["v"][p0:p0 + lp, hh], s["v"][b:b + lk, hh]]).float()
                    kp = torch.cat([s["k_pe"][p0:p0 + lp], s["k_pe"][b:b + lk]]).float()
                    q = s["q"][a:a + lq, hh].float().transpose(0, 1)
                    x = torch.matmul(q[..., :NOPE], k.permute(1, 2, 0))
                    x += torch.matmul(q[..., NOPE:], kp.t())
                    x *= SM_SCALE
                    if keep is not None:
                        x.masked_fill_(~keep, -math.inf)
                    m = x.amax(-1, keepdim=True)
                    p = x.sub_(m).exp_()
                    z = p.sum(-1, keepdim=True)
                    y = torch.matmul(p, v.transpose(0, 1)) / z
                    o[a:a + lq, hh] = y.transpose(0, 1).to(torch.bfloat16)
                    lse[a:a + lq, hh] = (m + z.log())[..., 0].transpose(0, 1)
            a += lq
            b += lk
        p0 += lp
    return o, lse


_own = dict(linear=_own_linear, decode=_own_decode, prefill=_own_prefill)
_plain = dict(linear=_plain_linear, decode=_plain_decode, prefill=_plain_prefill)


# ------------------------------------------------------------------ exact
def exact(case, seed):
    s = prepare(case, seed)
    return dict(linear=_exact_linear, decode=_exact_decode, prefill=_exact_prefill)[case["op"]](s)


def _exact_linear(s):
    w = s["w"].double()
    out = torch.empty(s["x"].shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for a in range(0, out.shape[0], 1024):
        y = s["x"][a:a + 1024].double() @ w.t()
        if s["bias"] is not None:
            y = y + s["bias"].double()
        act = s["case"]["act"]
        if act == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        elif act == "silu":
            y = y * torch.sigmoid(y)
        elif act == "gelu":
            y = y * 0.5 * torch.erfc(-y / math.sqrt(2))
        elif act == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        if s["residual"] is not None:
            y = y + s["residual"][a:a + 1024].double()
        out[a:a + 1024] = y
    return out


def _exact_decode(s):
    T, h, _ = s["q"].shape
    r, rows = s["rank"], s["rows"]
    o = torch.zeros(T, h, r, dtype=torch.float64, device="cuda")
    lse = torch.full((T, h), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"]):
        if n == 0:
            continue
        k = _cache_rows(s, b, n, torch.float64)
        for t in range(b * rows, (b + 1) * rows):
            x = torch.einsum("hd,nd->hn", s["q"][t].double(), k) * SM_SCALE
            lse[t] = torch.logsumexp(x, 1)
            o[t] = torch.exp(x - lse[t][:, None]) @ k[:, :r]
    return o, lse


def _exact_prefill(s):
    tq, h, _ = s["q"].shape
    o = torch.zeros(tq, h, VDIM, dtype=torch.float64, device="cuda")
    lse = torch.full((tq, h), -math.inf, dtype=torch.float64, device="cuda")
    cu_p, gs = _cu(s["pre"]), s["group_list"]
    cu_q, cu_k = _cu(s["lq"]), _cu(s["lk"])
    for g, lp in enumerate(s["pre"]):
        for i in range(gs[g], gs[g + 1]):
            lq, lk = s["lq"][i], s["lk"][i]
            if lq == 0:
                continue
            at = torch.cat([torch.arange(cu_p[g], cu_p[g + 1], device="cuda"),
                            torch.arange(cu_k[i], cu_k[i + 1], device="cuda") + cu_p[-1]])
            rows = slice(cu_q[i], cu_q[i + 1])
            hide = None
            if s["causal"]:
                j = torch.arange(lp + lk, device="cuda")[None, :] - (lp + lk - lq)
                hide = j > torch.arange(lq, device="cuda")[:, None]
            for head in range(h):
                q = s["q"][rows, head].double()
                x = (q[:, :NOPE] @ s["k"][at, head].double().t()
                     + q[:, NOPE:] @ s["k_pe"][at].double().t()) * SM_SCALE
                if hide is not None:
                    x[hide] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[rows, head] = z
                o[rows, head] = torch.exp(x - z[:, None]) @ s["v"][at, head].double()
    return o, lse
