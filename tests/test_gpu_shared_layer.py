"""Layers of a model that answers several questions about one text, as a server
runs them: the projections of `linear`, the cache write, prompt attention behind
the shared prefix, then decode steps behind it out of one graph, with the
sequences growing from page to page.

Against the layer in 64 bits, on the rows that the cache holds.  The call rounds
to bf16 q, the absorbed q, P, the latent output, y, the residual sum, the MLP's
inner activations and the second sum: eight roundings, of at most 2^-8 in norm.
Weights of variance 1 / fan-in pass a relative change on with a factor of about
one, so do scores of unit variance, and silu's slope is at most 1.1: the layer's
output is within 9 * 2^-8 of the definition in norm.  (The expanded form rounds k
and v in place of the absorbed q and the latent output: as many.)
"""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self, g, D, H, R, F):
        self.D, self.H, self.R = D, H, R
        self.wq, self.bq = normal(g, H * 192, D, scale=D ** -0.5), normal(g, H * 192, scale=0.1)
        self.wc = normal(g, R + 64, D, scale=D ** -0.5)
        self.wkv = normal(g, H * 256, R, scale=R ** -0.5)
        self.wo = normal(g, D, H * 128, scale=(H * 128) ** -0.5)
        self.w1, self.w2 = normal(g, F, D, scale=D ** -0.5), normal(g, D, F, scale=F ** -0.5)

    def rows(self, x, err):
        """q [T, H, 192] and the cache rows' two parts, as views of one product."""
        q = mla.linear(x, self.wq, bias=self.bq, err_count=err).view(len(x), self.H, 192)
        c = mla.linear(x, self.wc, err_count=err)
        return q, c[:, :self.R], c[:, self.R:]

    def rest(self, x, y, err):
        """Output projection and MLP, added to x in place."""
        mla.linear(y.view(len(x), self.H * 128), self.wo, residual=x, out=x, err_count=err)
        h = mla.linear(x, self.w1, activation="silu", err_count=err)
        mla.linear(h, self.w2, residual=x, out=x, err_count=err)

    def reference(self, x, keys):
        """Row t of x against keys[t] [n, R + 64], all in 64 bits."""
        d = lambda t: t.double()  # noqa: E731
        q = (d(x) @ d(self.wq).t() + d(self.bq)).view(len(x), self.H, 192)
        w = d(self.wkv).view(self.H, 256, self.R)
        y = torch.empty(len(x), self.H, 128, dtype=torch.float64, device="cuda")
        for t, k in enumerate(keys):
            kv = torch.einsum("hdr,nr->nhd", w, k[:, :self.R])
            s = torch.einsum("hd,nhd->hn", q[t, :, :128], kv[..., :128]) + q[t, :, 128:] @ k[:, self.R:].t()
            y[t] = torch.einsum("hn,nhd->hd", torch.softmax(s * SCALE, 1), kv[..., 128:])
        x = d(x) + y.view(len(x), -1) @ d(self.wo).t()
        return x + torch.nn.functional.silu(x @ d(self.w1).t()) @ d(self.w2).t()


def close(got, ref):
    diff = float((got.double() - ref).norm() / ref.norm())
    assert diff <= 9 * 2.0 ** -8, diff


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("R,H,bs,D", [(512, 16, 64, 1024), (256, 5, 16, 520)])
def test_questions_about_one_text(cuda_dev, R, H, bs, D, fmt):
    g = torch.Generator("cuda").manual_seed(R + H)
    layer = Layer(g, D, H, R, 2 * D + 8)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    prefix, new = 5 * bs, [40, 1, 0, 3 * bs, 77]  # whole pages; one padded sequence
    B, T, maxb = len(new), sum(new), 12
    cache = torch.zeros(8 * maxb, bs, R + 64, dtype=torch.bfloat16, device="cuda")
    scale = None
    if fmt != "bf16":
        cache, scale = cache.to(FP8[fmt]), torch.tensor([0.05], device="cuda")
    perm = torch.randperm(8 * maxb, generator=g, device="cuda").to(torch.int32)
    shared = prefix // bs
    own = perm[shared:shared + B * (maxb - shared)].view(B, -1)
    table = torch.cat([perm[:shared].expand(B, -1), own], 1).contiguous()

    def slots(b, first, n):
        t = torch.arange(first, first + n, device="cuda")
        return table[b, t // bs].long() * bs + t % bs

    def stored(b, n):
        c = cache.view(torch.uint8)[table[b].long()].reshape(maxb * bs, -1)[:n] if scale is not None \
            else cache[table[b].long()].reshape(maxb * bs, -1)[:n]
        return c.double() if scale is None else c.view(cache.dtype).float().double() * scale.double()

    # the text itself, written once
    x = normal(g, prefix, D)
    _, kv_c, k_pe = layer.rows(x, err)
    mla.cache_write(kv_c, k_pe, cache, slots(0, 0, prefix), scale=scale, err_count=err)

    # the questions' prompts: own keys behind the prefix's, gathered from the cache
    x = normal(g, T, D)
    start = x.clone()
    q, kv_c, k_pe = layer.rows(x, err)
    where = torch.cat([slots(b, prefix, n) for b, n in enumerate(new)])
    mla.cache_write(kv_c, k_pe, cache, where, scale=scale, err_count=err)
    ends = [prefix]
    for n in new:
        ends.append(ends[-1] + n)
    kv = torch.cat([table[0, :shared], own.reshape(-1)])  # one table row a run of rows
    runs = torch.zeros(B + 1, max(shared, maxb - shared), dtype=torch.int32, device="cuda")
    runs[0, :shared], runs[1:, :maxb - shared] = kv[:shared], own
    gc, gp = mla.gather_cache(cache, runs, i32([0] + ends), ends[-1], kv_lora_rank=R,
                              kv_scale=scale, err_count=err)
    k, v = mla.expand_kv(gc, layer.wkv, H, err_count=err)
    cu_q = i32([e - prefix for e in ends])
    for splits in (1, (2, 2), mla.mla_prefill_shared_num_kv_splits(T, B, 1, H, prefix, max(new), 152)):
        x.copy_(start)
        o, _ = mla.prefill_shared(q, k, v, gp, cu_q, i32(ends), i32([0, B]), i32([0, prefix]), SCALE,
                                  num_kv_splits=splits, err_count=err)
        layer.rest(x, o, err)
        keys = [stored(b, prefix + i + 1) for b, n in enumerate(new) for i in range(n)]
        torch.cuda.synchronize()
        assert err.item() == 0
        ref = layer.reference(start, keys)
        if fmt == "bf16":
            close(x, ref)
        else:  # gathered rows are rounded once more: the ninth
            assert float((x.double() - ref).norm() / ref.norm()) <= 10 * 2.0 ** -8

    # answers: one graph, replayed as the sequences grow
    lens = i32([prefix + n if n else 0 for n in new])
    slot = torch.zeros(B, dtype=torch.int64, device="cuda")
    x, xin = normal(g, B, D), normal(g, B, D)
    gs, pre = i32([0, B]), i32([prefix])

    def step():
        x.copy_(xin)
        q, kv_c, k_pe = layer.rows(x, err)
        mla.cache_write(kv_c, k_pe, cache, slot, scale=scale, err_count=err)
        ql = mla.absorb_q(q[..., :128], layer.wkv, err_count=err)
        o, _ = mla.decode_shared((ql, q[..., 128:]), cache, table, lens, gs, pre, SCALE,
                                 kv_lora_rank=R, kv_scale=scale, err_count=err)
        layer.rest(x, mla.project_v(o, layer.wkv, err_count=err), err)

    live = [b for b, n in enumerate(new) if n]
    at = [prefix + n for n in new]

    def fill():
        for b in range(B):
            slot[b] = slots(b, at[b], 1)[0] if b in live else -1
            lens[b] = at[b] + 1 if b in live else 0

    fill()
    kept = cache.clone()
    step()
    cache.copy_(kept)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    cache.copy_(kept)
    for i in range(bs + 3):
        fill()
        xin.copy_(normal(g, B, D))
        gr.replay()
        at = [n + 1 for n in at]
        if i % 9 == 0 or i > bs - 2:
            torch.cuda.synchronize()
            ref = layer.reference(xin[live], [stored(b, at[b]) for b in live])
            close(x[live], ref)
            dead = [b for b in range(B) if b not in live]  # nothing to attend to: y is 0
            none = layer.reference(xin[dead], [torch.zeros(1, R + 64, dtype=torch.float64,
                                                           device="cuda")] * len(dead))
            close(x[dead], none)
    assert err.item() == 0


def make_calls(seed=1):
    """name -> call(stream), each returning the tensors it allocated."""
    g = torch.Generator("cuda").manual_seed(seed)
    x, w, r = normal(g, 200, 1024), normal(g, 640, 1024, scale=1 / 32), normal(g, 200, 640)
    xl, wl = normal(g, 4000, 512), normal(g, 1536, 512, scale=1 / 23)
    H, T, pre = 8, 300, 2000
    q, kv, kp = normal(g, T, H, 192), normal(g, pre + T, H, 256), normal(g, pre + T, 64)
    cu_q, cu_k = i32([0, 100, 130, T]), i32([pre, pre + 100, pre + 130, pre + T])
    gs, cp = i32([0, 3]), i32([0, pre])
    cache, dq = normal(g, 80, 64, 576), normal(g, 6, 16, 576)
    table = torch.arange(6 * 40, device="cuda").remainder(80).to(torch.int32).view(6, 40)
    table[:, :20] = table[0, :20].clone()
    lens, dg, dp = i32([2000, 1300, 1280, 2560, 0, 1999]), i32([0, 6]), i32([1280])

    def prefill(s, splits):
        return mla.prefill_shared(q, kv[..., :128], kv[..., 128:], kp, cu_q, cu_k, gs, cp, SCALE,
                                  num_kv_splits=splits, stream=s)
    return {
        "linear": lambda s: (mla.linear(x, w, residual=r, activation="silu", stream=s),),
        "linear_large": lambda s: (mla.linear(xl, wl, activation="gelu", stream=s),),
        "prefill_shared": lambda s: prefill(s, 1),
        "prefill_shared_split": lambda s: prefill(s, 4),
        "prefill_shared_apart": lambda s: prefill(s, (2, 2)),
        "decode_shared": lambda s: mla.decode_shared(dq, cache, table, lens, dg, dp, SCALE, stream=s),
        "decode_shared_pair": lambda s: mla.decode_shared((dq[..., :512], dq[..., 512:]), cache, table,
                                                          lens, dg, dp, SCALE, stream=s),
    }


NAMES = ["linear", "linear_large", "prefill_shared", "prefill_shared_split", "prefill_shared_apart",
         "decode_shared", "decode_shared_pair"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_the_launch_streams_memory(cuda_dev, name):
    call = make_calls()[name]
    ref = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        # blocks of the outputs' sizes, free in the current stream's pool but
        # still to be written by what is queued there
        freed = [torch.empty_like(x) for x in ref]
        torch.cuda._sleep(20_000_000)
        for x in freed:
            x.zero_()
        ptrs = {x.data_ptr() for x in freed}
        del freed, x
        side.wait_stream(torch.cuda.current_stream())
        out = call(side)
        assert not ptrs & {x.data_ptr() for x in out}
        torch.cuda.synchronize()
        for x, r in zip(out, ref):
            assert torch.equal(x, r)
        del out, x


@pytest.mark.parametrize("name", NAMES)
def test_two_calls_at_once(cuda_dev, name):
    """Workspaces are let go when a call returns, with its kernels still queued;
    another call runs at once, on a stream of its own."""
    calls = [make_calls(s)[name] for s in (1, 2)]
    want = [[x.clone() for x in c(None)] for c in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        torch.cuda._sleep(1_000_000 * (i % 3))
        got = [calls[0](None), calls[1](side)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_replayed_at_once(cuda_dev, name):
    """One captured on a stream that joins the capture, each with its own memory."""
    calls = [make_calls(s)[name] for s in (1, 2)]
    want = [[x.clone() for x in c(None)] for c in calls]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i, c in enumerate(calls):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            if i:
                side[i].wait_stream(torch.cuda.current_stream())
            outs.append(c(side[i] if i else None))
            if i:
                torch.cuda.current_stream().wait_stream(side[i])
        graphs.append(gr)
    for o in outs:
        for x in o:
            x.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, s in zip(graphs, side):
            with torch.cuda.stream(s):
                gr.replay()
        calls[0](None)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_host_threads(cuda_dev):
    """Four host threads, each on a stream of its own."""
    import threading
    sets = [make_calls(i + 1) for i in range(4)]
    refs = [{n: [x.clone() for x in c[n](None)] for n in NAMES} for c in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        try:
            with torch.cuda.stream(s):
                for _ in range(10):
                    for n in NAMES:
                        out = sets[i][n](None)
                        if not all(torch.equal(x, r) for x, r in zip(out, refs[i][n])):
                            wrong.append((i, n))
        except Exception as e:  # noqa: BLE001 - reported below
            wrong.append((i, repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


@pytest.mark.parametrize("name", ["prefill_shared_split", "prefill_shared_apart", "decode_shared"])
def test_workspaces_do_not_pile_up(cuda_dev, name):
    call = make_calls()[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    active = lambda: torch.cuda.memory_stats()["active_bytes.all.current"]  # noqa: E731
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    keep = [call(side)]
    used = sum(x.nbytes for x in keep[0])
    torch.cuda._sleep(400_000_000)
    start = active()
    for _ in range(8):
        keep.append(call(side))
    grown = active() - start
    torch.cuda.synchronize()
    assert grown <= 8 * (used + 8 * 512), (grown, used)
