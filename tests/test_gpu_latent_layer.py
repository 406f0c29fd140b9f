"""The calls of a latent-attention layer together, as a server runs them: two
steps of prompt chunks and single tokens through batch tables, the cache
write, the gather, the kv_b products and the prompt attention; then decode
steps in the absorbed form on the same cache.

The paged path is compared bit for bit with the same kernels on contiguous
rows kept aside: it may differ in nothing but where the rows lie.  The two
forms compute the same function with other roundings: expanded rounds the
cached row, k, v, P and o, absorbed ql, P, the latent output and y, nine
in all; each moves what it rounds by at most 2^-8 in norm, and scores of unit
variance pass a relative change of the keys on with a factor of about one, so
the two are within 9 * 2^-8 of each other in norm.
"""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Server:
    """Requests, their pages and a cache, with every row also kept aside."""

    def __init__(self, R, H, bs, fmt, B, maxb, nb, seed):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.R, self.H, self.bs, self.nb, self.B = R, H, bs, nb, B
        self.w = normal(self.g, H * 256, R, scale=R ** -0.5)
        dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
        self.cache = torch.zeros(nb, bs, R + 64, dtype=torch.bfloat16, device="cuda")
        self.cache[:] = float("nan")
        self.cache = self.cache.to(dt)
        self.scale = None if fmt == "bf16" else torch.tensor([0.05], device="cuda")
        self.table = torch.full((B + 3, maxb), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(nb, generator=self.g, device="cuda").to(torch.int32)
        self.count = i32([nb])
        self.rows = i32(np.random.default_rng(seed).permutation(B + 3)[:B])
        self.ctx = i32(np.zeros(B))
        self.kept = [torch.empty(0, R + 64, dtype=torch.bfloat16, device="cuda") for _ in range(B)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, new, pad=0):
        T = int(sum(new))
        t = mla.batch_build(i32(new), self.ctx, self.table, self.free, self.count, self.bs, self.nb,
                            T + pad, req_ids=self.rows, free_count_out=self.count,
                            err_count=self.err)
        kv_c, k_pe = normal(self.g, T + pad, self.R), normal(self.g, T + pad, 64)
        mla.cache_write(kv_c, k_pe, self.cache, t.slot_mapping, scale=self.scale, err_count=self.err)
        row = torch.cat([kv_c, k_pe], 1)
        if self.scale is not None:
            row = ((row.float() / self.scale).to(self.cache.dtype).float() * self.scale).to(torch.bfloat16)
        a = 0
        for b, n in enumerate(new):
            self.kept[b] = torch.cat([self.kept[b], row[a:a + n]])
            a += n
        self.ctx = t.seq_lens
        return t, T

    def expanded(self, t, T, q):
        n = int(t.cu_seqlens_k[-1].item())
        kv_c, k_pe = mla.gather_cache(self.cache, t.block_table, t.cu_seqlens_k, n,
                                      kv_lora_rank=self.R, kv_scale=self.scale, err_count=self.err)
        k, v = mla.expand_kv(kv_c, self.w, self.H, err_count=self.err)
        S = mla.mla_prefill_num_kv_splits(T, self.B, self.H, int(t.seq_lens.max().item()), 152)
        o, lse = mla.prefill(q, k, v, k_pe, t.cu_seqlens_q, t.cu_seqlens_k, SCALE, num_kv_splits=S,
                             err_count=self.err)
        plain = torch.cat(self.kept)
        assert torch.equal(torch.cat([kv_c, k_pe], 1), plain)
        pk, pv = mla.expand_kv(plain[:, :self.R].contiguous(), self.w, self.H)
        assert torch.equal(k, pk) and torch.equal(v, pv)
        cu_q = i32(np.concatenate([[0], np.cumsum(np.diff(t.cu_seqlens_q.cpu().numpy()))]))
        cu_k = i32(np.concatenate([[0], np.cumsum([len(r) for r in self.kept])]))
        po, plse = mla.prefill(q, pk, pv, plain[:, self.R:].contiguous(), cu_q, cu_k, SCALE,
                               num_kv_splits=S)
        assert torch.equal(o, po) and torch.equal(lse, plse)
        return o, lse

    def absorbed(self, t, q):
        """One query row per request against its whole sequence."""
        ql = mla.absorb_q(q[..., :128], self.w, err_count=self.err)
        S = mla.mla_num_kv_splits(int(t.seq_lens.max().item()), 152)
        o, lse = mla.decode((ql, q[..., 128:].contiguous()), self.cache, t.block_table, t.seq_lens, SCALE, S,
                            kv_lora_rank=self.R, kv_scale=self.scale, err_count=self.err)
        return mla.project_v(o, self.w, err_count=self.err), lse


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("R,H,bs", [(512, 16, 64), (256, 5, 16)])
def test_a_servers_steps(cuda_dev, R, H, bs, fmt):
    B = 5
    s = Server(R, H, bs, fmt, B, maxb=-(-900 // bs), nb=B * (-(-900 // bs)) + 4, seed=R + H)
    for new, pad in (([130, 1, 0, 300, 64], 0), ([70, 1, 257, 3, 1], 9)):
        t, T = s.step(new, pad)
        q = normal(s.g, T, H, 192)
        s.expanded(t, T, q)
    # single tokens: both forms, on the same cache
    for _ in range(2):
        t, T = s.step([1] * B)
        q = normal(s.g, B, H, 192)
        o, lse = s.expanded(t, T, q)
        y, lse2 = s.absorbed(t, q)
        torch.cuda.synchronize()
        diff = float((o.double() - y.double()).norm() / o.double().norm())
        assert diff <= 9 * 2.0 ** -8, diff
        assert float((lse - lse2).abs().max()) <= 9 * 2.0 ** -8 * float(lse.abs().max())
    assert s.err.item() == 0


def test_layer_captured_in_one_graph(cuda_dev):
    """A decode step of the whole layer captured once and replayed as the
    sequences grow, page by page; the tables are built inside the graph."""
    B, H, R, bs = 6, 16, 512, 16
    s = Server(R, H, bs, "bf16", B, maxb=40, nb=300, seed=3)
    s.step([30, 1, 100, 16, 15, 64])
    ctx = s.ctx.clone()
    new, kv_c, k_pe = i32(np.ones(B)), normal(s.g, B, R), normal(s.g, B, 64)
    q = normal(s.g, B, H, 192)
    bt = torch.zeros(B, 40, dtype=torch.int32, device="cuda")
    out = {}

    def layer():
        t = mla.batch_build(new, ctx, s.table, s.free, s.count, bs, s.nb, B, req_ids=s.rows,
                            block_table=bt, free_count_out=s.count, err_count=s.err)
        mla.cache_write(kv_c, k_pe, s.cache, t.slot_mapping, err_count=s.err)
        ql = mla.absorb_q(q[..., :128], s.w)
        o, lse = mla.decode(torch.cat([ql, q[..., 128:]], 2), s.cache, t.block_table, t.seq_lens, SCALE,
                            2, kv_lora_rank=R, err_count=s.err)
        out["y"], out["lse"] = mla.project_v(o, s.w), lse
        ctx.copy_(t.seq_lens)

    start = (ctx.clone(), s.table.clone(), s.free.clone(), s.count.clone(), s.cache.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    for dst, src in zip((ctx, s.table, s.free, s.count, s.cache), start):
        dst.copy_(src)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for dst, src in zip((ctx, s.table, s.free, s.count, s.cache), start):
        dst.copy_(src)
    for step in range(20):
        kv_c.copy_(normal(s.g, B, R)), k_pe.copy_(normal(s.g, B, 64)), q.copy_(normal(s.g, B, H, 192))
        g.replay()
        for b in range(B):
            s.kept[b] = torch.cat([s.kept[b], torch.cat([kv_c[b:b + 1], k_pe[b:b + 1]], 1)])
        if step % 6 == 5:
            plain = torch.cat(s.kept)
            k, v = mla.expand_kv(plain[:, :R].contiguous(), s.w, H)
            o, lse = mla.prefill(q, k, v, plain[:, R:].contiguous(), i32(np.arange(B + 1)),
                                 i32(np.concatenate([[0], np.cumsum([len(r) for r in s.kept])])), SCALE)
            diff = float((out["y"].double() - o.double()).norm() / o.double().norm())
            assert diff <= 9 * 2.0 ** -8, (step, diff)
    assert s.err.item() == 0 and ctx.tolist() == [len(r) for r in s.kept]


def test_two_captured_layers_and_streams_do_not_mix(cuda_dev):
    """Two prompt attentions captured with workspaces of their own, replayed at
    once on two streams, each bit for bit what it is alone."""
    g = torch.Generator("cuda").manual_seed(4)
    cases = []
    for n, keys, H in ((3, 9000, 16), (200, 6000, 3)):
        q, kv, kp = normal(g, n, H, 192), normal(g, keys, H, 256), normal(g, keys, 64)
        a = (q, kv[..., :128], kv[..., 128:], kp, i32([0, n]), i32([0, keys]), SCALE)
        want = mla.prefill(*a, num_kv_splits=5)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            got = mla.prefill(*a, num_kv_splits=5)
        cases.append((gr, want, got, torch.cuda.Stream(), a))  # a graph reads its inputs' memory
    torch.cuda.synchronize()
    for _ in range(20):
        for gr, _, _, st, _ in cases:
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for _, want, got, _, _ in cases:
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_python_calls_check_their_tensors(cuda_dev):
    bf = torch.bfloat16
    w = torch.zeros(2 * 256, 512, dtype=bf, device="cuda")
    x = torch.zeros(3, 2, 128, dtype=bf, device="cuda")
    cu = i32([0, 3])
    kp = torch.zeros(3, 64, dtype=bf, device="cuda")
    q = torch.zeros(3, 2, 192, dtype=bf, device="cuda")
    cases = [
        lambda: mla.absorb_q(x.float(), w), lambda: mla.absorb_q(x, w.half()),
        lambda: mla.absorb_q(x[:, :1], w), lambda: mla.absorb_q(x.cpu(), w),
        lambda: mla.absorb_q(x, w, out=torch.zeros(3, 2, 256, dtype=bf, device="cuda")),
        lambda: mla.absorb_q(torch.zeros(3, 128, 2, dtype=bf, device="cuda").transpose(1, 2), w),
        lambda: mla.absorb_q(x, w, err_count=torch.zeros(1, device="cuda")),
        lambda: mla.project_v(x, w), lambda: mla.expand_kv(kp, w, 2), lambda: mla.expand_kv(kp, w, 0),
        lambda: mla.expand_kv(w[:3], w, 2, k_nope=x),
        lambda: mla.prefill(q, x, x, kp, cu.long(), cu, 0.1),
        lambda: mla.prefill(q, x, x[:2], kp, cu, cu, 0.1),
        lambda: mla.prefill(x, x, x, kp, cu, cu, 0.1),
        lambda: mla.prefill(q, x, x, kp, cu, i32([0, 1, 3]), 0.1),
        lambda: mla.prefill(q, x, x, kp, cu, cu, 0.1, lse=torch.zeros(2, 3, device="cuda").t()),
        lambda: mla.gather_cache(torch.zeros(2, 16, 576, dtype=bf, device="cuda"), i32([[0]]), cu, 3,
                                 kv_cache_dtype="fp8"),
        lambda: mla.gather_cache(torch.zeros(2, 16, 576, dtype=bf, device="cuda"), i32([[0]]), cu),
        lambda: mla.batch_build(cu, cu, i32([[0]]), cu, i32([1]), 16, 4),
        lambda: mla.batch_build(cu, i32([1]), i32([[0]]), cu, i32([1]), 16, 4, 5),
        lambda: mla.batch_build(cu, cu, i32([[0]]).long(), cu, i32([1]), 16, 4, 5),
    ]
    for i, f in enumerate(cases):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
    for f in (lambda: mla.prefill(q, x, x, kp, cu, cu, 0.0),
              lambda: mla.prefill(q, x, x, kp, cu, cu, 0.1, num_kv_splits=65),
              lambda: mla.prefill(q, x, x, kp, cu, cu, 0.1, num_kv_splits=2,
                                  workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
              lambda: mla.batch_build(cu, cu, i32([[0], [0]]), cu, i32([1]), 0, 4, 5)):
        with pytest.raises(mla.MlaError):
            f()
    torch.cuda.synchronize()
