"""GPU tests of the prompt attention against the definition in 64 bits.

Tolerances, from the arithmetic.  A score is a sum of 192 products, exact in
fp32, added in fp32 (each addition off by at most 2^-23 of a partial sum,
truncation included): off by at most ds = 192 * 2^-23 * S, S the largest
sm_scale * sum |q k| of the batch, and the exponent s * c - m * c by another
2^-23 (|s| + |m|) <= 2^-22 S.  So a weight is off by a factor within 1 +- e, e =
1.01 (ds + 2^-22 S) + 2^-21 (the exponential itself).  P is then rounded to bf16
(2^-8), the sum of weights is not; P.V adds n terms in fp32 (n 2^-23), and the
result is rounded to bf16 (2^-8).  With A = sum softmax |v|:
  |o - ref| <= (1 + 2^-8) A (2^-8 + 2 e + 2 n 2^-23) + 2^-8 |ref|
  |lse - ref| <= ds + 2^-22 S + e + n 2^-23 + 2^-22 |ref|
Splits add one more weight each: the same e again.
"""
import math

import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Case:
    def __init__(self, lq, lk, H, seed=0, tail_q=0, tail_k=0, scale=1.0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.lq, self.lk, self.H = lq, lk, H
        T, Tk = sum(lq) + tail_q, sum(lk) + tail_k
        self.q = normal(g, T, H, 192, scale=scale)
        self.kv = normal(g, Tk, H, 256, scale=scale)
        self.k_pe = normal(g, Tk, 64, scale=scale)
        self.k, self.v = self.kv[..., :128], self.kv[..., 128:]
        self.cu_q, self.cu_k = cu(lq), cu(lk)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, causal, splits=1, **kw):
        o, lse = mla.prefill(kw.pop("q", self.q), kw.pop("k", self.k), kw.pop("v", self.v),
                             self.k_pe, self.cu_q, self.cu_k, kw.pop("sm", SCALE), causal=causal,
                             num_kv_splits=splits, err_count=self.err, **kw)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        return o, lse

    def check(self, o, lse, causal, splits=1, sm=SCALE):
        a = b = 0
        for lq, lk in zip(self.lq, self.lk):
            if lq:
                self._check(o[a:a + lq], lse[a:a + lq], a, lq, b, lk, causal, splits, sm)
            a, b = a + lq, b + lk

    def _check(self, o, lse, a, lq, b, lk, causal, splits, sm):
        q = self.q[a:a + lq].double().transpose(0, 1)
        k = torch.cat([self.k[b:b + lk].double(),
                       self.k_pe[b:b + lk, None].double().expand(lk, self.H, 64)], 2).permute(1, 2, 0)
        v = self.v[b:b + lk].double().transpose(0, 1)
        x = q @ k * sm
        allowed = torch.ones(lq, lk, dtype=torch.bool, device="cuda")
        if causal:
            allowed = torch.ones_like(allowed).tril(lk - lq)
        S = float((q.abs() @ k.abs() * sm).max()) if lk else 0.0
        x = x.masked_fill(~allowed, -math.inf)
        ref_lse = torch.logsumexp(x, 2) if lk else x.new_full((self.H, lq), -math.inf)
        p = torch.exp(x - torch.where(ref_lse == -math.inf, 0.0, ref_lse)[..., None])
        ref = (p @ v).transpose(0, 1)
        A = (p @ v.abs()).transpose(0, 1)
        ref_lse = ref_lse.transpose(0, 1)
        ds = 192 * 2.0 ** -23 * S
        e = (1.01 * (ds + 2.0 ** -22 * S) + 2.0 ** -21) * (2 if splits > 1 else 1)
        n = lk + 64
        bound = (1 + 2.0 ** -8) * A * (2.0 ** -8 + 2 * e + 2 * n * 2.0 ** -23) + 2.0 ** -8 * ref.abs()
        err = (o.double() - ref).abs()
        assert bool((err <= bound).all()), ("o", float((err - bound).max()), float(err.max()))
        empty = ref_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty)
        assert bool((o[empty] == 0).all())
        lerr = (lse.double() - ref_lse).abs()[~empty]
        lb = (ds + 2.0 ** -22 * S + e + n * 2.0 ** -23 + 2.0 ** -22 * ref_lse.abs())[~empty]
        assert bool((lerr <= lb).all()), ("lse", float((lerr - lb).max()))


LENS = [
    ([1], [1]), ([1], [128]), ([1], [129]), ([5], [5]), ([127], [127]), ([128], [128]),
    ([129], [129]), ([256], [256]), ([257], [257]), ([300], [377]), ([200], [100]), ([3], [0]),
    ([1, 37, 130], [1, 37, 130]), ([0, 60, 0, 300], [10, 60, 0, 900]),
    ([255, 1, 513], [700, 2000, 513]), ([640], [1280]), ([2, 2, 2, 2], [130, 127, 4000, 1]),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk", LENS)
def test_lengths(cuda_dev, lq, lk, causal):
    c = Case(lq, lk, 3, seed=sum(lq) + sum(lk))
    c.check(*c.run(causal), causal)


@pytest.mark.parametrize("H", [1, 2, 8, 9, 16, 33])
def test_heads(cuda_dev, H):
    c = Case([70, 300, 129], [500, 300, 200], H, seed=H)
    c.check(*c.run(True), True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("splits", [2, 3, 7, 64])
def test_splits(cuda_dev, splits, causal):
    c = Case([1, 4, 0, 200, 3], [3000, 130, 5, 777, 0], 4, seed=splits)
    c.check(*c.run(causal, splits), causal, splits)


def test_long_prompt(cuda_dev):
    c = Case([3001], [3001], 2, seed=3)
    c.check(*c.run(True), True)


@pytest.mark.parametrize("splits", [1, 3])
def test_query_pair_strides_and_bystanders(cuda_dev, splits):
    """Every tensor a view of a wider or longer one: same bits, and the rows
    of no sequence and the columns between are left as they were."""
    c = Case([70, 200], [300, 200], 5, seed=1, tail_q=40, tail_k=13)
    o, lse = c.run(True, splits)
    c.check(o, lse, True, splits)
    nan = float("nan")
    T, Tk, H = c.q.shape[0], c.k.shape[0], 5
    qn = torch.full((T, H, 144), nan, dtype=torch.bfloat16, device="cuda")
    qn[..., 8:136] = c.q[..., :128]
    qp = torch.full((H, T, 64), nan, dtype=torch.bfloat16, device="cuda")
    qp[:] = c.q[..., 128:].transpose(0, 1)
    k = c.k.transpose(0, 1).contiguous()          # head-major
    v = torch.full((Tk, H, 136), nan, dtype=torch.bfloat16, device="cuda")
    v[..., :128] = c.v
    out = torch.full((T, H, 192), 5.0, dtype=torch.bfloat16, device="cuda")
    l2 = torch.full((T, H), 5.0, device="cuda")
    c.run(True, splits, q=(qn[..., 8:136], qp.transpose(0, 1)), k=k.transpose(0, 1),
          v=v[..., :128], out=out[..., :128], lse=l2)
    n = 270
    assert torch.equal(out[:n, :, :128], o[:n]) and torch.equal(l2[:n], lse[:n])
    assert bool((out[n:] == 5).all()) and bool((out[..., 128:] == 5).all())
    assert bool((l2[n:] == 5).all())


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_masked_keys_hold_does_not_matter(cuda_dev, bad, splits):
    """Rows past the sequences, and keys that only later rows attend to."""
    c = Case([150, 20], [150, 333], 3, seed=9, tail_k=200)
    o, lse = c.run(True, splits)
    c.kv[483:], c.k_pe[483:] = bad, bad           # behind the last sequence
    o2, lse2 = c.run(True, splits)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.kv[150 - 30:150] = bad                      # keys 120.. of the first sequence
    c.k_pe[150 - 30:150] = bad
    o2, lse2 = c.run(True, splits)
    keep = torch.ones(170, dtype=torch.bool)
    keep[120:150] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[keep], lse2[keep])
    assert not bool(torch.isfinite(o2[120:150]).any())


@pytest.mark.parametrize("splits", [1, 2])
def test_values_that_are_not_finite_reach_their_own_rows_and_dims(cuda_dev, splits):
    c = Case([300], [300], 2, seed=10)
    o, lse = c.run(True, splits)
    nan, inf = float("nan"), float("inf")
    for key, h, d, x in ((17, 0, 5, nan), (140, 1, 70, inf), (140, 1, 127, -inf), (299, 0, 0, nan),
                         (260, 1, 33, inf), (270, 1, 33, -inf)):
        c.v[key, h, d] = x
    o2, lse2 = c.run(True, splits)
    want = o.clone()
    want[17:, 0, 5] = nan
    want[140:, 1, 70] = inf
    want[140:, 1, 127] = -inf
    want[299:, 0, 0] = nan
    want[260:270, 1, 33] = inf
    want[270:, 1, 33] = nan
    fin = torch.isfinite(want)
    assert torch.equal(torch.isnan(o2), torch.isnan(want))
    assert torch.equal(o2[~torch.isnan(want)], want[~torch.isnan(want)]) and bool(fin.any())
    assert torch.equal(lse, lse2)


@pytest.mark.parametrize("splits", [1, 3])
def test_growing_and_large_scores(cuda_dev, splits):
    """Scores that grow along the keys (the running maximum moves in every
    tile) and reach hundreds; and a scale of 20."""
    c = Case([260], [1500], 2, seed=12)
    ramp = torch.linspace(0, 6, 1500, device="cuda")[:, None, None]
    c.kv[..., :128] = (c.q[:1, :, :128].float() * ramp).to(torch.bfloat16)
    c.q[:, :, :128] = c.q[:1, :, :128]
    c.check(*c.run(False, splits), False, splits)
    c.check(*c.run(True, splits), True, splits)
    d = Case([140], [400], 1, seed=13)
    d.check(*d.run(True, splits, sm=20.0), True, splits, sm=20.0)


def test_deterministic_other_stream_and_graph(cuda_dev):
    c = Case([500, 3], [900, 2000], 6, seed=14)
    for splits in (1, 4):
        o, lse = c.run(True, splits)
        for _ in range(3):
            o2, lse2 = c.run(True, splits)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        side = torch.cuda.Stream()
        o2, lse2 = c.run(True, splits, stream=side)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        out, l2 = torch.empty_like(o), torch.empty_like(lse)
        ws = torch.empty(max(1, mla.mla_prefill_workspace_bytes(*lse.shape, splits, 128)),
                         dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mla.prefill(c.q, c.k, c.v, c.k_pe, c.cu_q, c.cu_k, SCALE, num_kv_splits=splits,
                        workspace=ws, out=out, lse=l2)
        # other lengths in the same buffers
        c.cu_q.copy_(cu([400, 103]))
        c.cu_k.copy_(cu([1900, 900]))
        c.lq, c.lk = [400, 103], [1900, 900]
        g.replay()
        torch.cuda.synchronize()
        c.check(out, l2, True, splits)
        c.lq, c.lk = [500, 3], [900, 2000]
        c.cu_q.copy_(cu(c.lq)), c.cu_k.copy_(cu(c.lk))


def test_a_row_does_not_depend_on_the_batch(cuda_dev):
    c = Case([300], [700], 4, seed=15)
    o, lse = c.run(True)
    d = Case([77, 300, 5], [100, 700, 5], 4, seed=16)
    d.q[77:377], d.kv[100:800], d.k_pe[100:800] = c.q, c.kv, c.k_pe
    o2, lse2 = d.run(True)
    assert torch.equal(o2[77:377], o) and torch.equal(lse2[77:377], lse)


def test_bad_lengths_are_clamped_and_counted(cuda_dev):
    c = Case([100], [100], 2, seed=17)
    c.cu_q.copy_(torch.tensor([0, 1000], dtype=torch.int32))
    c.cu_k.copy_(torch.tensor([-5, 200], dtype=torch.int32))
    o, lse = mla.prefill(c.q, c.k, c.v, c.k_pe, c.cu_q, c.cu_k, SCALE, err_count=c.err)
    torch.cuda.synchronize()
    assert c.err.item() == 1
    c.check(o, lse, True)


def test_offsets_past_32_bits(cuda_dev):
    """Keys and values behind 2^31 elements."""
    H, Tk = 128, 67000
    kv = torch.zeros(Tk, H, 256, dtype=torch.bfloat16, device="cuda")
    c = Case([3, 2], [66000, 1000], 1, seed=18)
    kv[:, H - 1:] = c.kv
    q = torch.zeros(5, H, 192, dtype=torch.bfloat16, device="cuda")
    q[:, H - 1:] = c.q
    o, lse = mla.prefill(q, kv[..., :128], kv[..., 128:], c.k_pe, c.cu_q, c.cu_k, SCALE,
                         num_kv_splits=4, err_count=c.err)
    torch.cuda.synchronize()
    c.check(o[:, H - 1:], lse[:, H - 1:].contiguous(), True, 4)


def test_no_rows(cuda_dev):
    c = Case([0], [5], 2)
    o, lse = c.run(True)
    assert o.shape == (0, 2, 128) and lse.shape == (0, 2)
