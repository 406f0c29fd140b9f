"""GPU tests of the prompt attention behind shared prefixes against the
definition in 64 bits.  Tolerances as derived for the prompt attention: a score
is off by at most ds = 192 2^-23 S, a weight by a factor within 1 +- e, e = 1.01
(ds + 2^-22 S) + 2^-21, P by 2^-8, the sum over n keys by n 2^-23, the result by
2^-8; joining parts takes one more weight each, the same e again.
"""
import math

import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)
NAN = float("nan")


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def cu(lens, first=0):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]) + first, dtype=torch.int32,
                        device="cuda")


class Case:
    """Prefix keys of each group, then `gap` rows of nothing, then the sequences'."""

    def __init__(self, groups, prefix, lq, lk, H, seed=0, gap=0, tail=0, before=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.groups, self.prefix, self.lq, self.lk, self.H = groups, prefix, lq, lk, H
        self.p0, self.k0, self.r0 = before, before + sum(prefix) + gap, before
        T, Tk = before + sum(lq) + tail, self.k0 + sum(lk) + tail
        self.q = normal(g, T, H, 192)
        kv = normal(g, Tk, H, 256)
        self.k, self.v = kv[..., :128], kv[..., 128:]
        self.k_pe = normal(g, Tk, 64)
        self.cu_q, self.cu_k = cu(lq, before), cu(lk, self.k0)
        self.gs = torch.tensor(groups, dtype=torch.int32, device="cuda")
        self.cu_p = cu(prefix, self.p0)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, causal=True, splits=(1, 1), **kw):
        o, lse = mla.prefill_shared(kw.pop("q", self.q), self.k, self.v, self.k_pe, self.cu_q,
                                    self.cu_k, self.gs, self.cu_p, SCALE, causal=causal,
                                    num_kv_splits=splits, err_count=self.err, **kw)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        return o, lse

    def keys_of(self, b):
        """Key rows of sequence b: its prefix's, its own."""
        pre = torch.empty(0, dtype=torch.long, device="cuda")
        for g in range(len(self.prefix)):
            if self.groups[g] <= b < self.groups[g + 1]:
                p = self.p0 + sum(self.prefix[:g])
                pre = torch.arange(p, p + self.prefix[g], device="cuda")
        k = self.k0 + sum(self.lk[:b])
        return pre, torch.arange(k, k + self.lk[b], device="cuda")

    def check(self, o, lse, causal=True):
        a = self.r0
        for b, (lq, lk) in enumerate(zip(self.lq, self.lk)):
            rows = slice(a, a + lq)
            a += lq
            if lq == 0:
                continue
            pre, own = self.keys_of(b)
            at = torch.cat([pre, own])
            n, lp = at.numel(), pre.numel()
            q = self.q[rows].double().transpose(0, 1)
            k = torch.cat([self.k[at].double(),
                           self.k_pe[at, None].double().expand(n, self.H, 64)], 2).permute(1, 2, 0)
            v = self.v[at].double().transpose(0, 1)
            ok = torch.ones(lq, n, dtype=torch.bool, device="cuda")
            if causal:
                ok[:, lp:] = torch.ones(lq, lk, dtype=torch.bool, device="cuda").tril(lk - lq)
            x = (q @ k * SCALE).masked_fill(~ok, -math.inf)
            ref_lse = torch.logsumexp(x, 2) if n else x.new_full((self.H, lq), -math.inf)
            p = torch.exp(x - torch.where(ref_lse == -math.inf, 0.0, ref_lse)[..., None])
            p = torch.where(ok, p, 0.0)
            # a value outside the mask does not count, whatever it is
            used = ok.any(0)
            v = torch.where(used[None, :, None], v, torch.zeros_like(v))
            ref, A = (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1)
            ref_lse = ref_lse.transpose(0, 1)
            S = float((q.abs() @ k.abs() * SCALE).nan_to_num(0).max()) if n else 0.0
            ds = 192 * 2.0 ** -23 * S
            e = 2 * (1.01 * (ds + 2.0 ** -22 * S) + 2.0 ** -21)
            bo = (1 + 2.0 ** -8) * A * (2.0 ** -8 + 2 * e + 2 * n * 2.0 ** -23) \
                + 2.0 ** -8 * ref.abs()
            assert bool(((o[rows].double() - ref).abs() <= bo).all()), (b, lq, lk)
            empty = ref_lse == -math.inf
            assert torch.equal(lse[rows] == -math.inf, empty)
            assert bool((o[rows][empty] == 0).all())
            bl = ds + 2.0 ** -22 * S + e + n * 2.0 ** -23 + 2.0 ** -22 * ref_lse.abs()
            d = torch.where(empty, 0.0, lse[rows].double() - ref_lse).abs()
            assert bool((d <= torch.where(empty, 1.0, bl)).all())


CASES = [
    # groups, prefixes, rows, own keys, heads
    ([0, 1], [1], [1], [1], 1),
    ([0, 3], [700], [1, 40, 7], [1, 40, 7], 16),
    ([0, 2, 3], [127, 129], [5, 130, 300], [5, 200, 300], 5),
    ([0, 5], [128], [0, 3, 0, 17, 1], [0, 3, 9, 40, 1], 3),
    ([0, 1, 1, 4], [50, 999, 1], [64, 2, 3, 4], [64, 5, 0, 4], 7),       # an empty group
    ([0, 2, 4], [0, 300], [10, 20, 30, 40], [10, 0, 30, 100], 2),        # an empty prefix
    ([1, 3], [257], [33, 20, 1, 70], [50, 20, 1, 70], 4),                # sequences of no group
    ([0, 4], [4100], [257, 512, 1, 255], [257, 600, 300, 255], 4),
    ([0, 70], [333], [i % 9 for i in range(70)], [i % 9 + (i % 4) * 31 for i in range(70)], 2),
    ([3 * i for i in range(71)], [5 * i for i in range(70)], [i % 3 + 1 for i in range(210)],
     [i % 3 + 1 + i % 50 for i in range(210)], 1),
    ([0, 2], [2000], [30, 9], [4, 0], 3),                                # fewer own keys than rows
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
@pytest.mark.parametrize("causal,splits", [(True, (1, 1)), (True, (3, 2)), (False, (2, 1)),
                                           (False, (1, 3)), (True, (1, 0)), (True, (3, 0)),
                                           (False, (1, 0)), (False, (2, 0))])
def test_matches_64_bits(cuda_dev, case, causal, splits):
    c = Case(*case, seed=len(case[2]))
    c.check(*c.run(causal, splits), causal)


def test_many_parts_and_the_rule(cuda_dev):
    c = Case([0, 2, 5], [9000, 3333], [3, 11, 2, 60, 1], [3, 2500, 900, 60, 4000], 8)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = mla.mla_prefill_shared_num_kv_splits(77, 5, 2, 8, 9000, 4000, sms)
    assert n[0] > 1
    for s in (n, (64, 64), (40, 1), n[0], (1, 0), (7, 0)):
        c.check(*c.run(True, s))


def test_rows_of_no_sequence_and_gaps_are_left(cuda_dev):
    c = Case([0, 2], [200], [20, 300], [20, 310], 3, gap=40, tail=50, before=7)
    c.k[:7], c.v[:7], c.k_pe[:7] = NAN, NAN, NAN          # keys of nobody
    c.k[207:247], c.v[207:247] = NAN, NAN
    c.k[-50:], c.v[-50:] = NAN, NAN
    o = torch.full((c.q.shape[0], 3, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.q.shape[0], 3), 7.0, device="cuda")
    for s in ((1, 1), (2, 2), (1, 0), (3, 0)):
        c.check(*c.run(True, s, out=o, lse=lse))
        assert bool((o[:7] == 7).all()) and bool((o[-50:] == 7).all())
        assert bool((lse[:7] == 7).all()) and bool((lse[-50:] == 7).all())


@pytest.mark.parametrize("bad", [NAN, math.inf])
@pytest.mark.parametrize("splits", [(1, 1), (1, 0), (2, 0)])
def test_masked_keys_have_no_influence(cuda_dev, bad, splits):
    c = Case([0, 2], [130], [40, 150], [60, 400], 2)
    o, lse = c.run(True, splits)
    # the last own key of sequence 0: only its last row attends to it
    at = c.k0 + 59
    c.v[at, :, 3] = bad
    c.k[at, :, 5] = NAN
    o2, lse2 = c.run(True, splits)
    keep = torch.arange(190, device="cuda") != 39
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])
    assert not bool(o2[39, :, 3].isfinite().any())
    # one of the prefix's last keys (its last tile is cut): every row
    c.v[at, :, 3] = 0
    c.k[at, :, 5] = 0
    c.v[c.p0 + 129, 1, 7] = bad
    o3, _ = c.run(True, splits)
    assert not bool(o3[:, 1, 7].isfinite().any()) and bool(o3[:, 0].isfinite().all())


def test_many_short_sequences(cuda_dev):
    """More sequences in a block than lengths kept in shared memory."""
    lq = [(i * 7) % 5 for i in range(300)]
    c = Case([0, 100, 300], [300, 129], lq, [n + (i % 3) * 40 for i, n in enumerate(lq)], 2, seed=3)
    for s in ((1, 0), (2, 0), (1, 1)):
        c.check(*c.run(True, s))
        c.check(*c.run(False, s), False)


def test_equals_prefill_of_the_joined_keys(cuda_dev):
    """One sequence: the shared call and prefill over prefix and own keys."""
    c = Case([0, 1], [1024], [256], [256], 4)
    a, la = c.run()
    b, lb = mla.prefill(c.q, c.k, c.v, c.k_pe, cu([256]), cu([1280]), SCALE)
    assert bool(((a.double() - b.double()).abs() <= 2.0 ** -6 * b.double().abs() + 2e-3).all())
    assert bool(((la - lb).abs() < 1e-5).all())


def test_pair_of_q_strides_and_determinism(cuda_dev):
    c = Case([0, 2], [500], [33, 70], [40, 70], 6)
    o, lse = c.run(True, (2, 0))
    again = c.run(True, (2, 0))
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    wide = torch.zeros(103, 8, 160, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 1:7, 16:144]
    pair = (c.q[..., :128].contiguous(), c.q[..., 128:])
    got, _ = c.run(True, (2, 0), q=pair, out=out)
    assert torch.equal(got, o)
    wide[:, 1:7, 16:144] = 0
    assert not bool(wide.any())


def test_bad_lengths_are_clamped_and_counted(cuda_dev):
    c = Case([0, 2], [100], [8, 8], [8, 8], 2)
    c.cu_p[1] = 1 << 20  # past the keys
    c.gs[1] = 99         # past the sequences
    for s in (1, (1, 1)):
        c.err.zero_()
        o, lse = mla.prefill_shared(c.q, c.k, c.v, c.k_pe, c.cu_q, c.cu_k, c.gs, c.cu_p, SCALE,
                                    num_kv_splits=s, err_count=c.err)
        assert c.err.item() > 0 and bool(o.isfinite().all())


@pytest.mark.parametrize("splits", [(2, 1), (1, 0), (2, 0)])
def test_captured(cuda_dev, splits):
    c = Case([0, 2], [700], [16, 16], [48, 48], 4)
    o = torch.empty(32, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(32, 4, device="cuda")
    c.run(True, splits, out=o, lse=lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.prefill_shared(c.q, c.k, c.v, c.k_pe, c.cu_q, c.cu_k, c.gs, c.cu_p, SCALE,
                           num_kv_splits=splits, out=o, lse=lse)
    # other lengths in the same buffers
    d = Case([0, 2], [650], [20, 12], [70, 30], 4, seed=9)
    for dst, src in ((c.q, d.q), (c.k_pe[:d.k_pe.shape[0]], d.k_pe), (c.k[:d.k.shape[0]], d.k),
                     (c.v[:d.v.shape[0]], d.v), (c.cu_q, d.cu_q), (c.cu_k, d.cu_k),
                     (c.gs, d.gs), (c.cu_p, d.cu_p)):
        dst.copy_(src)
    g.replay()
    d.check(o, lse)
