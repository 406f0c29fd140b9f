"""GPU tests of the decode behind shared prefixes against the definition in 64
bits.

Tolerances, from the arithmetic.  A score is a sum of R + 64 products, exact in
fp32 (fp8 codes are exact in bf16, their scale goes into the factor of the score),
added in fp32: off by at most ds = (R + 64) 2^-23 S, S the largest sm_scale * sum |q k|;
factor, exponent and its difference to the maximum by another 2^-21 S.  So a weight
is off by a factor within 1 +- e, e = 1.01 (ds + 2^-21 S) + 2^-21 (the exponential),
and joining parts takes one more weight each.  P is rounded to bf16 (2^-8), the sum of
weights is not; P.V adds n terms in fp32 (n 2^-23), and the result is rounded to bf16
(2^-8) after a multiplication or two (2^-22).
"""
import math

import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """Groups of sequences with whole pages of the prefix in common; the page that a
    prefix ends in is each sequence's own copy.  lens < prefix: read from pages of
    its own."""

    def __init__(self, groups, prefix, lens, H, R=512, fmt="bf16", bs=64, rows=1, seed=0,
                 scale=0.05, extra=0, spare=5):
        g = torch.Generator("cuda").manual_seed(seed)
        self.groups, self.prefix, self.lens, self.H, self.R = groups, prefix, lens, H, R
        self.fmt, self.bs, self.rows = fmt, bs, rows
        D, B = R + 64, len(lens)
        group = [max([i for i in range(len(prefix)) if groups[i] <= b < groups[i + 1]],
                     default=None) for b in range(B)]
        self.group = group
        whole = [p // bs for p in prefix]
        need, at = [], sum(whole)
        first = [sum(whole[:i]) for i in range(len(whole))]
        for b, n in enumerate(lens):
            i = group[b]
            need.append(-(-n // bs) - (whole[i] if i is not None and n >= prefix[i] else 0))
        nb = sum(whole) + sum(need) + spare
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        maxb = max([1] + [-(-n // bs) for n in lens]) + extra
        cache = torch.randn(nb, bs, D, generator=g, device="cuda").bfloat16()
        self.table = torch.full((B, maxb), -7, dtype=torch.int32, device="cuda")
        for b, n in enumerate(lens):
            i, k = group[b], 0
            if i is not None and n >= prefix[i]:
                k = whole[i]
                self.table[b, :k] = perm[first[i]:first[i] + k]
            self.table[b, k:k + need[b]] = perm[at:at + need[b]]
            if i is not None and n >= prefix[i] and prefix[i] % bs:
                leader = min(x for x in range(groups[i], groups[i + 1]) if lens[x] >= prefix[i])
                if leader != b:
                    src = cache[self.table[leader, k].long(), :prefix[i] % bs].clone()
                    cache[perm[at].long(), :prefix[i] % bs] = src
            at += need[b]
        self.scale = None
        if fmt != "bf16":
            cache = (cache.float() / scale).to(FP8[fmt])
            self.scale = torch.tensor([scale], device="cuda")
        self.cache = cache
        self.q = torch.randn(B * rows, H, D, generator=g, device="cuda").bfloat16()
        self.seq_lens, self.gs, self.pre = i32(lens), i32(groups), i32(prefix)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, sm=SCALE, **kw):
        o, lse = mla.decode_shared(kw.pop("q", self.q), self.cache, self.table, self.seq_lens,
                                   self.gs, self.pre, sm, kv_lora_rank=self.R,
                                   kv_scale=self.scale, err_count=self.err, **kw)
        torch.cuda.synchronize()
        assert self.err.item() == 0
        return o, lse

    def keys(self, b):
        n = self.lens[b]
        blocks = self.table[b, :-(-n // self.bs)].long()
        c = self.cache
        if c.dtype != torch.bfloat16:
            c = c.view(torch.uint8)[blocks].reshape(-1, self.R + 64)[:n].view(c.dtype)
            return c.to(torch.float32).double() * self.scale.double()
        return c[blocks].reshape(-1, self.R + 64)[:n].double()

    def check(self, o, lse, sm=SCALE):
        for b, n in enumerate(self.lens):
            rows = slice(b * self.rows, (b + 1) * self.rows)
            if n == 0:
                assert bool((o[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())
                continue
            k = self.keys(b)
            q = self.q[rows].double().reshape(-1, self.R + 64)
            x = q @ k.t() * sm
            S = float((q.abs() @ k.abs().t()).max() * abs(sm))
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            ref, A = p @ k[:, :self.R], p @ k[:, :self.R].abs()
            ds = (self.R + 64) * 2.0 ** -23 * S
            e = 2 * (1.01 * (ds + 2.0 ** -21 * S) + 2.0 ** -21)
            bound = (1 + 2.0 ** -8) * A * (2.0 ** -8 + 2 * e + 2 * n * 2.0 ** -23) \
                + (2.0 ** -8 + 2.0 ** -21) * ref.abs()
            got = o[rows].double().reshape(-1, self.R)
            assert bool(((got - ref).abs() <= bound).all()), (b, float(((got - ref).abs() / bound).max()))
            bl = ds + 2.0 ** -21 * S + e + n * 2.0 ** -23 + 2.0 ** -21 * z.abs()
            assert bool(((lse[rows].double().reshape(-1) - z).abs() <= bl).all()), b


CASES = [
    # groups, prefixes, lengths, heads, more
    (([0, 1], [128], [128], 16), {}),
    (([0, 2], [128], [128, 129], 1), {}),
    (([0, 4], [512], [513, 520, 575, 512], 16), {}),
    (([0, 3], [100], [101, 300, 227], 5), {}),                       # shorter than a tile
    (([0, 3], [0], [1, 64, 200], 16), {}),
    (([0, 7], [700], [701, 0, 900, 0, 30, 1000, 0], 16), {}),        # padded, one shorter
    (([0, 3], [400], [0, 399, 0], 16), {}),                          # nobody has the prefix
    (([0, 5], [1000], [5, 0, 1000, 1001, 2000], 7), dict(rows=3)),   # the first ones are shorter
    (([0, 2, 2, 6], [300, 64, 1500], [333, 400, 1501, 1600, 1777, 1500], 128), {}),
    (([1, 3, 5], [256, 384], [90, 300, 260, 384, 500, 77], 32), {}),  # some of no group
    (([0, 40], [2050], [2050 + 13 * i for i in range(40)], 16), {}),
    (([0, 64], [8192], [8200 + 7 * i for i in range(64)], 16), {}),
    (([0, 3], [4096], [4100, 4097, 9000], 96), {}),
    (([0, 30], [640], [641 + i for i in range(30)], 20), dict(rows=2)),
    (([4 * i for i in range(26)], [150 + 9 * i for i in range(25)],
      [500 + 3 * i for i in range(100)], 2), {}),
    (([0, 1, 2], [5000, 4000], [5003, 4500], 128), {}),               # groups of one
]


@pytest.mark.parametrize("fmt,R", [("bf16", 512), ("bf16", 256), ("e4m3", 512), ("e4m3", 256),
                                   ("e5m2", 512)])
@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_matches_64_bits(cuda_dev, case, fmt, R):
    args, kw = case
    c = Case(*args, R=R, fmt=fmt, seed=len(args[2]), **kw)
    c.check(*c.run())


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("fmt,R", [("bf16", 512), ("e4m3", 256)])
def test_page_sizes(cuda_dev, bs, fmt, R):
    c = Case([0, 5, 9], [777, 1025], [790, 900, 777, 1100, 0, 1026, 1300, 1025, 2000], 16, R=R,
             fmt=fmt, bs=bs, seed=bs, extra=3)
    c.check(*c.run())


def test_scores_of_any_scale(cuda_dev):
    c = Case([0, 3], [256], [300, 270, 400], 16)
    for sm in (-0.05, 0.0, 3.0, 1e-6):
        c.check(*c.run(sm=sm), sm=sm)


def test_growing_maximum(cuda_dev):
    """Every tile's largest score beyond the last one's: O is rescaled each time."""
    c = Case([0, 3], [1024], [1300, 1100, 1024], 16, seed=3)
    ramp = torch.linspace(0.2, 6, 21, device="cuda")
    for b in range(3):
        n = c.lens[b]
        for p in range(-(-n // 64)):
            blk = c.table[b, p].long()
            c.cache[blk] = c.cache[blk].sign() * ramp[p].bfloat16()
    c.check(*c.run())


def test_ends_of_pages_have_no_influence(cuda_dev):
    c = Case([0, 3], [200], [210, 333, 250], 16, seed=5)
    o, lse = c.run()
    used = torch.zeros(c.cache.shape[0], 64, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.lens):
        for p in range(-(-n // 64)):
            used[c.table[b, p].long(), :min(64, n - 64 * p)] = True
    c.cache[~used] = float("nan")
    o2, lse2 = c.run()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_row_that_is_not_finite_stays_alone(cuda_dev):
    c = Case([0, 4], [256], [300, 280, 100, 290], 16, seed=6)
    o, lse = c.run()
    c.q[1, 3, 5] = float("nan")
    blk = c.table[3, 4].long()
    c.cache[blk, 10] = float("inf")   # an own token of the last sequence
    blk = c.table[2, 0].long()
    c.cache[blk, 0] = float("nan")    # the sequence that is shorter than the prefix
    o2, lse2 = c.run()
    assert torch.equal(o2[0], o[0]) and torch.equal(lse2[0], lse[0])
    others = torch.arange(16, device="cuda") != 3
    assert torch.equal(o2[1][others], o[1][others])
    assert bool(o2[1, 3].isnan().all()) and bool(o2[2].isnan().all())
    assert bool(lse2[3].isnan().all() | lse2[3].isinf().all()) or not bool(o2[3].isfinite().all())


def test_pair_of_q_and_determinism(cuda_dev):
    c = Case([0, 20], [3000], [3001 + 11 * i for i in range(20)], 16, seed=7)
    o, lse = c.run()
    a = c.run()
    assert torch.equal(o, a[0]) and torch.equal(lse, a[1])
    b = c.run(q=(c.q[..., :512].contiguous(), c.q[..., 512:]))
    assert torch.equal(o, b[0]) and torch.equal(lse, b[1])


def test_close_to_decode(cuda_dev):
    c = Case([0, 12], [1500], [1501 + 31 * i for i in range(12)], 32, seed=8)
    o, lse = c.run()
    o2, lse2 = mla.decode(c.q, c.cache, c.table.clamp(min=0), c.seq_lens, SCALE, 4)
    assert float((o.float() - o2.float()).abs().max()) < 2e-2
    assert float((lse - lse2).abs().max()) < 1e-4


def test_bad_ids_and_lengths_are_counted(cuda_dev):
    c = Case([0, 2], [128], [200, 190], 16, seed=9)
    c.table[1, 2] = 10 ** 6
    args = (c.q, c.cache, c.table, c.seq_lens, c.gs, c.pre, SCALE)
    o, lse = mla.decode_shared(*args, err_count=c.err)
    assert c.err.item() == 1
    # its tokens read as zeros
    z = c.cache[c.table[1, :2].long()].reshape(-1, 576).double()
    k = torch.cat([z, z.new_zeros(62, 576)])
    x = c.q[1].double() @ k.t() * SCALE
    ref = torch.softmax(x, 1) @ k[:, :512]
    assert float((o[1].double() - ref).abs().max()) < 2e-2
    c.table[1, 2] = 0
    c.err.zero_()
    c.seq_lens[0] = 10 ** 6
    c.pre[0] = -3
    c.gs[1] = 99
    c.table.clamp_(min=0)
    mla.decode_shared(*args, err_count=c.err)
    assert c.err.item() == 2


def test_refusals(cuda_dev):
    c = Case([0, 2], [128], [200, 190], 16)
    a = dict(q=c.q, kv_cache=c.cache, block_table=c.table, seq_lens=c.seq_lens, group_seqs=c.gs,
             prefix_lens=c.pre, sm_scale=SCALE)
    for over in (dict(q=c.q.float()), dict(q=c.q[..., :512]), dict(block_table=c.table[:1]),
                 dict(group_seqs=c.gs[:1]), dict(prefix_lens=c.gs), dict(seq_lens=c.seq_lens.long()),
                 dict(kv_lora_rank=576), dict(out=c.q[..., :512]),
                 dict(kv_cache=c.cache.float())):
        with pytest.raises(ValueError):
            mla.decode_shared(**{**a, **over})
    need = mla.mla_decode_shared_workspace_bytes(
        2, 16, 2, 1, 512, torch.cuda.get_device_properties(0).multi_processor_count)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    mla.decode_shared(**a, workspace=ws)
    with pytest.raises(mla.MlaError, match="WORKSPACE"):
        mla.decode_shared(**a, workspace=ws[:need - 256])
    with pytest.raises(mla.MlaError):
        mla.decode_shared(**a, workspace=ws[16:])


def test_captured_and_replayed_with_other_lengths(cuda_dev):
    c = Case([0, 8], [900], [1000 + i for i in range(8)], 16, seed=11, extra=40, spare=100)
    o = torch.empty(8, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(8, 16, device="cuda")
    c.run(out=o, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.decode_shared(c.q, c.cache, c.table, c.seq_lens, c.gs, c.pre, SCALE, out=o, lse=lse)
    for other in (([0, 8], [300], [0, 350, 301, 1000, 7, 0, 300, 999], 16),
                  ([0, 5], [1200], [1300 + 40 * i for i in range(5)] + [0, 60, 700], 16)):
        d = Case(*other, seed=len(other[1]) + other[1][0])
        c.cache[:d.cache.shape[0]].copy_(d.cache)
        c.table[:, :d.table.shape[1]].copy_(d.table)
        for x, y in ((c.q, d.q), (c.seq_lens, d.seq_lens), (c.gs, d.gs), (c.pre, d.pre)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        d.check(o, lse)


@pytest.mark.parametrize("fmt,R", [("e4m3", 512), ("e5m2", 256)])
def test_every_finite_code(cuda_dev, fmt, R):
    """Subnormal codes and the largest ones among them; those that are not finite
    give NaN or infinities for their sequence alone."""
    c = Case([0, 3], [256], [300, 260, 400], 8, R=R, fmt=fmt, seed=12, scale=2.0 ** -7)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes = codes[codes.view(FP8[fmt]).float().isfinite()]
    g = torch.Generator("cuda").manual_seed(4)
    raw = codes[torch.randint(len(codes), c.cache.shape, generator=g, device="cuda")]
    # the largest codes alone would leave one key to every softmax
    small = codes[codes.view(FP8[fmt]).float().abs() < 16]
    raw[..., 8:] = small[torch.randint(len(small), raw[..., 8:].shape, generator=g, device="cuda")]
    c.cache = raw.view(FP8[fmt])
    c.q[..., :8] = 0
    sm = SCALE
    c.check(*c.run(sm=sm), sm=sm)
    o, lse = c.run(sm=sm)
    raw[c.table[2, 5].long(), 3, 40] = 0x7F   # a NaN in an own token of the last one
    o2, lse2 = c.run(sm=sm)
    assert torch.equal(o[:2], o2[:2]) and torch.equal(lse[:2], lse2[:2])
    assert not bool(o2[2].isfinite().all())


def test_many_sequences(cuda_dev):
    """More parts than one warp lists by itself."""
    lens = [(37 * i) % 500 + (300 if i % 3 else 0) for i in range(700)]
    c = Case([0, 250, 250, 600, 640], [256, 100, 130, 384], lens, 2, seed=13, bs=128)
    c.check(*c.run())
    many = [128 + i % 70 for i in range(1200)]
    c = Case([2 * i for i in range(601)], [128] * 600, many, 1, R=256, seed=14)
    c.check(*c.run())


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
def test_scores_of_minus_infinity(cuda_dev, fmt):
    """Whole tiles of them, the first ones among them, have no weight."""
    c = Case([0, 3], [512], [700, 900, 520], 16, fmt=fmt, seed=14)
    c.q[..., 520] = c.q[..., 520].abs() + 0.1
    kept = c.keys

    def put(b, first, last):
        for t in range(first, last):
            c.cache[c.table[b, t // 64].long(), t % 64, 520] = -math.inf

    put(0, 0, 128), put(0, 256, 300), put(1, 512, 700)
    o, lse = c.run()
    for b, n in enumerate(c.lens):
        k = kept(b)
        out = torch.isinf(k[:, 520])
        k[:, 520] = torch.where(out, 0.0, k[:, 520])
        x = c.q[b].double() @ k.t() * SCALE
        x[:, out] = -math.inf
        z = torch.logsumexp(x, 1)
        ref = torch.exp(x - z[:, None]) @ k[:, :512]
        # P and o are rounded to bf16, 2^-8 each; the sums' share is far smaller
        bound = 2 ** -7 * 1.1 * torch.exp(x - z[:, None]) @ k[:, :512].abs() + 1e-4
        assert bool(((o[b].double() - ref).abs() <= bound).all()), b
        assert float((lse[b].double() - z).abs().max()) < 1e-3


@pytest.mark.parametrize("fmt,R", [("bf16", 512), ("e4m3", 256)])
@pytest.mark.parametrize("groups,prefix,lens", [
    ([0, 5], [222], [300, 171, 222, 130, 128]),
    ([0, 4, 9], [383, 129], [382, 383, 256, 500, 128, 129, 128, 700, 129]),
    ([0, 6], [1000], [999, 1000, 896, 897, 1100, 1023])])
def test_longer_than_the_shared_tiles_shorter_than_the_prefix(cuda_dev, groups, prefix, lens, fmt, R):
    """Those are decoded by themselves: their first tokens are their own."""
    c = Case(groups, prefix, lens, 16, R=R, fmt=fmt, seed=sum(lens))
    c.check(*c.run())
