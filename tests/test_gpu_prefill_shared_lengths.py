"""GPU tests of cumulative lengths outside the tensors in prefill_shared: clamped
and counted once a sequence as by prefill, whichever way own keys are worked on."""
import math

import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)
T, TK, H, PRE = 60, 400, 3, 150
CU_Q = [0, 10, 10, 33, 60]
CU_K = [150, 200, 210, 300, 400]

BAD = [  # (cu_q, cu_k, sequences that count)
    (CU_Q, CU_K, 0),
    (CU_Q, [-5, 200, 210, 300, 400], 1),
    (CU_Q, [150, 200, 210, 300, 900], 1),
    (CU_Q, [150, 200, 210, 500, 900], 2),
    (CU_Q, [-9, -5, 210, 300, 1 << 30], 3),
    ([0, 10, 10, 33, 71], CU_K, 1),
    ([0, 10, 10, 61, 1 << 30], CU_K, 2),          # the last one has no rows
    ([0, 10, 10, 61, 1 << 30], [-1, 200, 210, 300, 401], 3),
    ([-4, 10, 10, 33, 60], CU_K, 1),
    ([-40, -3, 10, 33, 64], [0, 200, 210, 300, 400], 3),
]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def clamped(cu, n):
    return [min(max(x, 0), n) for x in cu]


class Batch:
    def __init__(self):
        g = torch.Generator("cuda").manual_seed(2)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.q, self.k, self.v = normal(T, H, 192), normal(TK, H, 128), normal(TK, H, 128)
        self.k_pe = normal(TK, 64)
        self.err = i32([0])

    def run(self, cu_q, cu_k, splits, causal, prefix=PRE, groups=(0, 3)):
        self.err.zero_()
        out = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(T, H, device="cuda")
        mla.prefill_shared(self.q, self.k, self.v, self.k_pe, i32(cu_q), i32(cu_k),
                           i32(list(groups)), i32([0, prefix]), SCALE, causal=causal,
                           num_kv_splits=splits, out=out, lse=lse, err_count=self.err)
        return out, lse, self.err.item()


@pytest.mark.parametrize("splits", [(1, 0), (2, 0), (1, 1), (3, 2)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cu_q,cu_k,count", BAD)
def test_lengths_are_clamped_and_counted(cuda_dev, cu_q, cu_k, count, causal, splits):
    b = Batch()
    o, lse, err = b.run(cu_q, cu_k, splits, causal)
    ref, ref_lse, none = b.run(clamped(cu_q, T), clamped(cu_k, TK), splits, causal)
    assert none == 0
    assert torch.equal(o, ref) and torch.equal(lse, ref_lse)
    assert err == count


@pytest.mark.parametrize("splits", [(1, 0), (1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cu_q,cu_k,count", BAD)
def test_as_prefill_without_a_prefix(cuda_dev, cu_q, cu_k, count, causal, splits):
    b = Batch()
    o, lse, err = b.run(cu_q, cu_k, splits, causal, prefix=0)
    out, plse = torch.zeros_like(o), torch.zeros_like(lse)
    b.err.zero_()
    mla.prefill(b.q, b.k, b.v, b.k_pe, i32(cu_q), i32(cu_k), SCALE, causal=causal, out=out, lse=plse,
                err_count=b.err)
    assert b.err.item() == err == count
    assert torch.equal(lse == -math.inf, plse == -math.inf)
    # Each is off from 64 bits by what test_gpu_prefill_shared.py derives: P's and the
    # output's rounding, 2^-8 each, weights' factors within 1 +- e, of means that the
    # largest |v| bounds; and by ds in a score, so in the lse.
    k = torch.cat([b.k.double(), b.k_pe.double()[:, None].expand(TK, H, 64)], 2)
    S = float(torch.einsum("ihd,jhd->hij", b.q.double().abs(), k.abs()).max()) * SCALE
    ds = 192 * 2.0 ** -23 * S
    e = 2 * (1.01 * (ds + 2.0 ** -22 * S) + 2.0 ** -21)
    v = float(b.v.abs().max())
    one = (1 + 2.0 ** -8) * (2 * 2.0 ** -8 + 2 * e + 2 * TK * 2.0 ** -23) * v
    assert bool(((o.double() - out.double()).abs() <= 2 * one).all())
    dead = lse == -math.inf
    bl = ds + 2.0 ** -22 * S + e + TK * 2.0 ** -23 + 2.0 ** -22 * (S + math.log(TK))
    assert float((lse - plse)[~dead].abs().max()) <= 2 * bl


@pytest.mark.parametrize("splits", [(1, 0), (1, 1)])
def test_prefixes_are_counted_once(cuda_dev, splits):
    b = Batch()
    assert b.run(CU_Q, CU_K, splits, True, prefix=500)[2] == 1
    # many sequences, most of them past the rows; none of a group
    n = 300
    assert b.run(list(range(n + 1)), [400] * (n + 1), splits, True, groups=(0, 0))[2] == n - T


@pytest.mark.parametrize("causal", [True, False])
def test_starts_that_decrease_stay_in_the_tensors(cuda_dev, causal):
    """Not allowed, so only the first sequence's rows are told; its keys end where the
    tensors do, and a later sequence's start far before them."""
    b = Batch()
    b.v[TK - 1, 0, 5] = math.inf  # of the first sequence's last key: read again for its rows
    cu_q, cu_k = [0, 20, 20, 60], [TK - 100, TK, 10, TK]
    o, lse, err = b.run(cu_q, cu_k, (1, 0), causal, groups=(0, 3))
    ref, ref_lse, _ = b.run([0, 20], cu_k[:2], (1, 0), causal, groups=(0, 1))
    assert err == 1  # the empty sequence whose end lies before its start
    assert torch.equal(lse[:20], ref_lse[:20])
    assert torch.equal(o[:20].isfinite(), ref[:20].isfinite())
