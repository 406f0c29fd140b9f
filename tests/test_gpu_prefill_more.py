"""GPU tests of the prompt attention's rarer paths, with the definition in 64
bits, the cases and the tolerances of test_gpu_prefill."""
import math

import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_prefill import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [np.bool_(True), np.bool_(False), np.int64(1), 0])
def test_causal_as_any_truth_value(cuda_dev, causal):
    c = Case([70], [200], 2, seed=21)
    o, lse = c.run(causal)
    want = c.run(bool(causal))
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for bad in (None, "yes", 0.5):
        with pytest.raises(TypeError):
            c.run(bad)


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("n", [63, 64, 65, 130, 400])
def test_many_sequences(cuda_dev, n, splits):
    """From 64 sequences on their lengths are read from global memory; a step
    of a server has one row for most of them and none for some."""
    rng = np.random.default_rng(n)
    lq = rng.choice([0, 1, 1, 1, 1, 2, 7], n)
    lq[n // 2], lq[n - 1] = 300, 129
    lk = lq + rng.choice([0, 1, 100, 127, 300], n)
    lk[3] = 0
    c = Case(lq.tolist(), lk.tolist(), 3, seed=n, tail_q=5, tail_k=7)
    c.check(*c.run(True, splits), True, splits)
    c.check(*c.run(False, splits), False, splits)


@pytest.mark.parametrize("lq,lk,H", [([300, 40], [8900, 100], 33), ([100, 257], [17000, 300], 20),
                                     ([5], [30000], 9)])
def test_heads_that_a_group_does_not_divide(cuda_dev, lq, lk, H):
    """Few heads' keys at a time once many heads' do not fit in L2: groups of
    14 (of 33), 8 (of 20) and 8 (of 9), the last one part empty."""
    c = Case(lq, lk, H, seed=H)
    for splits in (1, 2):
        c.check(*c.run(True, splits), True, splits)


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("cols,at", [(144, 8), (136, 0), (152, 16)])
def test_output_rows_on_16_byte_boundaries(cuda_dev, cols, at, splits):
    """An output whose rows are not all on 32-byte boundaries: first address,
    head stride, row stride.  Same bits, nothing beside it written."""
    H = 3
    c = Case([70, 300, 1], [300, 300, 500], H, seed=cols)
    want = c.run(True, splits)
    c.check(*want, True, splits)
    out = torch.full((371, H, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = c.run(True, splits, out=out[..., at:at + 128])
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert bool((out[..., :at] == 7).all()) and bool((out[..., at + 128:] == 7).all())


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("sm", [1e5, 1e6, 1e8, 1e9, 1e15, 1e30])
def test_scores_beyond_any_range_of_their_weights(cuda_dev, sm, sign, splits):
    """Scores that are whole numbers times sm: exact, and so far apart that a
    row's weights are those of its largest keys, in equal parts.

    Tolerance: o as in test_gpu_prefill with no error of the scores, so e =
    2^-21: (1 + 2^-8) A (2^-8 + 2 e + 2 n 2^-23) + 2^-8 |ref|.  lse: c, m c (or m
    sm), the sum and its product with ln 2 are rounded once each, and so is the
    m c that the weights and their sum carry: below 2^-20 |ref| in all.
    Joining splits sees no more than their lse holds, so rows whose largest
    keys lie in several of them are left out there."""
    g = torch.Generator("cuda").manual_seed(7)
    T, K, H = 150, 700, 2
    whole = lambda *s: torch.randint(-8, 9, s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, kv, kp = whole(T, H, 192), whole(K, H, 256), whole(K, 64)
    if sign < 0:  # every score of a row below zero
        q, kp = q.abs() + 1, -kp.abs()
        kv[..., :128] = -kv[..., :128].abs() - 1
    kv[..., 128:] = torch.randn(K, H, 128, generator=g, device="cuda").to(torch.bfloat16)
    cu_q = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, K], dtype=torch.int32, device="cuda")
    for causal in (True, False):
        o, lse = mla.prefill(q, kv[..., :128], kv[..., 128:], kp, cu_q, cu_k, sm, causal=causal,
                             num_kv_splits=splits)
        k = torch.cat([kv[..., :128].double(), kp[:, None].double().expand(K, H, 64)], 2)
        x = torch.einsum("thd,khd->thk", q.double(), k)
        if causal:
            open_ = torch.ones(T, K, dtype=torch.bool, device="cuda").tril(K - T)
            x = x.masked_fill(~open_[:, None], -math.inf)
        top = x.amax(2, keepdim=True)
        first = x == top
        count = first.sum(2, keepdim=True).double()
        v = kv[..., 128:].double()
        ref = torch.einsum("thk,khd->thd", first / count, v)
        A = torch.einsum("thk,khd->thd", first / count, v.abs())
        ref_lse = (top * float(torch.tensor(sm, dtype=torch.float32)) + count.log())[..., 0]
        keep = torch.ones(T, H, dtype=torch.bool, device="cuda")
        if splits > 1:
            per = 256  # ceil(700 / 3) in whole tiles of 128
            parts = torch.stack([first[..., a:a + per].any(2) for a in range(0, K, per)]).sum(0)
            keep = parts == 1
        assert int(keep.sum()) > T * H // 2
        bound = ((1 + 2.0 ** -8) * A * (2.0 ** -8 + 2 * 2.0 ** -21 + 2 * K * 2.0 ** -23)
                 + 2.0 ** -8 * ref.abs())
        err = (o.double() - ref).abs()
        assert bool((err <= bound)[keep].all()), float((err - bound)[keep].max())
        lerr = (lse.double() - ref_lse).abs()
        assert bool((lerr <= 2.0 ** -20 * ref_lse.abs() + K * 2.0 ** -23)[keep].all())
