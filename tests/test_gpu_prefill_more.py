"""GPU tests of the prompt attention's rarer paths, with the definition in 64
bits, the cases and the tolerances of test_gpu_prefill."""
import numpy as np
import pytest
import torch

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
