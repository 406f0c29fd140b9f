"""GPU tests of the activations of mla.linear where their results are small: down to
the last bf16 value they keep their relative precision.

Tolerance: (32 + z^2 + 4 |u|) 2^-23 of the value for fp32 arithmetic, as derived in
test_gpu_linear.py, with 16 units more for a scaled exponent's rounding (2^-21) and a
power multiplied twice; a factor below the normal range is rounded by 2^-150, its
product with z by 2^-150, the result to bf16 by 2^-8 of the value or, below the normal
range, half of its steps there, 2^-134.
"""
import math

import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_linear import act64

pytestmark = pytest.mark.gpu

# from where the results are 1e-30 to where they are 0
ENDS = {"silu": (-110.0, -70.0), "gelu": (-15.0, -11.0), "gelu_tanh": (-11.5, -8.5)}


@pytest.mark.parametrize("act", list(ENDS))
@pytest.mark.parametrize("T,N,K", [(1, 4001, 8), (200, 4001, 64), (2000, 4001, 64), (300, 1000, 6000)])
def test_small_results(cuda_dev, act, T, N, K):
    lo, hi = ENDS[act]
    # multiples of 2^-9, as the sum of a bf16 weight and a bf16 bias
    z = (torch.linspace(lo, hi, N, device="cuda", dtype=torch.float64) * 512).round() / 512
    w0 = z.bfloat16()
    b = (z - w0.double()).bfloat16()
    assert torch.equal(w0.double() + b.double(), z)
    x = torch.zeros(T, (K + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :K]
    w = torch.zeros(N, (K + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :K]
    x[:, K - 1] = 1
    w[:, K - 1] = w0
    y = mla.linear(x, w, bias=b, activation=act)
    assert torch.equal(y, y[:1].expand(T, N))
    ref, u = act64(act, z)
    err = (32 + z * z + 4 * u.abs()) * 2.0 ** -23 * ref.abs() + (1 + z.abs()) * 2.0 ** -150
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -134 + (1 + 2.0 ** -7) * err
    d = (y[0].double() - ref).abs()
    worst = int((d / bound).argmax())
    assert bool((d <= bound).all()), (float(z[worst]), float(y[0, worst]), float(ref[worst]))
    # both sides of the normal range's end, and zeros, are among them
    assert bool((ref.abs() < 2.0 ** -135).any()) and bool((ref.abs() > 2.0 ** -120).any())


def test_ends(cuda_dev):
    z = [0.0, -0.0, 1e-36, -1e-36, 1e38, 3e38, -1e30, -3e38]
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = torch.tensor(z)
    ref = w[:, 0].double()
    for act in ENDS:
        y = mla.linear(x, w, activation=act)[0].double()
        assert bool((y[:2] == 0).all()) and bool((y[6:] == 0).all())
        assert bool(((y[2:4] - 0.5 * ref[2:4]).abs() <= 2.0 ** -8 * 0.5 * ref[2:4].abs()).all())
        assert torch.equal(y[4:6], ref[4:6])
        for end, want in ((math.inf, math.inf), (math.nan, math.nan)):
            b = torch.full((8,), end, dtype=torch.bfloat16, device="cuda")
            assert bool(torch.equal(mla.linear(x, w, bias=b, activation=act)[0].float().nan_to_num(7.0),
                                    torch.full((8,), want, device="cuda").nan_to_num(7.0)))
