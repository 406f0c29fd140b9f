"""GPU tests of the product with bias, activation and residual against the
formula in 64 bits.

Tolerance, from the arithmetic.  The sum: K products of bf16 values, exact in
fp32, added in fp32 in any order, also with truncating steps: off by at most K
2^-23 s, s = sum |x w|; the bias adds one more step.  The activations' slopes
are below 1.2.  Their own errors, relative to act(z): expf's fast form is off by
(2 + 1.2 |u|) 2^-23 of its value at u, plus |u| 2^-22 for u's own rounding, the
reciprocal by 2^-23; the normal tail's polynomial (eight steps on values up to 2.7),
reciprocal and exponential by 12 units, plus z^2 2^-23 for its argument's rounding
(its logarithmic slope is below |z| + 1); so (16 + z^2 + 4 |u|) 2^-23 |act|
covers each, with u the exponent's argument.  The residual adds one rounding,
bf16 one of at most 2^-8 of the value.
"""
import math

import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

ACTS = (None, "relu", "silu", "gelu", "gelu_tanh")


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def rows(g, T, N, pad=0):
    """[T, N] whose rows start on 16 bytes, with `pad` x 8 further columns."""
    return normal(g, T, (N + 7) // 8 * 8 + 8 * pad)[:, :N]


def act64(name, z):
    """(act(z), the exponent's argument)."""
    if name is None:
        return z, torch.zeros_like(z)
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z), torch.zeros_like(z)
    if name == "silu":
        return z * torch.sigmoid(z), z
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2)), torch.zeros_like(z)
    u = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(u), u


def check(y, x, w, bias=None, act=None, res=None):
    K = x.shape[1]
    z = x.double() @ w.double().t()
    s = x.double().abs() @ w.double().abs().t()
    if bias is not None:
        z = z + bias.double()
        s = s + bias.double().abs()
    a, u = act64(act, z)
    ref = a if res is None else a + res.double()
    err = 1.2 * (K + 1) * 2.0 ** -23 * s + (16 + z * z + 4 * u.abs()) * 2.0 ** -23 * a.abs()
    if res is not None:
        err = err + 2.0 ** -23 * (a.abs() + res.double().abs())
    bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -7) * err + 1e-30
    d = (y.double() - ref).abs()
    assert bool((d <= bound).all()), float((d / bound).max())


SHAPES = [(1, 8, 8), (1, 64, 8192), (1, 7168, 512), (2, 65, 63), (3, 1, 1), (7, 255, 100), (16, 5120, 2048),
          (31, 257, 65), (64, 2048, 5120), (65, 1000, 512), (127, 129, 4096), (128, 128, 64),
          (129, 640, 1536), (200, 7, 72), (300, 2049, 1), (1000, 6136, 200), (1500, 4104, 128),
          (2311, 1288, 640), (5000, 72, 520)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("bias,act,residual", [(False, None, False), (True, "silu", True)])
def test_matches_64_bits(cuda_dev, T, N, K, bias, act, residual):
    g = torch.Generator("cuda").manual_seed(T * 7 + N * 3 + K)
    x, w = rows(g, T, K), rows(g, N, K)
    b = normal(g, N) if bias else None
    r = rows(g, T, N) if residual else None
    check(mla.linear(x, w, bias=b, activation=act, residual=r), x, w, b, act, r)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,N,K", [(5, 200, 96), (140, 328, 256), (700, 3000, 64)])
def test_activations(cuda_dev, act, T, N, K):
    g = torch.Generator("cuda").manual_seed(T + N + K)
    # sums of a few units, and some far out on both sides
    x, w = normal(g, T, K), (normal(g, N, K).float() / math.sqrt(K) * 3).bfloat16()
    b = normal(g, N)
    b[::7] = 30.0
    b[3::7] = -30.0
    b[5::7] = -6.0
    check(mla.linear(x, w, bias=b, activation=act), x, w, b, act)
    r = normal(g, T, N)
    check(mla.linear(x, w, bias=b, activation=act, residual=r), x, w, b, act, r)


@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (33, 136, 320), (150, 264, 64), (900, 2560, 192)])
def test_strided_and_in_place(cuda_dev, T, N, K):
    g = torch.Generator("cuda").manual_seed(N)
    x, w = rows(g, T, K, 3), rows(g, N, K, 1)
    b = normal(g, N + 8)[8:]
    full = normal(g, T, N + 24)
    keep = full.clone()
    out = full[:, 8:8 + N]  # columns of a wider buffer
    check(mla.linear(x, w, bias=b, activation="relu", out=out), x, w, b, "relu")
    assert torch.equal(full[:, :8], keep[:, :8]) and torch.equal(full[:, 8 + N:], keep[:, 8 + N:])
    stream = rows(g, T, N, 1)
    before = stream.clone()
    got = mla.linear(x, w, residual=stream, out=stream)
    assert got.data_ptr() == stream.data_ptr()
    check(stream, x, w, res=before)
    # the same bits into a tensor of its own
    assert torch.equal(mla.linear(x, w, residual=before), stream)


@pytest.mark.parametrize("T,N,K", [(40, 160, 704), (300, 1024, 128)])
def test_rows_and_columns_do_not_mix(cuda_dev, T, N, K):
    """What is not finite in one row of x, one row of W, behind K or behind a
    row's end stays out of the others."""
    g = torch.Generator("cuda").manual_seed(T)
    xb, wb = normal(g, T, K + 8), normal(g, N, K + 8)
    clean = mla.linear(xb[:, :K], wb[:, :K])
    xb[:, K:] = float("nan")
    wb[:, K:] = float("inf")
    assert torch.equal(mla.linear(xb[:, :K], wb[:, :K]), clean)
    xb[T // 2] = float("nan")
    wb[N // 3] = float("inf")
    got = mla.linear(xb[:, :K], wb[:, :K])
    rows_ok = torch.arange(T, device="cuda") != T // 2
    cols_ok = torch.arange(N, device="cuda") != N // 3
    assert torch.equal(got[rows_ok][:, cols_ok], clean[rows_ok][:, cols_ok])
    assert bool(got[T // 2].isnan().all())
    assert not bool(got[:, N // 3].isfinite().any())


def test_ends_of_the_activations(cuda_dev):
    """Large sums: 0 or the sum itself on both sides, infinities kept apart."""
    x = torch.zeros(1, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1
    z = torch.tensor([1e30, -1e30, 100.0, -100.0, -200.0, 0.0, float("inf"), 3e38],
                     device="cuda").bfloat16()
    w = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    w[:, 0] = z
    w[6, 0] = 0
    b = torch.zeros(8, dtype=torch.bfloat16, device="cuda")
    b[6] = float("inf")
    for act in ACTS:
        y = mla.linear(x, w, bias=b, activation=act)[0].double()
        ref = act64(act, z.double())[0]
        assert bool(((y - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-30)[:6].all()), (act, y)
        assert float(y[6]) == math.inf and float(y[7]) > 2.9e38


def test_refusals(cuda_dev):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        mla.linear(x.float(), w)
    with pytest.raises(ValueError):
        mla.linear(x, w[:, :32])
    with pytest.raises(ValueError):
        mla.linear(x, w, bias=x[0])
    with pytest.raises(ValueError):
        mla.linear(x, w, residual=x)
    with pytest.raises(ValueError):
        mla.linear(x, w, out=torch.zeros(4, 16, device="cuda"))
    with pytest.raises(ValueError):
        mla.linear(x.t().contiguous().t(), w)
    with pytest.raises(mla.MlaError):
        mla.linear(x[:, 1:], w[:, 1:])  # rows do not start on 16 bytes
    with pytest.raises(mla.MlaError):
        mla.linear(x, w, out=x[:, :16])
    assert mla.linear(x[:0], w).shape == (0, 16)


def test_captured(cuda_dev):
    g = torch.Generator("cuda").manual_seed(5)
    for T, N, K in ((3, 640, 2048), (200, 640, 256)):
        x, w, r = normal(g, T, K), normal(g, N, K), normal(g, T, N)
        out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
        mla.linear(x, w, residual=r, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mla.linear(x, w, residual=r, out=out)
        x.copy_(normal(g, T, K))
        r.copy_(normal(g, T, N))
        graph.replay()
        check(out, x, w, res=r)


@pytest.mark.parametrize("T,N,K", [(442, 3120, 3001), (300, 2500, 4000), (1000, 1223, 4001), (700, 1000, 6000),
                                   (257, 4090, 9000)])
@pytest.mark.parametrize("bias,act,residual", [(False, None, False), (True, "gelu_tanh", True)])
def test_split_sums(cuda_dev, T, N, K, bias, act, residual):
    """Few large tiles and long sums: two to four pairs a tile."""
    g = torch.Generator("cuda").manual_seed(T + N)
    x, w = rows(g, T, K, 1), rows(g, N, K)
    w *= 1 / math.sqrt(K)  # (in place: its rows start on 16 bytes)
    b = normal(g, N) if bias else None
    r = rows(g, T, N, 2) if residual else None
    y = mla.linear(x, w, bias=b, activation=act, residual=r)
    check(y, x, w, b, act, r)
    assert torch.equal(mla.linear(x, w, bias=b, activation=act, residual=r), y)
    full = normal(g, T, (N + 7) // 8 * 8 + 24)
    keep = full.clone()
    out = full[:, 8:8 + N]
    mla.linear(x, w, bias=b, activation=act, residual=r, out=out)
    assert torch.equal(out, y)
    assert torch.equal(full[:, :8], keep[:, :8]) and torch.equal(full[:, 8 + N:], keep[:, 8 + N:])
    if residual:
        mla.linear(x, w, bias=b, activation=act, residual=r, out=r)
        assert torch.equal(r, y)
    # a row and a column that are not finite stay alone
    x[T // 2, 3], w[N // 3, K - 1] = float("nan"), float("inf")
    z = mla.linear(x, w, bias=b)
    ref = mla.linear(x, w, bias=b).isfinite()
    assert torch.equal(z.isfinite(), ref) and not bool(ref[T // 2].any()) and not bool(ref[:, N // 3].any())
    ref[T // 2], ref[:, N // 3] = True, True
    assert bool(ref.all())
