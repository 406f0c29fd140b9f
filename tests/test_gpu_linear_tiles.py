"""GPU tests of mla.linear with several tiles for each pair of CTAs, which go on in
accumulators that have been used: every width of a pair's tile, with four and more tiles
a pair, odd sizes, strided and in place.  Tolerances as in test_gpu_linear.py."""
import math

import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_linear import check, normal, rows
from test_linear_plan import linear_plan

pytestmark = pytest.mark.gpu

SHAPES = [  # tokens, out_features, in_features; columns of a tile
    (7999, 5111, 504, 256), (20001, 1000, 72, 256), (6001, 4104, 1000, 256),
    (80001, 185, 136, 192), (80003, 192, 65, 192), (80001, 121, 72, 128),
]


def plan_is(T, N, K, bn):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms < 140 or sms > 160:
        pytest.skip("other tiles on other devices")
    assert linear_plan(T, N, K, sms).key() == ("pair", bn, 1)
    assert -(-T // 256) * -(-N // bn) >= 4 * (sms // 2)


@pytest.mark.parametrize("T,N,K,bn", SHAPES)
@pytest.mark.parametrize("bias,act,residual", [(False, None, False), (True, None, True),
                                               (True, "silu", True), (True, "gelu", False)])
def test_many_tiles(cuda_dev, T, N, K, bn, bias, act, residual):
    plan_is(T, N, K, bn)
    g = torch.Generator("cuda").manual_seed(T + N)
    x, w = rows(g, T, K, 1), rows(g, N, K)
    w *= 1 / math.sqrt(K)  # (in place: its rows start on 16 bytes)
    b = normal(g, N) if bias else None
    r = rows(g, T, N, 2) if residual else None
    y = mla.linear(x, w, bias=b, activation=act, residual=r)
    check(y, x, w, b, act, r)
    assert torch.equal(mla.linear(x, w, bias=b, activation=act, residual=r), y)
    # columns of a wider buffer; what lies beside them stays
    full = normal(g, T, (N + 7) // 8 * 8 + 24)
    keep = full.clone()
    mla.linear(x, w, bias=b, activation=act, residual=r, out=full[:, 8:8 + N])
    assert torch.equal(full[:, 8:8 + N], y)
    assert torch.equal(full[:, :8], keep[:, :8]) and torch.equal(full[:, 8 + N:], keep[:, 8 + N:])
    if residual:
        mla.linear(x, w, bias=b, activation=act, residual=r, out=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("T,N,K,bn", [SHAPES[0], SHAPES[3]])
def test_what_is_not_finite_stays_in_its_row_and_column(cuda_dev, T, N, K, bn):
    plan_is(T, N, K, bn)
    g = torch.Generator("cuda").manual_seed(N)
    x, w = rows(g, T, K), rows(g, N, K)
    clean = mla.linear(x, w)
    x[T - 300, 3], w[N // 3, K - 1] = float("nan"), float("inf")
    got = mla.linear(x, w)
    finite = got.isfinite()
    assert not bool(finite[T - 300].any()) and not bool(finite[:, N // 3].any())
    got[T - 300], got[:, N // 3] = clean[T - 300], clean[:, N // 3]
    assert torch.equal(got, clean)


def test_captured(cuda_dev):
    T, N, K, bn = SHAPES[1]
    plan_is(T, N, K, bn)
    g = torch.Generator("cuda").manual_seed(5)
    x, w, r = normal(g, T, K), normal(g, N, K), normal(g, T, N)
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    mla.linear(x, w, residual=r, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mla.linear(x, w, residual=r, out=out)
        mla.linear(x, w, residual=out, out=out)
    x.copy_(normal(g, T, K))
    r.copy_(normal(g, T, N))
    graph.replay()
    one = mla.linear(x, w, residual=r)
    check(one, x, w, res=r)
    assert torch.equal(out, mla.linear(x, w, residual=one))
