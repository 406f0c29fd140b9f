"""GPU tests of the products with the kv_b weight against numpy in 64 bits.

Tolerance, from the arithmetic: the sums run over K = 128, 256 or 512 products
of bf16 values, exact in fp32, added in fp32; each addition is off by at most
2^-24 of a partial sum, so the sum by at most K * 2^-24 * sum |a b| (a bound
that holds for any order, also for a tree whose steps truncate: twice that).
The result is rounded once to bf16, off by at most 2^-8 of its value.  With s
= sum |a b|: |y - ref| <= 2^-8 |ref| + (1 + 2^-8) K 2^-23 s.
"""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

OPS = ("expand", "absorb", "project")


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def reference(op, x, w, H, R):
    """(value, sum of |products|) in 64 bits."""
    W = w.double().view(H, 256, R)
    x = x.double()
    def prod(a, b):
        if op == "expand":
            return torch.einsum("tr,hpr->thp", a, b)
        if op == "absorb":
            return torch.einsum("thp,hpr->thr", a, b[:, :128])
        return torch.einsum("thr,hjr->thj", a, b[:, 128:])
    return prod(x, W), prod(x.abs(), W.abs())


def call(op, x, w, H, **kw):
    if op == "expand":
        k, v = mla.expand_kv(x, w, H, **kw)
        return torch.cat([k, v], 2)
    return (mla.absorb_q if op == "absorb" else mla.project_v)(x, w, **kw)


def check(op, got, x, w, H, R):
    ref, s = reference(op, x, w, H, R)
    K = 128 if op == "absorb" else R
    bound = 2.0 ** -8 * ref.abs() + (1 + 2.0 ** -8) * K * 2.0 ** -23 * s
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("T,H,R", [
    (1, 1, 512), (1, 16, 256), (3, 5, 512), (31, 128, 256), (64, 16, 512), (127, 7, 512),
    (128, 3, 256), (129, 16, 512), (130, 128, 512), (1000, 3, 512), (4097, 2, 256), (700, 33, 256),
])
def test_matches_64_bits(cuda_dev, op, T, H, R):
    g = torch.Generator("cuda").manual_seed(T * 1000 + H + R)
    n = {"expand": (T, R), "absorb": (T, H, 128), "project": (T, H, R)}[op]
    x, w = normal(g, *n), normal(g, H * 256, R)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(op, call(op, x, w, H, err_count=err), x, w, H, R)
    assert err.item() == 0


@pytest.mark.parametrize("T,H,R", [(5, 4, 512), (200, 9, 256), (3, 1, 256)])
def test_strided_views_and_bystanders(cuda_dev, T, H, R):
    """Column slices of wider tensors, head-major outputs, a padded weight:
    same values bit for bit, and nothing else is written."""
    g = torch.Generator("cuda").manual_seed(5)
    w = normal(g, H * 256, R)
    wide_w = torch.full((H * 256, R + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_w[:, :R] = w
    q = torch.full((T + 2, H, 208), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:T, :, 8:136] = normal(g, T, H, 128)
    dense = mla.absorb_q(q[:T, :, 8:136].contiguous(), w)
    out = torch.full((T + 3, H, R + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.absorb_q(q[:T, :, 8:136], wide_w[:, :R], out=out[:T, :, :R])
    assert torch.equal(out[:T, :, :R], dense)
    assert bool((out[T:] == 3).all()) and bool((out[:, :, R:] == 3).all())
    hm = torch.full((H, T + 1, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    o = normal(g, H, T, R)
    mla.project_v(o.transpose(0, 1), w, out=hm[:, :T].transpose(0, 1))
    assert torch.equal(hm[:, :T].transpose(0, 1),
                       mla.project_v(o.transpose(0, 1).contiguous(), w))
    assert bool((hm[:, T] == 3).all())
    c = torch.full((T, R + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    c[:, :R] = normal(g, T, R)
    k = torch.full((T + 1, H, 192), 3.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full((T + 1, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    mla.expand_kv(c[:, :R], wide_w[:, :R], H, k_nope=k[:T, :, :128], v=v[:T])
    dk, dv = mla.expand_kv(c[:, :R].contiguous(), w, H)
    assert torch.equal(k[:T, :, :128], dk) and torch.equal(v[:T], dv)
    assert bool((k[T] == 3).all()) and bool((k[:, :, 128:] == 3).all()) and bool((v[T] == 3).all())


def test_special_values_stay_in_their_rows(cuda_dev):
    g = torch.Generator("cuda").manual_seed(6)
    H, R, T = 2, 512, 140
    w = normal(g, H * 256, R)
    o = normal(g, T, H, R)
    o[3, 1, 7] = float("nan")
    o[130, 0, 5] = float("inf")
    y = mla.project_v(o, w)
    bad = torch.zeros(T, H, dtype=torch.bool, device="cuda")
    bad[3, 1] = bad[130, 0] = True
    assert not bool(torch.isfinite(y[bad]).any())
    assert bool(torch.isfinite(y[~bad]).all())


def test_other_stream_and_graph(cuda_dev):
    g = torch.Generator("cuda").manual_seed(7)
    w, x = normal(g, 16 * 256, 512), normal(g, 70, 16, 128)
    ref = mla.absorb_q(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = mla.absorb_q(x, w, stream=side)
    side.synchronize()
    assert torch.equal(y, ref)
    out = torch.empty_like(ref)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        mla.absorb_q(x, w, out=out)
    x.copy_(normal(g, 70, 16, 128))
    gr.replay()
    assert torch.equal(out, mla.absorb_q(x, w))


def test_no_tokens(cuda_dev):
    w = torch.zeros(4 * 256, 256, dtype=torch.bfloat16, device="cuda")
    k, v = mla.expand_kv(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w, 4)
    assert k.shape == v.shape == (0, 4, 128)


@pytest.mark.parametrize("T,H,R", [(2047, 128, 256), (1537, 64, 512)])
def test_many_tiles(cuda_dev, T, H, R):
    """Sizes past the changes of tile width and of CTA pairs, sampled heads."""
    g = torch.Generator("cuda").manual_seed(8)
    w = normal(g, H * 256, R)
    W = w.view(H, 256, R)
    for op, shape in (("absorb", (T, H, 128)), ("expand", (T, R)), ("project", (T, H, R))):
        x = normal(g, *shape)
        y = call(op, x, w, H)
        for h in (0, H // 2, H - 1):
            xs = x if op == "expand" else x[:, h:h + 1]
            check(op, y[:, h:h + 1], xs, W[h].contiguous(), 1, R)
