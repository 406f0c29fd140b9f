"""Outputs of the calls around the decode that would lie over an input or each
other are refused on the host before any launch (so those run without a GPU);
columns of one buffer that do not meet are taken and hold the same bits."""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_latent_abi import (ABSORB, EXPAND, GATHER, PREFILL, PROJECT, RELEASE, args, at,
                             lib)  # noqa: F401

# strides in elements, addresses in bytes: at(5) holds [10][16][256] of bf16
ROW, HEAD = 16 * 256, 256


@pytest.mark.parametrize("over", [
    dict(v=at(5)),                                    # one buffer for both
    dict(v=at(5) + 2 * 120),                          # columns that meet
    dict(v=at(5) + 2 * HEAD),                         # the next head's k_nope
    dict(v=at(5) + 2 * (3 * ROW + 2 * HEAD)),
    dict(v=at(5) - 2 * (2 * ROW + HEAD)),
    dict(v=at(5) + 2 * ROW, vhs=512, vrs=2 * 16 * 256, krs=2 * 16 * 256),   # other head strides
    dict(k=at(5), krs=16 * 128, khs=128, v=at(5) + 2 * 4096),   # k_nope dense
    dict(H=1, khs=0, vhs=0, v=at(5) + 2 * 64),
    dict(T=1, v=at(5) + 2 * HEAD),
    dict(khs=10 * 256, krs=256, vhs=10 * 256, vrs=256, v=at(5) + 2 * 256),  # head-major
    # over rows of kv_c that lie apart
    dict(c=at(1), cs=ROW, k=at(1) + 2 * 512, v=at(1) + 2 * 384, krs=ROW, khs=128, vrs=ROW, vhs=128, H=1),
    dict(c=at(1), cs=1024, k=at(1) + 2 * 256, krs=1024, khs=128, H=1),
    dict(c=at(1), cs=ROW, k=at(1) + 2 * (ROW - 128), krs=ROW, khs=256, H=2),
])
def test_expand_outputs(lib, over):  # noqa: F811
    assert lib.mla_expand_kv(*args(EXPAND, over)) == 1


@pytest.mark.parametrize("fn,base,over", [
    # out among q_nope's columns [10][16][192], and among o's [10][16][512]
    ("mla_absorb_q", ABSORB, dict(hs=1024, rs=16 * 1024, out=at(1) + 2 * 64, ohs=1024, ors=16 * 1024)),
    ("mla_absorb_q", ABSORB, dict(hs=1024, rs=16 * 1024, out=at(1) - 2 * 504, ohs=1024, ors=16 * 1024)),
    ("mla_project_v", PROJECT, dict(out=at(1) + 2 * 384, ohs=512, ors=16 * 512)),
    ("mla_project_v", PROJECT, dict(out=at(1) + 2 * 512 * 16)),
    ("mla_project_v", PROJECT, dict(hs=640, rs=16 * 640, out=at(1) + 2 * 632, ohs=640, ors=16 * 640)),
])
def test_head_product_outputs(lib, fn, base, over):  # noqa: F811
    assert getattr(lib, fn)(*args(base, over)) == 1


@pytest.mark.parametrize("over", [
    dict(cnt_out=at(2)), dict(cnt_out=at(2) + 12), dict(cnt_out=at(1) + 4), dict(cnt_out=at(4)),
    dict(cnt_out=at(4) + (9 * 8 + 7) * 4), dict(cnt_out=at(5)), dict(cnt_out=at(5) + 196),
    dict(ids=at(5) + 100),
])
def test_release_outputs(lib, over):  # noqa: F811
    assert lib.mla_blocks_release(*args(RELEASE, over)) == 1


@pytest.mark.parametrize("over", [
    # kv_c and k_pe over each other: rows of one buffer, columns that meet
    dict(k_pe=at(4)), dict(k_pe=at(4) + 2 * 512 * 99), dict(cs=576, k_pe=at(4) + 2 * 504, ps=576),
    dict(cs=576, k_pe=at(4) + 2 * (576 * 3 + 64), ps=576),
    # over the cache's blocks, dense and with room between them, and over what names the rows
    dict(kv_c=at(1)), dict(kv_c=at(1) + 2 * 64 * 576 * 5), dict(k_pe=at(1) + 2 * 64 * 576 * 8 - 16),
    dict(bstride=2 * 64 * 576, kv_c=at(1) + 2 * 64 * 576, cs=512), dict(k_pe=at(2)),
    dict(kv_c=at(2) + 16), dict(k_pe=at(3)), dict(starts=at(4) + 1024), dict(kvd=1, scale=at(5) + 4),
])
def test_gather_outputs(lib, over):  # noqa: F811
    assert lib.mla_gather_cache(*args(GATHER, over)) == 1


QROW = 16 * 192


@pytest.mark.parametrize("over", [
    # o in q's columns, at another offset and in other rows; in q_pe's
    dict(o=at(1) + 2 * 32, ors=QROW, ohs=192), dict(o=at(1) + 2 * (2 * QROW + 128), ors=QROW, ohs=192),
    dict(o=at(1) + 2 * QROW), dict(o=at(1) - 2 * 1024),
    dict(qpe=at(9), qprs=QROW, qphs=192, o=at(9) + 2 * 48, ors=QROW, ohs=192),
    # among the keys and values [30][16][256], over k_pe and the lengths
    dict(o=at(2) + 2 * ROW, ors=ROW, ohs=HEAD), dict(o=at(2) + 2 * (5 * ROW + 120), ors=ROW, ohs=HEAD),
    dict(o=at(2) + 2 * 4096), dict(o=at(3)), dict(o=at(3) + 2 * 64 * 29), dict(o=at(4)),
    dict(o=at(5) - 2 * 2048), dict(o=at(8)), dict(o=at(6)), dict(o=at(6) + 10 * 16 * 2 * 129 * 4 - 16),
    # lse and the workspace
    dict(lse=at(1) + 64), dict(lse=at(2) + 4), dict(lse=at(3)), dict(lse=at(4) + 8), dict(lse=at(5) + 8),
    dict(lse=at(6) + 400), dict(lse=at(7) + 10 * 16 * 256 - 4), dict(lse=at(7) - 636),
    dict(ws=at(1) + 32), dict(ws=at(2)), dict(ws=at(3)), dict(ws=at(4)), dict(ws=at(5) - 160000),
    dict(ws=at(7) + 32), dict(ws=at(8)),
])
def test_prefill_outputs(lib, over):  # noqa: F811
    assert lib.mla_prefill(*args(PREFILL, over)) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("splits", [1, 3])
def test_prefill_into_columns_of_its_inputs(cuda_dev, splits):
    """q, k, v and o as columns of one buffer; a workspace that is not needed
    may be anything."""
    g = torch.Generator("cuda").manual_seed(3)
    T, H = 200, 5
    buf = torch.randn(T, H, 192 + 256 + 128, generator=g, device="cuda").to(torch.bfloat16)
    kp = torch.randn(T, 64, generator=g, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 70, T], dtype=torch.int32, device="cuda")
    q, k, v, o = buf[..., :192], buf[..., 192:320], buf[..., 320:448], buf[..., 448:]
    want = mla.prefill(q.contiguous(), k.contiguous(), v.contiguous(), kp, cu, cu, 0.07,
                       num_kv_splits=splits)
    ws = torch.empty(mla.mla_prefill_workspace_bytes(T, H, splits, 128), dtype=torch.uint8,
                     device="cuda") if splits > 1 else q.contiguous()
    got = mla.prefill(q, k, v, kp, cu, cu, 0.07, num_kv_splits=splits, out=o, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 1), (1, 16), (37, 1), (200, 5), (1000, 16)])
def test_products_into_columns_of_one_buffer(cuda_dev, T, H):
    g = torch.Generator("cuda").manual_seed(T + H)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    R = 512
    c, w = normal(T, R), normal(H * 256, R)
    k, v = mla.expand_kv(c, w, H)
    halves = torch.zeros(T, H, 256, dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros(T, R + 2 * H * 128, dtype=torch.bfloat16, device="cuda")  # kv_c too
    flat[:, :R] = c
    heads = torch.zeros(H, T, 256, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    f = flat[:, R:].view(T, 2, H, 128) if T == 1 else flat[:, R:].unflatten(1, (2, H, 128))
    for x, kk, vv in ((c, halves[..., :128], halves[..., 128:]), (flat[:, :R], f[:, 0], f[:, 1]),
                      (c, heads[..., :128], heads[..., 128:]), (c, heads[..., 128:], heads[..., :128])):
        mla.expand_kv(x, w, H, k_nope=kk, v=vv)
        assert torch.equal(kk, k) and torch.equal(vv, v)
    buf = torch.zeros(T, H, 192 + R + 128, dtype=torch.bfloat16, device="cuda")
    buf[..., :192] = normal(T, H, 192)
    ql = mla.absorb_q(buf[..., :128], w, out=buf[..., 192:192 + R])
    y = mla.project_v(ql, w, out=buf[..., 192 + R:])
    assert torch.equal(ql, mla.absorb_q(buf[..., :128].contiguous(), w))
    assert torch.equal(y, mla.project_v(ql.contiguous(), w))


@pytest.mark.gpu
def test_an_unneeded_workspace_inside_an_input_is_taken(cuda_dev):
    q = torch.randn(20, 3, 192, device="cuda").to(torch.bfloat16)
    kv, kp = torch.randn(20, 3, 256, device="cuda").to(torch.bfloat16), q[:, 0, :64].contiguous()
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    want = mla.prefill(q, kv[..., :128], kv[..., 128:], kp, cu, cu, 0.07)
    got = mla.prefill(q, kv[..., :128], kv[..., 128:], kp, cu, cu, 0.07, workspace=q[5:])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
