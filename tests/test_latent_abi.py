"""The C entry points around the decode (batch tables, gather, kv_b products,
prompt attention) reject bad arguments on the host before any launch, and the
Python calls bad tensors; so these run without a GPU."""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from mla_paged_kv_concat_gb300 import _lib, build

FAKE = 1 << 12  # an aligned non-null host address; validation never dereferences


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def at(i):
    """Distinct fake buffers, far apart."""
    return FAKE + (i << 24)


def args(base, over):
    a = dict(base)
    for k in over:
        assert k in a, k
    a.update(over)
    return list(a.values())


BATCH = dict(ids=at(1), ql=at(2), ctx=at(3), n=4, table=at(4), ts=8, rows=10, maxb=8, bs=16, nb=100,
             free=at(5), cap=50, cnt=at(6), cnt_out=at(7), T=20, bt=at(8), bts=8, sl=at(9),
             cuq=at(10), cuk=at(11), pos=at(12), slot=at(13), err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ql=None), 1), (dict(ctx=None), 1), (dict(table=None), 1), (dict(free=None), 1),
    (dict(cnt=None), 1), (dict(cnt_out=None), 1), (dict(bt=None), 1), (dict(sl=None), 1),
    (dict(cuq=None), 1), (dict(cuk=None), 1), (dict(pos=None), 1), (dict(slot=None), 1),
    (dict(n=-1), 1), (dict(n=8193), 2), (dict(rows=0), 1), (dict(maxb=0), 1), (dict(bs=0), 1),
    (dict(bs=1025), 1), (dict(nb=0), 1), (dict(cap=-1), 1), (dict(T=-1), 1),
    (dict(ts=7), 1), (dict(bts=7), 1), (dict(maxb=1 << 20, ts=1 << 20, bts=1 << 20, bs=1024), 1),
    (dict(maxb=(1 << 20) + 1, ts=1 << 21, bts=1 << 21, bs=1024), 2),
    (dict(ctx=at(3) + 2), 1), (dict(pos=at(12) + 4), 1), (dict(slot=at(13) + 4), 1),
    # outputs over inputs or each other
    (dict(sl=at(3)), 1), (dict(sl=at(2) + 8), 1), (dict(bt=at(4) + 64), 1), (dict(cuq=at(9)), 1),
    (dict(cuk=at(10) + 16), 1), (dict(slot=at(12)), 1), (dict(cnt_out=at(5)), 1),
    (dict(cuq=at(1)), 1),
])
def test_batch_build_refusals(lib, over, code):
    # the 2^20-page row makes the two tables' fake buffers overlap: refused too
    assert lib.mla_batch_build(*args(BATCH, over)) == code


RELEASE = dict(ids=at(1), held=at(2), n=4, table=at(4), ts=8, rows=10, maxb=8, bs=16, nb=100,
               free=at(5), cap=50, cnt=at(6), cnt_out=at(6), err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(held=None), 1), (dict(table=None), 1), (dict(free=None), 1), (dict(cnt=None), 1),
    (dict(cnt_out=None), 1), (dict(n=-1), 1), (dict(n=9000), 2), (dict(bs=0), 1), (dict(ts=7), 1),
    (dict(n=8192, maxb=1 << 18, ts=1 << 18, bs=1), 2), (dict(cnt=at(5) + 4), 1),
    (dict(held=at(5) + 8), 1), (dict(table=at(5) - 128), 1), (dict(cnt_out=at(6) + 1), 1),
])
def test_blocks_release_refusals(lib, over, code):
    assert lib.mla_blocks_release(*args(RELEASE, over)) == code


GATHER = dict(cache=at(1), kvd=0, nb=8, bs=64, bstride=64 * 576, R=512, P=64, bt=at(2), bts=4,
              maxb=4, cu=at(3), starts=None, seqs=2, T=100, scale=None, kv_c=at(4), cs=512,
              k_pe=at(5), ps=64, err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(cache=None), 1), (dict(bt=None), 1), (dict(cu=None), 1), (dict(kv_c=None), 1),
    (dict(k_pe=None), 1), (dict(kvd=1), 1), (dict(kvd=2), 1), (dict(kvd=3, scale=at(6)), 1),
    (dict(R=384), 2), (dict(P=32), 2), (dict(T=-1), 1), (dict(seqs=-1), 1), (dict(nb=0), 1),
    (dict(bs=0), 1), (dict(bs=1025), 1), (dict(maxb=0), 1), (dict(bts=3), 1),
    (dict(bstride=64 * 576 - 8), 1), (dict(bstride=64 * 576 + 4), 1), (dict(cache=at(1) + 8), 1),
    (dict(cs=508), 1), (dict(cs=516), 1), (dict(ps=63), 1), (dict(kv_c=at(4) + 8), 1),
    (dict(k_pe=at(5) + 2), 1), (dict(cu=at(3) + 1), 1),
])
def test_gather_refusals(lib, over, code):
    assert lib.mla_gather_cache(*args(GATHER, over)) == code


EXPAND = dict(c=at(1), cs=512, T=10, w=at(2), ws=512, H=16, R=512, nope=128, vd=128, k=at(5),
              krs=16 * 256, khs=256, v=at(5) + 256, vrs=16 * 256, vhs=256, err=None, stream=None)
ABSORB = dict(x=at(1), rs=16 * 192, hs=192, T=10, w=at(2), ws=512, H=16, R=512, nope=128, vd=128,
              out=at(5), ors=16 * 512, ohs=512, err=None, stream=None)
PROJECT = dict(x=at(1), rs=16 * 512, hs=512, T=10, w=at(2), ws=512, H=16, R=512, nope=128, vd=128,
               out=at(5), ors=16 * 128, ohs=128, err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(c=None), 1), (dict(w=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(T=-1), 1),
    (dict(H=0), 1), (dict(H=1025), 1), (dict(R=384), 2), (dict(nope=64), 2), (dict(vd=64), 2),
    (dict(cs=504), 1), (dict(cs=516), 1), (dict(ws=504), 1), (dict(ws=520 + 4), 1),
    (dict(ws=(1 << 20) + 8), 1), (dict(c=at(1) + 8), 1), (dict(w=at(2) + 2), 1),
    (dict(k=at(5) + 8), 1), (dict(khs=120), 1), (dict(khs=0), 1), (dict(krs=-8), 1),
    (dict(krs=1 << 39), 1), (dict(krs=2048, khs=256), 1),   # rows that overlap
    (dict(k=at(1)), 1), (dict(v=at(2) + 16 * 256 * 512 * 2 - 16), 1),
])
def test_expand_refusals(lib, over, code):
    assert lib.mla_expand_kv(*args(EXPAND, over)) == code


@pytest.mark.parametrize("fn,base", [("mla_absorb_q", ABSORB), ("mla_project_v", PROJECT)])
@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(T=-1), 1), (dict(H=0), 1),
    (dict(R=100), 2), (dict(nope=192), 2), (dict(hs=100), 1), (dict(rs=4), 1), (dict(ohs=64), 1),
    (dict(ors=132), 1), (dict(x=at(1) + 4), 1), (dict(out=at(5) + 8), 1), (dict(out=at(1)), 1),
    (dict(out=at(2) + 1024), 1), (dict(err=FAKE + 2), 1),
])
def test_head_product_refusals(lib, fn, base, over, code):
    assert getattr(lib, fn)(*args(base, over)) == code


PREFILL = dict(q=at(1), qrs=16 * 192, qhs=192, qpe=None, qprs=0, qphs=0, T=10, H=16, k=at(2),
               krs=16 * 256, khs=256, v=at(2) + 256, vrs=16 * 256, vhs=256, kpe=at(3), kps=64,
               Tk=30, nope=128, rope=64, vd=128, cuq=at(4), cuk=at(5), seqs=2, causal=1,
               scale=0.07, S=2, ws=at(6), wsb=10 * 16 * 2 * 129 * 4, o=at(7), ors=16 * 128, ohs=128,
               lse=at(8), err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(kpe=None), 1),
    (dict(cuq=None), 1), (dict(cuk=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(T=-1), 1), (dict(Tk=-1), 1), (dict(seqs=-1), 1), (dict(H=0), 1), (dict(H=1025), 1),
    (dict(S=0), 1), (dict(S=65), 1), (dict(nope=64), 2), (dict(rope=32), 2), (dict(vd=512), 2),
    (dict(seqs=65536), 2), (dict(T=(1 << 30) + 1), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(qhs=184), 1), (dict(qpe=at(9), qprs=1024, qphs=56), 1), (dict(qpe=at(9) + 2, qprs=1024, qphs=64), 1),
    (dict(khs=100), 1), (dict(vrs=12), 1), (dict(kps=60), 1), (dict(kps=68), 1),
    (dict(q=at(1) + 8), 1), (dict(kpe=at(3) + 8), 1), (dict(o=at(7) + 8), 1), (dict(lse=at(8) + 2), 1),
    (dict(ors=64, ohs=128), 1), (dict(ors=1024, ohs=128), 1), (dict(o=at(1)), 1), (dict(o=at(2)), 1),
    (dict(ws=None), 1), (dict(ws=at(6) + 16), 1), (dict(wsb=100), 3),
    (dict(T=1 << 29, seqs=1000, H=1024, qrs=1024 * 192, ors=1024 * 128), 1),
])
def test_prefill_refusals(lib, over, code):
    assert lib.mla_prefill(*args(PREFILL, over)) == code


def test_too_many_units_are_refused(lib):
    """One CTA per block slot, head and split: more than a grid holds."""
    over = dict(T=1 << 20, seqs=65535, H=1024, qhs=192, qrs=1024 * 192, khs=256, krs=1024 * 256,
                vhs=256, vrs=1024 * 256, ohs=128, ors=1024 * 128, S=64, wsb=(1 << 64) - 1)
    assert lib.mla_prefill(*args(PREFILL, over)) == 2


def test_zero_work_is_a_noop(lib):
    assert lib.mla_gather_cache(*args(GATHER, dict(T=0, cache=None))) == 0
    assert lib.mla_gather_cache(*args(GATHER, dict(seqs=0, cu=None))) == 0
    assert lib.mla_expand_kv(*args(EXPAND, dict(T=0, c=None))) == 0
    assert lib.mla_absorb_q(*args(ABSORB, dict(T=0, x=None))) == 0
    assert lib.mla_project_v(*args(PROJECT, dict(T=0, x=None))) == 0
    assert lib.mla_prefill(*args(PREFILL, dict(T=0, q=None))) == 0
    assert lib.mla_prefill(*args(PREFILL, dict(seqs=0, cuq=None))) == 0


def test_split_rule_and_workspace():
    f = mla.mla_prefill_num_kv_splits
    assert f(8192, 1, 16, 8192, 152) == 1          # the blocks fill the SMs
    assert f(256, 1, 16, 32768, 152) == 9          # 16 units: nine parts each
    assert f(16, 1, 16, 4096, 152) == 4            # none under 1024 keys
    assert f(24, 8, 16, 32768, 152) == 8           # few rows: lengths evened out
    assert f(24, 8, 16, 4096, 152) == 2
    assert f(64, 64, 16, 4096, 152) == 1
    assert f(1000, 1, 16, 1000, 152) == 1
    assert f(1, 1, 1, 1 << 40, 152) == 64
    assert f(0, 1, 16, 100, 152) == f(5, 0, 16, 100, 152) == f(5, 1, 16, 0, 152) == 1
    g = mla.mla_prefill_workspace_bytes
    assert g(10, 16, 1, 128) == 0 and g(10, 16, 3, 128) == 10 * 16 * 3 * 129 * 4
    assert g(2 ** 31 - 1, 2 ** 31 - 1, 64, 128) == (1 << 64) - 1


def test_python_calls_refuse_tensors_off_the_gpu(lib):
    bf, i32 = torch.bfloat16, torch.int32
    w = torch.zeros(512, 512, dtype=bf)
    z = torch.zeros(3, dtype=i32)
    calls = [
        lambda: mla.absorb_q(torch.zeros(3, 2, 128, dtype=bf), w),
        lambda: mla.project_v(torch.zeros(3, 2, 512, dtype=bf), w),
        lambda: mla.expand_kv(torch.zeros(3, 512, dtype=bf), w, 2),
        lambda: mla.prefill(torch.zeros(3, 2, 192, dtype=bf), torch.zeros(3, 2, 128, dtype=bf),
                            torch.zeros(3, 2, 128, dtype=bf), torch.zeros(3, 64, dtype=bf), z, z, 0.1),
        lambda: mla.gather_cache(torch.zeros(2, 16, 576, dtype=bf), torch.zeros(2, 4, dtype=i32), z, 3),
        lambda: mla.batch_build(z, z, torch.zeros(3, 4, dtype=i32), z, z[:1], 16, 3, 5),
        lambda: mla.blocks_release(z, torch.zeros(3, 4, dtype=i32), z, z[:1], 16, 3),
    ]
    for f in calls:
        with pytest.raises(ValueError, match="must be a CUDA tensor"):
            f()
    with pytest.raises(TypeError, match="must be a tensor"):
        mla.absorb_q(None, w)
