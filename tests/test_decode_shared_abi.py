"""mla_decode_shared rejects bad arguments on the host before any launch; so
these run without a GPU."""
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


BASE = dict(q=at(1), qs=16 * 576, qh=576, qp=None, qps=0, qph=0, T=8, H=16, cache=at(2), kvd=0,
            nb=100, bs=64, bstride=64 * 576, R=512, P=64, bt=at(3), bts=10, maxb=10, lens=at(4),
            B=4, gs=at(5), pre=at(6), G=2, sm=0.07, scale=None, ws=at(7), wsb=1 << 40, o=at(8),
            lse=at(9), err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(G=0), 1), (dict(G=-1), 1), (dict(G=1025), 2), (dict(T=8193, B=8193), 2),
    (dict(q=None), 1), (dict(cache=None), 1), (dict(bt=None), 1), (dict(lens=None), 1),
    (dict(gs=None), 1), (dict(pre=None), 1), (dict(o=None), 1), (dict(lse=None), 1),
    (dict(gs=at(5) + 2), 1), (dict(pre=at(6) + 1), 1), (dict(err=at(10) + 1), 1),
    (dict(B=3), 1), (dict(B=0), 1), (dict(H=0), 1), (dict(H=129), 1), (dict(bs=48), 2),
    (dict(R=384), 2), (dict(P=32), 2), (dict(kvd=1), 1), (dict(kvd=7), 1), (dict(qs=8), 1),
    (dict(qh=568), 1), (dict(q=at(1) + 8), 1), (dict(bts=9), 1), (dict(bstride=100), 1),
    (dict(maxb=(1 << 24) + 1, bts=1 << 25), 2),                       # past 2^30 tokens
    (dict(maxb=1 << 24, bts=1 << 24, T=8192, B=8192), 2),    # past 2^30 tiles
])
def test_decode_shared_refusals(lib, over, code):
    a = dict(BASE)
    a.update(over)
    assert lib.mla_decode_shared(*a.values()) == code


def test_no_rows(lib):
    assert lib.mla_decode_shared(*dict(BASE, T=0, B=0).values()) == 0


def test_workspace_size(lib):
    f = mla.mla_decode_shared_workspace_bytes
    # 128 fp32 vectors of R for each block of 128 vectors, own and shared, and twice
    # for each pair of CTAs
    n = f(64, 16, 64, 1, 512, 152)
    assert n >= (64 + 8 + 152) * 128 * 512 * 4 and n < (64 + 8 + 160) * 128 * 520 * 4
    assert f(64, 16, 64, 1, 256, 152) < n < f(64, 16, 64, 40, 512, 152)
    for bad in ((0, 16, 64, 1, 512, 152), (64, 0, 64, 1, 512, 152), (64, 16, 0, 1, 512, 152),
                (64, 16, 64, 0, 512, 152), (64, 16, 64, 1, 384, 152), (64, 16, 64, 1, 512, 1),
                (64, 16, 64, 1025, 512, 152), (8193, 1, 8193, 1, 512, 152)):
        assert f(*bad) == 0


def test_python_refusals():
    z = torch.zeros(2, 2, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mla.decode_shared(z, z, z, z, z, z, 0.1)
