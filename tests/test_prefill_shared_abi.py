"""mla_prefill_shared rejects bad arguments on the host before any launch; so
these run without a GPU."""
import ctypes

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


T, H = 10, 4
WS = T * H * 3 * 129 * 4
BASE = dict(q=at(1), qs=H * 192, qh=192, qp=None, qps=0, qph=0, T=T, H=H, k=at(2), ks=H * 256,
            kh=256, v=at(2) + 256, vs=H * 256, vh=256, kp=at(4), kps=64, Tk=100, nope=128, rope=64,
            vd=128, cuq=at(5), cuk=at(6), B=3, gs=at(7), cup=at(8), G=1, causal=1, sm=0.07, pre=2,
            own=1, ws=at(9), wsb=WS, o=at(10), os=H * 128, oh=128, lse=at(11), err=None,
            stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(gs=None), 1), (dict(cup=None), 1), (dict(G=0), 1), (dict(G=-1), 1), (dict(G=65536), 2),
    (dict(gs=at(7) + 2), 1), (dict(cup=at(8) + 1), 1), (dict(pre=0), 1), (dict(pre=65), 1),
    (dict(own=-1), 1), (dict(own=65), 1), (dict(ws=None), 1), (dict(ws=at(9) + 16), 1),
    (dict(wsb=WS - 1), 3), (dict(pre=3), 3), (dict(own=2), 3), (dict(q=None), 1), (dict(k=None), 1),
    (dict(vd=64), 2), (dict(sm=0.0), 1), (dict(cuq=None), 1), (dict(lse=None), 1),
    # outputs over the groups' arrays
    (dict(o=at(7)), 1), (dict(lse=at(8)), 1), (dict(ws=at(7)), 1), (dict(lse=at(10)), 1),
])
def test_prefill_shared_refusals(lib, over, code):
    a = dict(BASE)
    a.update(over)
    assert lib.mla_prefill_shared(*a.values()) == code


def test_nothing_to_do(lib):
    assert lib.mla_prefill_shared(*dict(BASE, T=0).values()) == 0
    assert lib.mla_prefill_shared(*dict(BASE, B=0).values()) == 0


def test_split_rule(lib):
    rule = mla.mla_prefill_shared_num_kv_splits
    # 256-row blocks of the prefix leave SMs idle: parts of at least 256 keys
    pre, own = rule(60, 3, 1, 16, 8192, 60, 152)
    assert 5 <= pre <= 9 and own == 1
    pre, own = rule(60, 3, 1, 16, 1000, 60, 152)
    assert 2 <= pre <= 3 and own == 1
    assert rule(60, 3, 1, 16, 500, 0, 152) == (1, 0)
    # many rows: one part; a few rows each with long keys of their own: apart
    assert rule(8213, 40, 1, 32, 4000, 300, 152) == (1, 0)
    assert rule(16, 8, 1, 16, 8192, 30000, 152)[1] > 0
    for a in ((10, 2, 1, 1, 10 ** 6, 10 ** 6, 152), (0, 0, 0, 0, 0, 0, 0), (5, 5, 5, 5, 5, 5, 5)):
        pre, own = rule(*a)
        assert 1 <= pre <= 64 and 0 <= own <= 64
    assert lib.mla_prefill_shared_num_kv_splits(8213, 40, 1, 32, 4000, 300, 152, None) == 1


def test_python_refusals():
    z = torch.zeros(2, 2, 192, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        mla.prefill_shared(z, z, z, z, z, z, z, z, 0.1)
