"""mla_linear rejects bad arguments on the host before any launch, and the
Python call bad tensors; so these run without a GPU."""
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


BASE = dict(x=at(1), xs=128, T=10, K=128, w=at(2), ws=128, N=64, bias=at(3), act=0, res=at(4),
            rs=64, y=at(5), ys=64, err=None, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(T=-1), 1), (dict(K=0), 1),
    (dict(N=0), 1), (dict(act=-1), 1), (dict(act=5), 1), (dict(T=(1 << 30) + 1), 2),
    (dict(K=(1 << 20) + 1, xs=1 << 21, ws=1 << 21), 2), (dict(N=(1 << 20) + 1), 2),
    (dict(xs=120), 1), (dict(ws=120), 1), (dict(ys=56), 1), (dict(rs=56), 1),
    (dict(xs=132), 1), (dict(ws=132), 1), (dict(ys=68), 1), (dict(rs=68), 1), (dict(xs=0), 1),
    (dict(x=at(1) + 8), 1), (dict(w=at(2) + 2), 1), (dict(bias=at(3) + 8), 1),
    (dict(res=at(4) + 4), 1), (dict(y=at(5) + 8), 1), (dict(err=at(6) + 1), 1),
    # y over an input, and over a residual that it is not
    (dict(y=at(1) + 64), 1), (dict(y=at(2)), 1), (dict(y=at(3)), 1), (dict(y=at(4) + 128), 1),
    (dict(y=at(4), ys=72), 1), (dict(xs=1 << 39), 1),
])
def test_linear_refusals(lib, over, code):
    a = dict(BASE)
    a.update(over)
    assert lib.mla_linear(*a.values()) == code


def test_linear_no_tokens(lib):
    a = dict(BASE, T=0, x=None, y=None)
    assert lib.mla_linear(*a.values()) == 0


def test_python_refusals():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation"):
        mla.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="CUDA tensor"):
        mla.linear(x, w)
    with pytest.raises(TypeError):
        mla.linear(None, w)
