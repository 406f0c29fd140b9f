"""The rule that chooses mla_linear's kernel and tile, on the CPU: over devices of any
number of SMs and over all kinds of shapes it gives a plan that the kernels take."""
import ctypes
import itertools
import subprocess
import sys

import pytest

from mla_paged_kv_concat_gb300 import build

PAIR, FEW = 0, 1


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("form", "bn", "splits", "a_rows", "b_rows")]

    def key(self):
        return ("few" if self.form == FEW else "split" if self.splits > 1 else "pair", self.bn,
                self.splits)


def linear_plan(tokens, n, k, sms):
    f = ctypes.CDLL(build.LIB)["_ZN3mla11linear_planEiiii"]
    f.restype, f.argtypes = Plan, [ctypes.c_int] * 4
    return f(tokens, n, k, sms)


TOKENS = (1, 16, 17, 33, 65, 128, 129, 256, 257, 300, 1000, 1024, 1025, 4096, 1 << 30)
N = (1, 8, 129, 1000, 6136, 1 << 20)
K = (1, 64, 65, 184, 2048, 6000, 1 << 20)


@pytest.mark.parametrize("sms", [*range(1, 21), 74, 132, 148, 152, 160])
def test_every_shape_has_a_plan(sms):
    build.build()
    # in a process of its own: a division by zero would end it
    code = (f"import sys; sys.path[:0] = {sys.path!r}\n"
            "from test_linear_plan import check\n"
            f"check({sms})\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:] or r.returncode


def check(sms):
    for t, n, k in itertools.product(TOKENS, N, K):
        p, at = linear_plan(t, n, k, sms), (t, n, k, sms)
        nk = -(-k // 64)
        assert 1 <= p.splits <= nk, at
        if p.form == FEW:
            assert t <= 1024 and p.bn in (16, 32, 64, 128) and p.splits in (1, 2, 3, 4, 8), at
            assert p.a_rows == p.bn and p.b_rows == 128 and p.splits <= sms, at
            assert p.bn == 128 or p.bn >= t, at
        else:
            assert p.form == PAIR and t > 128 and p.a_rows == 128 and p.b_rows == p.bn // 2, at
            if p.splits > 1:
                assert p.bn == 256 and p.splits <= 4 and 2 * p.splits <= sms, at
                assert -(-t // 256) * -(-n // 256) * 2 * p.splits < 1 << 31, at  # the grid
            else:
                assert p.bn in (128, 192, 256), at
