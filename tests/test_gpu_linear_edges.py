"""GPU tests that mla.linear writes nothing but its output where out_features is no
multiple of 8: columns behind a row, and what lies behind the last one, stay."""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_linear import check, normal, rows

pytestmark = pytest.mark.gpu

SHAPES = [  # pairs of CTAs with tiles of 256, 192 and 128 columns, split sums, few tokens
    (8000, 5104, 64), (1000, 6128, 200), (1500, 4096, 128), (5000, 120, 72), (2000, 0, 40),
    (300, 0, 16), (1000, 1216, 4000), (442, 3120, 3000), (300, 2496, 512), (64, 640, 512), (3, 0, 512),
]


@pytest.mark.parametrize("more", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_what_lies_behind_stays(cuda_dev, T, N, K, more):
    N += more
    g = torch.Generator("cuda").manual_seed(T + N)
    x, w, b = rows(g, T, K), rows(g, N, K), normal(g, N)
    S = (N + 7) // 8 * 8 + 16
    # rows at a stride of S, from 8 columns on; the buffer goes on behind the last row
    buf = normal(g, T * S + 64)
    keep = buf.clone()
    out = buf.as_strided((T, N), (S, 1), 8)
    kept = torch.ones_like(buf, dtype=torch.bool)
    kept.as_strided((T, N), (S, 1), 8)[:] = False
    for act, res in ((None, None), ("silu", None), ("relu", rows(g, T, N, 1)), (None, out)):
        before = None if res is None else res.clone()
        mla.linear(x, w, bias=b, activation=act, residual=res, out=out)
        assert torch.equal(buf[kept].view(torch.int16), keep[kept].view(torch.int16)), act
        check(out, x, w, b, act, before)
