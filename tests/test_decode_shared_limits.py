"""What mla_decode_shared counts in 32 bits is bounded on the host; these run
without a GPU."""
import pytest

import mla_paged_kv_concat_gb300 as mla
from test_decode_shared_abi import BASE, lib  # noqa: F401

SHAPES = [  # sequences, rows of each, heads: 2^29 query vectors
    (8192, 1 << 16, 1), (8192, 1 << 9, 128), (64, 1 << 16, 128),
]


@pytest.mark.parametrize("B,rows,H", SHAPES)
def test_query_vectors(lib, B, rows, H):  # noqa: F811
    def call(n):
        a = dict(BASE, q=1 << 44, o=1 << 45, lse=1 << 46, T=B * n, B=B, H=H, qs=H * 576, maxb=1,
                 wsb=0)
        return lib.mla_decode_shared(*a.values())

    assert B * rows * H == 1 << 29
    assert call(rows) in (3, 4)  # passes: too small a workspace, or no device
    assert call(rows + 1) == 2
    size = mla.mla_decode_shared_workspace_bytes
    assert size(B * rows, H, B, 1, 256, 152) > (1 << 29) * 256 * 4
    assert size(B * (rows + 1), H, B, 1, 256, 152) == 0
