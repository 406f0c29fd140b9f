"""GPU tests of the batch tables at their limits: sums of lengths past 32 bits,
the stack's height read and written by one release."""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_batch import Pool, i32

pytestmark = pytest.mark.gpu

MAX = 2 ** 31 - 1


@pytest.mark.parametrize("new,ctx,ids", [
    ([MAX, MAX, 1], [16, 16, 16], None),
    ([MAX, 5, MAX, 1, 0, 40, 3, MAX, 1], [16, 0, 64, 16, 16, 3, 0, 0, 16], [8, 0, 3, 1, 9, 2, 7, 4, 5]),
    ([1] * 300 + [MAX] * 3 + [1] * 700, [16] * 1003, None),
])
@pytest.mark.parametrize("alias", [False, True])
def test_query_lengths_that_sum_past_32_bits(cuda_dev, new, ctx, ids, alias):
    """Lengths beyond the row are clamped and counted; every other entry gets
    its own pages, and no page is in a row and still on the stack."""
    B, bs, maxb, T = len(new), 16, 4, 500
    pool = Pool(B + 2, maxb, bs, 4 * B + 10, seed=B)
    rows = np.arange(B) if ids is None else np.asarray(ids)
    for r, c in zip(rows, ctx):
        pool.hold(r, c)
    table, free, count = i32(pool.table), i32(pool.free), i32([pool.count])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bt0 = np.full((B, maxb), -7, np.int32)
    out = mla.batch_build(i32(new), i32(ctx), table, free, count, bs, pool.num_blocks, T,
                          req_ids=None if ids is None else i32(ids), block_table=i32(bt0),
                          free_count_out=count if alias else None, err_count=err)
    torch.cuda.synchronize()
    bt, seq, _, cu_k, pos, slot, errs = pool.build(rows, np.asarray(new, np.int64), ctx, T, bt0)
    cu_q = np.minimum(np.concatenate([[0], np.cumsum(np.asarray(new, np.int64))]), MAX)
    np.testing.assert_array_equal(out.cu_seqlens_q.cpu().numpy(), cu_q)
    for got, want in ((out.block_table, bt), (table, pool.table), (out.seq_lens, seq),
                      (out.cu_seqlens_k, cu_k), (out.positions, pos), (out.slot_mapping, slot)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert out.free_count.item() == pool.count and err.item() == errs
    held = np.concatenate([table[r, :-(-int(n) // bs)].cpu().numpy() for r, n in zip(rows, seq)])
    live = np.concatenate([held, pool.free[:pool.count]])
    assert len(set(live.tolist())) == len(live)


@pytest.mark.parametrize("B,pages", [(1, 1), (64, 100), (8192, 60)])
def test_release_in_place_is_release_apart(cuda_dev, B, pages):
    """The height is read by every CTA and written by one before the others
    end: the same stack as with an output of its own, however it is run."""
    bs, nb = 16, B * pages + 50
    perm = torch.randperm(nb, device="cuda", dtype=torch.int32)
    table, held = perm[:B * pages].view(B, pages).contiguous(), i32([pages * bs] * B)
    free0 = torch.full((nb,), -9, dtype=torch.int32, device="cuda")
    free0[:50] = perm[B * pages:]
    want = torch.cat([perm[B * pages:], perm[:B * pages]])
    for _ in range(20):
        for apart in (False, True):
            free, count = free0.clone(), i32([50])
            out = mla.blocks_release(held, table, free, count, bs, nb,
                                     free_count_out=torch.empty_like(count) if apart else None)
            assert torch.equal(free, want) and out.item() == nb
            assert count.item() == (50 if apart else nb)
