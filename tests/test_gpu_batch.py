"""GPU tests of the batch tables: block tables, slot maps, positions and
cumulative lengths from request lengths, pages off and back onto the stack of
free ones, against a plain Python walk over the requests.  Everything is an
integer, so everything has to be equal."""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu


class Pool:
    """Host model of the requests' table and the stack of free pages."""

    def __init__(self, rows, maxb, bs, num_blocks, seed=0):
        rng = np.random.default_rng(seed)
        self.bs, self.num_blocks, self.maxb = bs, num_blocks, maxb
        self.free = rng.permutation(num_blocks).astype(np.int32)
        self.count = num_blocks
        self.table = np.full((rows, maxb), -1, np.int32)

    def hold(self, row, tokens):
        n = -(-tokens // self.bs)
        for i in range(n):
            self.count -= 1
            self.table[row, i] = self.free[self.count]

    def build(self, ids, new, ctx, T, bt):
        """The walk: tables, errors; updates the pool."""
        cap = self.maxb * self.bs
        B, errs = len(new), 0
        pos, slot = np.zeros(T, np.int64), np.full(T, -1, np.int64)
        seq = np.zeros(B, np.int64)
        t = 0
        for b in range(B):
            n, c = max(int(new[b]), 0), min(max(int(ctx[b]), 0), cap)
            s = min(c + n, cap)
            errs += new[b] < 0 or c != ctx[b] or c + n > cap
            ok = 0 <= ids[b] < len(self.table)
            old, pages = -(-c // self.bs), -(-s // self.bs)
            row = self.table[ids[b]] if ok else np.full(self.maxb, -1, np.int32)
            if ok:
                for i in range(old, pages):
                    self.count -= 1
                    row[i] = self.free[self.count] if self.count >= 0 else -1
                    if not 0 <= row[i] < self.num_blocks:
                        row[i] = -1
                        errs += 1
            bt[b, :pages] = row[:pages]
            for j in range(n):
                if t + j >= T:
                    break
                p = c + j
                pos[t + j] = p
                if ok and p < s and 0 <= row[p // self.bs] < self.num_blocks:
                    slot[t + j] = row[p // self.bs] * self.bs + p % self.bs
                else:
                    errs += 1
            t += n
            seq[b] = s
        errs += t > T
        self.count = max(self.count, 0)
        nq = np.maximum(np.asarray(new, np.int64), 0)
        cu = lambda x: np.concatenate([[0], np.cumsum(x)]).astype(np.int32)  # noqa: E731
        return bt, seq.astype(np.int32), cu(nq), cu(seq), pos, slot, errs


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


def run(pool, ids, new, ctx, T, alias, stream=None):
    B = len(new)
    table, free = i32(pool.table), i32(pool.free)
    count = i32([pool.count])
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bt0 = np.full((B, pool.maxb), -7, np.int32)
    out = mla.batch_build(i32(new), i32(ctx), table, free, count, pool.bs, pool.num_blocks, T,
                          req_ids=None if ids is None else i32(ids), block_table=i32(bt0),
                          free_count_out=count if alias else None, err_count=err)
    torch.cuda.synchronize()
    want = pool.build(np.arange(B) if ids is None else ids, new, ctx, T, bt0)
    for name, got, ref in zip(out._fields[:6], out, want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    np.testing.assert_array_equal(table.cpu().numpy(), pool.table)
    assert out.free_count.item() == pool.count
    assert err.item() == want[-1]
    return out


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,bs,max_new,max_ctx,pad,seed", [
    (1, 64, 1, 0, 0, 1), (1, 1, 7, 3, 5, 2), (3, 16, 40, 70, 0, 3), (64, 64, 1, 4096, 0, 4),
    (257, 16, 33, 300, 100, 5), (300, 128, 3, 5000, 1, 6), (2, 1024, 5000, 3000, 9, 7),
    (1000, 48, 2, 400, 0, 8), (8192, 16, 2, 50, 3, 9),
    # rows of several pieces, 16-byte aligned and not
    (5, 1, 1000, 4000, 7, 10), (5, 1, 1001, 4000, 0, 11),
])
def test_matches_the_walk(cuda_dev, B, bs, max_new, max_ctx, pad, seed, alias):
    rng = np.random.default_rng(seed)
    new = rng.integers(0, max_new + 1, B)
    if max_new == 1:
        new[:] = 1
    ctx = rng.integers(0, max_ctx + 1, B)
    maxb = -(-(max_ctx + max_new) // bs)
    rows = B + 5
    pool = Pool(rows, maxb, bs, int((-(-(ctx + new) // bs)).sum()) + 3, seed)
    ids = rng.permutation(rows)[:B]
    for b in range(B):
        pool.hold(ids[b], int(ctx[b]))
    run(pool, ids, new, ctx, int(new.sum()) + pad, alias)


def test_no_requests_and_no_tokens(cuda_dev):
    pool = Pool(4, 4, 16, 20)
    out = run(pool, None, np.zeros(0, int), np.zeros(0, int), 5, False)
    assert out.slot_mapping.tolist() == [-1] * 5 and out.cu_seqlens_q.tolist() == [0]
    run(pool, None, np.zeros(3, int), np.zeros(3, int), 0, True)


def test_more_tokens_than_rows(cuda_dev):
    run(Pool(3, 8, 16, 30), None, np.array([50, 7, 20]), np.array([0, 0, 0]), 60, False)


@pytest.mark.parametrize("alias", [False, True])
def test_stack_runs_empty(cuda_dev, alias):
    """The last requests' pages cannot be taken: -1 and counted, height 0."""
    pool = Pool(400, 8, 16, 200)
    run(pool, None, np.full(400, 20), np.zeros(400, int), 8000, alias)
    assert pool.count == 0


def test_bad_lengths_rows_and_ids(cuda_dev):
    pool = Pool(6, 4, 16, 40)
    for r in (0, 1, 3):
        pool.hold(r, 20)
    pool.table[3, 1] = 40          # a page id outside the pool in a row's held part
    pool.free[pool.count - 2] = -5  # and one on the stack
    run(pool, np.array([0, 6, -1, 1, 3, 5]), np.array([10, 4, 3, 100, 8, -2]),
        np.array([20, 20, 5, 20, 20, 400]), 200, False)


def test_steps_in_place_then_release(cuda_dev):
    """A prompt, decode steps with the stack's height in place, and the pages
    back: no page is held twice, and in the end all are free again."""
    rng = np.random.default_rng(11)
    B, bs, maxb, nb = 40, 16, 12, 300
    free, count = i32(rng.permutation(nb)), i32([nb])
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = i32(np.zeros(B))
    first = rng.integers(1, 60, B)
    for step in range(20):
        new = i32(first if step == 0 else np.ones(B))
        t = mla.batch_build(new, lens, table, free, count, bs, nb, int(new.sum().item()),
                            free_count_out=count, err_count=err)
        lens = t.seq_lens
        held = torch.cat([t.block_table[b, :-(-int(n) // bs)] for b, n in enumerate(lens.tolist())])
        live = torch.cat([held, free[:count.item()]])
        assert sorted(live.tolist()) == list(range(nb))
    before = free[:count.item()].tolist()
    ids = rng.permutation(B)
    want = before + [int(x) for b in ids for x in table[b, :-(-int(lens[b]) // bs)].tolist()]
    mla.blocks_release(lens[torch.from_numpy(ids).cuda()].contiguous(), table, free, count, bs, nb,
                       req_ids=i32(ids), err_count=err)
    assert count.item() == nb and err.item() == 0
    assert free.tolist() == want


@pytest.mark.parametrize("B,pages,seed", [(1, 1, 1), (7, 40, 2), (600, 30, 3), (8192, 3, 4)])
def test_release_leaves_bad_entries_out(cuda_dev, B, pages, seed):
    rng = np.random.default_rng(seed)
    bs, nb = 16, 100000
    table = rng.integers(0, nb, (B + 2, pages)).astype(np.int32)
    bad = rng.random(table.shape) < 0.2
    table[bad] = rng.choice([-1, nb, nb + 9], size=int(bad.sum()))
    lens = rng.integers(0, pages * bs + 1, B)
    ids = rng.permutation(B + 2)[:B]
    ids[0] = B + 2  # outside the table
    want, errs = [5, 6, 7], 1
    for b in range(1, B):
        e = table[ids[b], :-(-int(lens[b]) // bs)]
        ok = (e >= 0) & (e < nb)
        want += e[ok].tolist()
        errs += int((~ok).sum())
    cap = len(want) - 4 if len(want) > 20 else len(want)  # four do not fit
    errs += len(want) - cap
    free = torch.full((cap + 8,), -9, dtype=torch.int32, device="cuda")
    free[:3] = i32([5, 6, 7])
    count, err = i32([3]), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = mla.blocks_release(i32(lens), i32(table), free[:cap], count, bs, nb, req_ids=i32(ids),
                             free_count_out=torch.empty_like(count), err_count=err)
    assert out.item() == cap and count.item() == 3
    assert free.tolist() == want[:cap] + [-9] * 8
    assert err.item() == errs


def test_captured_and_replayed(cuda_dev):
    """A captured step replays over new lengths, the height in place."""
    B, bs, nb = 300, 16, 4000
    pool = Pool(B, 20, bs, nb, 3)
    new, ctx = i32(np.ones(B)), i32(np.zeros(B))
    table, free, count = i32(pool.table), i32(pool.free), i32([nb])
    bt = torch.zeros(B, 20, dtype=torch.int32, device="cuda")
    outs = dict(block_table=bt, seq_lens=torch.empty_like(ctx), positions=torch.empty(
        400, dtype=torch.int64, device="cuda"), slot_mapping=torch.empty(
        400, dtype=torch.int64, device="cuda"), cu_seqlens_q=i32(np.zeros(B + 1)),
        cu_seqlens_k=i32(np.zeros(B + 1)), free_count_out=count)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        mla.batch_build(new, ctx, table, free, count, bs, nb, **outs)
    side.synchronize()
    table.copy_(i32(pool.table)), count.fill_(nb)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.batch_build(new, ctx, table, free, count, bs, nb, **outs)
    c = np.zeros(B, int)
    for step in range(4):
        n = np.random.default_rng(step).integers(0, 2, B)
        new.copy_(i32(n)), ctx.copy_(i32(c))
        g.replay()
        torch.cuda.synchronize()
        ref = pool.build(np.arange(B), n, c, 400, bt.cpu().numpy().copy())
        np.testing.assert_array_equal(outs["slot_mapping"].cpu().numpy(), ref[5])
        np.testing.assert_array_equal(table.cpu().numpy(), pool.table)
        assert count.item() == pool.count
        c = c + n
