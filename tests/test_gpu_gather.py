"""GPU tests of the gather of cached rows: bit for bit the cached values (bf16
cache), or bf16(value * scale) with the product in fp32 (fp8 caches)."""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu


def make(R, fmt, bs, lens, seed, block_pad=0):
    g = torch.Generator().manual_seed(seed)
    d = R + 64
    pages = [-(-n // bs) for n in lens]
    nb = sum(pages) + 3
    flat = torch.randn(nb, bs * d + block_pad, generator=g) * 3
    flat[:, 5] = float("nan")
    if fmt == "bf16":
        cache = flat.to(torch.bfloat16)
    else:
        cache = (flat / 0.05).to({"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt])
    view = cache[:, :bs * d].unflatten(1, (bs, d))
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(pages + [1]) + 1), nb + 5, dtype=torch.int32)
    a = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[a:a + n]
        a += n
    return cache, view, table


def want_rows(view, table, b, pos, scale):
    bs = view.shape[1]
    rows = torch.stack([view[table[b, p // bs].item()].view(torch.uint8).view(bs, -1)[p % bs]
                        for p in pos]).view(view.dtype)
    return rows if view.dtype == torch.bfloat16 else (rows.float() * scale).to(torch.bfloat16)


def bits(x):
    return x.contiguous().view(torch.int16)


def same(a, b):
    n = torch.isnan(b.float())
    assert torch.equal(torch.isnan(a.float()), n)
    assert torch.equal(bits(a)[~n], bits(b)[~n])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2"])
@pytest.mark.parametrize("R,bs,lens,pad", [
    (512, 64, [1], 0), (512, 16, [70, 0, 3, 129], 64), (256, 64, [0, 200, 31, 33], 0),
    (256, 1, [5, 40], 16), (512, 100, [333, 1], 0), (256, 1024, [1500], 128),
])
def test_rows_bit_for_bit(cuda_dev, R, bs, lens, pad, fmt):
    cache, view, table = make(R, fmt, bs, lens, R + bs, pad)
    dcache = cache.cuda()
    dview = dcache[:, :bs * (R + 64)].unflatten(1, (bs, R + 64))
    starts = [n // 3 for n in lens]
    for use_starts in (False, True):
        take = [n - s if use_starts else n for n, s in zip(lens, starts)]
        cu = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
        T = int(cu[-1])
        scale = torch.tensor([0.05], dtype=torch.float32)
        buf = torch.full((T + 4, R + 72), 7.0, dtype=torch.bfloat16, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kv_c, k_pe = mla.gather_cache(
            dview, table.cuda(), torch.from_numpy(cu).cuda(), kv_c=buf[:, :R], k_pe=buf[:, R:R + 64],
            seq_starts=torch.tensor(starts, dtype=torch.int32).cuda() if use_starts else None,
            kv_lora_rank=R, kv_scale=None if fmt == "bf16" else scale.cuda(), err_count=err)
        torch.cuda.synchronize()
        assert err.item() == 0
        got = buf.cpu()
        assert torch.all(got[T:] == 7) and torch.all(got[:, R + 64:] == 7)
        for b in range(len(lens)):
            s = starts[b] if use_starts else 0
            if take[b]:
                ref = want_rows(view, table, b, range(s, s + take[b]), scale)
                same(got[cu[b]:cu[b + 1], :R + 64], ref)


def test_bad_pages_and_positions_are_zeros_and_counted(cuda_dev):
    cache, view, table = make(256, "bf16", 16, [40, 20], 5)
    table[0, 1] = cache.shape[0]
    table[1, 0] = -1
    cu = torch.tensor([0, 40, 100], dtype=torch.int32)  # 60 rows of a sequence with 64 slots
    starts = torch.tensor([0, 30], dtype=torch.int32)
    table[1, 1:] = 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c, p = mla.gather_cache(view.cuda(), table.cuda(), cu.cuda(), 100, seq_starts=starts.cuda(),
                            err_count=err)
    cap = table.shape[1] * 16
    zero = [t for t in range(16, 32)] + [40 + j for j in range(60) if 30 + j < 16 or 30 + j >= cap]
    got = torch.cat([c, p], 1).cpu()
    assert err.item() == len(zero)
    assert torch.all(bits(got[zero]) == 0)
    rest = [t for t in range(40) if t not in zero]
    same(got[rest], want_rows(view, table, 0, rest, None))


def test_offsets_past_32_bits(cuda_dev):
    """Pages behind 2^32 bytes and 2^31 elements of the cache."""
    R, bs, d = 512, 64, 576
    nb = (1 << 32) // (bs * d) + 40
    cache = torch.empty(nb, bs, d, dtype=torch.bfloat16, device="cuda")
    ids = [nb - 1, 3, nb - 30]
    for i, b in enumerate(ids):
        cache[b] = torch.randn(bs, d, device="cuda", generator=torch.Generator("cuda").manual_seed(i))
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3 * bs - 7], dtype=torch.int32, device="cuda")
    c, p = mla.gather_cache(cache, table, cu, 3 * bs - 7)
    assert torch.equal(torch.cat([c, p], 1), cache[ids].reshape(-1, d)[:3 * bs - 7])
