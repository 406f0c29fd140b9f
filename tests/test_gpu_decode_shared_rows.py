"""GPU test of decode_shared with more than 2^24 query rows: rows and heads of a
vector do not share 32 bits.  Tolerances as derived in test_gpu_decode_shared.py.
"""
import math

import pytest
import torch

import mla_paged_kv_concat_gb300 as mla

pytestmark = pytest.mark.gpu

SCALE = 1 / math.sqrt(192)


def test_rows_past_2_to_the_24(cuda_dev):
    B, rows, R, bs, n = 8192, 2049, 256, 128, 130  # a prefix of one tile, two own tokens
    T, D = B * rows, R + 64
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 55 GB")
    g = torch.Generator("cuda").manual_seed(24)
    cache = torch.randn(2, bs, D, generator=g, device="cuda").bfloat16()
    q = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    first = (1 << 24) - 500  # what is looked at: rows on both sides, to the last
    q[first:] = torch.randn(T - first, 1, D, generator=g, device="cuda").bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[0, 1]]).expand(B, 2).contiguous()
    err = i32([0])
    o, lse = mla.decode_shared(q, cache, table, i32([n] * B), i32([0, B]), i32([128]), SCALE,
                               kv_lora_rank=R, err_count=err)
    assert err.item() == 0
    k = cache.reshape(-1, D)[:n].double()
    x = q[first:, 0].double()
    S = float((x.abs() @ k.abs().t()).max() * SCALE)
    x = x @ k.t() * SCALE
    z = torch.logsumexp(x, 1)
    p = torch.exp(x - z[:, None])
    ref, A = p @ k[:, :R], p @ k[:, :R].abs()
    ds = D * 2.0 ** -23 * S
    e = 2 * (1.01 * (ds + 2.0 ** -21 * S) + 2.0 ** -21)
    bound = (1 + 2.0 ** -8) * A * (2.0 ** -8 + 2 * e + 2 * n * 2.0 ** -23) \
        + (2.0 ** -8 + 2.0 ** -21) * ref.abs()
    bad = ((o[first:, 0].double() - ref).abs() > bound).any(1)
    bl = ds + 2.0 ** -21 * S + e + n * 2.0 ** -23 + 2.0 ** -21 * z.abs()
    bad |= (lse[first:, 0].double() - z).abs() > bl
    wrong = (torch.nonzero(bad)[:4, 0] + first).tolist()
    # rows of zeros, in front: the mean of the keys' values
    mean = k[:, :R].mean(0)
    front = (o[:first:100003, 0].double() - mean).abs()
    del q, o, lse
    torch.cuda.empty_cache()
    assert not wrong, wrong
    assert bool((front <= (1 + 2.0 ** -8) * k[:, :R].abs().mean(0) * (2.0 ** -8 + 4 * n * 2.0 ** -23)
                 + (2.0 ** -8 + 2.0 ** -21) * mean.abs()).all())
