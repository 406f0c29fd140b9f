"""GPU tests of the gather of cached rows with many sequences, whose lengths
are then searched in global memory."""
import numpy as np
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_gpu_gather import make, same, want_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [255, 256, 257, 1000])
def test_many_sequences(cuda_dev, n, fmt):
    rng = np.random.default_rng(n)
    lens = rng.choice([0, 1, 5, 16, 17, 40], n).tolist()
    lens[0], lens[n - 1] = 0, 33
    R, bs = 256, 16
    cache, view, table = make(R, fmt, bs, lens, n)
    starts = [x // 3 for x in lens]
    take = [x - s for x, s in zip(lens, starts)]
    cu = np.concatenate([[0], np.cumsum(take)]).astype(np.int32)
    T = int(cu[-1])
    scale = torch.tensor([0.05])
    kv_c = torch.full((T + 3, R), 7.0, dtype=torch.bfloat16, device="cuda")
    k_pe = torch.full((T + 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    mla.gather_cache(cache.cuda()[:, :bs * (R + 64)].unflatten(1, (bs, R + 64)), table.cuda(),
                     torch.from_numpy(cu).cuda(), kv_c=kv_c, k_pe=k_pe, kv_lora_rank=R,
                     seq_starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                     kv_scale=None if fmt == "bf16" else scale.cuda(), err_count=err)
    torch.cuda.synchronize()
    assert err.item() == 0
    got = torch.cat([kv_c, k_pe], 1).cpu()
    assert torch.all(got[T:] == 7)
    ref = torch.cat([want_rows(view, table, b, range(s, s + m), scale)
                     for b, (s, m) in enumerate(zip(starts, take)) if m])
    same(got[:T], ref)
