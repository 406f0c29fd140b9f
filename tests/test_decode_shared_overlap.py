"""Outputs and workspaces of mla_decode_shared that would lie over an input or
each other are refused on the host before any launch."""
import pytest
import torch

import mla_paged_kv_concat_gb300 as mla
from test_decode_shared_abi import BASE, at, lib  # noqa: F401

# BASE: q [8][16][576] at at(1), cache 100 blocks of 64 x 576 at at(2), table [4][10] at at(3),
# 4 lengths, 3 group_seqs, 2 prefix_lens at at(4) to at(6); o [8][16][512] at at(8), lse at at(9)
Q, BLOCK, O = 8 * 16 * 576 * 2, 64 * 576 * 2, 8 * 16 * 512 * 2
SPLIT = dict(qh=512, qs=16 * 512, qp=at(11), qps=16 * 64, qph=64)


@pytest.mark.parametrize("over", [
    dict(o=at(1)), dict(o=at(1) + Q - 16), dict(o=at(1) - O + 16), dict(lse=at(1) + 100),
    dict(SPLIT, o=at(11)), dict(SPLIT, lse=at(11) + 8 * 16 * 64 * 2 - 4),
    dict(o=at(2) + 99 * BLOCK), dict(lse=at(2) + 100 * BLOCK - 4),
    dict(o=at(3)), dict(lse=at(3) + 4 * 10 * 4 - 4), dict(lse=at(4)), dict(lse=at(4) + 12),
    dict(lse=at(5)), dict(lse=at(5) + 8), dict(lse=at(6) + 4),
    dict(o=at(8), lse=at(8) + 1024), dict(lse=at(8) + O - 4), dict(o=at(9)),
    dict(kvd=1, scale=at(10), lse=at(10)),
])
def test_outputs(lib, over):  # noqa: F811
    assert lib.mla_decode_shared(*dict(BASE, **over).values()) == 1


@pytest.mark.parametrize("over", [
    {}, dict(o=at(1) + Q), dict(o=at(1) - O), dict(lse=at(2) + 100 * BLOCK),
    dict(lse=at(3) + 4 * 10 * 4), dict(lse=at(4) + 16), dict(lse=at(6) + 8), dict(lse=at(8) + O),
    # between the cache's blocks, between a table's rows, in dims that q does not hold
    dict(bstride=64 * 576 + 16384, o=at(2) + BLOCK, T=4, B=4, H=8, qs=8 * 576),
    dict(bts=1000, lse=at(3) + 40, T=4, B=4, H=16), dict(SPLIT, o=at(1) + 8 * 16 * 512 * 2),
    dict(kvd=0, scale=at(10), lse=at(10)),  # a scale that a bf16 cache does not read
])
def test_side_by_side(lib, over):  # noqa: F811
    """Passes: too small a workspace, or no device."""
    assert lib.mla_decode_shared(*dict(BASE, wsb=0, **over).values()) in (3, 4)


@pytest.mark.gpu
def test_workspace(cuda_dev):
    B, H, R, bs = 4, 16, 512, 64
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator("cuda").manual_seed(1)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    need = mla.mla_decode_shared_workspace_bytes(B, H, B, 1, R, sms)
    buf = torch.zeros(need + (1 << 20), dtype=torch.uint8, device="cuda")
    ws = buf[:need]

    def behind(t, back=0):
        """A copy of t in buf, its first `back` bytes inside the workspace."""
        n = t.numel() * t.element_size()
        at = (need + 255) // 256 * 256 - back
        buf[at:at + n] = t.contiguous().view(-1).view(torch.uint8)
        return buf[at:at + n].view(t.dtype).view(t.shape)

    q = torch.randn(B, H, R + 64, generator=g, device="cuda").bfloat16()
    cache = torch.randn(20, bs, R + 64, generator=g, device="cuda").bfloat16()
    a = dict(q=q, kv_cache=cache, block_table=i32([[0, 1, 2]] * B), seq_lens=i32([140, 150, 130, 0]),
             group_seqs=i32([0, B]), prefix_lens=i32([128]))
    out = dict(out=torch.zeros(B, H, R, dtype=torch.bfloat16, device="cuda"),
               lse=torch.zeros(B, H, device="cuda"))
    ref = mla.decode_shared(**a, sm_scale=0.07, kv_lora_rank=R)
    for name in [*a, *out]:
        if name == "kv_cache":
            continue
        for back in (0, 256):
            args = {**a, **out}
            args[name] = behind(args[name], back)
            if back:
                with pytest.raises(mla.MlaError):
                    mla.decode_shared(**args, sm_scale=0.07, kv_lora_rank=R, workspace=ws)
            else:
                o, lse = mla.decode_shared(**args, sm_scale=0.07, kv_lora_rank=R, workspace=ws)
                assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1]), name
