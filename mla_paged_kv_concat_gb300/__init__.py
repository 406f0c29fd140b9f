"""MLA decode over a paged latent KV cache, GB300-native (sm_103a).

Thin Python binding over the C ABI of ``libmla.so`` (``include/mla.h``):

* ``mla_cache_write``, ``mla_decode``, ``mla_decode_ex``,
  ``mla_num_kv_splits``, ``mla_decode_workspace_bytes`` — the C entry points
  under the same names, taking raw device pointers (ints) and a stream handle.
* ``mla_norm_rope_cache_write`` and ``norm_rope_cache_write(...)`` — the cache
  write fused with the RMSNorm of kv_c and the rotary embedding of k_pe / q_pe.
* ``DecodePlan`` — ``mla_plan_create`` / ``mla_plan_run``: a validated step
  over fixed tensors whose ``run()`` only launches kernels (CUDA-graph safe).
* ``mla_lse_merge`` and ``lse_merge(...)`` — the cross-shard LSE merge of
  per-shard (o, lse) pairs (decode context parallelism).
* ``batch_build(...)`` and ``blocks_release(...)`` — a step's block table, slot
  map, positions and cumulative lengths from its requests' lengths, pages
  taken off and put back onto a stack of free ones.
* ``gather_cache(...)`` — cached rows of a ragged batch as contiguous bf16.
* ``expand_kv(...)``, ``absorb_q(...)`` and ``project_v(...)`` — the products
  with the kv_b weight of the expanded and the absorbed form.
* ``prefill(...)`` — attention of the expanded form over ragged prompts.
* ``cache_write(...)`` and ``decode(...)`` — torch-tensor conveniences that
  only marshal pointers, strides and the current CUDA stream; every step of
  the computation runs in the library's CUDA kernels.

PyTorch supplies device memory and streams; nothing here computes the method.
"""
from __future__ import annotations

from typing import NamedTuple

from . import _lib
from ._lib import (MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_FP8_E5M2, MLA_PATH_AUTO,
                   MLA_PATH_MMA_SYNC, MLA_PATH_TCGEN05, MlaError, load)

__all__ = [
    "mla_cache_write", "mla_decode", "mla_decode_ex", "mla_num_kv_splits",
    "mla_decode_workspace_bytes", "mla_lse_merge", "mla_norm_rope_cache_write",
    "cache_write", "norm_rope_cache_write", "decode", "lse_merge", "DecodePlan",
    "mla_batch_build", "mla_blocks_release", "mla_gather_cache",
    "mla_expand_kv", "mla_absorb_q", "mla_project_v", "expand_kv", "absorb_q", "project_v",
    "mla_prefill", "mla_prefill_num_kv_splits", "mla_prefill_workspace_bytes", "prefill",
    "batch_build", "blocks_release", "gather_cache", "BatchTables",
    "MlaError", "load",
    "MLA_KV_BF16", "MLA_KV_FP8_E4M3", "MLA_KV_FP8_E5M2", "MLA_PATH_AUTO", "MLA_PATH_MMA_SYNC",
    "MLA_PATH_TCGEN05",
]


# ---------------------------------------------------------------- raw C ABI
def mla_cache_write(*args) -> int:
    return load().mla_cache_write(*args)


def mla_decode(*args) -> int:
    return load().mla_decode(*args)


def mla_decode_ex(*args) -> int:
    return load().mla_decode_ex(*args)


def mla_norm_rope_cache_write(*args) -> int:
    return load().mla_norm_rope_cache_write(*args)


def mla_lse_merge(*args) -> int:
    return load().mla_lse_merge(*args)


def mla_batch_build(*args) -> int:
    return load().mla_batch_build(*args)


def mla_blocks_release(*args) -> int:
    return load().mla_blocks_release(*args)


def mla_gather_cache(*args) -> int:
    return load().mla_gather_cache(*args)


def mla_expand_kv(*args) -> int:
    return load().mla_expand_kv(*args)


def mla_absorb_q(*args) -> int:
    return load().mla_absorb_q(*args)


def mla_project_v(*args) -> int:
    return load().mla_project_v(*args)


def mla_prefill(*args) -> int:
    return load().mla_prefill(*args)


def mla_prefill_num_kv_splits(num_tokens: int, num_seqs: int, num_heads: int, max_kv_len: int,
                              sm_count: int) -> int:
    return load().mla_prefill_num_kv_splits(num_tokens, num_seqs, num_heads, max_kv_len, sm_count)


def mla_prefill_workspace_bytes(num_tokens: int, num_heads: int, num_kv_splits: int,
                                v_dim: int) -> int:
    return load().mla_prefill_workspace_bytes(num_tokens, num_heads, num_kv_splits, v_dim)


def mla_num_kv_splits(max_seq_len: int, sm_count: int) -> int:
    return int(load().mla_num_kv_splits(int(max_seq_len), int(sm_count)))


def mla_decode_workspace_bytes(num_rows: int, num_heads: int, num_kv_splits: int,
                               kv_lora_rank: int) -> int:
    return int(load().mla_decode_workspace_bytes(num_rows, num_heads, num_kv_splits,
                                                 kv_lora_rank))


# ---------------------------------------------------------------- torch glue
def _torch():
    import torch
    return torch


def _stream_ptr(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _kv_dtype(kv_cache, kv_cache_dtype: str | None) -> int:
    torch = _torch()
    if kv_cache_dtype in (None, "auto"):
        if kv_cache.dtype == torch.bfloat16:
            return MLA_KV_BF16
        if kv_cache.dtype in (torch.uint8, torch.float8_e4m3fn):
            return MLA_KV_FP8_E4M3
        if kv_cache.dtype == torch.float8_e5m2:
            return MLA_KV_FP8_E5M2
        raise ValueError(f"unsupported cache dtype {kv_cache.dtype}")
    if kv_cache_dtype in ("fp8", "fp8_e4m3"):
        return MLA_KV_FP8_E4M3
    if kv_cache_dtype == "fp8_e5m2":
        return MLA_KV_FP8_E5M2
    if kv_cache_dtype == "bf16":
        return MLA_KV_BF16
    raise ValueError(f"unsupported kv_cache_dtype {kv_cache_dtype!r}")


def _cache_geom(kv_cache):
    """(num_blocks, block_size, D, block_stride) of a [NB, bs, D] cache view."""
    nb, bs, d = kv_cache.shape
    assert kv_cache.stride(2) == 1 and kv_cache.stride(1) == d, "cache rows must be dense"
    return nb, bs, d, kv_cache.stride(0)


def cache_write(kv_c, k_pe, kv_cache, slot_mapping, kv_cache_dtype: str | None = None,
                scale=None, err_count=None, stream=None) -> None:
    """Write [kv_c | k_pe] rows into ``kv_cache`` at ``slot_mapping`` (in place).

    Same operands as the pages' concat_and_cache_mla(kv_c, k_pe, kv_cache,
    slot_mapping, kv_cache_dtype, scale); ``scale`` is a device fp32 tensor
    (fp8 caches only).
    """
    kvd = _kv_dtype(kv_cache, kv_cache_dtype)
    nb, bs, d, bstride = _cache_geom(kv_cache)
    assert kv_c.stride(1) == 1 and k_pe.stride(1) == 1
    R, P = kv_c.shape[1], k_pe.shape[1]
    assert R + P == d
    st = load().mla_cache_write(
        kv_c.data_ptr(), kv_c.stride(0), k_pe.data_ptr(), k_pe.stride(0),
        slot_mapping.data_ptr(), slot_mapping.numel(), R, P, kv_cache.data_ptr(), nb, bs,
        bstride, kvd, scale.data_ptr() if scale is not None else None,
        err_count.data_ptr() if err_count is not None else None, _stream_ptr(stream))
    _lib.check(st, "mla_cache_write")


def norm_rope_cache_write(kv_c, k_pe, kv_cache, slot_mapping, gamma, eps: float, positions,
                          cos_sin_table, q_pe=None, kv_cache_dtype: str | None = None,
                          scale=None, err_count=None, stream=None) -> None:
    """RMSNorm(kv_c) * gamma and the non-NeoX rotation of k_pe by position,
    written into ``kv_cache`` at ``slot_mapping``; ``q_pe`` [T, H, 64] (bf16,
    may be the rope columns of q) is rotated in place when given.

    ``gamma`` bf16 [R]; ``positions`` int64 [T]; ``cos_sin_table`` fp32
    [max_position, 64] (cos | sin); ``scale`` a device fp32 tensor (fp8
    caches only).
    """
    kvd = _kv_dtype(kv_cache, kv_cache_dtype)
    nb, bs, d, bstride = _cache_geom(kv_cache)
    assert kv_c.stride(1) == 1 and k_pe.stride(1) == 1 and cos_sin_table.stride(1) == 1
    R, P = kv_c.shape[1], k_pe.shape[1]
    assert R + P == d and cos_sin_table.shape[1] == P
    if q_pe is not None:
        assert q_pe.stride(2) == 1 and q_pe.shape[0] >= slot_mapping.numel()
    st = load().mla_norm_rope_cache_write(
        kv_c.data_ptr(), kv_c.stride(0), k_pe.data_ptr(), k_pe.stride(0),
        slot_mapping.data_ptr(), slot_mapping.numel(), R, P, kv_cache.data_ptr(), nb, bs,
        bstride, kvd, scale.data_ptr() if scale is not None else None, gamma.data_ptr(),
        float(eps), positions.data_ptr(), cos_sin_table.data_ptr(), cos_sin_table.shape[0],
        q_pe.data_ptr() if q_pe is not None else None,
        q_pe.stride(0) if q_pe is not None else 0, q_pe.stride(1) if q_pe is not None else 0,
        q_pe.shape[1] if q_pe is not None else 0,
        err_count.data_ptr() if err_count is not None else None, _stream_ptr(stream))
    _lib.check(st, "mla_norm_rope_cache_write")


def decode(q, kv_cache, block_table, seq_lens, sm_scale: float, num_kv_splits: int, *,
           kv_lora_rank: int | None = None, kv_cache_dtype: str | None = None,
           kv_scale=None, workspace=None, out=None, lse=None, err_count=None,
           stream=None, path: int = MLA_PATH_AUTO):
    """MLA decode; returns (o [rows, H, R] bf16, lse [rows, H] fp32).

    ``q`` [rows, H, R+P] bf16, or the pair (q_nope [rows, H, R], q_pe
    [rows, H, P]) read in place without a concatenation; rows =
    len(seq_lens) * rows_per_seq.  ``kv_cache`` [NB, bs, R+P];
    ``block_table`` int32 [seqs, max_blocks]; ``seq_lens`` int32 [seqs];
    ``kv_scale`` device fp32 tensor for fp8 caches; ``workspace`` a device
    buffer of at least ``mla_decode_workspace_bytes`` bytes (allocated here
    when omitted and needed).
    """
    if isinstance(q, (tuple, list)):
        q_nope, q_pe = q
        plan = DecodePlan(q_nope, kv_cache, block_table, seq_lens, sm_scale, num_kv_splits,
                          q_pe=q_pe, kv_cache_dtype=kv_cache_dtype, kv_scale=kv_scale,
                          workspace=workspace, out=out, lse=lse, err_count=err_count,
                          path=path)
        try:
            plan.run(stream)
        finally:
            plan.close()
        return plan.out, plan.lse
    torch = _torch()
    kvd = _kv_dtype(kv_cache, kv_cache_dtype)
    nb, bs, d, bstride = _cache_geom(kv_cache)
    rows, H, dq = q.shape
    assert dq == d and q.stride(2) == 1
    R = kv_lora_rank if kv_lora_rank is not None else d - 64
    P = d - R
    seqs = seq_lens.numel()
    if out is None:
        out = torch.empty(rows, H, R, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty(rows, H, dtype=torch.float32, device=q.device)
    need = mla_decode_workspace_bytes(rows, H, num_kv_splits, R)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = load().mla_decode_ex(
        q.data_ptr(), q.stride(0), q.stride(1), rows, H, kv_cache.data_ptr(), kvd, nb, bs,
        bstride, R, P, block_table.data_ptr(), block_table.stride(0), block_table.shape[1],
        seq_lens.data_ptr(), seqs, float(sm_scale),
        kv_scale.data_ptr() if kv_scale is not None else None, int(num_kv_splits), ws_ptr,
        ws_bytes, out.data_ptr(), lse.data_ptr(),
        err_count.data_ptr() if err_count is not None else None, _stream_ptr(stream),
        int(path))
    _lib.check(st, "mla_decode")
    return out, lse


class DecodePlan:
    """A validated, prepared decode step over fixed tensors (``mla_plan_*``).

    ``run()`` only launches kernels, so it can be captured into a CUDA graph
    and replayed after new values are copied into the same tensors.  The
    tensors are kept referenced for the plan's life.

    ``q``: [rows, H, R+P] bf16, or dims [0, R) when ``q_pe`` [rows, H, P] is
    given.  ``write``: optional dict(kv_c, k_pe, slot_mapping) of the step's
    new tokens, written before stage 1; ``norm_rope``: optional dict(gamma,
    eps, positions, cos_sin_table, rotate_q) that makes that write the fused
    RMSNorm + rotary write (rotate_q also rotates the query's rope dims in
    place).
    """

    def __init__(self, q, kv_cache, block_table, seq_lens, sm_scale: float, num_kv_splits: int,
                 *, q_pe=None, kv_cache_dtype: str | None = None, kv_scale=None,
                 workspace=None, out=None, lse=None, err_count=None,
                 path: int = MLA_PATH_AUTO, write=None, norm_rope=None):
        import ctypes
        torch = _torch()
        kvd = _kv_dtype(kv_cache, kv_cache_dtype)
        nb, bs, d, bstride = _cache_geom(kv_cache)
        rows, H, dq = q.shape
        assert q.stride(2) == 1
        if q_pe is not None:
            R, P = dq, q_pe.shape[2]
            assert q_pe.shape[:2] == (rows, H) and q_pe.stride(2) == 1
        else:
            R, P = d - 64, 64
            assert dq == d
        assert R + P == d
        if out is None:
            out = torch.empty(rows, H, R, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = torch.empty(rows, H, dtype=torch.float32, device=q.device)
        need = mla_decode_workspace_bytes(rows, H, num_kv_splits, R)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        self.out, self.lse = out, lse
        self._keep = [q, q_pe, kv_cache, block_table, seq_lens, kv_scale, workspace, out, lse,
                      err_count, write, norm_rope]
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        dd = _lib.DecodeDesc(
            q=q.data_ptr(), q_row_stride=q.stride(0), q_head_stride=q.stride(1),
            q_pe=ptr(q_pe), q_pe_row_stride=q_pe.stride(0) if q_pe is not None else 0,
            q_pe_head_stride=q_pe.stride(1) if q_pe is not None else 0,
            num_rows=rows, num_heads=H, kv_cache=kv_cache.data_ptr(), kv_dtype=kvd,
            num_blocks=nb, block_size=bs, block_stride=bstride, kv_lora_rank=R, rope_dim=P,
            kv_scale=ptr(kv_scale), block_table=block_table.data_ptr(),
            block_table_stride=block_table.stride(0), max_blocks_per_seq=block_table.shape[1],
            seq_lens=seq_lens.data_ptr(), num_seqs=seq_lens.numel(), sm_scale=float(sm_scale),
            num_kv_splits=int(num_kv_splits), workspace=ptr(workspace),
            workspace_bytes=workspace.numel() * workspace.element_size()
            if workspace is not None else 0,
            o=out.data_ptr(), lse=lse.data_ptr(), err_count=ptr(err_count), path=int(path))
        if write is not None:
            kv_c, k_pe, slots = write["kv_c"], write["k_pe"], write["slot_mapping"]
            assert kv_c.stride(1) == 1 and k_pe.stride(1) == 1
            dd.kv_c, dd.kv_c_row_stride = kv_c.data_ptr(), kv_c.stride(0)
            dd.k_pe, dd.k_pe_row_stride = k_pe.data_ptr(), k_pe.stride(0)
            dd.slot_mapping, dd.num_tokens = slots.data_ptr(), slots.numel()
            if norm_rope is not None:
                tab = norm_rope["cos_sin_table"]
                assert tab.stride(1) == 1 and tab.shape[1] == P
                dd.gamma = norm_rope["gamma"].data_ptr()
                dd.eps = float(norm_rope["eps"])
                dd.positions = norm_rope["positions"].data_ptr()
                dd.cos_sin_table, dd.max_position = tab.data_ptr(), tab.shape[0]
                dd.rotate_q = int(bool(norm_rope.get("rotate_q", False)))
        handle = ctypes.c_void_p()
        _lib.check(load().mla_plan_create(ctypes.byref(dd), ctypes.byref(handle)),
                   "mla_plan_create")
        self._handle = handle.value

    def run(self, stream=None):
        """Launch the step on ``stream`` (default: the current torch stream)."""
        assert self._handle is not None, "plan closed"
        _lib.check(load().mla_plan_run(self._handle, _stream_ptr(stream)), "mla_plan_run")
        return self.out, self.lse

    def close(self):
        if getattr(self, "_handle", None) is not None:
            load().mla_plan_destroy(self._handle)
            self._handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def lse_merge(o_parts, lse_parts, *, out=None, lse=None, stream=None):
    """Cross-shard LSE merge; returns (o [rows, H, R] bf16, lse [rows, H] fp32).

    ``o_parts`` bf16 [G, rows, H, R] and ``lse_parts`` fp32 [G, rows, H]: the
    (o, lse) of G disjoint KV token shards of the same query vectors, each
    part dense in (rows, H, R) / (rows, H); lse = -inf marks an empty part.
    """
    torch = _torch()
    G, rows, H, R = o_parts.shape
    assert lse_parts.shape == (G, rows, H)
    assert o_parts.stride()[1:] == (H * R, R, 1) and lse_parts.stride()[1:] == (H, 1)
    if out is None:
        out = torch.empty(rows, H, R, dtype=torch.bfloat16, device=o_parts.device)
    if lse is None:
        lse = torch.empty(rows, H, dtype=torch.float32, device=o_parts.device)
    st = load().mla_lse_merge(
        o_parts.data_ptr(), o_parts.stride(0), lse_parts.data_ptr(), lse_parts.stride(0), G,
        rows, H, R, out.data_ptr(), lse.data_ptr(), _stream_ptr(stream))
    _lib.check(st, "mla_lse_merge")
    return out, lse


# ------------------------------------------------------- prompts and batches
def _check(cond: bool, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _cuda(stream, **tensors):
    """Checks that every tensor given is on the current CUDA device (where the
    kernels run); returns that device."""
    torch = _torch()
    for name, t in tensors.items():
        _check(t is None or t.is_cuda, f"{name} must be a CUDA tensor")
    dev = torch.device("cuda", torch.cuda.current_device())
    for name, t in tensors.items():
        _check(t is None or t.device == dev, f"{name} is not on the current device {dev}")
    _check(stream is None or stream.device == dev, f"the stream is not on the current device {dev}")
    return dev


def _empty(stream, *shape, dtype, device):
    """A new tensor for a kernel that runs on `stream`."""
    torch = _torch()
    t = torch.empty(*shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


def _typed(t, dtype, shape, name):
    """Checks dtype and shape (None: any size) and unit last stride."""
    if t is None:
        return
    _check(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
    _check(t.dim() == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)),
           f"{name} has shape {tuple(t.shape)}, not {shape}")
    _check(t.numel() == 0 or t.shape[-1] == 1 or t.stride(-1) == 1,
           f"{name} must have unit last stride")


def _ptr(t):
    return t.data_ptr() if t is not None else None


class BatchTables(NamedTuple):
    """A step's tables, from :func:`batch_build`."""
    block_table: object    # int32 [reqs, max_blocks]
    seq_lens: object       # int32 [reqs]
    cu_seqlens_q: object   # int32 [reqs + 1]
    cu_seqlens_k: object   # int32 [reqs + 1]
    positions: object      # int64 [tokens]
    slot_mapping: object   # int64 [tokens]
    free_count: object     # int32 [1]


def batch_build(query_lens, context_lens, req_block_table, free_blocks, free_count,
                block_size: int, num_blocks: int, num_tokens: int | None = None, *, req_ids=None,
                block_table=None, seq_lens=None, cu_seqlens_q=None, cu_seqlens_k=None,
                positions=None, slot_mapping=None, free_count_out=None, err_count=None,
                stream=None) -> BatchTables:
    """Build a step's tables from int32 [B] ``query_lens`` (new tokens) and
    ``context_lens`` (cached tokens) of its requests.

    ``req_block_table`` int32 [rows, max_blocks] holds each running request's
    pages (row ``req_ids[b]``, or b) and gets the new ones, taken off the top
    of the stack ``free_blocks`` int32 [n] of height ``free_count`` int32 [1].
    ``num_tokens``: rows of positions and slot_mapping (padding rows get slot
    -1); needed unless one of the two is given.  Outputs are allocated when
    not given; a block table allocated here starts as zeros.
    ``free_count_out`` may be ``free_count`` (updated in place).
    """
    torch = _torch()
    i32, i64 = torch.int32, torch.int64
    dev = _cuda(stream, query_lens=query_lens, context_lens=context_lens,
                req_block_table=req_block_table, free_blocks=free_blocks, free_count=free_count,
                req_ids=req_ids, block_table=block_table, seq_lens=seq_lens,
                cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k, positions=positions,
                slot_mapping=slot_mapping, free_count_out=free_count_out, err_count=err_count)
    _check(query_lens.dim() == 1, "query_lens must have one dimension")
    B = query_lens.shape[0]
    if num_tokens is None:
        given = positions if positions is not None else slot_mapping
        _check(given is not None, "num_tokens is needed when no token output is given")
        num_tokens = given.shape[0]
    _typed(req_block_table, i32, (None, None), "req_block_table")
    rows, maxb = req_block_table.shape
    if block_table is None:
        with torch.cuda.stream(stream):
            block_table = torch.zeros(B, maxb, dtype=i32, device=dev)
    mk = lambda t, n, d: t if t is not None else _empty(stream, n, dtype=d, device=dev)  # noqa: E731
    seq_lens = mk(seq_lens, B, i32)
    cu_seqlens_q, cu_seqlens_k = mk(cu_seqlens_q, B + 1, i32), mk(cu_seqlens_k, B + 1, i32)
    positions, slot_mapping = mk(positions, num_tokens, i64), mk(slot_mapping, num_tokens, i64)
    free_count_out = mk(free_count_out, 1, i32)
    for t, d, shape, name in (
            (query_lens, i32, (B,), "query_lens"), (context_lens, i32, (B,), "context_lens"),
            (req_ids, i32, (B,), "req_ids"), (free_blocks, i32, (None,), "free_blocks"),
            (free_count, i32, (1,), "free_count"), (free_count_out, i32, (1,), "free_count_out"),
            (block_table, i32, (B, maxb), "block_table"), (seq_lens, i32, (B,), "seq_lens"),
            (cu_seqlens_q, i32, (B + 1,), "cu_seqlens_q"),
            (cu_seqlens_k, i32, (B + 1,), "cu_seqlens_k"),
            (positions, i64, (num_tokens,), "positions"),
            (slot_mapping, i64, (num_tokens,), "slot_mapping"),
            (err_count, i32, (1,), "err_count")):
        _typed(t, d, shape, name)
    st = load().mla_batch_build(
        _ptr(req_ids), query_lens.data_ptr(), context_lens.data_ptr(), B,
        req_block_table.data_ptr(), req_block_table.stride(0), rows, maxb, int(block_size),
        int(num_blocks), free_blocks.data_ptr(), free_blocks.numel(), free_count.data_ptr(),
        free_count_out.data_ptr(), int(num_tokens), block_table.data_ptr(),
        block_table.stride(0), seq_lens.data_ptr(), cu_seqlens_q.data_ptr(),
        cu_seqlens_k.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(), _ptr(err_count),
        _stream_ptr(stream))
    _lib.check(st, "mla_batch_build")
    return BatchTables(block_table, seq_lens, cu_seqlens_q, cu_seqlens_k, positions,
                       slot_mapping, free_count_out)


def blocks_release(held_lens, req_block_table, free_blocks, free_count, block_size: int,
                   num_blocks: int, *, req_ids=None, free_count_out=None, err_count=None,
                   stream=None):
    """Put the pages of finished requests (int32 [B] ``held_lens`` tokens each,
    rows ``req_ids`` of ``req_block_table``) back onto the stack
    ``free_blocks``; returns the new height (``free_count_out``, by default
    ``free_count`` updated in place)."""
    torch = _torch()
    i32 = torch.int32
    if free_count_out is None:
        free_count_out = free_count
    _cuda(stream, held_lens=held_lens, req_block_table=req_block_table, free_blocks=free_blocks,
          free_count=free_count, req_ids=req_ids, free_count_out=free_count_out,
          err_count=err_count)
    _typed(held_lens, i32, (None,), "held_lens")
    B = held_lens.shape[0]
    for t, shape, name in ((req_block_table, (None, None), "req_block_table"),
                           (req_ids, (B,), "req_ids"), (free_blocks, (None,), "free_blocks"),
                           (free_count, (1,), "free_count"),
                           (free_count_out, (1,), "free_count_out"),
                           (err_count, (1,), "err_count")):
        _typed(t, i32, shape, name)
    rows, maxb = req_block_table.shape
    st = load().mla_blocks_release(
        _ptr(req_ids), held_lens.data_ptr(), B, req_block_table.data_ptr(),
        req_block_table.stride(0), rows, maxb, int(block_size), int(num_blocks),
        free_blocks.data_ptr(), free_blocks.numel(), free_count.data_ptr(),
        free_count_out.data_ptr(), _ptr(err_count), _stream_ptr(stream))
    _lib.check(st, "mla_blocks_release")
    return free_count_out


def gather_cache(kv_cache, block_table, cu_seqlens, num_tokens: int | None = None, *,
                 kv_lora_rank: int | None = None, seq_starts=None,
                 kv_cache_dtype: str | None = None, kv_scale=None, kv_c=None, k_pe=None,
                 err_count=None, stream=None):
    """Cached rows of a ragged batch as (kv_c bf16 [T, R], k_pe bf16 [T, P]).

    Output row t of sequence b (``cu_seqlens`` int32 [B + 1]) is its cached
    token ``seq_starts[b] + t - cu_seqlens[b]`` (``seq_starts`` int32 [B], by
    default 0).  ``num_tokens`` rows are allocated unless kv_c and k_pe are
    given; rows past ``cu_seqlens[B]`` are left as they were.  fp8 caches are
    multiplied by the device scalar ``kv_scale``.
    """
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    dev = _cuda(stream, kv_cache=kv_cache, block_table=block_table, cu_seqlens=cu_seqlens,
                seq_starts=seq_starts, kv_scale=kv_scale, kv_c=kv_c, k_pe=k_pe,
                err_count=err_count)
    kvd = _kv_dtype(kv_cache, kv_cache_dtype)
    _check(kv_cache.element_size() == (2 if kvd == MLA_KV_BF16 else 1),
           "kv_cache_dtype does not fit the cache")
    nb, bs, d, bstride = _cache_geom(kv_cache)
    R = kv_lora_rank if kv_lora_rank is not None else d - 64
    P = d - R
    _typed(block_table, i32, (None, None), "block_table")
    B = block_table.shape[0]
    if num_tokens is None:
        _check(kv_c is not None, "num_tokens is needed when kv_c is not given")
        num_tokens = kv_c.shape[0]
    if kv_c is None:
        kv_c = _empty(stream, num_tokens, R, dtype=bf, device=dev)
    if k_pe is None:
        k_pe = _empty(stream, num_tokens, P, dtype=bf, device=dev)
    for t, dt, shape, name in ((cu_seqlens, i32, (B + 1,), "cu_seqlens"),
                               (seq_starts, i32, (B,), "seq_starts"),
                               (kv_c, bf, (num_tokens, R), "kv_c"),
                               (k_pe, bf, (num_tokens, P), "k_pe"),
                               (err_count, i32, (1,), "err_count")):
        _typed(t, dt, shape, name)
    _check(kv_scale is None or (kv_scale.dtype == torch.float32 and kv_scale.numel() == 1),
           "kv_scale must be one float32")
    st = load().mla_gather_cache(
        kv_cache.data_ptr(), kvd, nb, bs, bstride, R, P, block_table.data_ptr(),
        block_table.stride(0), block_table.shape[1], cu_seqlens.data_ptr(), _ptr(seq_starts), B,
        int(num_tokens), _ptr(kv_scale), kv_c.data_ptr(), kv_c.stride(0), k_pe.data_ptr(),
        k_pe.stride(0), _ptr(err_count), _stream_ptr(stream))
    _lib.check(st, "mla_gather_cache")
    return kv_c, k_pe


NOPE_DIM = 128  # head dims of the expanded form: keys without the rope part
V_DIM = 128     # and values


def _strides(t):
    """(row, head) strides of a [T, H, D] tensor; those of dimensions of size
    1, which torch leaves arbitrary, as in a dense tensor."""
    T, H, D = t.shape
    hs = t.stride(1) if H > 1 else D
    rs = t.stride(0) if T > 1 else (H * hs if H > 1 else D)
    return rs, hs


def _kv_b(w_kv_b, num_heads: int):
    """Checks the kv_b weight [H * 256, R]; returns R."""
    torch = _torch()
    _typed(w_kv_b, torch.bfloat16, (num_heads * (NOPE_DIM + V_DIM), None), "w_kv_b")
    return w_kv_b.shape[1]


def expand_kv(kv_c, w_kv_b, num_heads: int, *, k_nope=None, v=None, err_count=None,
              stream=None):
    """Keys and values of latents ``kv_c`` [T, R]: (k_nope, v), bf16
    [T, H, 128] each; ``w_kv_b`` [H * 256, R] is the kv_b projection's weight
    (per head 128 rows of W_UK, then 128 of W_UV).  Allocated as the two
    halves of one [T, H, 256] buffer unless both are given."""
    torch = _torch()
    bf = torch.bfloat16
    dev = _cuda(stream, kv_c=kv_c, w_kv_b=w_kv_b, k_nope=k_nope, v=v, err_count=err_count)
    R = _kv_b(w_kv_b, num_heads)
    _typed(kv_c, bf, (None, R), "kv_c")
    T = kv_c.shape[0]
    _check((k_nope is None) == (v is None), "give both k_nope and v, or neither")
    if k_nope is None:
        kv = _empty(stream, T, num_heads, NOPE_DIM + V_DIM, dtype=bf, device=dev)
        k_nope, v = kv[..., :NOPE_DIM], kv[..., NOPE_DIM:]
    _typed(k_nope, bf, (T, num_heads, NOPE_DIM), "k_nope")
    _typed(v, bf, (T, num_heads, V_DIM), "v")
    _typed(err_count, torch.int32, (1,), "err_count")
    st = load().mla_expand_kv(
        kv_c.data_ptr(), kv_c.stride(0) if T > 1 else R, T, w_kv_b.data_ptr(), w_kv_b.stride(0),
        num_heads, R, NOPE_DIM, V_DIM, k_nope.data_ptr(), *_strides(k_nope), v.data_ptr(),
        *_strides(v), _ptr(err_count), _stream_ptr(stream))
    _lib.check(st, "mla_expand_kv")
    return k_nope, v


def _head_product(fn, x, w_kv_b, n_in, n_out, out, err_count, stream):
    torch = _torch()
    bf = torch.bfloat16
    dev = _cuda(stream, x=x, w_kv_b=w_kv_b, out=out, err_count=err_count)
    _check(x.dim() == 3, "the input must be [tokens, heads, dims]")
    T, H, _ = x.shape
    R = _kv_b(w_kv_b, H)
    n_in, n_out = n_in or R, n_out or R
    _typed(x, bf, (T, H, n_in), "the input")
    if out is None:
        out = _empty(stream, T, H, n_out, dtype=bf, device=dev)
    _typed(out, bf, (T, H, n_out), "out")
    _typed(err_count, torch.int32, (1,), "err_count")
    st = getattr(load(), fn)(
        x.data_ptr(), *_strides(x), T, w_kv_b.data_ptr(), w_kv_b.stride(0), H, R, NOPE_DIM,
        V_DIM, out.data_ptr(), *_strides(out), _ptr(err_count), _stream_ptr(stream))
    _lib.check(st, fn)
    return out


def absorb_q(q_nope, w_kv_b, *, out=None, err_count=None, stream=None):
    """The latent query ql_nope [T, H, R] of ``q_nope`` [T, H, 128] (any row
    and head strides: a column slice of q will do): ``decode``'s query is then
    the pair (ql_nope, q_pe).  ``w_kv_b`` as in :func:`expand_kv`."""
    return _head_product("mla_absorb_q", q_nope, w_kv_b, NOPE_DIM, None, out, err_count, stream)


def project_v(o, w_kv_b, *, out=None, err_count=None, stream=None):
    """Values [T, H, 128] of ``decode``'s latent output ``o`` [T, H, R];
    ``w_kv_b`` as in :func:`expand_kv`."""
    return _head_product("mla_project_v", o, w_kv_b, None, V_DIM, out, err_count, stream)


def prefill(q, k_nope, v, k_pe, cu_seqlens_q, cu_seqlens_k, sm_scale: float, *,
            causal: bool = True, num_kv_splits: int = 1, workspace=None, out=None, lse=None,
            err_count=None, stream=None):
    """Attention of the expanded form; returns (o [T, H, 128] bf16, lse [T, H]
    fp32).

    ``q`` [T, H, 192] bf16 (128 dims, then 64 rope dims), or the pair (q_nope
    [T, H, 128], q_pe [T, H, 64]); ``k_nope`` and ``v`` [Tk, H, 128] as
    :func:`expand_kv` gives them, ``k_pe`` [Tk, 64]; ``cu_seqlens_q`` and
    ``cu_seqlens_k`` int32 [seqs + 1].  Causal rows are the last tokens of
    their sequence's keys.  ``num_kv_splits``: parts of the key axis, from
    ``mla_prefill_num_kv_splits``; the workspace they need is allocated here
    when not given.
    """
    torch = _torch()
    bf, i32 = torch.bfloat16, torch.int32
    q, q_pe = q if isinstance(q, (tuple, list)) else (q, None)
    dev = _cuda(stream, q=q, q_pe=q_pe, k_nope=k_nope, v=v, k_pe=k_pe, cu_seqlens_q=cu_seqlens_q,
                cu_seqlens_k=cu_seqlens_k, workspace=workspace, out=out, lse=lse,
                err_count=err_count)
    _check(q.dim() == 3 and k_pe.dim() == 2, "q must be [tokens, heads, dims], k_pe [keys, 64]")
    T, H, _ = q.shape
    Tk, P = k_pe.shape
    B = cu_seqlens_q.shape[0] - 1
    if out is None:
        out = _empty(stream, T, H, V_DIM, dtype=bf, device=dev)
    if lse is None:
        lse = _empty(stream, T, H, dtype=torch.float32, device=dev)
    for t, d, shape, name in ((q, bf, (T, H, NOPE_DIM + (P if q_pe is None else 0)), "q"),
                              (q_pe, bf, (T, H, P), "q_pe"),
                              (k_nope, bf, (Tk, H, NOPE_DIM), "k_nope"),
                              (v, bf, (Tk, H, V_DIM), "v"), (k_pe, bf, (Tk, P), "k_pe"),
                              (cu_seqlens_q, i32, (B + 1,), "cu_seqlens_q"),
                              (cu_seqlens_k, i32, (B + 1,), "cu_seqlens_k"),
                              (out, bf, (T, H, V_DIM), "out"),
                              (lse, torch.float32, (T, H), "lse"),
                              (err_count, i32, (1,), "err_count")):
        _typed(t, d, shape, name)
    _check(B >= 0 and lse.is_contiguous(), "lse must be contiguous, cu_seqlens_q not empty")
    need = mla_prefill_workspace_bytes(T, H, num_kv_splits, V_DIM)
    if need and workspace is None:
        workspace = _empty(stream, need, dtype=torch.uint8, device=dev)
    _check(workspace is None or workspace.is_contiguous(), "workspace must be contiguous")
    st = load().mla_prefill(
        q.data_ptr(), *_strides(q), _ptr(q_pe), *(_strides(q_pe) if q_pe is not None else (0, 0)),
        T, H, k_nope.data_ptr(), *_strides(k_nope), v.data_ptr(), *_strides(v), k_pe.data_ptr(),
        k_pe.stride(0) if Tk > 1 else P, Tk, NOPE_DIM, P, V_DIM, cu_seqlens_q.data_ptr(),
        cu_seqlens_k.data_ptr(), B, int(bool(causal)), float(sm_scale), int(num_kv_splits),
        _ptr(workspace), workspace.numel() * workspace.element_size() if workspace is not None else 0,
        out.data_ptr(), *_strides(out), lse.data_ptr(), _ptr(err_count), _stream_ptr(stream))
    _lib.check(st, "mla_prefill")
    return out, lse
