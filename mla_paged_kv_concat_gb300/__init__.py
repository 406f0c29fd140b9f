"""MLA decode over a paged latent KV cache, GB300-native (sm_103a).

Thin Python binding over the C ABI of ``libmla.so`` (``include/mla.h``):

* ``mla_cache_write``, ``mla_decode``, ``mla_decode_ex``,
  ``mla_num_kv_splits``, ``mla_decode_workspace_bytes`` — the C entry points
  under the same names, taking raw device pointers (ints) and a stream handle.
* ``mla_norm_rope_cache_write`` and ``norm_rope_cache_write(...)`` — the cache
  write fused with the RMSNorm of kv_c and the rotary embedding of k_pe / q_pe.
* ``decode_shared(...)`` — the decode of a batch whose sequences share prefixes,
  a prefix read once for all of them.
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
* ``linear(...)`` — a projection with bias, activation and residual.
* ``prefill(...)`` — attention of the expanded form over ragged prompts.
* ``prefill_shared(...)`` — the same for sequences that share prefixes.
* ``cache_write(...)`` and ``decode(...)`` — torch-tensor conveniences that
  only marshal pointers, strides and the current CUDA stream; every step of
  the computation runs in the library's CUDA kernels.

PyTorch supplies device memory and streams; nothing here computes the method.
"""
from __future__ import annotations

from typing import NamedTuple

from . import _lib
from ._lib import (MLA_ACT_GELU, MLA_ACT_GELU_TANH, MLA_ACT_NONE, MLA_ACT_RELU, MLA_ACT_SILU,
                   MLA_KV_BF16, MLA_KV_FP8_E4M3, MLA_KV_FP8_E5M2, MLA_PATH_AUTO,
                   MLA_PATH_MMA_SYNC, MLA_PATH_TCGEN05, MlaError, load)

__all__ = [
    "mla_cache_write", "mla_decode", "mla_decode_ex", "mla_num_kv_splits",
    "mla_decode_workspace_bytes", "mla_lse_merge", "mla_norm_rope_cache_write",
    "cache_write", "norm_rope_cache_write", "decode", "lse_merge", "DecodePlan",
    "mla_batch_build", "mla_blocks_release", "mla_gather_cache",
    "mla_expand_kv", "mla_absorb_q", "mla_project_v", "expand_kv", "absorb_q", "project_v",
    "mla_prefill", "mla_prefill_num_kv_splits", "mla_prefill_workspace_bytes", "prefill",
    "batch_build", "blocks_release", "gather_cache", "BatchTables", "mla_linear", "linear",
    "mla_prefill_shared", "mla_prefill_shared_num_kv_splits", "prefill_shared",
    "mla_decode_shared", "mla_decode_shared_workspace_bytes", "decode_shared",
    "MlaError", "load",
    "MLA_KV_BF16", "MLA_KV_FP8_E4M3", "MLA_KV_FP8_E5M2", "MLA_PATH_AUTO", "MLA_PATH_MMA_SYNC",
    "MLA_PATH_TCGEN05", "MLA_ACT_NONE", "MLA_ACT_RELU", "MLA_ACT_SILU", "MLA_ACT_GELU",
    "MLA_ACT_GELU_TANH",
]


# ---------------------------------------------------------------- raw C ABI
def mla_cache_write(*args) -> int:
    return load().mla_cache_write(*args)


def mla_decode(*args) -> int:
    return load().mla_decode(*args)


def mla_decode_ex(*args) -> int:
    return load().mla_decode_ex(*args)


def mla_decode_shared(*args) -> int:
    return load().mla_decode_shared(*args)


def mla_decode_shared_workspace_bytes(num_rows: int, num_heads: int, num_seqs: int,
                                      num_groups: int, kv_lora_rank: int, sm_count: int) -> int:
    return int(load().mla_decode_shared_workspace_bytes(num_rows, num_heads, num_seqs, num_groups,
                                                        kv_lora_rank, sm_count))


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


def mla_linear(*args) -> int:
    return load().mla_linear(*args)


def mla_prefill(*args) -> int:
    return load().mla_prefill(*args)


def mla_prefill_num_kv_splits(num_tokens: int, num_seqs: int, num_heads: int, max_kv_len: int,
                              sm_count: int) -> int:
    return load().mla_prefill_num_kv_splits(num_tokens, num_seqs, num_heads, max_kv_len, sm_count)


def mla_prefill_shared(*args) -> int:
    return load().mla_prefill_shared(*args)


def mla_prefill_shared_num_kv_splits(num_tokens: int, num_seqs: int, num_groups: int,
                                     num_heads: int, max_prefix_len: int, max_kv_len: int,
                                     sm_count: int) -> tuple[int, int]:
    """(parts of a prefix's keys, parts of a sequence's own keys or 0: those
    together with the prefix's)."""
    import ctypes
    own = ctypes.c_int()
    pre = load().mla_prefill_shared_num_kv_splits(num_tokens, num_seqs, num_groups, num_heads,
                                                  max_prefix_len, max_kv_len, sm_count,
                                                  ctypes.byref(own))
    return pre, own.value


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


def _empty(stream, *shape, dtype, device, returned=True):
    """Memory of the stream that a call runs on.  A block of the current
    stream's pool may still be in use by work queued there, which a kernel on
    another stream does not wait for.  What is returned may be used on the
    caller's own current stream too, so its block is not given out again
    before that."""
    torch = _torch()
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    current = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = torch.empty(*shape, dtype=dtype, device=device)
    if returned and current != stream:
        t.record_stream(current)
    return t


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
    when omitted and needed).  What is allocated here is memory of the stream
    that the call runs on (``stream``, by default the current one).
    """
    if isinstance(q, (tuple, list)):
        q_nope, q_pe = q
        plan = DecodePlan(q_nope, kv_cache, block_table, seq_lens, sm_scale, num_kv_splits,
                          q_pe=q_pe, kv_cache_dtype=kv_cache_dtype, kv_scale=kv_scale,
                          workspace=workspace, out=out, lse=lse, err_count=err_count,
                          path=path, _stream=stream)
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
        out = _empty(stream, rows, H, R, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = _empty(stream, rows, H, dtype=torch.float32, device=q.device)
    need = mla_decode_workspace_bytes(rows, H, num_kv_splits, R)
    if need and workspace is None:
        workspace = _empty(stream, need, dtype=torch.uint8, device=q.device, returned=False)
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


def decode_shared(q, kv_cache, block_table, seq_lens, group_seqs, prefix_lens, sm_scale: float, *,
                  kv_lora_rank: int | None = None, kv_cache_dtype: str | None = None,
                  kv_scale=None, workspace=None, out=None, lse=None, err_count=None, stream=None):
    """:func:`decode` for sequences that share prefixes; returns (o [rows, H, R]
    bf16, lse [rows, H] fp32).

    Group g is the sequences ``group_seqs[g]`` to ``group_seqs[g + 1]`` (int32
    [groups + 1]); the first ``prefix_lens[g]`` (int32 [groups]) tokens of each are
    the same, through whichever of their block tables they are read.  Sequences
    shorter than that (padded rows of length 0) or of no group are decoded by
    themselves.  Other arguments as :func:`decode`; ``workspace`` a device buffer of
    ``mla_decode_shared_workspace_bytes`` bytes, 256-byte aligned (allocated here
    when omitted).  The work is shared out on the device: the call can be captured
    and replayed with other lengths.
    """
    q, q_pe = q if isinstance(q, (tuple, list)) else (q, None)
    return _bind().decode_shared(
        q, q_pe, kv_cache, -1 if kv_cache_dtype is None else _kv_dtype(kv_cache, kv_cache_dtype),
        block_table, seq_lens, group_seqs, prefix_lens, sm_scale,
        -1 if kv_lora_rank is None else kv_lora_rank, kv_scale, workspace, out, lse, err_count,
        stream)


class DecodePlan:
    """A validated, prepared decode step over fixed tensors (``mla_plan_*``).

    ``run()`` only launches kernels, so it can be captured into a CUDA graph
    and replayed after new values are copied into the same tensors.  The
    tensors are kept referenced for the plan's life; those not given are
    allocated here, on the current stream: another stream waits for that one
    before its first ``run``.

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
                 path: int = MLA_PATH_AUTO, write=None, norm_rope=None, _stream=None):
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
            out = _empty(_stream, rows, H, R, dtype=torch.bfloat16, device=q.device)
        if lse is None:
            lse = _empty(_stream, rows, H, dtype=torch.float32, device=q.device)
        need = mla_decode_workspace_bytes(rows, H, num_kv_splits, R)
        if need and workspace is None:
            workspace = _empty(_stream, need, dtype=torch.uint8, device=q.device, returned=False)
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
    What is allocated here is memory of the stream that the call runs on.
    """
    torch = _torch()
    G, rows, H, R = o_parts.shape
    assert lse_parts.shape == (G, rows, H)
    assert o_parts.stride()[1:] == (H * R, R, 1) and lse_parts.stride()[1:] == (H, 1)
    if out is None:
        out = _empty(stream, rows, H, R, dtype=torch.bfloat16, device=o_parts.device)
    if lse is None:
        lse = _empty(stream, rows, H, dtype=torch.float32, device=o_parts.device)
    st = load().mla_lse_merge(
        o_parts.data_ptr(), o_parts.stride(0), lse_parts.data_ptr(), lse_parts.stride(0), G,
        rows, H, R, out.data_ptr(), lse.data_ptr(), _stream_ptr(stream))
    _lib.check(st, "mla_lse_merge")
    return out, lse


# ------------------------------------------------------- prompts and batches
_bind_module = None


def _bind():
    """The compiled binding (csrc/bind.cpp): it checks the tensors (dtype,
    shape, unit last stride, on the current device; ValueError), allocates
    outputs that are not given and calls the library (MlaError).

    A call runs on ``stream``, by default the current one, and what it
    allocates (outputs, workspace) is that stream's memory.  With another
    stream than the current one the caller makes it wait for the inputs, keeps
    those until it is done with them, and makes the current one wait for it
    before the outputs are used there."""
    global _bind_module
    if _bind_module is None:
        _torch()
        load()
        from . import _calls
        _bind_module = _calls
    return _bind_module


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
    return BatchTables(*_bind().batch_build(
        query_lens, context_lens, req_block_table, free_blocks, free_count, block_size,
        num_blocks, -1 if num_tokens is None else num_tokens, req_ids, block_table, seq_lens,
        cu_seqlens_q, cu_seqlens_k, positions, slot_mapping, free_count_out, err_count, stream))


def blocks_release(held_lens, req_block_table, free_blocks, free_count, block_size: int,
                   num_blocks: int, *, req_ids=None, free_count_out=None, err_count=None,
                   stream=None):
    """Put the pages of finished requests (int32 [B] ``held_lens`` tokens each,
    rows ``req_ids`` of ``req_block_table``) back onto the stack
    ``free_blocks``; returns the new height (``free_count_out``, by default
    ``free_count`` updated in place)."""
    return _bind().blocks_release(held_lens, req_block_table, free_blocks, free_count, block_size,
                                  num_blocks, req_ids, free_count_out, err_count, stream)


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
    return _bind().gather_cache(
        kv_cache, -1 if kv_cache_dtype is None else _kv_dtype(kv_cache, kv_cache_dtype),
        block_table, cu_seqlens, -1 if num_tokens is None else num_tokens,
        -1 if kv_lora_rank is None else kv_lora_rank, seq_starts, kv_scale, kv_c, k_pe,
        err_count, stream)


def expand_kv(kv_c, w_kv_b, num_heads: int, *, k_nope=None, v=None, err_count=None,
              stream=None):
    """Keys and values of latents ``kv_c`` [T, R]: (k_nope, v), bf16
    [T, H, 128] each; ``w_kv_b`` [H * 256, R] is the kv_b projection's weight
    (per head 128 rows of W_UK, then 128 of W_UV).  Allocated unless both are
    given (they may be the halves of one [T, H, 256] buffer)."""
    return _bind().expand_kv(kv_c, w_kv_b, num_heads, k_nope, v, err_count, stream)


def absorb_q(q_nope, w_kv_b, *, out=None, err_count=None, stream=None):
    """The latent query ql_nope [T, H, R] of ``q_nope`` [T, H, 128] (any row
    and head strides: a column slice of q will do): ``decode``'s query is then
    the pair (ql_nope, q_pe).  ``w_kv_b`` as in :func:`expand_kv`."""
    return _bind().absorb_q(q_nope, w_kv_b, out, err_count, stream)


def project_v(o, w_kv_b, *, out=None, err_count=None, stream=None):
    """Values [T, H, 128] of ``decode``'s latent output ``o`` [T, H, R];
    ``w_kv_b`` as in :func:`expand_kv`."""
    return _bind().project_v(o, w_kv_b, out, err_count, stream)


_ACTIVATIONS = {None: MLA_ACT_NONE, "relu": MLA_ACT_RELU, "silu": MLA_ACT_SILU,
                "gelu": MLA_ACT_GELU, "gelu_tanh": MLA_ACT_GELU_TANH}


def linear(x, weight, *, bias=None, activation: str | None = None, residual=None, out=None,
           err_count=None, stream=None):
    """``act(x @ weight.T + bias) + residual`` as bf16 [T, N], rounded once.

    ``x`` bf16 [T, K], ``weight`` bf16 [N, K] as a linear layer stores it,
    ``bias`` bf16 [N], ``residual`` bf16 [T, N] (any row strides that are
    multiples of 8); ``activation``: None, "relu", "silu", "gelu" (x Phi(x)) or
    "gelu_tanh".  ``out`` may be ``residual`` (updated in place).  What is allocated
    here has rows of N rounded up to a multiple of 8.
    """
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unsupported activation {activation!r}")
    return _bind().linear(x, weight, bias, _ACTIVATIONS[activation], residual, out, err_count,
                          stream)


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
    ``mla_prefill_num_kv_splits`` (few rows against long contexts take up to
    six times as long in the one part of the default); the workspace they need
    is allocated here when not given.
    """
    q, q_pe = q if isinstance(q, (tuple, list)) else (q, None)
    return _bind().prefill(q, q_pe, k_nope, v, k_pe, cu_seqlens_q, cu_seqlens_k, sm_scale, causal,
                           num_kv_splits, workspace, out, lse, err_count, stream)


def prefill_shared(q, k_nope, v, k_pe, cu_seqlens_q, cu_seqlens_k, group_seqs, cu_prefix,
                   sm_scale: float, *, causal: bool = True, num_kv_splits=1, workspace=None,
                   out=None, lse=None, err_count=None, stream=None):
    """:func:`prefill` for sequences that share prefixes; returns (o, lse).

    Group g is the sequences ``group_seqs[g]`` to ``group_seqs[g + 1]`` (int32
    [groups + 1]); their rows all attend to the key rows ``cu_prefix[g]`` to
    ``cu_prefix[g + 1]`` (int32 [groups + 1]) of ``k_nope``, ``v`` and ``k_pe``,
    besides their own keys there (``cu_seqlens_k``, masked as by ``causal``).
    ``num_kv_splits``: parts of the prefixes' keys and of the sequences' own (0:
    those together with the prefix's), a pair from
    ``mla_prefill_shared_num_kv_splits``, or the first of them alone (the default
    takes up to ten times as long where many short sequences have long keys of
    their own).
    """
    q, q_pe = q if isinstance(q, (tuple, list)) else (q, None)
    pre, own = num_kv_splits if isinstance(num_kv_splits, (tuple, list)) else (num_kv_splits, 0)
    return _bind().prefill_shared(q, q_pe, k_nope, v, k_pe, cu_seqlens_q, cu_seqlens_k, group_seqs,
                                  cu_prefix, sm_scale, causal, pre, own, workspace, out, lse,
                                  err_count, stream)
