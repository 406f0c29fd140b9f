// C entry points (declared in include/mla.h) around the decode: batch tables,
// the gather of cached rows, the products with the kv_b weight and the prompt
// attention.  Host-side validation and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include "../../include/mla.h"
#include "abi.cuh"
#include "kernels.cuh"
#include "tensors.cuh"

namespace {

using mla::aligned16;
using mla::aligned4;
using mla::aligned8;
using mla::cuda_fail;
using mla::Heads;
using mla::heads_disjoint;
using mla::heads_map;
using mla::heads_ok;
using mla::intersect;
using mla::make_map;
using mla::Runs;
using mla::runs;

// Whether [a, a + na) and [b, b + nb) (bytes) share a byte.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
         y < x + static_cast<uintptr_t>(na);
}

// The arguments that building and releasing share.
mla_status fill_batch(const int32_t* req_ids, const int32_t* context_lens, int num_reqs,
                      const int32_t* req_block_table, int64_t req_block_table_stride,
                      int num_table_rows, int max_blocks_per_req, int block_size,
                      int num_blocks, const int32_t* free_blocks, int free_capacity,
                      const int32_t* free_count, int32_t* free_count_out, int* err_count,
                      mla::BatchParams* p) {
  if (num_reqs < 0 || num_table_rows < 1 || max_blocks_per_req < 1 || block_size < 1 ||
      block_size > 1024 || num_blocks < 1 || free_capacity < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_reqs > mla::kMaxBatchReqs ||
      static_cast<int64_t>(max_blocks_per_req) * block_size > (int64_t{1} << 30))
    return MLA_ERR_UNSUPPORTED;
  if (req_block_table_stride < max_blocks_per_req) return MLA_ERR_INVALID_ARG;
  if ((num_reqs > 0 && (!context_lens || !req_block_table)) ||
      (free_capacity > 0 && !free_blocks) || !free_count || !free_count_out)
    return MLA_ERR_INVALID_ARG;
  if (!aligned4(req_ids) || !aligned4(context_lens) || !aligned4(req_block_table) ||
      !aligned4(free_blocks) || !aligned4(free_count) || !aligned4(free_count_out) ||
      !aligned4(err_count))
    return MLA_ERR_INVALID_ARG;
  memset(p, 0, sizeof *p);
  p->req_ids = req_ids;
  p->context_lens = context_lens;
  p->num_reqs = num_reqs;
  p->req_table = const_cast<int32_t*>(req_block_table);
  p->rt_stride = req_block_table_stride;
  p->num_table_rows = num_table_rows;
  p->capacity = max_blocks_per_req * block_size;
  p->block_size = block_size;
  p->num_blocks = num_blocks;
  p->free_blocks = free_blocks;
  p->free_capacity = free_capacity;
  p->free_count = free_count;
  p->free_count_out = free_count_out;
  p->err_count = err_count;
  return MLA_OK;
}

constexpr int kNopeDim = 128, kVDim = 128;

mla_status latent_proj(int mode, Heads in, int in_heads, int tokens, const void* w,
                       int64_t w_stride, int heads, int R, int nope, int vdim, Heads out0,
                       Heads out1, int* err_count, void* stream) {
  if (tokens < 0 || heads < 1 || heads > 1024 || nope < 1 || vdim < 1) return MLA_ERR_INVALID_ARG;
  if ((R != 512 && R != 256) || nope != kNopeDim || vdim != kVDim) return MLA_ERR_UNSUPPORTED;
  if (tokens == 0) return MLA_OK;
  const bool two = mode == mla::kProjExpand;
  if (!heads_ok(in, tokens, in_heads) || !heads_ok(out0, tokens, heads) ||
      (two && !heads_ok(out1, tokens, heads)) || !w || !aligned16(w) || w_stride % 8 != 0 ||
      w_stride < R || w_stride > (int64_t{1} << 20) || !aligned4(err_count))
    return MLA_ERR_INVALID_ARG;
  if (!heads_disjoint(out0, tokens, heads) || (two && !heads_disjoint(out1, tokens, heads)))
    return MLA_ERR_INVALID_ARG;
  // the rows the product leaves out count as well
  const Runs r_w = runs(w, 2 * ((static_cast<int64_t>(heads) * (nope + vdim) - 1) * w_stride + R));
  // outputs may lie between an input's rows or each other's (columns of one
  // buffer)
  const Runs r_in = runs(in, tokens, in_heads), r0 = runs(out0, tokens, heads);
  const Runs r1 = two ? runs(out1, tokens, heads) : r0;
  if (intersect(r0, r_w) || intersect(r0, r_in) ||
      (two && (intersect(r1, r_w) || intersect(r1, r_in) || intersect(r0, r1))))
    return MLA_ERR_INVALID_ARG;
  int sms = 0;
  cudaError_t e = mla::device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  mla::ProjParams p = {};
  p.tokens = tokens;
  p.heads = heads;
  p.k = in.cols;
  p.cols = two ? nope + vdim : out0.cols;
  p.w_row0 = mode == mla::kProjProject ? nope : 0;
  p.bn = mla::proj_tile_cols(mode, tokens, heads, p.cols, sms);
  p.pair = mla::proj_pairs(mode, tokens, heads, p.k, sms);
  p.a_rows = tokens < 128 ? tokens : 128;
  p.err_count = err_count;
  mla::ProjMaps m;
  mla_status st = heads_map(&m.a, in, tokens, in_heads, p.a_rows);
  if (st == MLA_OK)
    st = make_map(&m.b, w, R, nope + vdim, heads, w_stride, w_stride * (nope + vdim),
                  p.pair ? 128 : mode == mla::kProjAbsorb ? 64 : p.bn, 1);
  if (st == MLA_OK) st = heads_map(&m.c0, out0, tokens, heads, 32);
  if (st == MLA_OK) st = heads_map(&m.c1, two ? out1 : out0, tokens, heads, 32);
  if (st != MLA_OK) return st;
  e = mla::launch_latent_proj(p, m, mode, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

// Groups of sequences that share a prefix, for the prompt attention.
struct Groups {
  const int32_t *seqs = nullptr, *cu_prefix = nullptr;
  int num = 0, splits = 0;
};

mla_status prefill(const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* q_pe,
                   int64_t q_pe_row_stride, int64_t q_pe_head_stride, int num_tokens,
                   int num_heads, const void* k_nope, int64_t k_row_stride, int64_t k_head_stride,
                   const void* v, int64_t v_row_stride, int64_t v_head_stride, const void* k_pe,
                   int64_t k_pe_row_stride, int num_kv_tokens, int nope_dim, int rope_dim,
                   int v_dim, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                   int num_seqs, const Groups& groups, int causal, float sm_scale,
                   int num_kv_splits, void* workspace, size_t workspace_bytes, void* o,
                   int64_t o_row_stride, int64_t o_head_stride, float* lse, int* err_count,
                   void* stream) {
  const int parts = num_kv_splits + groups.splits;
  if (num_tokens < 0 || num_kv_tokens < 0 || num_seqs < 0 || num_heads < 1 || num_heads > 1024 ||
      num_kv_splits < (groups.num > 0 ? 0 : 1) || num_kv_splits > 64 || groups.num < 0 ||
      (groups.num > 0 && (groups.splits < 1 || groups.splits > 64)) || nope_dim < 1 || rope_dim < 1 || v_dim < 1 ||
      !(sm_scale >= 1e-30f && sm_scale <= 1e30f))
    return MLA_ERR_INVALID_ARG;
  if (nope_dim != kNopeDim || v_dim != kVDim || rope_dim != 64 || num_seqs > 65535 ||
      groups.num > 65535 ||
      num_tokens > (1 << 30) || num_kv_tokens > (1 << 30))
    return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  const Heads hq{q, q_row_stride, q_head_stride, q_pe ? nope_dim : nope_dim + rope_dim};
  const Heads hqp = q_pe ? Heads{q_pe, q_pe_row_stride, q_pe_head_stride, rope_dim}
                         : Heads{q ? static_cast<const uint16_t*>(q) + nope_dim : nullptr,
                                 q_row_stride, q_head_stride, rope_dim};
  const Heads hk{k_nope, k_row_stride, k_head_stride, nope_dim};
  const Heads hv{v, v_row_stride, v_head_stride, v_dim};
  const Heads hkp{k_pe, k_pe_row_stride, 0, rope_dim};
  const Heads ho{o, o_row_stride, o_head_stride, v_dim};
  if (!heads_ok(hq, num_tokens, num_heads) || !heads_ok(hqp, num_tokens, num_heads) ||
      !heads_ok(ho, num_tokens, num_heads) || !heads_disjoint(ho, num_tokens, num_heads))
    return MLA_ERR_INVALID_ARG;
  if (num_kv_tokens > 0 &&
      (!heads_ok(hk, num_kv_tokens, num_heads) || !heads_ok(hv, num_kv_tokens, num_heads) ||
       !heads_ok(hkp, num_kv_tokens, 1)))
    return MLA_ERR_INVALID_ARG;
  if (!cu_seqlens_q || !cu_seqlens_k || !lse || !aligned4(cu_seqlens_q) ||
      !aligned4(cu_seqlens_k) || !aligned4(lse) || !aligned4(err_count) ||
      (groups.num > 0 && (!groups.seqs || !groups.cu_prefix || !aligned4(groups.seqs) ||
                          !aligned4(groups.cu_prefix))))
    return MLA_ERR_INVALID_ARG;
  const size_t need = mla_prefill_workspace_bytes(num_tokens, num_heads, parts, v_dim);
  if (need > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 31u) != 0)
      return MLA_ERR_INVALID_ARG;
    if (workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  // one CTA per 256-row block slot, head and split
  if ((num_tokens / 256 + static_cast<int64_t>(num_seqs)) * 2 * num_heads * num_kv_splits +
          (num_tokens / 256 + static_cast<int64_t>(groups.num) + 2) * 2 * num_heads * groups.splits >
      INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  const int64_t n_cu = (static_cast<int64_t>(num_seqs) + 1) * 4;
  const int64_t n_groups = groups.num > 0 ? (static_cast<int64_t>(groups.num) + 1) * 4 : 0;
  Runs in[9] = {runs(hq, num_tokens, num_heads),  runs(hqp, num_tokens, num_heads),
                runs(cu_seqlens_q, n_cu),         runs(cu_seqlens_k, n_cu),
                runs(groups.seqs, n_groups),      runs(groups.cu_prefix, n_groups)};
  int n_in = 6;
  if (num_kv_tokens > 0) {
    in[n_in++] = runs(hk, num_kv_tokens, num_heads);
    in[n_in++] = runs(hv, num_kv_tokens, num_heads);
    in[n_in++] = runs(hkp, num_kv_tokens, 1);
  }
  // what is not written (a workspace that is not needed) overlaps nothing
  const Runs out[3] = {runs(ho, num_tokens, num_heads),
                       runs(lse, static_cast<int64_t>(num_tokens) * num_heads * 4),
                       runs(workspace, need > INT64_MAX ? INT64_MAX : static_cast<int64_t>(need))};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (intersect(out[i], in[j])) return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (intersect(out[i], out[j])) return MLA_ERR_INVALID_ARG;
  }
  mla::PrefillParams p = {};
  p.num_tokens = num_tokens;
  p.num_kv = num_kv_tokens;
  p.heads = num_heads;
  p.num_seqs = num_seqs;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.pe_col = q_pe ? 0 : nope_dim;
  p.causal = causal != 0;
  p.sm_scale = sm_scale;
  p.num_splits = parts;
  p.num_groups = groups.num;
  p.prefix_splits = groups.splits;
  p.group_seqs = groups.seqs;
  p.cu_prefix = groups.cu_prefix;
  p.v = static_cast<const uint16_t*>(v);
  p.v_row_stride = v_row_stride;
  p.v_head_stride = num_heads > 1 ? v_head_stride : 0;
  p.o = static_cast<uint16_t*>(o);
  p.o_row_stride = o_row_stride;
  p.o_head_stride = num_heads > 1 ? o_head_stride : 0;
  p.o_aligned32 = (reinterpret_cast<uintptr_t>(o) & 31u) == 0 && o_row_stride % 16 == 0 &&
                  p.o_head_stride % 16 == 0;
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = need ? p.ws_o + static_cast<size_t>(num_tokens) * num_heads * parts * v_dim
                  : nullptr;
  p.err_count = err_count;
  mla::PrefillMaps m;
  memset(&m, 0, sizeof m);
  mla_status st = heads_map(&m.q, hq, num_tokens, num_heads, 128);
  if (st == MLA_OK && q_pe) st = heads_map(&m.q_pe, hqp, num_tokens, num_heads, 128);
  if (num_kv_tokens > 0) {
    if (st == MLA_OK) st = heads_map(&m.k, hk, num_kv_tokens, num_heads, 128);
    if (st == MLA_OK) st = heads_map(&m.k_pe, hkp, num_kv_tokens, 1, 128);
    if (st == MLA_OK) st = heads_map(&m.v, hv, num_kv_tokens, num_heads, 64);
  }
  if (st != MLA_OK) return st;
  cudaError_t e = mla::launch_prefill(p, m, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

mla_status mla_batch_build(const int32_t* req_ids, const int32_t* query_lens,
                           const int32_t* context_lens, int num_reqs,
                           int32_t* req_block_table, int64_t req_block_table_stride,
                           int num_table_rows, int max_blocks_per_req, int block_size,
                           int num_blocks, const int32_t* free_blocks, int free_capacity,
                           const int32_t* free_count, int32_t* free_count_out,
                           int num_tokens, int32_t* block_table, int64_t block_table_stride,
                           int32_t* seq_lens, int32_t* cu_seqlens_q, int32_t* cu_seqlens_k,
                           int64_t* positions, int64_t* slot_mapping, int* err_count,
                           void* stream) {
  mla::BatchParams p;
  mla_status st =
      fill_batch(req_ids, context_lens, num_reqs, req_block_table, req_block_table_stride,
                 num_table_rows, max_blocks_per_req, block_size, num_blocks, free_blocks,
                 free_capacity, free_count, free_count_out, err_count, &p);
  if (st != MLA_OK) return st;
  if (num_tokens < 0 || (num_reqs > 0 && block_table_stride < max_blocks_per_req))
    return MLA_ERR_INVALID_ARG;
  if ((num_reqs > 0 && (!query_lens || !block_table || !seq_lens)) || !cu_seqlens_q ||
      !cu_seqlens_k || (num_tokens > 0 && (!positions || !slot_mapping)))
    return MLA_ERR_INVALID_ARG;
  if (!aligned4(query_lens) || !aligned4(block_table) || !aligned4(seq_lens) ||
      !aligned4(cu_seqlens_q) || !aligned4(cu_seqlens_k) || !aligned8(positions) ||
      !aligned8(slot_mapping))
    return MLA_ERR_INVALID_ARG;
  // every CTA reads the lengths, the stack and the rows' old pages again
  // while others already write: no output may lie over them
  const int64_t n4 = static_cast<int64_t>(num_reqs) * 4;
  const struct { const void* p; int64_t n; } in[] = {
      {req_ids, req_ids ? n4 : 0},
      {query_lens, n4},
      {context_lens, n4},
      {free_blocks, static_cast<int64_t>(free_capacity) * 4},
      {free_count, free_count == free_count_out ? 0 : 4}};
  const int64_t rt_bytes =
      ((num_table_rows - 1) * req_block_table_stride + max_blocks_per_req) * 4;
  const struct { const void* p; int64_t n; } out[] = {
      {req_block_table, num_reqs ? rt_bytes : 0},
      {block_table,
       num_reqs ? ((num_reqs - 1) * block_table_stride + max_blocks_per_req) * 4 : 0},
      {seq_lens, n4},
      {cu_seqlens_q, n4 + 4},
      {cu_seqlens_k, n4 + 4},
      {positions, static_cast<int64_t>(num_tokens) * 8},
      {slot_mapping, static_cast<int64_t>(num_tokens) * 8},
      {free_count_out, 4}};
  constexpr int kIn = sizeof in / sizeof in[0], kOut = sizeof out / sizeof out[0];
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < kIn; ++j)
      if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return MLA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return MLA_ERR_INVALID_ARG;
  }
  p.query_lens = query_lens;
  p.num_tokens = num_tokens;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.seq_lens = seq_lens;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.positions = positions;
  p.slot_mapping = slot_mapping;
  int sms = 0;
  cudaError_t e = mla::device_sm_count(&sms);
  if (e == cudaSuccess) e = mla::launch_batch_build(p, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

mla_status mla_blocks_release(const int32_t* req_ids, const int32_t* held_lens, int num_reqs,
                              const int32_t* req_block_table, int64_t req_block_table_stride,
                              int num_table_rows, int max_blocks_per_req, int block_size,
                              int num_blocks, int32_t* free_blocks, int free_capacity,
                              const int32_t* free_count, int32_t* free_count_out,
                              int* err_count, void* stream) {
  mla::BatchParams p;
  mla_status st =
      fill_batch(req_ids, held_lens, num_reqs, req_block_table, req_block_table_stride,
                 num_table_rows, max_blocks_per_req, block_size, num_blocks, free_blocks,
                 free_capacity, free_count, free_count_out, err_count, &p);
  if (st != MLA_OK) return st;
  if (static_cast<int64_t>(num_reqs) * max_blocks_per_req > INT32_MAX)
    return MLA_ERR_UNSUPPORTED;
  const int64_t n4 = static_cast<int64_t>(num_reqs) * 4;
  // the stack is written while other CTAs still read the rows, and the new
  // height before the last of them ends
  const int64_t stack = static_cast<int64_t>(free_capacity) * 4;
  const struct { const void* p; int64_t n; } in[] = {
      {free_count, free_count == free_count_out ? 0 : 4},
      {held_lens, n4},
      {req_ids, req_ids ? n4 : 0},
      {req_block_table,
       num_reqs ? ((num_table_rows - 1) * req_block_table_stride + max_blocks_per_req) * 4 : 0}};
  if (overlap(free_blocks, stack, free_count_out, 4)) return MLA_ERR_INVALID_ARG;
  for (const auto& x : in)
    if (overlap(free_blocks, stack, x.p, x.n) || overlap(free_count_out, 4, x.p, x.n))
      return MLA_ERR_INVALID_ARG;
  p.free_out = free_blocks;
  cudaError_t e = mla::launch_blocks_release(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

mla_status mla_gather_cache(const void* kv_cache, mla_kv_dtype kv_dtype, int num_blocks,
                            int block_size, int64_t block_stride, int kv_lora_rank,
                            int rope_dim, const int32_t* block_table,
                            int64_t block_table_stride, int max_blocks_per_seq,
                            const int32_t* cu_seqlens, const int32_t* seq_starts,
                            int num_seqs, int num_tokens, const float* kv_scale, void* kv_c,
                            int64_t kv_c_row_stride, void* k_pe, int64_t k_pe_row_stride,
                            int* err_count, void* stream) {
  if (num_tokens < 0 || num_seqs < 0 || num_blocks < 1 || block_size < 1 || block_size > 1024 ||
      max_blocks_per_seq < 1)
    return MLA_ERR_INVALID_ARG;
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3 && kv_dtype != MLA_KV_FP8_E5M2)
    return MLA_ERR_INVALID_ARG;
  if ((kv_lora_rank != 512 && kv_lora_rank != 256) || rope_dim != 64) return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0) return MLA_OK;
  const bool fp8 = kv_dtype != MLA_KV_BF16;
  if (!kv_cache || !block_table || !cu_seqlens || !kv_c || !k_pe || (fp8 && !kv_scale))
    return MLA_ERR_INVALID_ARG;
  const int64_t elt = fp8 ? 1 : 2;
  if (block_stride < static_cast<int64_t>(block_size) * (kv_lora_rank + rope_dim) ||
      (block_stride * elt) % 16 != 0 || !aligned16(kv_cache) ||
      block_table_stride < max_blocks_per_seq)
    return MLA_ERR_INVALID_ARG;
  if (kv_c_row_stride < kv_lora_rank || k_pe_row_stride < rope_dim || kv_c_row_stride % 8 != 0 ||
      k_pe_row_stride % 8 != 0 || !aligned16(kv_c) || !aligned16(k_pe) ||
      !aligned4(block_table) || !aligned4(cu_seqlens) || !aligned4(seq_starts) ||
      !aligned4(kv_scale) || !aligned4(err_count))
    return MLA_ERR_INVALID_ARG;
  const Runs out[2] = {runs(kv_c, num_tokens, kv_c_row_stride * 2, 1, 0, int64_t{kv_lora_rank} * 2),
                       runs(k_pe, num_tokens, k_pe_row_stride * 2, 1, 0, int64_t{rope_dim} * 2)};
  const Runs in[5] = {
      runs(kv_cache, num_blocks, block_stride * elt, 1, 0,
           static_cast<int64_t>(block_size) * (kv_lora_rank + rope_dim) * elt),
      runs(block_table, num_seqs, block_table_stride * 4, 1, 0, int64_t{max_blocks_per_seq} * 4),
      runs(cu_seqlens, (static_cast<int64_t>(num_seqs) + 1) * 4),
      runs(seq_starts, static_cast<int64_t>(num_seqs) * 4), runs(fp8 ? kv_scale : nullptr, 4)};
  if (intersect(out[0], out[1])) return MLA_ERR_INVALID_ARG;
  for (const Runs& o : out)
    for (const Runs& x : in)
      if (intersect(o, x)) return MLA_ERR_INVALID_ARG;
  mla::GatherParams p = {};
  p.cache = kv_cache;
  p.block_stride = block_stride;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.capacity = static_cast<int64_t>(max_blocks_per_seq) * block_size;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.cu = cu_seqlens;
  p.starts = seq_starts;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.scale = kv_scale;
  p.e5m2 = kv_dtype == MLA_KV_FP8_E5M2;
  p.kv_c = static_cast<uint16_t*>(kv_c);
  p.kv_c_stride = kv_c_row_stride;
  p.k_pe = static_cast<uint16_t*>(k_pe);
  p.k_pe_stride = k_pe_row_stride;
  p.err_count = err_count;
  cudaError_t e = mla::launch_gather_cache(p, kv_lora_rank, fp8, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

mla_status mla_expand_kv(const void* kv_c, int64_t kv_c_row_stride, int num_tokens,
                         const void* w_kv_b, int64_t w_row_stride, int num_heads,
                         int kv_lora_rank, int nope_dim, int v_dim, void* k_nope,
                         int64_t k_row_stride, int64_t k_head_stride, void* v,
                         int64_t v_row_stride, int64_t v_head_stride, int* err_count,
                         void* stream) {
  return latent_proj(mla::kProjExpand, {kv_c, kv_c_row_stride, 0, kv_lora_rank}, 1, num_tokens,
                     w_kv_b, w_row_stride, num_heads, kv_lora_rank, nope_dim, v_dim,
                     {k_nope, k_row_stride, k_head_stride, nope_dim},
                     {v, v_row_stride, v_head_stride, v_dim}, err_count, stream);
}

mla_status mla_absorb_q(const void* q_nope, int64_t q_row_stride, int64_t q_head_stride,
                        int num_tokens, const void* w_kv_b, int64_t w_row_stride,
                        int num_heads, int kv_lora_rank, int nope_dim, int v_dim,
                        void* ql_nope, int64_t ql_row_stride, int64_t ql_head_stride,
                        int* err_count, void* stream) {
  return latent_proj(mla::kProjAbsorb, {q_nope, q_row_stride, q_head_stride, nope_dim}, num_heads,
                     num_tokens, w_kv_b, w_row_stride, num_heads, kv_lora_rank, nope_dim, v_dim,
                     {ql_nope, ql_row_stride, ql_head_stride, kv_lora_rank}, {}, err_count,
                     stream);
}

mla_status mla_project_v(const void* o, int64_t o_row_stride, int64_t o_head_stride,
                         int num_tokens, const void* w_kv_b, int64_t w_row_stride,
                         int num_heads, int kv_lora_rank, int nope_dim, int v_dim, void* y,
                         int64_t y_row_stride, int64_t y_head_stride, int* err_count,
                         void* stream) {
  return latent_proj(mla::kProjProject, {o, o_row_stride, o_head_stride, kv_lora_rank}, num_heads,
                     num_tokens, w_kv_b, w_row_stride, num_heads, kv_lora_rank, nope_dim, v_dim,
                     {y, y_row_stride, y_head_stride, v_dim}, {}, err_count, stream);
}

mla_status mla_linear(const void* x, int64_t x_row_stride, int num_tokens, int in_features,
                      const void* w, int64_t w_row_stride, int out_features, const void* bias,
                      int activation, const void* residual,
                      int64_t residual_row_stride, void* y, int64_t y_row_stride,
                      int* err_count, void* stream) {
  if (num_tokens < 0 || in_features < 1 || out_features < 1 || activation < MLA_ACT_NONE ||
      activation > MLA_ACT_GELU_TANH)
    return MLA_ERR_INVALID_ARG;
  constexpr int kMost = 1 << 20;
  if (num_tokens > (1 << 30) || in_features > kMost || out_features > kMost)
    return MLA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MLA_OK;
  const Heads hx{x, x_row_stride, 0, in_features}, hw{w, w_row_stride, 0, in_features};
  const Heads hr{residual, residual_row_stride, 0, out_features};
  const Heads hy{y, y_row_stride, 0, out_features};
  if (!heads_ok(hx, num_tokens, 1) || !heads_ok(hw, out_features, 1) ||
      !heads_ok(hy, num_tokens, 1) || (residual && !heads_ok(hr, num_tokens, 1)) ||
      !aligned16(bias) || !aligned4(err_count))
    return MLA_ERR_INVALID_ARG;
  const Runs ry = runs(hy, num_tokens, 1);
  if (intersect(ry, runs(hx, num_tokens, 1)) || intersect(ry, runs(hw, out_features, 1)) ||
      intersect(ry, runs(bias, 2 * int64_t{out_features})))
    return MLA_ERR_INVALID_ARG;
  // the warp that stores y's element has the residual's before it does, and no other
  // warp reads that one
  const bool in_place = residual == y && (residual_row_stride == y_row_stride || num_tokens == 1);
  if (residual && !in_place && intersect(ry, runs(hr, num_tokens, 1))) return MLA_ERR_INVALID_ARG;
  int sms = 0;
  cudaError_t e = mla::device_sm_count(&sms);
  if (e != cudaSuccess) return cuda_fail(e);
  const mla::LinearPlan plan = mla::linear_plan(num_tokens, out_features, in_features, sms);
  mla::LinearParams p = {};
  p.tokens = num_tokens;
  p.n = out_features;
  p.k = in_features;
  p.act = activation;
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual);
  p.res_stride = residual_row_stride;
  p.y = static_cast<uint16_t*>(y);
  p.y_stride = y_row_stride;
  p.form = plan.form;
  p.bn = plan.bn;
  p.splits = plan.splits;
  p.err_count = err_count;
  mla::LinearMaps m;
  mla_status st = make_map(&m.a, x, in_features, 1, num_tokens, x_row_stride, x_row_stride, 1,
                           plan.a_rows);
  if (st == MLA_OK)
    st = make_map(&m.b, w, in_features, 1, out_features, w_row_stride, w_row_stride, 1,
                  plan.b_rows);
  if (st == MLA_OK)
    st = make_map(&m.c, y, out_features < 8 ? 8 : out_features & ~7, 1, num_tokens, y_row_stride,
                  y_row_stride, 1, 32);
  if (st != MLA_OK) return st;
  e = mla::launch_linear(p, m, sms, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_OK : cuda_fail(e);
}

// Measured on GB300, 16 heads (us at S = 1 / the rule's S / twice that): one
// sequence of 256 rows, 32768 keys: 437 / 75 (9) / 92; two of 500 rows, 4596 keys:
// 72 / 53 (2) / 63; contexts of 4096 to 32768 keys, eight of 1 to 5 rows: 382 / 218 (8)
// / 228; of 1000 to 30000 keys, 16 of 1 to 8 rows: 465 / 325 (4) / 323; of 500 to 16000
// keys, one row each, 32: 388 / 351 (2) / 344, 40: 469 / 437 (2) / 434, 56: 659 / 629 (2)
// / 630; of 4096 keys each, one row, 48: 309 / 299 (2) / 292, 56: 315 / 337 (2) / 338 (the
// rule's worst, it does not see that the lengths are equal), 64: 364 (1) / 383; 1000
// rows, 1000 keys: 23 (1) / 26.  With 4 for 6 below the first three ragged ones took
// 225 (5), 336 (3) and 351 (2).
int mla_prefill_num_kv_splits(int num_tokens, int num_seqs, int num_heads, int64_t max_kv_len,
                              int sm_count) {
  if (num_tokens < 1 || num_seqs < 1 || num_heads < 1 || max_kv_len < 1 || sm_count < 1) return 1;
  // 256-row blocks there are at least, one CTA each per head
  const int64_t by_rows = (static_cast<int64_t>(num_tokens) + 255) / 256;
  const int64_t blocks = num_seqs > by_rows && num_seqs <= num_tokens ? num_seqs : by_rows;
  const int64_t units = blocks * num_heads;
  int64_t s = sm_count / units, most = max_kv_len / 1024;
  if (s < 2) {
    // Nearly every SM has a unit.  With few rows a sequence its length is what
    // a unit takes; parts of it even out lengths that differ.
    s = 1;
    const int64_t parts = 6 * static_cast<int64_t>(sm_count);
    if (num_tokens <= 64 * static_cast<int64_t>(num_seqs) && units < parts) {
      s = (parts + units - 1) / units;
      most = max_kv_len / 2048;
    }
  }
  if (s > most) s = most;
  if (s > 64) s = 64;
  return s < 1 ? 1 : static_cast<int>(s);
}

size_t mla_prefill_workspace_bytes(int num_tokens, int num_heads, int num_kv_splits, int v_dim) {
  if (num_tokens <= 0 || num_heads <= 0 || num_kv_splits <= 1 || v_dim <= 0) return 0;
  size_t n = static_cast<size_t>(num_tokens);
  const size_t f[4] = {static_cast<size_t>(num_heads), static_cast<size_t>(num_kv_splits),
                       static_cast<size_t>(v_dim) + 1, sizeof(float)};
  for (size_t x : f)
    if (__builtin_mul_overflow(n, x, &n)) return SIZE_MAX;
  return n;
}

mla_status mla_prefill(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                       const void* q_pe, int64_t q_pe_row_stride, int64_t q_pe_head_stride,
                       int num_tokens, int num_heads, const void* k_nope, int64_t k_row_stride,
                       int64_t k_head_stride, const void* v, int64_t v_row_stride,
                       int64_t v_head_stride, const void* k_pe, int64_t k_pe_row_stride,
                       int num_kv_tokens, int nope_dim, int rope_dim, int v_dim,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int num_seqs,
                       int causal, float sm_scale, int num_kv_splits, void* workspace,
                       size_t workspace_bytes, void* o, int64_t o_row_stride,
                       int64_t o_head_stride, float* lse, int* err_count, void* stream) {
  return prefill(q, q_row_stride, q_head_stride, q_pe, q_pe_row_stride, q_pe_head_stride, num_tokens,
                 num_heads, k_nope, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride,
                 k_pe, k_pe_row_stride, num_kv_tokens, nope_dim, rope_dim, v_dim, cu_seqlens_q,
                 cu_seqlens_k, num_seqs, Groups{}, causal, sm_scale, num_kv_splits, workspace,
                 workspace_bytes, o, o_row_stride, o_head_stride, lse, err_count, stream);
}

// The least estimated time, in microseconds as measured on GB300: a unit takes 4 for its
// start and end and 1.5 for 128 keys (2 where it has a second tile of query rows), half
// as much again where the own keys of several sequences are masked; the units share the
// SMs, the last ones overhang by half of the longest; a join takes 3.5 and 2.3e-4 for
// a row and head of each part.  Own keys together with the prefix's (first loop) or
// apart (second).  Measured (us: one part together / this rule's / the best of eleven
// tried, before rows without keys in a tile took less in windows of several sequences; today's
// first two behind it), 16 heads: three sequences of 20 rows, 1000 keys before them, 20 of
// their own 21.0 / 15.2 (3 and 1) / 14.5 (20.5 / 14.8), 300 of their own 36.2 / 15.4 (3, 1) /
// 15.4 (36.0 / 15.0); one of 200 rows, 4000 and 200 keys 69.3 / 25.5 (8, 1) / 25.5 (68.0 /
// 24.5); eight of 60 rows, 4000 and 60 keys 73.0 / 38.5 (4, 0) / 37.0 (70.0 / 36.5), 700 and 60
// keys 28.6 / 28.6 / 23.8 (the worst found; 25.3 / 25.3); 64 single rows, 8192 and 1000 keys
// 1178 / 128 (8, 1) / 126 (1215 / 128); 48 of 48 rows, 8192 and 48 keys 144 / 144 / 144, apart
// 180 (132 / 132, 183); 32 heads, eight of 1000 rows, 4096 and 1000 keys 533 / 533 / 533, apart
// 633 (543 / 543, 618).
int mla_prefill_shared_num_kv_splits(int num_tokens, int num_seqs, int num_groups, int num_heads,
                                     int64_t max_prefix_len, int64_t max_kv_len, int sm_count,
                                     int* num_kv_splits) {
  if (num_kv_splits) *num_kv_splits = 0;
  if (num_tokens < 1 || num_seqs < 1 || num_groups < 1 || num_heads < 1 || max_prefix_len < 1 ||
      sm_count < 1)
    return 1;
  const int64_t by_rows = (static_cast<int64_t>(num_tokens) + 255) / 256;
  const int64_t blocks = num_groups > by_rows ? num_groups : by_rows;
  const double units = static_cast<double>(blocks) * num_heads;
  const double rows = static_cast<double>(num_tokens) / num_seqs;  // of a sequence
  const double tile = num_tokens > 128 * blocks ? 2.0 : 1.5;
  const double record = static_cast<double>(num_tokens) * num_heads * 2.3e-4;
  auto tiles = [](int64_t keys, int parts) {
    return static_cast<double>((keys - 1) / (int64_t{128} * parts) + 1);
  };
  auto span = [&](double work, double count, double longest) {
    return count <= sm_count ? longest : work / sm_count + longest / 2;
  };
  // own keys that a unit of 256 rows passes over: its sequences' all, of which the
  // masks cut all tiles but those before a long sequence's rows
  double own = 0;
  if (max_kv_len > 0) {
    const double seqs = static_cast<double>((num_seqs - 1) / num_groups + 1);
    const double window = static_cast<double>(max_kv_len) / 128 *
                          (rows >= 256 ? 1 : 256 / rows < seqs ? 256 / rows : seqs);
    own = tile * (window + (rows >= 256 && window > 2 ? 2 : window) / 2);
  }
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 64 && (s == 1 || max_prefix_len / s >= 256); ++s) {
    const double part = 4 + tiles(max_prefix_len, s) * tile;
    double cost = span(units * (s * part + own), units * s, part + own);
    if (s > 1) cost += 3.5 + s * record;
    // units without rows, at most two a head and part, take their turns, too
    if (s > 1 && (num_tokens / 256 + num_groups + 2.0) * num_heads * s > sm_count) cost += 3;
    if (s == 1 || cost < least) {
      best = s;
      least = cost;
    }
  }
  if (!num_kv_splits || max_kv_len < 1) return best;
  const int parts = mla_prefill_num_kv_splits(num_tokens, num_seqs, num_heads, max_kv_len, sm_count);
  const double own_units =
      static_cast<double>(num_seqs > by_rows ? num_seqs : by_rows) * num_heads * parts;
  const double own_part = 4 + tiles(max_kv_len, parts) * (rows > 128 ? 2.0 : 1.5);
  for (int s = 1; s <= 64 && (s == 1 || max_prefix_len / s >= 256); ++s) {
    const double part = 4 + tiles(max_prefix_len, s) * tile;
    const double cost = span(units * s * part + own_units * own_part, units * s + own_units,
                             part > own_part ? part : own_part) +
                        3.5 + (s + parts) * record;
    if (cost < least) {
      best = s;
      *num_kv_splits = parts;
      least = cost;
    }
  }
  return best;
}

mla_status mla_prefill_shared(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* q_pe,
    int64_t q_pe_row_stride, int64_t q_pe_head_stride, int num_tokens, int num_heads,
    const void* k_nope, int64_t k_row_stride, int64_t k_head_stride, const void* v,
    int64_t v_row_stride, int64_t v_head_stride, const void* k_pe, int64_t k_pe_row_stride,
    int num_kv_tokens, int nope_dim, int rope_dim, int v_dim, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int num_seqs, const int32_t* group_seqs,
    const int32_t* cu_prefix, int num_groups, int causal, float sm_scale, int num_prefix_splits,
    int num_kv_splits, void* workspace, size_t workspace_bytes, void* o, int64_t o_row_stride,
    int64_t o_head_stride, float* lse, int* err_count, void* stream) {
  if (num_groups < 1) return MLA_ERR_INVALID_ARG;
  const Groups groups{group_seqs, cu_prefix, num_groups, num_prefix_splits};
  return prefill(q, q_row_stride, q_head_stride, q_pe, q_pe_row_stride, q_pe_head_stride, num_tokens,
                 num_heads, k_nope, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride,
                 k_pe, k_pe_row_stride, num_kv_tokens, nope_dim, rope_dim, v_dim, cu_seqlens_q,
                 cu_seqlens_k, num_seqs, groups, causal, sm_scale, num_kv_splits, workspace,
                 workspace_bytes, o, o_row_stride, o_head_stride, lse, err_count, stream);
}

}  // extern "C"
