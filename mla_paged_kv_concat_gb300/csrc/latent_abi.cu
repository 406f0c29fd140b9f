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

namespace {

using mla::aligned16;
using mla::aligned4;
using mla::aligned8;
using mla::cuda_fail;

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
  const int64_t stack = static_cast<int64_t>(free_capacity) * 4;
  if (overlap(free_blocks, stack, free_count, 4) ||
      overlap(free_blocks, stack, free_count_out, 4) ||
      overlap(free_blocks, stack, held_lens, n4) ||
      overlap(free_blocks, stack, req_ids, req_ids ? n4 : 0) ||
      overlap(free_blocks, stack, req_block_table,
              num_reqs ? ((num_table_rows - 1) * req_block_table_stride + max_blocks_per_req) * 4
                       : 0))
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

}  // extern "C"
