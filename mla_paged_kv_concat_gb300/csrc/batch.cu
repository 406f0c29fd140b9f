// Batch tables on the GPU: block tables, slot map, positions and cumulative
// lengths of a step from its requests' lengths, with new pages taken off a
// stack of free pages; and the return of finished requests' pages.
//
// For request b with c cached and n new tokens and pages of bs tokens: the
// request holds ceil(c / bs) pages and needs ceil((c + n) / bs); the
// difference over all requests, in request and then page order, comes off
// the stack's top, so that page k of the batch's new pages is
// free[count - 1 - k].  Token j of request b sits at position c + j, in slot
// page * bs + (c + j) % bs.
//
// What bounds it: launch and memory latency for a decode step (a few KB),
// the copy of the page ids for large batches.  So it is one launch with no
// pass between its CTAs: every CTA forms the prefix sums of all requests
// itself (12 bytes a request, from L2), then takes whole requests' table rows
// and 256-token pieces of the slot map in turn.  A token's page is looked up
// where it comes from (the request's old row or the stack), never where
// another CTA writes it, so no order between CTAs matters.
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRelThreads = 512;
constexpr int kRelCtas = 8;  // one portable cluster

__device__ __forceinline__ int cdiv_pos(int a, int b) {  // a >= 0; no overflow near INT_MAX
  return a / b + (a % b != 0);
}

__device__ __forceinline__ int sat32(long long x) {
  return x > 2147483647ll ? 2147483647 : static_cast<int>(x);
}

// A request's lengths, clamped to what its table row can hold.
struct Req {
  int row;    // row of the requests' table, -1 when the id is out of range
  int n;      // new tokens
  int ctx;    // cached tokens
  int seq;    // cached + new, at most the capacity
  bool bad;   // something was clamped
};

__device__ __forceinline__ Req load_req(const BatchParams& p, int b) {
  Req r;
  const int q = p.query_lens ? __ldg(p.query_lens + b) : 0, c = __ldg(p.context_lens + b);
  const int id = p.req_ids ? __ldg(p.req_ids + b) : b;
  r.row = id >= 0 && id < p.num_table_rows ? id : -1;
  r.n = q < 0 ? 0 : q;
  r.ctx = c < 0 ? 0 : (c > p.capacity ? p.capacity : c);
  const long long s = static_cast<long long>(r.ctx) + r.n;
  r.seq = s > p.capacity ? p.capacity : static_cast<int>(s);
  r.bad = q < 0 || r.ctx != c || s > p.capacity;
  return r;
}

// Turns a[1..n] into inclusive sums with a[0] = 0 (64-bit sums, stored
// saturated), over a block of NT threads; returns the total.  `part` holds
// one partial per warp.
template <int NT>
__device__ long long block_scan(int* a, int n, long long* part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + NT - 1) / NT;
  const int lo = 1 + min(n, tid * per), hi = 1 + min(n, (tid + 1) * per);
  long long s = 0;
  for (int i = lo; i < hi; ++i) s += a[i];
  long long inc = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const long long x = part[w];
    if (w < warp) before += x;
    total += x;
  }
  long long run = before + inc - s;
  for (int i = lo; i < hi; ++i) {
    run += a[i];
    a[i] = sat32(run);
  }
  if (tid == 0) a[0] = 0;
  __syncthreads();  // a[] complete; part[] may be used again
  return total;
}

// Adds up the threads' error counts into the caller's counter.
__device__ __forceinline__ void count_errors(int* err_count, int errs) {
  if (!err_count) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) errs += __shfl_xor_sync(0xffffffffu, errs, o);
  if ((threadIdx.x & 31) == 0 && errs) atomicAdd(err_count, errs);
}

__device__ __forceinline__ int stack_count(const BatchParams& p) {
  const int c = __ldg(p.free_count);
  return c < 0 ? 0 : (c > p.free_capacity ? p.free_capacity : c);
}

// `*p` of CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_load(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];"
               : "=r"(v)
               : "r"(tc::map_peer(smem_u32(p), rank))
               : "memory");
  return v;
}

// New page k of the batch, or -1 when the stack does not hold it or holds an
// id outside the pool there.
__device__ __forceinline__ int pop_page(const BatchParams& p, int count, long long k) {
  if (k >= count) return -1;
  const int id = __ldg(p.free_blocks + (count - 1 - k));
  return id >= 0 && id < p.num_blocks ? id : -1;
}

__global__ void __launch_bounds__(kThreads) batch_build_kernel(const BatchParams p) {
  extern __shared__ int sm[];
  __shared__ long long part[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int B = p.num_reqs, tid = threadIdx.x;
  const bool first = blockIdx.x == 0;
  int* cuq = sm;              // [B + 1] first token row of each request
  int* off = sm + B + 1;      // [B + 1] new pages before each request
  int* cuk = sm + 2 * (B + 1);  // [B + 1] cumulative lengths (CTA 0 only)
  int errs = 0;
  for (int b = tid; b < B; b += kThreads) {
    const Req r = load_req(p, b);
    cuq[b + 1] = r.n;
    off[b + 1] =
        r.row < 0 ? 0 : cdiv_pos(r.seq, p.block_size) - cdiv_pos(r.ctx, p.block_size);
    if (first) {
      cuk[b + 1] = r.seq;
      p.seq_lens[b] = r.seq;
      errs += r.bad ? 1 : 0;
    }
  }
  const int count = stack_count(p);
  __syncthreads();
  const long long total_q = block_scan<kThreads>(cuq, B, part);
  const long long total_new = block_scan<kThreads>(off, B, part);
  if (first) {
    block_scan<kThreads>(cuk, B, part);
    for (int b = tid; b <= B; b += kThreads) {
      p.cu_q[b] = cuq[b];
      p.cu_k[b] = cuk[b];
    }
    if (tid == 0) {
      if (total_q > p.num_tokens) ++errs;
      // with the same address for both counts another CTA may still have to
      // read the old one: a launch of its own writes it then
      if (!p.defer_count)
        *p.free_count_out = total_new > count ? 0 : count - static_cast<int>(total_new);
    }
  }

  // ---- table rows: old pages from the request's row, new ones off the stack
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    const Req r = load_req(p, b);
    const int pages = cdiv_pos(r.seq, p.block_size);
    const int old = r.row < 0 ? 0 : cdiv_pos(r.ctx, p.block_size);
    int32_t* dst = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
    int32_t* req = r.row < 0 ? nullptr : p.req_table + static_cast<int64_t>(r.row) * p.rt_stride;
    int done = 0;
    if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(req)) & 15u) == 0) {
      const int n4 = old >> 2;
      for (int i = tid; i < n4; i += kThreads)
        reinterpret_cast<int4*>(dst)[i] = reinterpret_cast<const int4*>(req)[i];
      done = n4 << 2;
    }
    const long long k0 = off[b];
    for (int i = done + tid; i < pages; i += kThreads) {
      int id;
      if (i < old) {
        id = req[i];
      } else {
        id = r.row < 0 ? -1 : pop_page(p, count, k0 + (i - old));
        if (id < 0 && r.row >= 0) ++errs;
        if (req) req[i] = id;
      }
      dst[i] = id;
    }
  }

  // ---- token rows
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + tid; t < p.num_tokens;
       t += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t pos = 0, slot = -1;
    if (t < total_q) {
      int a = 0, z = B - 1;  // the last request whose first row is <= t
      while (a < z) {
        const int m = (a + z + 1) >> 1;
        if (cuq[m] <= t) a = m; else z = m - 1;
      }
      const Req r = load_req(p, a);
      pos = static_cast<int64_t>(r.ctx) + (t - cuq[a]);
      if (r.row >= 0 && pos < r.seq) {
        const int page = static_cast<int>(pos) / p.block_size;
        const int old = cdiv_pos(r.ctx, p.block_size);
        const int id =
            page < old ? p.req_table[static_cast<int64_t>(r.row) * p.rt_stride + page]
                       : pop_page(p, count, static_cast<long long>(off[a]) + (page - old));
        if (id >= 0 && id < p.num_blocks)
          slot = static_cast<int64_t>(id) * p.block_size +
                 (static_cast<int>(pos) - page * p.block_size);
      }
      if (slot < 0) ++errs;
    }
    p.positions[t] = pos;
    p.slot_mapping[t] = slot;
  }
  count_errors(p.err_count, errs);
}

// free_count_out = free_count - the batch's new pages, in place.
__global__ void __launch_bounds__(kThreads) batch_count_kernel(const BatchParams p) {
  __shared__ long long part[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  long long s = 0;
  for (int b = threadIdx.x; b < p.num_reqs; b += kThreads) {
    const Req r = load_req(p, b);
    if (r.row >= 0) s += cdiv_pos(r.seq, p.block_size) - cdiv_pos(r.ctx, p.block_size);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) total += part[w];
    const int count = *p.free_count_out;
    const int c = count < 0 ? 0 : (count > p.free_capacity ? p.free_capacity : count);
    *p.free_count_out = total > c ? 0 : c - static_cast<int>(total);
  }
}

// Pages of the requests back onto the stack: the pages of all requests, in
// request and then page order, form one list; entries outside the pool (a
// page that could not be taken) are left out and counted.  Where an entry
// goes depends on the valid ones before it, so the list is cut into eight
// equal pieces, one for each CTA of a cluster: each counts its valid entries,
// reads the counts before it from the other CTAs' shared memory, and writes.
__global__ void __cluster_dims__(kRelCtas, 1, 1) __launch_bounds__(kRelThreads)
    blocks_release_kernel(const BatchParams p) {
  extern __shared__ int sm[];
  __shared__ long long part[kRelThreads / 32];
  __shared__ int warp_n[kRelThreads / 32];
  __shared__ int valid_here;
  griddep_wait();
  griddep_launch_dependents();
  const int B = p.num_reqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x;
  int* pre = sm;  // [B + 1] pages before each request
  int errs = 0;
  for (int b = tid; b < B; b += kRelThreads) {
    const Req r = load_req(p, b);
    pre[b + 1] = r.row < 0 ? 0 : cdiv_pos(r.ctx, p.block_size);
    if (rank == 0 && (r.bad || r.row < 0)) ++errs;
  }
  if (tid == 0) valid_here = 0;
  const int count = stack_count(p);
  __syncthreads();
  const long long total = block_scan<kRelThreads>(pre, B, part);
  const long long lo = total * rank / kRelCtas, hi = total * (rank + 1) / kRelCtas;
  auto entry = [&](long long i) -> int {
    if (i >= hi) return -1;
    int a = 0, z = B - 1;
    while (a < z) {
      const int m = (a + z + 1) >> 1;
      if (pre[m] <= i) a = m; else z = m - 1;
    }
    const int row = p.req_ids ? __ldg(p.req_ids + a) : a;
    const int id = p.req_table[static_cast<int64_t>(row) * p.rt_stride + (i - pre[a])];
    return id >= 0 && id < p.num_blocks ? id : -1;
  };
  int mine = 0;
  for (long long i = lo + tid; i < hi; i += kRelThreads) mine += entry(i) >= 0 ? 1 : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0 && mine) atomicAdd(&valid_here, mine);  // integer: any order, one result
  __syncthreads();
  tc::cluster_sync();
  long long before = 0, all = 0;
  for (int c = 0; c < kRelCtas; ++c) {
    const int v = cluster_load(&valid_here, c);
    if (c < rank) before += v;
    all += v;
  }
  // nobody leaves, and no count is written, before every CTA has read both
  tc::cluster_sync();
  const long long room = p.free_capacity - count;
  if (rank == 0 && tid == 0) {
    const long long kept = all < room ? all : room;
    *p.free_count_out = count + static_cast<int>(kept);
    errs += sat32(total - kept);
  }
  long long base = count + before;
  for (long long i0 = lo; i0 < hi; i0 += kRelThreads) {
    const int id = entry(i0 + tid);
    const uint32_t mask = __ballot_sync(0xffffffffu, id >= 0);
    if (lane == 0) warp_n[warp] = __popc(mask);
    __syncthreads();
    int pos = __popc(mask & ((1u << lane) - 1u)), step = 0;
#pragma unroll
    for (int w = 0; w < kRelThreads / 32; ++w) {
      const int n = warp_n[w];
      if (w < warp) pos += n;
      step += n;
    }
    if (id >= 0 && base + pos < p.free_capacity) p.free_out[base + pos] = id;
    base += step;
    __syncthreads();
  }
  count_errors(p.err_count, errs);
}

}  // namespace

cudaError_t launch_batch_build(const BatchParams& p_in, int sm_count, cudaStream_t stream) {
  BatchParams p = p_in;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(batch_build_kernel, 3 * (kMaxBatchReqs + 1) * 4, attr_done);
  if (e != cudaSuccess) return e;
  const int pieces = p.num_tokens / kThreads + (p.num_tokens % kThreads != 0);
  int grid = p.num_reqs > pieces ? p.num_reqs : pieces;
  if (grid > 4 * sm_count) grid = 4 * sm_count;
  if (grid < 1) grid = 1;
  p.defer_count = p.free_count == p.free_count_out && grid > 1;
  e = launch_overlapped(batch_build_kernel, dim3(grid), dim3(kThreads),
                        3 * (static_cast<size_t>(p.num_reqs) + 1) * 4, stream, p);
  if (e != cudaSuccess || !p.defer_count) return e;
  return launch_overlapped(batch_count_kernel, dim3(1), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_blocks_release(const BatchParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(blocks_release_kernel, (kMaxBatchReqs + 1) * 4, attr_done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(blocks_release_kernel, dim3(kRelCtas), dim3(kRelThreads),
                           (static_cast<size_t>(p.num_reqs) + 1) * 4, stream, p);
}

}  // namespace mla
