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
// for large batches the latency of the page ids' copy on top.  So it is one
// launch with no pass between its CTAs: each forms the prefix sums of all
// requests itself (12 bytes a request, from L2) and its warps then take units:
// 1024 ids of a request's row (eight 16-byte loads of a lane in flight, or 16
// of one id where a row is not aligned), or 32 token rows.  A token's page is
// looked up where it comes from (the request's old row or the stack), never
// where another warp writes it, so no order between units matters.  1000
// requests of up to 65536 tokens in pages of 16 (17 MB moved): 7.4 us (a CTA
// per row, with its own sums: 10-16; four CTAs of 64 registers on an SM, which
// spill: 10.4); a decode step of 64 requests 3.4 us.
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"  // cluster helpers

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPiece = 1024;  // ids of a table row in one unit
constexpr int kRelThreads = 512;
constexpr int kRelCtas = 8;  // one portable cluster

// a / block_size and its round-up for 0 <= a < 2^31, as a product with a
// reciprocal (see page_reciprocal): a division by a variable took half of the
// kernel's instructions.
__device__ __forceinline__ int page_of(const BatchParams& p, int a) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(a)) * p.page_mul) >>
                          p.page_shift);
}
__device__ __forceinline__ int pages_of(const BatchParams& p, int a) {
  return a == 0 ? 0 : page_of(p, a - 1) + 1;
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

__device__ __forceinline__ Req make_req(const BatchParams& p, int q, int c, int id) {
  Req r;
  r.row = id >= 0 && id < p.num_table_rows ? id : -1;
  r.n = q < 0 ? 0 : q;
  r.ctx = c < 0 ? 0 : (c > p.capacity ? p.capacity : c);
  const long long s = static_cast<long long>(r.ctx) + r.n;
  r.seq = s > p.capacity ? p.capacity : static_cast<int>(s);
  r.bad = q < 0 || r.ctx != c || s > p.capacity;
  return r;
}

__device__ __forceinline__ Req load_req(const BatchParams& p, int b) {
  return make_req(p, p.query_lens ? __ldg(p.query_lens + b) : 0, __ldg(p.context_lens + b),
                  p.req_ids ? __ldg(p.req_ids + b) : b);
}

// f(b, request) for four requests of [from, to) at b = first, first + step,
// ..., all loads in flight before the first is used.
template <typename F>
__device__ __forceinline__ void four_reqs(const BatchParams& p, int first, int step, int to, F&& f) {
  int q[4], c[4], id[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = first + k * step;
    const bool in = b < to;
    q[k] = in && p.query_lens ? __ldg(p.query_lens + b) : 0;
    c[k] = in ? __ldg(p.context_lens + b) : 0;
    id[k] = in && p.req_ids ? __ldg(p.req_ids + b) : b;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int b = first + k * step;
    if (b < to) f(b, make_req(p, q[k], c[k], id[k]));
  }
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

// A plain load: blocks_release_kernel may write this address before it ends.
__device__ __forceinline__ int stack_count(const BatchParams& p) {
  const int c = *p.free_count;
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

__device__ __forceinline__ int new_pages(const BatchParams& p, const Req& r) {
  return r.row < 0 ? 0 : pages_of(p, r.seq) - pages_of(p, r.ctx);
}

// Prefix sums over all requests in one pass, four neighbouring requests a
// thread and 1024 a step: g(b, request), then f(b, tokens before, X before)
// with X the new pages, or the lengths with kSeq.  Returns (all tokens, all X).
template <bool kSeq, typename G, typename F>
__device__ __forceinline__ longlong2 scan_reqs(const BatchParams& p, long long (*part)[kWarps],
                                               G&& g, F&& f) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  longlong2 total = make_longlong2(0, 0);
  for (int base = 0; base < p.num_reqs; base += 4 * kThreads) {
    const int b0 = base + 4 * tid;
    int n[4] = {0, 0, 0, 0}, x[4] = {0, 0, 0, 0};
    four_reqs(p, b0, 1, p.num_reqs, [&](int b, const Req& r) {
      n[b - b0] = r.n;
      x[b - b0] = kSeq ? r.seq : new_pages(p, r);
      g(b, r);
    });
    long long own_n = 0, own_x = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      own_n += n[k];
      own_x += x[k];
    }
    long long sn = own_n, sx = own_x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long un = __shfl_up_sync(0xffffffffu, sn, o);
      const long long ux = __shfl_up_sync(0xffffffffu, sx, o);
      if (lane >= o) {
        sn += un;
        sx += ux;
      }
    }
    if (lane == 31) {
      part[0][warp] = sn;
      part[1][warp] = sx;
    }
    __syncthreads();
    long long cn = total.x + sn - own_n, cx = total.y + sx - own_x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long wn = part[0][w], wx = part[1][w];
      if (w < warp) {
        cn += wn;
        cx += wx;
      }
      total.x += wn;
      total.y += wx;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (b0 + k < p.num_reqs) {
        f(b0 + k, cn, cx);
        cn += n[k];
        cx += x[k];
      }
    }
    __syncthreads();  // part[] may be written again
  }
  return total;
}

// Sum over the block of one value per thread.
__device__ long long block_sum(long long s, long long* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();  // part[] may still be read from the last call
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += part[w];
  return total;
}

__global__ void __launch_bounds__(kThreads, 3) batch_build_kernel(const BatchParams p) {
  extern __shared__ int sm[];
  __shared__ long long part[2][kWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int B = p.num_reqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int errs = 0;
  if (blockIdx.x == 0) {
    // ---- lengths and their sums
    const longlong2 total = scan_reqs<true>(
        p, part,
        [&](int b, const Req& r) {
          p.seq_lens[b] = r.seq;
          errs += r.bad ? 1 : 0;
        },
        [&](int b, long long n, long long seq) {
          p.cu_q[b] = sat32(n);
          p.cu_k[b] = sat32(seq);
        });
    if (tid == 0) {
      p.cu_q[B] = sat32(total.x);
      p.cu_k[B] = sat32(total.y);
      if (total.x > p.num_tokens) ++errs;
    }
    count_errors(p.err_count, errs);
    return;
  }
  int* cuq = sm;          // [B] first token row of each request
  int* off = sm + B;      // [B] new pages before each request
  int* ctx = sm + 2 * B;  // [B]
  int* row = sm + 3 * B;  // [B]
  const int count = stack_count(p);
  const longlong2 total = scan_reqs<false>(
      p, part,
      [&](int b, const Req& r) {
        ctx[b] = r.ctx;
        row[b] = r.row;
      },
      [&](int b, long long n, long long pages) {
        cuq[b] = sat32(n);
        off[b] = sat32(pages);
      });
  // With the same address for both counts another CTA may still have to read
  // the old one: a launch of its own writes it then.
  if (blockIdx.x == 1 && tid == 0 && !p.defer_count)
    *p.free_count_out = total.y > count ? 0 : count - static_cast<int>(total.y);
  const int64_t warps = static_cast<int64_t>(gridDim.x - 1) * kWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x - 1) * kWarps + warp; u < p.units; u += warps) {
    if (u < p.row_units) {
      // ---- a piece of a table row: old pages from the request's row, new
      // ones off the stack
      const int b = static_cast<int>(u / p.row_pieces);
      const int i0 = static_cast<int>(u % p.row_pieces) * kPiece;
      const int c = ctx[b], rw = row[b];
      // New tokens: a step of cuq, unless its sums have saturated.  (The length
      // kept beside ctx costs an SM its third CTA from 3800 requests on: 4500
      // of them 22.7 us against 17.4.)
      const long long n = total.x > INT32_MAX ? max(0, __ldg(p.query_lens + b))
                                              : (b + 1 < B ? cuq[b + 1] : total.x) - cuq[b];
      const int seq = c + n > p.capacity ? p.capacity : static_cast<int>(c + n);
      const int end = min(pages_of(p, seq), i0 + kPiece);
      const int old_all = rw < 0 ? 0 : pages_of(p, c), old = min(old_all, end);
      int32_t* dst = p.block_table + static_cast<int64_t>(b) * p.bt_stride;
      int32_t* req = rw < 0 ? nullptr : p.req_table + static_cast<int64_t>(rw) * p.rt_stride;
      int done = min(i0, end);
      if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(req)) & 15u) == 0) {
        const int n4 = old >> 2;
        int4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((i0 >> 2) + lane + k * 32 < n4)
            x[k] = reinterpret_cast<const int4*>(req)[(i0 >> 2) + lane + k * 32];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((i0 >> 2) + lane + k * 32 < n4)
            reinterpret_cast<int4*>(dst)[(i0 >> 2) + lane + k * 32] = x[k];
        done = max(done, n4 << 2);
      } else {
#pragma unroll 1
        for (; done < old; done += 512) {
          int x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (done + lane + k * 32 < old) x[k] = req[done + lane + k * 32];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (done + lane + k * 32 < old) dst[done + lane + k * 32] = x[k];
        }
        done = min(done, max(old, i0));
      }
      for (int i = done + lane; i < end; i += 32) {
        int id;
        if (i < old) {
          id = req[i];
        } else {
          id = rw < 0 ? -1 : pop_page(p, count, static_cast<long long>(off[b]) + (i - old_all));
          if (id < 0 && rw >= 0) ++errs;
          if (req) req[i] = id;
        }
        dst[i] = id;
      }
    } else {
      // ---- token rows
      const int64_t t = (u - p.row_units) * 32 + lane;
      if (t >= p.num_tokens) continue;
      int64_t pos = 0, slot = -1;
      if (t < total.x) {
        int a = 0, z = B - 1;  // the last request whose first row is <= t
        while (a < z) {
          const int m = (a + z + 1) >> 1;
          if (cuq[m] <= t) a = m; else z = m - 1;
        }
        const int c = ctx[a], rw = row[a];
        pos = static_cast<int64_t>(c) + (t - cuq[a]);
        if (rw >= 0 && pos < p.capacity) {
          const int page = page_of(p, static_cast<int>(pos)), old = pages_of(p, c);
          const int id = page < old
                             ? p.req_table[static_cast<int64_t>(rw) * p.rt_stride + page]
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
  }
  __syncwarp();
  count_errors(p.err_count, errs);
}

// free_count_out = free_count - the batch's new pages, in place.
__global__ void __launch_bounds__(kThreads) batch_count_kernel(const BatchParams p) {
  __shared__ long long part[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  long long s = 0;
  for (int i = threadIdx.x; i < p.num_reqs; i += 4 * kThreads)
    four_reqs(p, i, kThreads, p.num_reqs, [&](int, const Req& r) { s += new_pages(p, r); });
  const long long total = block_sum(s, part);
  if (threadIdx.x == 0) {
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
    pre[b + 1] = r.row < 0 ? 0 : pages_of(p, r.ctx);
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

// With s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1: m d = 2^(31+s) + e,
// 0 < e <= d <= 2^s, so a m / 2^(31+s) exceeds a / d by less than 1 / d for
// a < 2^31 and the floors are equal.
void page_reciprocal(BatchParams* p) {
  int s = 0;
  while ((1 << s) < p->block_size) ++s;
  p->page_shift = 31 + s;
  p->page_mul = static_cast<uint32_t>((uint64_t{1} << (31 + s)) / p->block_size + 1);
}

}  // namespace

cudaError_t launch_batch_build(const BatchParams& p_in, int sm_count, cudaStream_t stream) {
  BatchParams p = p_in;
  page_reciprocal(&p);
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(batch_build_kernel, 4 * kMaxBatchReqs * 4, attr_done);
  if (e != cudaSuccess) return e;
  // max_blocks is capacity / block_size
  p.row_pieces = (p.capacity / p.block_size + kPiece - 1) / kPiece;
  p.row_units = static_cast<int64_t>(p.num_reqs) * p.row_pieces;
  p.units = p.row_units + (static_cast<int64_t>(p.num_tokens) + 31) / 32;
  const int64_t ctas = (p.units + kWarps - 1) / kWarps, most = 3 * sm_count - 1;
  const int grid = 1 + static_cast<int>(ctas < 1 ? 1 : ctas < most ? ctas : most);
  p.defer_count = p.free_count == p.free_count_out;
  e = launch_overlapped(batch_build_kernel, dim3(grid), dim3(kThreads),
                        4 * static_cast<size_t>(p.num_reqs) * 4, stream, p);
  if (e != cudaSuccess || !p.defer_count) return e;
  return launch_overlapped(batch_count_kernel, dim3(1), dim3(kThreads), 0, stream, p);
}

cudaError_t launch_blocks_release(const BatchParams& p_in, cudaStream_t stream) {
  BatchParams p = p_in;
  page_reciprocal(&p);
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(blocks_release_kernel, (kMaxBatchReqs + 1) * 4, attr_done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(blocks_release_kernel, dim3(kRelCtas), dim3(kRelThreads),
                           (static_cast<size_t>(p.num_reqs) + 1) * 4, stream, p);
}

}  // namespace mla
