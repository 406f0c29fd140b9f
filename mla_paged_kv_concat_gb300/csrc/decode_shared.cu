// MLA decode for a batch whose sequences share prefixes: the cached rows of a
// prefix are read once for all query vectors of its group.
//
//   s_j = sm_scale * q . K_j,  o = sum_j softmax(s)_j K_j[0:R],  lse = ln sum e^s
//
// over all tokens j of the row's sequence, as in the plain decode.  The tokens
// are cut in two: the first floor(prefix / 128) * 128 of a group are passed over
// by the vectors (rows x heads) of all its sequences together, the others by each
// sequence's own vectors.  Each part leaves an unnormalised output, a maximum and
// a sum, and the last kernel joins them:
//   M = max m_i,  o = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// A sequence shorter than the shared part (a padded row of length 0 among them)
// takes no part in it: its own pass then starts at token 0, so that every vector
// of a shared pass attends to every token of it, and nothing is masked there.
//
// Work.  128 vectors x 128 tokens are 128 x 128 x (R + 64) products of Q K^T and
// 128 x R x 128 of P V.  An fp32 O of 128 x 512 fills all 512 columns of a CTA's
// TMEM, so the two CTAs of a cluster split the work by product: rank 0 (scores)
// holds Q (packed bf16 in TMEM, the rope part in shared memory), computes S and
// the softmax and sends P, in bf16, into rank 1's shared memory; rank 1 (values)
// holds O and accumulates P V.  Data flow one way, so the rank that computes
// scores runs ahead by the two P buffers and no round trip is on any tile's path.
// Per tile the tensor cores have 36 x 74 cycles (M = 128, N = 128) on rank 0 and
// 16 x 138 (N = 256) on rank 1.  Rank 1 reads the latent part of the rows again,
// from L2.
//   rank 0: Q 256 + S 2 x 128 TMEM columns; a ring of five 32 KiB boxes of K (128
//     dims x 128 tokens) and one of two rope boxes (16 KiB)
//   rank 1: O R TMEM columns; P 2 x 32 KiB; a ring of five 32 KiB boxes of V (256
//     dims x 64 tokens)
// An fp8 cache lands in staging boxes and four more warps of each CTA turn it into
// the bf16 boxes; its values are exact in bf16, and the scale is applied to the
// scores and to the joined output.
//
// Schedule.  A first kernel (one CTA) turns lengths into a list of all tiles: the
// groups' prefixes, then the sequences, each cut into blocks of 128 vectors.  Pair
// c of CTAs takes tiles [c C, (c + 1) C).  Blocks of one prefix are listed in
// chunks of C tiles side by side, so that pairs at work together read the same
// rows.  Unit u (chunk of a block) meets pair c in segment u + c, which is also
// its place in the workspace: list positions only grow, so no two are alike.
//
// Roles (320 threads, 448 with an fp8 cache): warps 0-7 softmax (rank 0) or
// rescaling and output of O (rank 1), thread = TMEM lane = vector, two warps a
// lane quarter (token or dim halves); warp 8 TMA, warp 9 MMA, 10-13 conversion.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int TT = 128;                 // tokens of a tile
constexpr int kBig = 32768;             // ring box
constexpr int kRope = 16384;            // rope box: 128 tokens x 64 dims
constexpr int kPBuf = 32768;            // P: two boxes of 128 vectors x 64 tokens
// Shared memory of rank 0 and rank 1.
constexpr int S_QPE = 0;
constexpr int S_ROPE = S_QPE + 16384;   // two boxes
constexpr int S_RING = S_ROPE + 2 * kRope;
constexpr int V_RING = 2 * kPBuf;
constexpr int kData = 229376;
constexpr int OFF_MISC = kData;         // rank 1: rescale factors, two buffers of 128
constexpr int OFF_BAR = OFF_MISC + 1024;
constexpr int OFF_TMEM = OFF_BAR + 512;
constexpr int kSmem = OFF_TMEM + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
template <bool FP8>
struct Ring {
  static constexpr int S_BOXES = FP8 ? 4 : 5, V_BOXES = FP8 ? 3 : 5;
  static constexpr int STAGES = FP8 ? 2 : 1, V_STAGES = FP8 ? 4 : 1;  // fp8 staging boxes
  static constexpr int S_STAGE = S_RING + S_BOXES * kBig;             // 16 KiB each
  static constexpr int S_RSTAGE = S_STAGE + (FP8 ? 2 * 16384 : 0);    // rope: 8 KiB
  static constexpr int S_RED = S_RSTAGE + (FP8 ? 8192 : 0);           // [2][2][128] fp32
  static constexpr int V_STAGE = V_RING + V_BOXES * kBig;
  static_assert(V_STAGE + (FP8 ? 4 * 16384 : 0) <= kData, "rank 1's shared memory");
  static_assert(S_RED + 2048 <= kData, "rank 0's shared memory");
};

constexpr uint32_t S_COL = 256;  // rank 0: Q below, S 2 x 128 columns
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleAt = 8.0f;  // log2 units

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ int clampi(int x, int lo, int hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  const bool ok = tc::mbar_wait_cluster(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- schedule
// Inclusive scan of a[0, n) by the block; values are not negative.
template <typename Op>
__device__ void block_scan(int* a, int n, int* tot, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int v = i < n ? a[i] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = op(v, t);
    }
    if (lane == 31) tot[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int w = tot[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w = op(w, t);
      }
      tot[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v = op(v, tot[warp - 1]);
    v = op(v, carry);
    if (i < n) a[i] = v;
    carry = op(carry, tot[31]);
    __syncthreads();
  }
}

// Where unit (chunk j, block g) of a part lies in the list.
__device__ __forceinline__ int chunk_tiles(const SharedPart& v, int C) {
  return v.blocks == 1 || v.tiles < C ? v.tiles : C;
}

__global__ void __launch_bounds__(1024) shared_schedule_kernel(const SharedParams p) {
  extern __shared__ int sm[];
  const int G = p.num_groups, B = p.num_seqs, V = G + B;
  int* ends = sm;             // [G + 1] first sequence of each group
  int* shared = ends + G + 1; // [G] tokens of its shared part
  int* lead = shared + G;     // [G] the sequence whose table they are read through
  int* pre = lead + G;        // [V + 1] tiles before a part
  int* unit = pre + V + 1;    // [V + 1] units before a part
  __shared__ int tot[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const int per = p.rows_per_seq * p.num_heads;  // vectors of a sequence
  const int own_blocks = cdiv(per, 128);
  auto length = [&](int b) { return clampi(__ldg(p.seq_lens + b), 0, p.capacity); };

  for (int g = threadIdx.x; g <= G; g += blockDim.x)
    ends[g] = clampi(__ldg(p.group_seqs + g), 0, B);
  __syncthreads();
  block_scan(ends, G + 1, tot, [](int a, int b) { return max(a, b); });
  for (int g = warp; g < G; g += 32) {
    const int raw = __ldg(p.prefix_lens + g);
    const int n = clampi(raw, 0, p.capacity) & ~(TT - 1);
    if (lane == 0 && (raw < 0 || raw > p.capacity) && p.err_count) atomicAdd(p.err_count, 1);
    int count = 0, first = B;
    for (int b = ends[g] + lane; b < ends[g + 1]; b += 32)
      if (length(b) >= n) {
        ++count;
        first = min(first, b);
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      count += __shfl_xor_sync(0xffffffffu, count, d);
      first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
    }
    if (lane == 0) {
      shared[g] = count > 1 ? n : 0;
      lead[g] = first;
    }
  }
  __syncthreads();
  // the parts: groups, then sequences
  auto part = [&](int v) {
    SharedPart x = {};
    x.group = -1;
    if (v < G) {
      x.row0 = ends[v] * p.rows_per_seq;
      x.vecs = (ends[v + 1] - ends[v]) * per;
      x.tok1 = shared[v];
      x.table = lead[v];
    } else {
      const int b = v - G;
      int a = 0, z = G;  // the last group that starts at or before b
      while (a < z) {
        const int m = (a + z + 1) >> 1;
        if (ends[m] <= b) a = m; else z = m - 1;
      }
      x.row0 = b * p.rows_per_seq;
      x.vecs = per;
      x.tok1 = length(b);
      x.table = b;
      if (a < G && b >= ends[a] && shared[a] > 0 && x.tok1 >= shared[a]) {
        x.group = a;
        x.tok0 = shared[a];
      }
    }
    x.tiles = cdiv(x.tok1 - x.tok0, TT);
    x.blocks = x.tiles ? cdiv(x.vecs, 128) : 0;
    return x;
  };
  for (int v = threadIdx.x; v < V; v += blockDim.x) {
    const SharedPart x = part(v);
    pre[v + 1] = x.tiles * x.blocks;
    if (v >= G) {
      const int raw = __ldg(p.seq_lens + v - G);
      if ((raw < 0 || raw > p.capacity) && p.err_count) atomicAdd(p.err_count, 1);
    }
  }
  if (threadIdx.x == 0) pre[0] = unit[0] = 0;
  __syncthreads();
  block_scan(pre + 1, V, tot, [](int a, int b) { return a + b; });
  const int total = pre[V];
  const int C = max(1, cdiv(total, p.pairs));
  for (int v = threadIdx.x; v < V; v += blockDim.x) {
    const SharedPart x = part(v);
    unit[v + 1] = x.blocks == 0 ? 0 : x.blocks * cdiv(x.tiles, chunk_tiles(x, C));
  }
  __syncthreads();
  block_scan(unit + 1, V, tot, [](int a, int b) { return a + b; });
  for (int v = threadIdx.x; v < V; v += blockDim.x) {
    SharedPart x = part(v);
    x.tile0 = pre[v];
    x.unit0 = unit[v];
    p.parts[v] = x;
  }
  if (threadIdx.x == 0) p.header[0] = C;
  // the segments of each pair
  for (int c = threadIdx.x; c < p.pairs; c += blockDim.x) {
    const int64_t lo64 = static_cast<int64_t>(c) * C;
    const int lo = lo64 < total ? static_cast<int>(lo64) : total;
    const int hi = lo + C < total ? lo + C : total;
    int2 mine = make_int2(0, 0);
    if (lo < hi) {
      int a = 0, z = V - 1;  // the last part that starts at or before lo
      while (a < z) {
        const int m = (a + z + 1) >> 1;
        if (pre[m] <= lo) a = m; else z = m - 1;
      }
      int t = lo;
      for (int v = a; t < hi; ++v) {
        if (pre[v + 1] <= t) continue;
        const SharedPart x = part(v);
        const int ch = chunk_tiles(x, C);
        while (t < hi && t < pre[v + 1]) {
          const int in = t - pre[v];
          const int j = in / (ch * x.blocks);
          const int len = min(ch, x.tiles - j * ch);
          const int y = in - j * ch * x.blocks, g = y / len, k = y - g * len;
          const int n = min(len - k, hi - t);
          SharedSegment s;
          s.table = x.table;
          s.row0 = x.row0;
          s.vec0 = g * 128;
          s.vecs = min(128, x.vecs - g * 128);
          s.tok0 = x.tok0 + (j * ch + k) * TT;
          s.tok1 = min(x.tok1, s.tok0 + n * TT);
          s.pad0 = s.pad1 = 0;
          const int slot = unit[v] + j * x.blocks + g + c;
          p.segments[slot] = s;
          if (mine.y == 0) mine.x = slot;
          ++mine.y;
          t += n;
        }
      }
    }
    p.pair_segments[c] = mine;
  }
}

// ---------------------------------------------------------------- conversion
// 16 fp8 codes to bf16, exactly.
__device__ __forceinline__ void fp8x16(const uint4& raw, bool e5m2, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t two = static_cast<uint16_t>(w[i >> 1] >> ((i & 1) * 16));
    const __half2_raw h =
        __nv_cvt_fp8x2_to_halfraw2(two, e5m2 ? __NV_E5M2 : __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    o[i] = pack_bf16x2(f.x, f.y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// One converting warp's part of `rows` x 64 dims: staging rows of 64 bytes to a
// swizzled box of 128-byte rows.
__device__ __forceinline__ void convert_box(const uint8_t* src, uint8_t* dst, int rows, int t,
                                            bool e5m2) {
#pragma unroll 4
  for (int i = t; i < rows * 4; i += 128) {
    const uint4 x = *reinterpret_cast<const uint4*>(src + i * 16);
    uint4 lo, hi;
    fp8x16(x, e5m2, lo, hi);
    const int r = i >> 2, c = (i & 3) * 2;
    *reinterpret_cast<uint4*>(dst + sw128(r, c)) = lo;
    *reinterpret_cast<uint4*>(dst + sw128(r, c + 1)) = hi;
  }
}

// ---------------------------------------------------------------- main kernel
template <int R, bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP8 ? 448 : 320, 1)
    decode_shared_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tmap) {
  using RG = Ring<FP8>;
  constexpr int KB = R / 128;   // 32 KiB boxes of K a tile
  constexpr int VB = R / 256;   // 256-dim parts of O
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  // The same places in both CTAs; each uses its own.
  uint64_t* full = bars;             // [5] ring box landed (converted)
  uint64_t* empty = full + 5;        // [5]
  uint64_t* rfull = empty + 5;       // [2] rank 0: rope box landed
  uint64_t* rempty = rfull + 2;      // [2]
  uint64_t* st_full = rempty + 2;    // [4] fp8 staging box landed
  uint64_t* st_empty = st_full + 4;  // [4]
  uint64_t* rs_full = st_empty + 4;  // rank 0: fp8 staging of a rope box
  uint64_t* rs_empty = rs_full + 1;
  uint64_t* s_full = rs_empty + 1;   // [2] rank 0: S of a tile of this parity
  uint64_t* s_free = s_full + 2;     // [2] rank 0: S read
  uint64_t* q_full = s_free + 2;     // rank 0: the segment's Q is in place
  uint64_t* q_free = q_full + 1;     // rank 0: the segment's last Q K^T is done
  uint64_t* p_free = q_free + 1;     // [2] rank 0: P buffer read by rank 1's products
  uint64_t* p_full = p_free + 2;     // [2] rank 1: P and rescale factors landed
  uint64_t* o_ready = p_full + 2;    // [2] rank 1: O rescaled for this tile's P
  uint64_t* pv_done = o_ready + 2;   // [2] rank 1
  uint64_t* o_free = pv_done + 2;    // rank 1: the segment's O has been read out
  static_assert((5 + 5 + 2 + 2 + 4 + 4 + 1 + 1 + 2 + 2 + 1 + 1 + 2 + 2 + 2 + 2 + 1) * 8 <= 512,
                "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);

  const uint32_t rank = tc::cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmap);
    for (int i = 0; i < 5; ++i) {
      mbar_init(&full[i], FP8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&rfull[i], FP8 ? 4 : 1);
      mbar_init(&rempty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 8);
      mbar_init(&p_free[i], 1);
      mbar_init(&p_full[i], 1);
      mbar_init(&o_ready[i], 8);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], 4);
    }
    mbar_init(rs_full, 1);
    mbar_init(rs_empty, 4);
    mbar_init(q_full, 8);
    mbar_init(q_free, 1);
    mbar_init(o_free, 8);
    fence_mbar_init();
    if (rank == 1)
      for (int i = 0; i < 2; ++i) mbar_arrive_expect_tx(&p_full[i], kPBuf + 512);
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer's barriers exist before any remote traffic
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int2 mine = p.pair_segments[blockIdx.x >> 1];
  const int H = p.num_heads;
  const int bs = p.block_size;
  const int box_rows = bs < 64 ? bs : 64;
  auto segment = [&](int k) -> SharedSegment {
    const int4* s = reinterpret_cast<const int4*>(p.segments + mine.x + k);
    SharedSegment r;
    reinterpret_cast<int4*>(&r)[0] = s[0];
    reinterpret_cast<int4*>(&r)[1] = s[1];
    return r;
  };
  bool ok = true;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    // Lane l loads (page l % 8, 64-dim part l / 8) of a K box, page l % 4 and
    // part l / 4 of a V box.  Page ids are read one tile before they are used.
    const int pages = TT / box_rows;  // of a tile: 2, 4 or 8
    constexpr int kRowBytes = FP8 ? 64 : 128;  // a row of a 64-dim part
    int nb = 0, nr = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int32_t* bt = p.block_table + static_cast<int64_t>(sg.table) * p.bt_stride;
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      auto id_of = [&](int t) -> int {
        const int tk = sg.tok0 + t * TT + (lane & 7) * box_rows;
        return lane < pages && t < tiles && tk < sg.tok1 ? __ldg(bt + tk / bs) : 0;
      };
      int id = id_of(0);
      for (int t = 0; t < tiles && ok; ++t) {
        const int next = id_of(t + 1);
        const int tok = sg.tok0 + t * TT;
        const int have = min(pages, cdiv(sg.tok1 - tok, box_rows));  // pages to load
        if (rank == 0 && lane < have && (id < 0 || id >= p.num_blocks) && p.err_count)
          atomicAdd(p.err_count, 1);
        // a box: `parts` 64-dim parts from dim `d0` on, pages [p0, p0 + np)
        auto load = [&](uint8_t* dst, uint64_t* bar, int parts, int part_bytes, int d0, int p0,
                        int np, int page, int part) {
          const int blk = __shfl_sync(0xffffffffu, id, (p0 + page) & 31);
          if (lane == 0)
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(parts * np * box_rows * kRowBytes));
          __syncwarp();
          if (page < np && part < parts) {
            const int tk = tok + (p0 + page) * box_rows;
            tma_load_3d(dst + part * part_bytes + page * box_rows * kRowBytes, &tmap, bar,
                        d0 + part * 64, tk % bs, blk);
          }
        };
        if (rank == 0) {
          for (int c = 0; c < KB && ok; ++c, ++nb) {
            const int st = FP8 ? nb % RG::STAGES : nb % RG::S_BOXES;
            const int use = FP8 ? nb / RG::STAGES : nb / RG::S_BOXES;
            ok = warp_wait(FP8 ? &st_empty[st] : &empty[st], (use & 1) ^ 1);
            if (!ok) break;
            uint8_t* dst = smem + (FP8 ? RG::S_STAGE + st * 16384 : S_RING + st * kBig);
            load(dst, FP8 ? &st_full[st] : &full[st], 2, TT * kRowBytes, c * 128, 0, have,
                 lane & 7, lane >> 3);
          }
          if (!ok) break;
          const int st = nr & 1;
          ok = FP8 ? warp_wait(rs_empty, st ^ 1) : warp_wait(&rempty[st], ((nr >> 1) & 1) ^ 1);
          if (!ok) break;
          load(smem + (FP8 ? RG::S_RSTAGE : S_ROPE + st * kRope), FP8 ? rs_full : &rfull[st], 1, TT * kRowBytes, R, 0, have, lane & 7, lane >> 3);
          ++nr;
        } else {
          const int half = pages / 2;
          for (int e = 0; e < 2 && e * half < have && ok; ++e)
            for (int d = 0; d < VB; ++d, ++nb) {
              const int st = FP8 ? nb % RG::V_STAGES : nb % RG::V_BOXES;
              const int use = FP8 ? nb / RG::V_STAGES : nb / RG::V_BOXES;
              ok = warp_wait(FP8 ? &st_empty[st] : &empty[st], (use & 1) ^ 1);
              if (!ok) break;
              uint8_t* dst = smem + (FP8 ? RG::V_STAGE + st * 16384 : V_RING + st * kBig);
              load(dst, FP8 ? &st_full[st] : &full[st], 4, 64 * kRowBytes, d * 256, e * half,
                   min(half, have - e * half), lane & 3, lane >> 2);
            }
        }
        id = next;
      }
    }
  } else if (FP8 && warp >= 10) {
    // ---------------------------------------------------------- conversion
    const int t = threadIdx.x - 320;
    const bool e5m2 = p.e5m2;
    int nb = 0, nr = 0;
    // staging box -> ring box, `parts` 64-dim parts of `rows` rows each
    auto turn = [&](uint64_t* sf, uint64_t* se, int su, const uint8_t* src, uint64_t* bf,
                    uint64_t* be, int bu, uint8_t* dst, int parts, int rows) -> bool {
      if (!warp_wait(sf, su & 1) || !warp_wait(be, (bu & 1) ^ 1)) return false;
      for (int c = 0; c < parts; ++c)
        convert_box(src + c * rows * 64, dst + c * rows * 128, rows, t, e5m2);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bf);
        mbar_arrive(se);
      }
      return true;
    };
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      for (int tok = sg.tok0; tok < sg.tok1 && ok; tok += TT) {
        if (rank == 0) {
          for (int c = 0; c < KB && ok; ++c, ++nb) {
            const int st = nb % RG::STAGES, bx = nb % RG::S_BOXES;
            ok = turn(&st_full[st], &st_empty[st], nb / RG::STAGES,
                      smem + RG::S_STAGE + st * 16384, &full[bx], &empty[bx], nb / RG::S_BOXES,
                      smem + S_RING + bx * kBig, 2, TT);
          }
          if (ok) {
            const int st = nr & 1;
            ok = turn(rs_full, rs_empty, nr, smem + RG::S_RSTAGE, &rfull[st], 
                      &rempty[st], nr >> 1, smem + S_ROPE + st * kRope, 1, TT);
            ++nr;
          }
        } else {
          for (int e = 0; e < 2 && tok + e * 64 < sg.tok1 && ok; ++e)
            for (int d = 0; d < VB && ok; ++d, ++nb) {
              const int st = nb % RG::V_STAGES, bx = nb % RG::V_BOXES;
              ok = turn(&st_full[st], &st_empty[st], nb / RG::V_STAGES,
                        smem + RG::V_STAGE + st * 16384, &full[bx], &empty[bx], nb / RG::V_BOXES,
                        smem + V_RING + bx * kBig, 4, 64);
            }
        }
      }
    }
  } else if (warp == 9 && rank == 0) {
    // ------------------------------------------------------------- Q K^T
    constexpr uint32_t idesc = tc::idesc_bf16(128, TT, 0, 0);
    const uint64_t dq = tc::smem_desc(smem_u32(smem + S_QPE), 16, 1024, tc::kLayoutSw128);
    int n = 0, nb = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      ok = warp_wait(q_full, k & 1);
      for (int t = 0; t < tiles && ok; ++t, ++n) {
        const uint32_t dS = tmem + S_COL + (n & 1) * TT;
        ok = warp_wait(&s_free[n & 1], ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < KB; ++c, ++nb) {
          const int bx = nb % RG::S_BOXES;
          ok = ok && warp_wait(&full[bx], (nb / RG::S_BOXES) & 1);
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint64_t db =
                tc::smem_desc(smem_u32(smem + S_RING + bx * kBig), 16, 1024, tc::kLayoutSw128);
#pragma unroll
            for (int s = 0; s < 8; ++s)
              tc::mma_ts(dS, tmem + c * 64 + s * 8,
                         db + static_cast<uint64_t>((s >> 2) * (16384 >> 4) + (s & 3) * 2), idesc,
                         (c > 0 || s > 0) ? 1u : 0u);
            tc::commit(&empty[bx]);
          }
          __syncwarp();
        }
        if (!ok) break;
        ok = warp_wait(&rfull[n & 1], (n >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint64_t db = tc::smem_desc(smem_u32(smem + S_ROPE + (n & 1) * kRope), 16, 1024,
                                            tc::kLayoutSw128);
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc::mma_ss(dS, dq + static_cast<uint64_t>(s * 2), db + static_cast<uint64_t>(s * 2),
                       idesc, 1u);
          tc::commit(&rempty[n & 1]);
          tc::commit(&s_full[n & 1]);
          if (t + 1 == tiles) tc::commit(q_free);
        }
        __syncwarp();
      }
    }
    // nothing of this CTA's still runs on the tensor core when TMEM is freed
    if (ok && mine.y > 0) ok = warp_wait(q_free, (mine.y - 1) & 1);
  } else if (warp == 9) {
    // --------------------------------------------------------------- P V
    constexpr uint32_t idesc = tc::idesc_bf16(128, 256, 0, 1);
    int n = 0, nb = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      if (k > 0) ok = warp_wait(o_free, (k - 1) & 1);
      for (int t = 0; t < tiles && ok; ++t, ++n) {
        ok = warp_wait(&o_ready[n & 1], (n >> 1) & 1);
        if (!ok) break;
        tc::fence_after_sync();
        const int left = sg.tok1 - (sg.tok0 + t * TT);  // tokens of the tile
#pragma unroll 1
        for (int e = 0; e < 2 && e * 64 < left && ok; ++e) {
          const uint64_t da = tc::smem_desc(smem_u32(smem + (n & 1) * kPBuf + e * 16384), 16, 1024,
                                            tc::kLayoutSw128);
#pragma unroll
          for (int d = 0; d < VB; ++d, ++nb) {
            const int bx = nb % RG::V_BOXES;
            ok = ok && warp_wait(&full[bx], (nb / RG::V_BOXES) & 1);
            if (!ok) break;
            uint8_t* box = smem + V_RING + bx * kBig;
            if (left < e * 64 + 64) {
              // Rows past the sequence's end hold other tokens, or what was
              // there before: zeros, since 0 * NaN is NaN (their P is 0).
              const int valid = left - e * 64;
              for (int i = lane; i < (64 - valid) * 32; i += 32) {
                const int r = valid + (i >> 5), rem = i & 31;
                *reinterpret_cast<uint4*>(box + (rem >> 3) * 8192 + r * 128 + (rem & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
              __syncwarp();
            }
            tc::fence_after_sync();
            if (tc::elect_one()) {
              // V is MN-major: the next 64 dims are 8 KiB on, 16 tokens 2 KiB
              const uint64_t db = tc::smem_desc(smem_u32(box), 8192, 1024, tc::kLayoutSw128);
#pragma unroll
              for (int s = 0; s < 4; ++s)
                tc::mma_ss(tmem + d * 256, da + static_cast<uint64_t>(s * 2),
                           db + static_cast<uint64_t>(s * 128), idesc,
                           (t > 0 || e > 0 || s > 0) ? 1u : 0u);
              tc::commit(&empty[bx]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        if (tc::elect_one()) {
          tc::commit(&pv_done[n & 1]);
          tc::commit_multicast(&p_free[n & 1], 1);  // rank 0 may send the tile after next's P
        }
        __syncwarp();
      }
    }
    if (ok && n > 0) ok = warp_wait(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
  } else if (rank == 0) {
    // ------------------------------------------------------------- softmax
    const int quad = warp & 3, h = warp >> 2;  // lane quarter, token half
    const int r = quad * 32 + lane;            // vector of the block
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const float c = p.sm_scale * (FP8 ? __ldg(p.kv_scale) : 1.f) * kLog2e;
    float* red = reinterpret_cast<float*>(smem + RG::S_RED);
    const uint32_t p_peer = tc::map_peer(smem_u32(smem), 1);
    const uint32_t a_peer = tc::map_peer(smem_u32(smem + OFF_MISC), 1);
    const uint32_t bar_peer = tc::map_peer(smem_u32(&p_full[0]), 1);
    // The meeting of the two warps of a quarter; one that gave up passes false
    // and both leave.
    auto meet = [&](bool good) -> bool { return named_bar_and(1 + quad, 64, good); };
    int n = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      // ---- Q: this vector's half of the latent dims into TMEM, of the rope dims
      // into the swizzled box, once the last segment's products have read theirs
      bool good = k == 0 || warp_wait(q_free, (k - 1) & 1);
      const bool live = r < sg.vecs;
      if (good) {
        tc::fence_after_sync();
        const int vec = sg.vec0 + r;
        const int row = live ? sg.row0 + vec / H : 0, hd = live ? vec % H : 0;
        const uint16_t* qn = p.q + row * p.q_row_stride + hd * p.q_head_stride + h * (R / 2);
        const uint16_t* qp = p.q_pe + row * p.q_pe_row_stride + hd * p.q_pe_head_stride + h * 32;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        uint4 pe[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) pe[j] = live ? __ldg(reinterpret_cast<const uint4*>(qp) + j) : zero;
#pragma unroll 2
        for (int d = 0; d < R / 128; ++d) {
          uint32_t x[32];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 y = live ? __ldg(reinterpret_cast<const uint4*>(qn + d * 64) + j) : zero;
            x[4 * j] = y.x;
            x[4 * j + 1] = y.y;
            x[4 * j + 2] = y.z;
            x[4 * j + 3] = y.w;
          }
          tc::st_32x32b_x32(tmem + lanes + h * (R / 4) + d * 32, x);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint4*>(smem + S_QPE + sw128(r, h * 4 + j)) = pe[j];
        tc::wait_st();
        tc::fence_before_sync();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < tiles; ++t, ++n) {
        const int b = n & 1;
        const uint32_t par = (n >> 1) & 1;
        uint32_t s[64];
        float mt = -INFINITY;
        if (good && warp_wait(&s_full[b], par)) {
          tc::fence_after_sync();
          const uint32_t col = tmem + lanes + S_COL + b * TT + h * 64;
          tc::ld_32x32b_x32(col, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
          tc::ld_32x32b_x32(col + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
          tc::wait_ld();
          tc::reg_fence(s);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[b]);
          const int left = sg.tok1 - (sg.tok0 + t * TT) - h * 64;  // tokens of this half
          float mx[4] = {mt, mt, mt, mt};
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * c);
          if (left < 64) {
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (j >= left) s[j] = 0xFF800000u;  // -inf
          }
#pragma unroll
          for (int j = 0; j < 64; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(s[j]));
          mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // the P buffer's last tile has been read by rank 1
          if (n >= 2 && !warp_wait_cluster(&p_free[b], par ^ 1)) good = false;
        } else {
          good = false;
        }
        // ---- the vector's maximum over both halves (by tile parity: the other
        // warp reads this tile's value before either writes the one after next's)
        float* rp = red + b * 256;
        rp[h * 128 + r] = mt;
        if (!meet(good)) {
          ok = false;
          break;
        }
        const float m_new = fmaxf(m, fmaxf(rp[r], rp[128 + r]));
        // O is rescaled only when the maximum has grown by more than 2^8
        float alpha = 1.f;
        if (m_new > m + kRescaleAt) {
          if (t > 0) alpha = ex2(m - m_new);
          l *= alpha;
          m = m_new;
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t dst = p_peer + b * kPBuf + h * 16384, bar = bar_peer + b * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = ex2(__uint_as_float(s[8 * j + 2 * e]) - m);
            const float a1 = ex2(__uint_as_float(s[8 * j + 2 * e + 1]) - m);
            sum[e] += a0 + a1;
            w[e] = pack_bf16x2(a0, a1);
          }
          tc::st_async_v4u(dst + sw128(r, j), w[0], w[1], w[2], w[3], bar);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        if (h == 0) tc::st_async_b32(a_peer + b * 512 + r * 4, __float_as_uint(alpha), bar);
      }
      if (!ok) break;
      // ---- the segment's maximum and sum
      if (!meet(good)) {
        ok = false;
        break;
      }
      float* rl = red;
      if (h == 1) rl[r] = l;
      meet(true);
      if (h == 0 && live)
        p.ml[static_cast<int64_t>(mine.x + k) * 128 + r] = make_float2(m, l + rl[r]);
      meet(true);
    }
    // rank 1's last arrivals here have landed before this CTA can leave
    for (int j = 1; j <= 2 && ok; ++j)
      if (n >= j) ok = warp_wait_cluster(&p_free[(n - j) & 1], ((n - j) >> 1) & 1);
  } else {
    // ------------------------------------------------------ O of rank 1
    const int quad = warp & 3, h = warp >> 2;  // lane quarter, half of the dims
    const int r = quad * 32 + lane;
    const uint32_t o_col = tmem + (static_cast<uint32_t>(quad * 32) << 16) + h * (R / 2);
    const float* factors = reinterpret_cast<const float*>(smem + OFF_MISC);
    int n = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      for (int t = 0; t < tiles && ok; ++t, ++n) {
        const int b = n & 1;
        ok = warp_wait_cluster(&p_full[b], (n >> 1) & 1);
        if (!ok) break;
        const float alpha = factors[b * 128 + r];
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&p_full[b], kPBuf + 512);  // the next use
        if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          ok = warp_wait(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int q = 0; q < R / 2; q += 32) {
            uint32_t o[32];
            tc::ld_32x32b_x32(o_col + q, o);
            tc::wait_ld();
            tc::reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st_32x32b_x32(o_col + q, o);
          }
          tc::wait_st();
        }
        fence_proxy_async_smem();  // P, written by rank 0, is the product's operand
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_ready[b]);
      }
      if (!ok) break;
      // ---- the segment's O
      ok = warp_wait(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1);
      if (!ok) break;
      tc::fence_after_sync();
      float* dst = p.partial + (static_cast<int64_t>(mine.x + k) * 128 + r) * R + h * (R / 2);
#pragma unroll 1
      for (int q = 0; q < R / 2; q += 32) {
        uint32_t o[32];
        tc::ld_32x32b_x32(o_col + q, o);
        tc::wait_ld();
        tc::reg_fence(o);
        if (r < sg.vecs) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + q + e),
                         "r"(o[e]), "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]),
                         "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                         : "memory");
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }
  if (!ok && lane == 0) gave_up(p.err_count);

  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer's buffers and barriers are used to the end
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// One warp for each vector: the segments of its sequence's part and of its
// group's, weighted by their maxima.  Lane j finds segment j; the outputs of a
// few are in flight together.
constexpr int kJoinWarps = 8;
constexpr int kInFlight = 4;

template <int R>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(const SharedParams p) {
  constexpr int NV = R / 128;  // float4 groups a lane
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t vec = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  const int H = p.num_heads;
  if (vec >= static_cast<int64_t>(p.num_rows) * H) return;
  const int row = static_cast<int>(vec / H);
  const int C = p.header[0];
  SharedPart part[2];
  part[0] = p.parts[p.num_groups + row / p.rows_per_seq];
  const bool two = part[0].group >= 0;
  part[1] = p.parts[two ? part[0].group : 0];
  int block[2], at[2], items[2], span[2];  // slots to look at: chunks x pairs a chunk can meet
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int v = static_cast<int>(vec - static_cast<int64_t>(part[i].row0) * H);
    block[i] = v >> 7;
    at[i] = v & 127;
    const bool any = part[i].blocks > 0 && (i == 0 || two);
    span[i] = part[i].blocks == 1 ? cdiv(part[i].tiles, C) + 1 : 2;
    items[i] = any ? cdiv(part[i].tiles, chunk_tiles(part[i], C)) * span[i] : 0;
  }
  const int n = items[0] + items[1];
  // record (slot * 128 + vector) of item i, or -1
  auto record = [&](int i) -> int64_t {
    if (i >= n) return -1;
    const int w = i >= items[0];
    const SharedPart& x = w ? part[1] : part[0];
    const int k = w ? i - items[0] : i, sp = w ? span[1] : span[0];
    const int g = w ? block[1] : block[0], ch = chunk_tiles(x, C);
    const int j = k / sp, len = min(ch, x.tiles - j * ch);
    const int first = x.tile0 + j * ch * x.blocks + g * len;
    const int c = first / C + (k - j * sp);
    if (static_cast<int64_t>(c) * C >= first + len) return -1;
    return static_cast<int64_t>(x.unit0 + j * x.blocks + g + c) * 128 + (w ? at[1] : at[0]);
  };
  int64_t rec = record(lane);
  float2 ml = rec >= 0 ? p.ml[rec] : make_float2(-INFINITY, 0.f);
  float M = ml.x;
  for (int i = lane + 32; i < n; i += 32) {
    const int64_t x = record(i);
    if (x >= 0) M = fmaxf(M, p.ml[x].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float4 acc[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    if (i0 > 0) {
      rec = record(i0 + lane);
      ml = rec >= 0 ? p.ml[rec] : make_float2(-INFINITY, 0.f);
    }
    const float w = rec >= 0 ? ex2(ml.x - M) : 0.f;
    den += w * ml.y;
    uint32_t mask = __ballot_sync(0xffffffffu, rec >= 0);
    while (mask) {
      int js[kInFlight];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        js[u] = mask ? __ffs(mask) - 1 : -1;
        mask &= mask ? mask - 1 : 0u;
      }
      float4 v[kInFlight][NV];
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const int64_t x = __shfl_sync(0xffffffffu, rec, js[u] < 0 ? 0 : js[u]);
        if (js[u] < 0) continue;
        const float4* src = reinterpret_cast<const float4*>(p.partial + x * R);
#pragma unroll
        for (int k = 0; k < NV; ++k) v[u][k] = src[k * 32 + lane];
      }
#pragma unroll
      for (int u = 0; u < kInFlight; ++u) {
        const float wj = __shfl_sync(0xffffffffu, w, js[u] < 0 ? 0 : js[u]);
        if (js[u] < 0) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          acc[k].x += wj * v[u][k].x;
          acc[k].y += wj * v[u][k].y;
          acc[k].z += wj * v[u][k].z;
          acc[k].w += wj * v[u][k].w;
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
  const float inv = n == 0 ? 0.f : (p.kv_scale ? __ldg(p.kv_scale) : 1.f) / den;
  uint2* o = reinterpret_cast<uint2*>(p.o + vec * R);
#pragma unroll
  for (int k = 0; k < NV; ++k)
    o[k * 32 + lane] = make_uint2(pack_bf16x2(acc[k].x * inv, acc[k].y * inv),
                                  pack_bf16x2(acc[k].z * inv, acc[k].w * inv));
  if (lane == 0) p.lse[vec] = n == 0 ? -INFINITY : (M + log2f(den)) * kLn2;
}

size_t align_up(size_t x) { return (x + 255) & ~size_t{255}; }

template <int R, bool FP8>
cudaError_t launch_main(const SharedParams& p, const CUtensorMap& tmap, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(decode_shared_kernel<R, FP8>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_shared_kernel<R, FP8>, dim3(2 * p.pairs), dim3(FP8 ? 448 : 320),
                           kSmem, stream, p, tmap);
}

}  // namespace

// Units are at most one more for each block than the pairs' shares, and a unit
// meets each further pair in one more segment.
size_t shared_layout(int num_rows, int num_heads, int num_seqs, int num_groups, int R, int pairs,
                     uint8_t* base, SharedParams* p) {
  const int64_t vecs = static_cast<int64_t>(num_rows) * num_heads;
  const int64_t own = static_cast<int64_t>(num_seqs) *
                      ((static_cast<int64_t>(num_rows / num_seqs) * num_heads + 127) / 128);
  const int64_t blocks = own + vecs / 128 + num_groups;
  const size_t slots = static_cast<size_t>(blocks + 2 * pairs + 1);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base ? base + at : nullptr;
    at += align_up(bytes);
    return q;
  };
  uint8_t* header = take(64 * sizeof(int));
  uint8_t* pair_segments = take(pairs * sizeof(int2));
  uint8_t* parts = take((static_cast<size_t>(num_groups) + num_seqs) * sizeof(SharedPart));
  uint8_t* segments = take(slots * sizeof(SharedSegment));
  uint8_t* ml = take(slots * 128 * sizeof(float2));
  uint8_t* partial = take(slots * 128 * sizeof(float) * R);
  if (p) {
    p->header = reinterpret_cast<int*>(header);
    p->pair_segments = reinterpret_cast<int2*>(pair_segments);
    p->parts = reinterpret_cast<SharedPart*>(parts);
    p->segments = reinterpret_cast<SharedSegment*>(segments);
    p->ml = reinterpret_cast<float2*>(ml);
    p->partial = reinterpret_cast<float*>(partial);
  }
  return at;
}

cudaError_t launch_decode_shared(const SharedParams& p, const CUtensorMap& tmap, int R, bool fp8,
                                 cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr int kMostSmem = (3 * (kMaxSharedGroups + 1) + 2 * (kMaxSharedGroups + kMaxSharedSeqs + 1)) * 4;
  static_assert(kMostSmem <= 226 * 1024, "the schedule's shared memory");
  cudaError_t e = set_smem_attr_once(shared_schedule_kernel, kMostSmem, attr_done);
  if (e != cudaSuccess) return e;
  const int G = p.num_groups, V = G + p.num_seqs;
  const size_t smem = (3 * static_cast<size_t>(G + 1) + 2 * static_cast<size_t>(V + 1)) * 4;
  e = launch_overlapped(shared_schedule_kernel, dim3(1), dim3(1024), smem, stream, p);
  if (e != cudaSuccess) return e;
  if (R == 512)
    e = fp8 ? launch_main<512, true>(p, tmap, stream) : launch_main<512, false>(p, tmap, stream);
  else
    e = fp8 ? launch_main<256, true>(p, tmap, stream) : launch_main<256, false>(p, tmap, stream);
  if (e != cudaSuccess) return e;
  const int64_t vecs = static_cast<int64_t>(p.num_rows) * p.num_heads;
  const dim3 grid(static_cast<unsigned>((vecs + kJoinWarps - 1) / kJoinWarps));
  return R == 512 ? launch_overlapped(shared_join_kernel<512>, grid, dim3(kJoinWarps * 32), 0,
                                      stream, p)
                  : launch_overlapped(shared_join_kernel<256>, grid, dim3(kJoinWarps * 32), 0,
                                      stream, p);
}

}  // namespace mla
