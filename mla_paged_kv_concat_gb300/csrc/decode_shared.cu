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
//   rank 0: Q R / 2 + S 2 x 128 TMEM columns; a ring of 11 boxes of 16 KiB (64 dims
//     x 128 tokens of K or 128 vectors of Q), 32 KiB of P on its way
//   rank 1: O R TMEM columns; P 2 x 32 KiB; a ring of five 32 KiB boxes of V (256
//     dims x 64 tokens)
// An fp8 cache lands in staging boxes and two groups of four warps of each CTA turn
// it into the bf16 boxes (on rank 0 one of them also loads Q); its values are exact in
// bf16, and the scale is applied to the scores and to the joined output.
//
// Schedule.  A first kernel (one CTA) turns the lengths into a list of all tiles: the
// groups' prefixes, then the sequences, each cut into blocks of 128 vectors.  Blocks
// of one prefix are listed in chunks side by side, so that pairs at work together
// read the same rows.  A unit (chunk of a block) has kStart places in the list
// before its tiles, for what its start and end take, and pair c of CTAs has the
// places [c C, (c + 1) C).  Unit u meets pair c in segment u + c, which is also its
// place in the workspace: list positions only grow, so no two are alike.
//
// Measured on GB300, one call out of a graph, and what bounds it:
//   128 sequences, 128 heads, three prefixes, bf16, R = 512   319 us  1.10 PFLOP/s: a tile
//       of 128 x 128 takes 1.76 us on rank 0, its 36 products 95 cycles each for 74 alone.
//       What holds them is not shown: the busiest SM's tensor pipe is 58 % and its tensor
//       memory 61 % busy, shared memory's operand reads 34 % on average
//   64 sequences behind 8192 tokens, 16 heads, bf16, R = 512   53.6  12 tiles a pair; lists
//       5, start and Q 5, O 4, join 8
//   45 sequences, 32 heads, two prefixes, E4M3, R = 256        57.0  conversion on rank 0,
//       2.1 us a tile
//   33 sequences of two rows behind 4097, 16 heads, E5M2, 512  47.4  the same, 3.3 us a tile
//   4 sequences behind 512, 16 heads, bf16, R = 512            22.5  three dependent kernels:
//       lists 4.3, start and Q 4.7, a tile 5, O 2, join 5
// The plain decode takes 408, 89, 84, 69 and 12.4 us on these.  It is the faster one
// where the tokens of all sequences together are few: with 16 heads about 150 thousand of
// a bf16 cache, 35 to 100 thousand of an fp8 one.  128 heads fill the 128 vectors alone, and
// sharing saves cache reads, no products: 64 sequences behind 4096 tokens 113 us against
// 112, with an E4M3 cache 138 against 410 (R = 512) and 93 against 75 (R = 256).
//
// Roles (384 threads, 512 with an fp8 cache): rank 0 warps 0-3 softmax, thread =
// TMEM lane = vector, 4-7 loading Q; rank 1 warps 0-7 rescaling and output of O, two
// a lane quarter (dim halves); warp 9 MMA, warps 8, 10, 11 TMA.  With an fp8 cache 8,
// 14, 15 TMA, 4-7 (besides Q) and 10-13 conversion, rank 1's output warps 0-3 alone.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int TT = 128;                 // tokens of a tile
constexpr int kKBox = 16384;            // rank 0's ring box: 64 dims x 128 tokens (or vectors)
constexpr int kVBox = 32768;            // rank 1's: 256 dims x 64 tokens
constexpr int kPBuf = 32768;            // P: two boxes of 128 vectors x 64 tokens
// Shared memory of rank 0 and rank 1.
constexpr int S_QPE = 0;
constexpr int S_OUT = S_QPE + kKBox;    // P on its way to rank 1, 8 KiB a warp
constexpr int S_RING = S_OUT + kPBuf;
constexpr int V_RING = 2 * kPBuf;
constexpr int kData = 229376;
constexpr int OFF_MISC = kData;         // rank 1: rescale factors, two buffers of 128
constexpr int OFF_BAR = OFF_MISC + 1024;
constexpr int OFF_TMEM = OFF_BAR + 512;
constexpr int kSmem = OFF_TMEM + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr int kMostBoxes = 11, kMostStages = 6;
template <bool FP8>
struct Ring {
  static constexpr int S_BOXES = FP8 ? 8 : 11, V_BOXES = FP8 ? 3 : 5;
  // fp8 staging boxes: 8 KiB on rank 0, 16 KiB on rank 1
  static constexpr int S_STAGES = FP8 ? 6 : 0, V_STAGES = FP8 ? 4 : 0;
  static constexpr int S_STAGE = S_RING + S_BOXES * kKBox;
  static constexpr int V_STAGE = V_RING + V_BOXES * kVBox;
  static_assert(S_STAGE + S_STAGES * 8192 <= kData, "rank 0's shared memory");
  static_assert(V_STAGE + V_STAGES * 16384 <= kData, "rank 1's shared memory");
  static_assert(S_BOXES <= kMostBoxes && S_STAGES <= kMostStages, "barriers");
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
// Packed fp32 pairs.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void mul2(uint32_t& a, uint32_t& b, float c) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(pack2(__uint_as_float(a), __uint_as_float(b))), "l"(pack2(c, c)));
  float x, y;
  unpack2(d, x, y);
  a = __float_as_uint(x);
  b = __float_as_uint(y);
}
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity) {
  const bool ok = tc::mbar_wait_cluster(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// ---------------------------------------------------------------- schedule
// Sum over the CTA, and inclusive sums of a[0, n) in place; `tot`: 32 shared values.
__device__ __forceinline__ int cta_sum(int v, int64_t* tot) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) tot[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) v += static_cast<int>(tot[w]);
  return v;
}
__device__ __forceinline__ void cta_scan(int64_t* a, int n, int64_t* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t carry = 0;
  for (int base = 0; base < n; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int64_t v = i < n ? a[i] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += t;
    }
    __syncthreads();
    if (lane == 31) tot[warp] = v;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
      if (w == warp) v += all;
      all += tot[w];
    }
    if (i < n) a[i] = v + carry;
    carry += all;
  }
  __syncthreads();
}

// Places that a unit has in the list before its tiles.  Measured (us, 1 / 2 / 3, the
// first four batches of the header): 338 / 317 / 317, 55.7 / 53.6 / 54.9, 58.4 / 57.0 /
// 57.2, 53.9 / 47.4 / 47.8.
constexpr int kStart = 2;

// Tiles of a unit of a part: chunks, or all where a single block has nobody beside it
// to read the same rows.  Up to 16 tiles of such a block go to a pair each where there are
// pairs to spare (chunks of one tile): joining a piece costs 0.3 us, a tile 1.9 (us, all
// together / one by one: four sequences behind 512 tokens 24.5 / 22.3, eight behind 1024
// 28.4 / 26.8, behind 4096 32.5 / 38.3).
__device__ __forceinline__ int unit_tiles(int blocks, int tiles, int chunk) {
  const bool whole = blocks == 1 && (chunk > 1 || tiles > 16);
  return whole || tiles < chunk ? tiles : chunk;
}

// The lists in shared memory (free again afterwards).
struct Lists {
  int64_t* before;    // [V + 1] places (low half) and units before a part: groups, then sequences
  int *tok0, *tok1;   // [V] a part's tokens
  int *ends, *lead;   // [G + 1] first sequence of each group; [G] the one whose table is read
  int* prefix;        // [G] all of a prefix: who takes part has it to the end
  int* group;         // [B] the group whose shared part a sequence takes part in, or -1
};

// The list; returns (tiles of a chunk, places of a pair).
__device__ __forceinline__ int2 make_list(const SharedParams& p, const Lists& lists, int64_t* tot) {
  const int G = p.num_groups, B = p.num_seqs, V = G + B;
  int64_t* before = lists.before;
  int *tok0 = lists.tok0, *tok1 = lists.tok1, *ends = lists.ends, *lead = lists.lead;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = p.rows_per_seq * p.num_heads;  // vectors of a sequence
  // first sequences that do not decrease, whatever the caller gave
  if (warp == 0) {
    int carry = 0;
    for (int base = 0; base <= G; base += 32) {
      int v = base + lane <= G ? ends[base + lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, d));
      v = max(v, carry);
      if (base + lane <= G) ends[base + lane] = v;
      carry = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  // what the sequences of a group can share, when there are two at least
  for (int g = warp; g < G; g += static_cast<int>(blockDim.x >> 5)) {
    const int n = lists.prefix[g];
    int count = 0, first = B;
    for (int b = ends[g] + lane; b < ends[g + 1]; b += 32)
      if (tok1[G + b] >= n) {
        ++count;
        first = min(first, b);
      }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      count += __shfl_xor_sync(0xffffffffu, count, d);
      first = min(first, __shfl_xor_sync(0xffffffffu, first, d));
    }
    __syncwarp();
    if (lane == 0) {
      if (count < 2) tok1[g] = 0;
      lead[g] = first;
    }
  }
  __syncthreads();
  // the group whose shared part sequence b takes part in, or -1
  auto group_of = [&](int b) {
    int a = 0, z = G;  // the last group that starts at or before b
    while (a < z) {
      const int m = (a + z + 1) >> 1;
      if (ends[m] <= b) a = m; else z = m - 1;
    }
    return a < G && b >= ends[a] && tok1[a] > 0 && tok1[G + b] >= lists.prefix[a] ? a : -1;
  };
  auto blocks_of = [&](int v) {
    return tok1[v] <= tok0[v] ? 0 : cdiv(v < G ? (ends[v + 1] - ends[v]) * per : per, 128);
  };
  auto tiles_of = [&](int v) { return cdiv(tok1[v] - tok0[v], TT); };
  int all_tiles = 0;
  for (int v = static_cast<int>(threadIdx.x); v < V; v += static_cast<int>(blockDim.x)) {
    if (v >= G) {
      const int g = group_of(v - G);
      lists.group[v - G] = g;
      tok0[v] = g < 0 ? 0 : tok1[g];
    }
    all_tiles += tiles_of(v) * blocks_of(v);
  }
  const int tiles = cta_sum(all_tiles, tot);  // at most 2^30
  // Chunks of a pair's share, which with its start is the share itself where that
  // comes out (found in a few steps: larger chunks are fewer starts).
  const int least = max(1, cdiv(tiles, p.pairs));
  int chunk = least, C = 1;
  for (int step = 0; step < 3; ++step) {
    int all_units = 0;
    for (int v = static_cast<int>(threadIdx.x); v < V; v += static_cast<int>(blockDim.x)) {
      const int n = blocks_of(v), t = tiles_of(v);
      if (n > 0) all_units += n * cdiv(t, unit_tiles(n, t, chunk));
    }
    C = max(1, cdiv(tiles + kStart * cta_sum(all_units, tot), p.pairs));
    const int next = max(least, C - kStart);
    if (next <= chunk || step == 2) break;
    chunk = next;
  }
  C = max(C, chunk + kStart);
  for (int v = static_cast<int>(threadIdx.x); v < V; v += static_cast<int>(blockDim.x)) {
    const int n = blocks_of(v), t = tiles_of(v);
    const int64_t units = n == 0 ? 0 : n * cdiv(t, unit_tiles(n, t, chunk));
    before[v + 1] = units << 32 | static_cast<int64_t>(t * n + kStart * units);
  }
  if (threadIdx.x == 0) before[0] = 0;
  __syncthreads();
  cta_scan(before + 1, V, tot);
  return make_int2(chunk, C);
}

// Segments of pair c: walks its places of the list.
__device__ __forceinline__ void walk(const SharedParams& p, const Lists& l, int chunk, int C, int c) {
  const int G = p.num_groups, V = G + p.num_seqs;
  const int per = p.rows_per_seq * p.num_heads;
  auto places = [&](int v) { return static_cast<int>(l.before[v] & 0xFFFFFFFF); };
  const int total = places(V);
  const int64_t lo64 = static_cast<int64_t>(c) * C;
  const int lo = lo64 < total ? static_cast<int>(lo64) : total;
  const int hi = total - lo > C ? lo + C : total;
  int a = 0, z = V - 1;  // the last part that starts at or before lo
  while (a < z) {
    const int m = (a + z + 1) >> 1;
    if (places(m) <= lo) a = m; else z = m - 1;
  }
  int2 mine = make_int2(0, 0);
  int t = lo;
  for (int v = a; t < hi; ++v) {
    const int end = places(v + 1);
    if (end <= t) continue;
    const int start = places(v), unit0 = static_cast<int>(l.before[v] >> 32);
    const int vecs = v < G ? (l.ends[v + 1] - l.ends[v]) * per : per, blocks = cdiv(vecs, 128);
    const int tiles = cdiv(l.tok1[v] - l.tok0[v], TT);
    const int ch = unit_tiles(blocks, tiles, chunk);
    const int whole = (ch + kStart) * blocks;  // places of a whole chunk
    while (t < hi && t < end) {
      const int in = t - start;
      const int j = in / whole;
      const int len = min(ch, tiles - j * ch);
      const int y = in - j * whole;
      const int g = y / (len + kStart), k = y - g * (len + kStart);  // place of the unit
      const int n = min(len + kStart - k, hi - t);
      const int k0 = max(k - kStart, 0), k1 = k + n - kStart;  // its tiles here
      if (k1 > k0) {
        SharedSegment s;
        s.table = v < G ? l.lead[v] : v - G;
        s.row0 = (v < G ? l.ends[v] : v - G) * p.rows_per_seq;
        s.vec0 = g * 128;
        s.vecs = min(128, vecs - g * 128);
        s.tok0 = l.tok0[v] + (j * ch + k0) * TT;
        s.tok1 = min(l.tok1[v], s.tok0 + (k1 - k0) * TT);
        s.pad0 = s.pad1 = 0;
        const int slot = unit0 + j * blocks + g + c;
        p.segments[slot] = s;
        if (mine.y == 0) mine.x = slot;
        ++mine.y;
      }
      t += n;
    }
  }
  p.pair_segments[c] = mine;
}

// What the join needs for sequence b.
__device__ __forceinline__ void fill_row(const SharedParams& p, const Lists& l, int chunk, int C,
                                         int b) {
  const int G = p.num_groups, per = p.rows_per_seq * p.num_heads;
  auto place = [&](int v) {
    SharedPlace x;
    x.first = static_cast<int>(l.before[v] & 0xFFFFFFFF);
    x.tiles = cdiv(l.tok1[v] - l.tok0[v], TT);
    x.blocks = x.tiles <= 0 ? 0 : cdiv(v < G ? (l.ends[v + 1] - l.ends[v]) * per : per, 128);
    x.chunk = x.blocks == 0 ? 1 : unit_tiles(x.blocks, x.tiles, chunk);
    x.unit0 = static_cast<int>(l.before[v] >> 32);
    x.row0 = (v < G ? l.ends[v] : v - G) * p.rows_per_seq;
    return x;
  };
  const int g = l.group[b];
  SharedRow x;
  x.own = place(G + b);
  x.group = place(g < 0 ? 0 : g);
  if (g < 0) x.group.blocks = 0;
  x.per_pair = C;
  x.pad = 0;
  p.rows[b] = x;
}

// One CTA.  (The same in every CTA of the main kernel instead saved its launch but
// not its time: 53 us for 56, and 25 for 23 in a short step.)
__global__ void __launch_bounds__(1024) shared_schedule_kernel(const SharedParams p) {
  extern __shared__ int64_t list_sm[];
  const int G = p.num_groups, B = p.num_seqs, V = G + B;
  Lists l;
  l.before = list_sm;
  int64_t* tot = l.before + V + 1;
  l.tok0 = reinterpret_cast<int*>(tot + 32);
  l.tok1 = l.tok0 + V;
  l.ends = l.tok1 + V;
  l.lead = l.ends + G + 1;
  l.prefix = l.lead + G;
  l.group = l.prefix + G;
  griddep_wait();
  griddep_launch_dependents();
  for (int g = threadIdx.x; g <= G; g += blockDim.x)
    l.ends[g] = clampi(__ldg(p.group_seqs + g), 0, B);
  for (int g = threadIdx.x; g < G; g += blockDim.x) {
    const int n = __ldg(p.prefix_lens + g);
    l.tok0[g] = 0;
    l.prefix[g] = clampi(n, 0, p.capacity);
    l.tok1[g] = l.prefix[g] & ~(TT - 1);
    if ((n < 0 || n > p.capacity) && p.err_count) atomicAdd(p.err_count, 1);
  }
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int n = __ldg(p.seq_lens + b);
    l.tok1[G + b] = clampi(n, 0, p.capacity);
    if ((n < 0 || n > p.capacity) && p.err_count) atomicAdd(p.err_count, 1);
  }
  __syncthreads();
  const int2 found = make_list(p, l, tot);
  // the pairs' segments by the first threads, the sequences' rows by the last
  for (int c = threadIdx.x; c < p.pairs; c += blockDim.x) walk(p, l, found.x, found.y, c);
  for (int b = blockDim.x - 1 - threadIdx.x; b < B; b += blockDim.x)
    fill_row(p, l, found.x, found.y, b);
}

size_t schedule_smem(int G, int V) {
  return (static_cast<size_t>(V) + 1 + 32) * 8 + (3 * static_cast<size_t>(V) + 2 * G + 1) * 4;
}

// ---------------------------------------------------------------- conversion
// A thread's part (t of 128) of an 8 KiB staging box, rows of 64 codes, to bf16
// (exactly) in swizzled 128-byte rows: four pieces of 16 codes.  Alone on an SM two
// groups of four warps take 270 cycles a box, 232 of them what loading 8 and storing
// 16 KiB takes; beside the other roles 400 to 450, of which a third are waits, fence and
// arrivals.  One piece at a time, the least code: with two the E4M3 batch of the header
// took 62.6 us for 61.0, with four 68.8.  (Moving the bits with integer operations
// instead of the conversion instructions: 330 to 530 cycles; the next box's codes asked
// for under this one's stores: 59.9 us for 57.5.)
template <bool E5M2>
__device__ __forceinline__ void convert_box(const uint8_t* src, uint8_t* dst, int t) {
  uint8_t* const d0 = dst + sw128(t >> 2, (t & 3) * 2);
  uint8_t* const d1 = dst + sw128(t >> 2, (t & 3) * 2 + 1);
#pragma unroll 1
  for (int at = t; at < 512; at += 128) {
    const uint4 raw = *reinterpret_cast<const uint4*>(src + at * 16);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t two = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) * 16));
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, E5M2 ? __NV_E5M2 : __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      o[e] = pack_bf16x2(f.x, f.y);
    }
    *reinterpret_cast<uint4*>(d0 + (at - t) * 32) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(d1 + (at - t) * 32) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// ---------------------------------------------------------------- main kernel
template <int R, bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FP8 ? 512 : 384, 1)
    decode_shared_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tmap) {
  using RG = Ring<FP8>;
  constexpr int NQ = R / 64;    // boxes of the latent dims: of Q, and of K a tile
  constexpr int VB = R / 256;   // 256-dim parts of O
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  // The same places in both CTAs; each uses its own.
  uint64_t* full = bars;                      // [kMostBoxes] ring box landed (converted)
  uint64_t* empty = full + kMostBoxes;        // [kMostBoxes]
  uint64_t* st_full = empty + kMostBoxes;     // [kMostStages] fp8 staging box landed
  uint64_t* st_empty = st_full + kMostStages; // [kMostStages]
  uint64_t* s_full = st_empty + kMostStages;  // [2] rank 0: S of a tile of this parity
  uint64_t* s_free = s_full + 2;              // [2] rank 0: S read
  uint64_t* q_full = s_free + 2;              // rank 0: the segment's Q is in place
  uint64_t* q_free = q_full + 1;              // rank 0: the segment's last Q K^T is done
  uint64_t* p_free = q_free + 1;              // [2] rank 0: P buffer read by rank 1's products
  uint64_t* p_full = p_free + 2;              // [2] rank 1: P and rescale factors landed
  uint64_t* o_ready = p_full + 2;             // [2] rank 1: O rescaled for this tile's P
  uint64_t* pv_done = o_ready + 2;            // [2] rank 1
  uint64_t* o_free = pv_done + 2;             // rank 1: the segment's O has been read out
  uint64_t* seg_filled = o_free + 1;          // rank 0: the segment's last K box has been filled
  static_assert((2 * kMostBoxes + 2 * kMostStages + 16) * 8 <= 512, "barriers");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);

  const uint32_t rank = tc::cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmap);
    for (int i = 0; i < kMostBoxes; ++i) {
      mbar_init(&full[i], FP8 ? 4 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kMostStages; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_free[i], 1);
      mbar_init(&p_full[i], 1);
      mbar_init(&o_ready[i], FP8 ? 4 : 8);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 4);
    mbar_init(q_free, 1);
    mbar_init(o_free, FP8 ? 4 : 8);
    mbar_init(seg_filled, FP8 ? 4 : 3);
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
  // ---------------------------------------------------- producer
  auto produce = [&]() {
    // Three warps share the boxes of the ring: one, at 0.28 us a box, did not keep
    // up.  Lane l loads page l of a K box, page l % 4 and 64-dim part l / 4 of a V
    // box.  Page ids are read one tile before they are used.
    const int which = warp == 8 ? 0 : FP8 ? warp - 13 : warp - 9;
    const int pages = TT / box_rows;  // of a tile: 2, 4 or 8
    const int my_page = lane & 7;
    const int v_page = lane & 3, v_part = lane >> 2;
    constexpr int kRowBytes = FP8 ? 64 : 128;  // a row of a 64-dim part
    int nb = 0;  // position in the ring (fp8: of the staging boxes, where Q has none)
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int32_t* bt = p.block_table + static_cast<int64_t>(sg.table) * p.bt_stride;
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      auto id_of = [&](int t) -> int {
        const int tk = sg.tok0 + t * TT + my_page * box_rows;
        return my_page < pages && t < tiles && tk < sg.tok1 ? __ldg(bt + tk / bs) : 0;
      };
      int id = id_of(0);
      if (!FP8 && rank == 0) nb += NQ;  // the segment's Q comes first
      for (int t = 0; t < tiles && ok; ++t) {
        const int next = id_of(t + 1);
        const int tok = sg.tok0 + t * TT;
        const int have = min(pages, cdiv(sg.tok1 - tok, box_rows));  // pages to load
        if (rank == 0) {
          if (which == 0 && lane < have && (id < 0 || id >= p.num_blocks) && p.err_count)
            atomicAdd(p.err_count, 1);
          constexpr int N = FP8 ? RG::S_STAGES : RG::S_BOXES;
          const int row = (tok + my_page * box_rows) % bs;
          for (int c = 0; c <= NQ && ok; ++c, ++nb) {  // the last box: the rope part
            if (nb % 3 != which) continue;
            const int st = nb % N;
            ok = warp_wait(FP8 ? &st_empty[st] : &empty[st], ((nb / N) & 1) ^ 1);
            if (!ok) break;
            uint64_t* bar = FP8 ? &st_full[st] : &full[st];
            if (lane == 0)
              mbar_arrive_expect_tx(bar, static_cast<uint32_t>(have * box_rows * kRowBytes));
            __syncwarp();
            if (lane < have)
              tma_load_3d(smem + (FP8 ? RG::S_STAGE + st * 8192 : S_RING + st * kKBox) +
                              lane * box_rows * kRowBytes,
                          &tmap, bar, c * 64, row, id);
          }
        } else {
          constexpr int N = FP8 ? RG::V_STAGES : RG::V_BOXES;
          const int half = pages / 2;
          for (int e = 0; e < 2 && e * half < have && ok; ++e) {
            const int np = min(half, have - e * half);
            const int blk = __shfl_sync(0xffffffffu, id, e * half + v_page);
            const int row = (tok + (e * half + v_page) * box_rows) % bs;
            for (int d = 0; d < VB; ++d, ++nb) {
              // (with the two groups of converting warps a staging box's fillers and
              // readers have to be the same ones every time)
              if (nb % (FP8 ? 2 : 3) != which) continue;
              const int st = nb % N;
              ok = warp_wait(FP8 ? &st_empty[st] : &empty[st], ((nb / N) & 1) ^ 1);
              if (!ok) break;
              uint64_t* bar = FP8 ? &st_full[st] : &full[st];
              if (lane == 0)
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(4 * np * box_rows * kRowBytes));
              __syncwarp();
              if (v_page < np && v_part < 4)
                tma_load_3d(smem + (FP8 ? RG::V_STAGE + st * 16384 : V_RING + st * kVBox) +
                                (v_part * 64 + v_page * box_rows) * kRowBytes,
                            &tmap, bar, d * 256 + v_part * 64, row, blk);
            }
          }
        }
        id = next;
      }
      if (!FP8 && rank == 0 && ok) {
        // A ring barrier's parity tells no more than one use apart, and the next
        // segment's Q boxes, which others fill, lie between this warp's last box
        // and its next: it waits for its share of them to be free, too, and only
        // then says that it is done here, so that none is filled before.
        ok = warp_wait(q_full, k & 1);
        if (k + 1 < mine.y)
          for (int c = 0; c < NQ && ok; ++c)
            if ((nb + c) % 3 == which)
              ok = warp_wait(&empty[(nb + c) % RG::S_BOXES],
                             (((nb + c) / RG::S_BOXES) & 1) ^ 1);
        if (lane == 0) mbar_arrive(seg_filled);
      }
    }
  };
  // ---------------------------------------------------- conversion
  // `count` boxes from staging box ns and ring box nb on (behind Q's), every other
  // one for each of two groups of four warps (t of 128): 8 KiB, twice on rank 1, rows
  // of 64 codes one after the other in both (two 64-dim parts of 64 rows lie as one of
  // 128).  Positions and phases are counted on: divisions by the rank's own ring sizes
  // took 0.14 us a box.
  auto convert_boxes = [&](int count, int ns, int nb, int group, int t) -> bool {
    const int stages = FP8 ? (rank == 0 ? RG::S_STAGES : RG::V_STAGES) : 1;
    const int boxes = rank == 0 ? RG::S_BOXES : RG::V_BOXES;
    const int first = (ns ^ group) & 1;
    int st = (ns + first) % stages, bx = (nb + first) % boxes;
    uint32_t sp = ((ns + first) / stages) & 1, bp = (((nb + first) / boxes) & 1) ^ 1;
#pragma unroll 1
    for (int i = first; i < count; i += 2) {
      bool r = mbar_try_wait(&st_full[st], sp);
      r = mbar_try_wait(&empty[bx], bp) && r;
      if (!__all_sync(0xffffffffu, r)) {
        r = mbar_wait(&st_full[st], sp) && mbar_wait(&empty[bx], bp);
        if (!__all_sync(0xffffffffu, r)) return false;
      }
      const uint8_t* src = smem + (rank == 0 ? RG::S_STAGE + st * 8192 : RG::V_STAGE + st * 16384);
      uint8_t* dst = smem + (rank == 0 ? S_RING + bx * kKBox : V_RING + bx * kVBox);
#pragma unroll 1
      for (int c = 0; c < (rank == 0 ? 1 : 2); ++c) {
        if (p.e5m2)
          convert_box<true>(src + c * 8192, dst + c * 16384, t);
        else
          convert_box<false>(src + c * 8192, dst + c * 16384, t);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane < 2) mbar_arrive(lane == 0 ? &full[bx] : &st_empty[st]);
      st += 2;
      if (st >= stages) {
        st -= stages;
        sp ^= 1;
      }
      bx += 2;
      if (bx >= boxes) {
        bx -= boxes;
        bp ^= 1;
      }
    }
    return true;
  };
  auto box_count = [&](const SharedSegment& sg) {
    const int tokens = sg.tok1 - sg.tok0;
    return rank == 0 ? cdiv(tokens, TT) * (NQ + 1) : cdiv(tokens, 64) * VB;
  };
  // ------------------------------------------------------- Q K^T
  auto scores = [&]() {
    constexpr uint32_t idesc = tc::idesc_bf16(128, TT, 0, 0);
    const uint64_t dq = tc::smem_desc(smem_u32(smem + S_QPE), 16, 1024, tc::kLayoutSw128);
    const uint64_t ring =
        tc::smem_desc(smem_u32(smem + S_RING), 16, 1024, tc::kLayoutSw128);
    int n = 0, bx = 0;       // tile, ring box
    uint32_t phase = 0;      // of the box's barrier
    auto skip = [&](int boxes) {
      bx += boxes;
      if (bx >= RG::S_BOXES) {
        bx -= RG::S_BOXES;
        phase ^= 1;
      }
    };
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      skip(NQ);  // Q's boxes
      ok = warp_wait(q_full, k & 1);
      for (int t = 0; t < tiles && ok; ++t, ++n) {
        const uint32_t dS = tmem + S_COL + (n & 1) * TT;
        ok = warp_wait(&s_free[n & 1], ((n >> 1) & 1) ^ 1);
        if (!ok) break;
        // Two boxes for each wait, vote and issuing block: those cost about as much as
        // the four instructions of a box.  The latent parts' loop is not unrolled
        // (the roles' code shares the instruction caches).
#pragma unroll 1
        for (int c = 0; c < NQ && ok; c += 2) {
          const int b0 = bx;
          const uint32_t ph0 = phase;
          skip(1);
          const int b1 = bx;
          const uint32_t ph1 = phase;
          skip(1);
          bool r = mbar_try_wait(&full[b0], ph0);
          r = mbar_try_wait(&full[b1], ph1) && r;
          if (!__all_sync(0xffffffffu, r)) {
            r = mbar_wait(&full[b0], ph0) && mbar_wait(&full[b1], ph1);
            ok = __all_sync(0xffffffffu, r);
          }
          if (!ok) break;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint64_t d0 = ring + static_cast<uint64_t>(b0 * (kKBox >> 4));
            const uint64_t d1 = ring + static_cast<uint64_t>(b1 * (kKBox >> 4));
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_ts(dS, tmem + c * 32 + s * 8, d0 + static_cast<uint64_t>(s * 2), idesc,
                         (c > 0 || s > 0) ? 1u : 0u);
            tc::commit(&empty[b0]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tc::mma_ts(dS, tmem + c * 32 + 32 + s * 8, d1 + static_cast<uint64_t>(s * 2), idesc, 1u);
            tc::commit(&empty[b1]);
          }
          __syncwarp();
        }
        if (!ok) break;
        const int b0 = bx;
        ok = warp_wait(&full[b0], phase);
        skip(1);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {  // the rope part
          const uint64_t d0 = ring + static_cast<uint64_t>(b0 * (kKBox >> 4));
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tc::mma_ss(dS, dq + static_cast<uint64_t>(s * 2), d0 + static_cast<uint64_t>(s * 2), idesc,
                       1u);
          tc::commit(&empty[b0]);
          tc::commit(&s_full[n & 1]);
          if (t + 1 == tiles) tc::commit(q_free);
        }
        __syncwarp();
      }
    }
    // nothing of this CTA's still runs on the tensor core when TMEM is freed
    if (ok && mine.y > 0) ok = warp_wait(q_free, (mine.y - 1) & 1);
  };
  // --------------------------------------------------------- P V
  auto values = [&]() {
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
            uint8_t* box = smem + V_RING + bx * kVBox;
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
  };
  // ----------------------------------------------------------- Q
  auto load_q = [&](int k, const SharedSegment& sg, int nb, bool ok) -> bool {
    // The latent dims come through the K ring, as boxes of 64 dims x 128 vectors
    // that are asked for together (loaded row by row straight into TMEM they took
    // 8.7 us), and go on into TMEM; the rope dims stay in shared memory.
    const int tq = threadIdx.x - 128, r = tq;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    // This thread copies 16 bytes (dims 8 (tq % 8) on) of vectors tq / 8 + 16 j:
    // their rows, counted from the block's first (at most 128 of them: rows of the
    // batch times 128 do not fit 32 bits), and heads, -1 for vectors that there are
    // not, which become zeros.
    const int row_in = sg.vec0 / H, row0 = sg.row0 + row_in;
    int place[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int v = (tq >> 3) + 16 * j;
      const int vec = sg.vec0 - row_in * H + v;
      const int row = vec / H;
      place[j] = v < sg.vecs ? row * 128 + (vec - row * H) : -1;
    }
    auto nope = [&](int j) {
      const int64_t row = row0 + (place[j] >> 7), hd = place[j] & 127;
      return p.q + (place[j] < 0 ? 0 : row * p.q_row_stride + hd * p.q_head_stride) + (tq & 7) * 8;
    };
    auto rope = [&](int j) {
      const int64_t row = row0 + (place[j] >> 7), hd = place[j] & 127;
      return p.q_pe + (place[j] < 0 ? 0 : row * p.q_pe_row_stride + hd * p.q_pe_head_stride) +
             (tq & 7) * 8;
    };
    if (k > 0) {  // on their way into L2 while the last segment goes on
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (place[j] < 0) continue;
        if ((tq & 7) < NQ)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(nope(j) + (tq & 7) * 56));
        if ((tq & 7) == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(rope(j)));
      }
    }
    // the boxes before these have been filled, and those that wait for these to be
    // free have seen them so
    if (ok && k > 0) ok = warp_wait(seg_filled, (k - 1) & 1);
    for (int c = 0; c < NQ && ok; ++c) {
      const int bx = (nb + c) % RG::S_BOXES;
      ok = warp_wait(&empty[bx], (((nb + c) / RG::S_BOXES) & 1) ^ 1);
      if (!ok) break;
      const uint32_t dst = smem_u32(smem + S_RING) + bx * kKBox;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        cp_async16(dst + sw128((tq >> 3) + 16 * j, tq & 7), nope(j) + c * 64,
                   place[j] < 0 ? 0u : 16u);
    }
    // the last segment's products have read their Q
    if (ok && k > 0) ok = warp_wait(q_free, (k - 1) & 1);
    if (ok) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        cp_async16(smem_u32(smem + S_QPE) + sw128((tq >> 3) + 16 * j, tq & 7), rope(j),
                   place[j] < 0 ? 0u : 16u);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    ok = named_bar_and(1, 128, ok);  // the four warps leave together
    if (!ok) return false;
    tc::fence_after_sync();
#pragma unroll 2
    for (int c = 0; c < NQ; ++c) {
      const uint8_t* src = smem + S_RING + ((nb + c) % RG::S_BOXES) * kKBox;
      uint32_t x[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 y = *reinterpret_cast<const uint4*>(src + sw128(r, j));
        x[4 * j] = y.x;
        x[4 * j + 1] = y.y;
        x[4 * j + 2] = y.z;
        x[4 * j + 3] = y.w;
      }
      tc::st_32x32b_x32(tmem + lanes + c * 32, x);
    }
    tc::wait_st();
    tc::fence_before_sync();
    // the ring's barriers count these boxes as filled and read, too
    if (FP8 ? lane < NQ : tq < NQ) mbar_arrive(&full[(nb + lane) % RG::S_BOXES]);
    named_bar_sync(1, 128);
    // read, before anyone is told that Q is there
    if (tq < NQ) mbar_arrive(&empty[(nb + tq) % RG::S_BOXES]);
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    return true;
  };
  // Q (the four warps of group 1, on rank 0), and with an fp8 cache the conversion by
  // both groups: one call of each, since copies of the code would share the
  // instruction caches.
  auto fill = [&](int group) {
    const int t = threadIdx.x - (group == 1 ? 128 : 320);
    int ns = 0, nb = 0;  // positions among the staging boxes and in the ring
    const bool q = rank == 0 && group == 1;
    // (a warp of these whose wait gave up still meets the others at Q's barrier)
    for (int k = 0; k < mine.y && (ok || q); ++k) {
      const SharedSegment sg = segment(k);
      if (rank == 0) {
        // group 0 does not follow the segment's Q boxes, and waits until they have been
        // filled and read: a ring barrier's parity tells no more than one use apart
        ok = q ? load_q(k, sg, nb, ok) : warp_wait(q_full, k & 1);
        if (!ok) break;
        nb += NQ;
      }
      const int count = box_count(sg);
      if (FP8) ok = convert_boxes(count, ns, nb, group, t);
      ns += count;
      nb += count;
      if (FP8 && rank == 0 && group == 0 && lane == 0) mbar_arrive(seg_filled);
    }
  };
  // ----------------------------------------------------- softmax
  auto softmax = [&]() {
    const int r = threadIdx.x;  // vector of the block, TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const float c = p.sm_scale * (FP8 ? __ldg(p.kv_scale) : 1.f) * kLog2e;
    const uint32_t p_peer = tc::map_peer(smem_u32(smem), 1) + warp * 4096;
    const uint32_t a_peer = tc::map_peer(smem_u32(smem + OFF_MISC), 1) + r * 4;
    const uint32_t bar_peer = tc::map_peer(smem_u32(&p_full[0]), 1);
    uint8_t* out = smem + S_OUT + warp * 8192;  // 32 vectors x 64 tokens, twice
    int n = 0;
    for (int k = 0; k < mine.y && ok; ++k) {
      const SharedSegment sg = segment(k);
      const int tiles = cdiv(sg.tok1 - sg.tok0, TT);
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < tiles; ++t, ++n) {
        const int b = n & 1;
        const uint32_t par = (n >> 1) & 1;
        ok = warp_wait(&s_full[b], par);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t col = tmem + lanes + S_COL + b * TT;
        const int left = sg.tok1 - (sg.tok0 + t * TT);  // tokens of the tile
        // S in one piece, or, beside the converting warps, in four that are read twice,
        // for the maximum and for the weights: the 11 KiB of straight code that 128
        // values take do not stay in the instruction caches then (E4M3, 256-wide latent
        // 67 us against 72; a bf16 cache 332 against 321 the other way round).
        constexpr int kPiece = FP8 ? 32 : TT;
        uint32_t s[kPiece];
        auto load = [&](int q0) {
#pragma unroll
          for (int q = 0; q < kPiece; q += 32)
            tc::ld_32x32b_x32(col + q0 + q, *reinterpret_cast<uint32_t(*)[32]>(&s[q]));
          tc::wait_ld();
          tc::reg_fence(s);
#pragma unroll
          for (int j = 0; j < kPiece; j += 2) mul2(s[j], s[j + 1], c);
          if (left < q0 + kPiece) {
#pragma unroll
            for (int j = 0; j < kPiece; ++j)
              if (q0 + j >= left) s[j] = 0xFF800000u;  // -inf
          }
        };
        auto s_read = [&]() {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[b]);
        };
        float mx[4] = {m, m, m, m};
#pragma unroll 1
        for (int q = 0; q < TT; q += kPiece) {
          load(q);
          if (!FP8) s_read();
#pragma unroll
          for (int j = 0; j < kPiece; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[j + 2 * e]), __uint_as_float(s[j + 2 * e + 1])));
        }
        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // O is rescaled only when the maximum has grown by more than 2^8
        float alpha = 1.f;
        if (m_new > m + kRescaleAt) {
          if (t > 0) alpha = ex2(m - m_new);
          l *= alpha;
          m = m_new;
        }
        const float base = m == -INFINITY ? 0.f : m;  // scores of -inf alone: weights of 0
        // the P buffer's last tile has been read by rank 1's products, the last
        // copies have read what they send
        if (n >= 2) ok = warp_wait_cluster(&p_free[b], par ^ 1);
        if (!ok) break;
        if (lane == 0) tc::bulk_wait_read();
        __syncwarp();
        const uint32_t bar = bar_peer + b * 8;
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int q0 = 0; q0 < TT; q0 += kPiece) {
          if (FP8) {
            load(q0);
            if (q0 + kPiece == TT) s_read();
          }
#pragma unroll
          for (int i0 = 0; i0 < kPiece; i0 += 32) {
            const int q = q0 + i0;
            uint8_t* box = out + (q >> 6) * 4096;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = i0 + j * 8 + e * 2;
                float x0, x1;
                unpack2(add2(pack2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), pack2(-base, -base)),
                        x0, x1);
                x0 = ex2(x0);
                x1 = ex2(x1);
                sum[e & 1] = add2(sum[e & 1], pack2(x0, x1));
                w[e] = pack_bf16x2(x0, x1);
              }
              *reinterpret_cast<uint4*>(box + sw128(lane, ((q & 32) >> 3) + j)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (q & 32) {  // a box of 64 tokens is complete
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0)
                tc::bulk_copy_to_peer(p_peer + b * kPBuf + (q >> 6) * 16384, box, 4096, bar);
            }
          }
        }
        float s0, s1, s2, s3;
        unpack2(sum[0], s0, s1);
        unpack2(sum[1], s2, s3);
        l += (s0 + s1) + (s2 + s3);
        tc::st_async_b32(a_peer + b * 512, __float_as_uint(alpha), bar);
      }
      if (!ok) break;
      if (r < sg.vecs) p.ml[static_cast<int64_t>(mine.x + k) * 128 + r] = make_float2(m, l);
    }
    if (lane == 0) tc::bulk_wait_read();
    // rank 1's last arrivals here have landed before this CTA can leave
    for (int j = 1; j <= 2 && ok; ++j)
      if (n >= j) ok = warp_wait_cluster(&p_free[(n - j) & 1], ((n - j) >> 1) & 1);
  };
  // ------------------------------------------------- O of rank 1
  auto output = [&]() {
    // two warps a lane quarter, each with half of the dims; one with an fp8 cache
    constexpr int kDims = FP8 ? R : R / 2;
    const int quad = warp & 3, h = warp >> 2;
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
          for (int q = 0; q < kDims; q += 32) {
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
      // [8-dim group][vector]: a warp's store is 1 KiB in one piece (rows of R
      // each took 9.5 us a block)
      float* dst = p.partial + static_cast<int64_t>(mine.x + k) * 128 * R +
                   (static_cast<int64_t>(h) * (R / 16) * 128 + r) * 8;
#pragma unroll 2
      for (int q = 0; q < kDims; q += 32) {
        uint32_t o[32];
        tc::ld_32x32b_x32(o_col + q, o);
        tc::wait_ld();
        tc::reg_fence(o);
        if (r < sg.vecs) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             dst + (q + e) * 128),
                         "r"(o[e]), "r"(o[e + 1]), "r"(o[e + 2]), "r"(o[e + 3]), "r"(o[e + 4]),
                         "r"(o[e + 5]), "r"(o[e + 6]), "r"(o[e + 7])
                         : "memory");
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  };

  // With an fp8 cache's 512 threads the softmax warps take registers of the
  // others (128 x 168 + 384 x 112 < 512 x 128).
  if (FP8 ? warp < 4 : warp < (rank == 0 ? 4 : 8)) {
    if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    if (rank == 0)
      softmax();
    else
      output();
  } else {
    if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    if (warp < 8 || (FP8 && warp >= 10 && warp < 14))
      fill(warp < 8 ? 1 : 0);
    else if (warp != 9)
      produce();
    else if (rank == 0)
      scores();
    else
      values();
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
// A CTA joins eight vectors of one sequence: the segments of its own part and of
// its group's, weighted by their maxima.  Thread = vector (lane % 8) and groups of
// eight dims, so that a warp reads pieces of 256 bytes; the segments' places,
// maxima and sums come in first, all at once.
constexpr int kJoin = 8;          // vectors
constexpr int kInFlight = 4;

template <int R>
__global__ void __launch_bounds__(256) shared_join_kernel(const SharedParams p) {
  constexpr int NV = R / 256;  // groups of 8 dims a thread
  extern __shared__ int sm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.num_heads, per = p.rows_per_seq * H, ctas = cdiv(per, kJoin);
  const int seq = static_cast<int>(blockIdx.x) / ctas;
  const int vec0 = (static_cast<int>(blockIdx.x) - seq * ctas) * kJoin;  // of the sequence
  int* rec = sm;                                        // [items][8] slot * 128 + vector, or -1
  float* m = reinterpret_cast<float*>(sm + p.most_items * kJoin);  // maxima, then weights
  float* l = m + p.most_items * kJoin;
  __shared__ float inverse[kJoin];
  griddep_wait();
  griddep_launch_dependents();
  const SharedRow at = p.rows[seq];
  const SharedPlace part[2] = {at.own, at.group};
  const int C = at.per_pair;
  int items[2], span[2];  // slots to look at: chunks x pairs that a chunk can meet
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    span[i] = cdiv(part[i].chunk, C) + 1;
    items[i] = part[i].blocks == 0 ? 0 : cdiv(part[i].tiles, part[i].chunk) * span[i];
  }
  const int n = items[0] + items[1];
  for (int i = threadIdx.x; i < n * kJoin; i += 256) {
    const int v = i & (kJoin - 1), item = i / kJoin;
    const int w = item >= items[0];
    const SharedPlace& x = w ? part[1] : part[0];
    const int k = w ? item - items[0] : item, sp = w ? span[1] : span[0];
    const int j = k / sp, len = min(x.chunk, x.tiles - j * x.chunk);
    // the vector among the part's: of its sequence alone, or of the group's
    const int u = vec0 + v + (w ? (seq * p.rows_per_seq - x.row0) * H : 0);
    const int g = u >> 7;
    const int tile0 = x.first + j * (x.chunk + kStart) * x.blocks + g * (len + kStart) + kStart;
    const int c = tile0 / C + (k - j * sp);
    int r = -1;
    if (vec0 + v < per && static_cast<int64_t>(c) * C < tile0 + len)
      r = (x.unit0 + j * x.blocks + g + c) * 128 + (u & 127);
    const float2 ml = r >= 0 ? p.ml[r] : make_float2(-INFINITY, 0.f);
    rec[i] = r;
    m[i] = ml.x;
    l[i] = ml.y;
  }
  __syncthreads();
  {  // warp v: the weights of vector v
    const int v = warp;
    float M = -INFINITY, den = 0.f;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, m[i * kJoin + v]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    for (int i = lane; i < n; i += 32) {
      const int a = i * kJoin + v;
      const float w = rec[a] >= 0 ? ex2(m[a] - M) : 0.f;
      den += w * l[a];
      m[a] = w;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
    if (lane == 0 && vec0 + v < per) {
      inverse[v] = n == 0 ? 0.f : (p.kv_scale ? __ldg(p.kv_scale) : 1.f) / den;
      p.lse[static_cast<int64_t>(seq) * per + vec0 + v] =
          n == 0 ? -INFINITY : (M + log2f(den)) * kLn2;
    }
  }
  __syncthreads();
  const int v = lane & 7;
  if (vec0 + v >= per) return;
  float acc[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
  const int group = warp * 4 + (lane >> 3);
  for (int i0 = 0; i0 < n; i0 += kInFlight) {
    float4 x[kInFlight][NV][2];
    float w[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int r = i0 + u < n ? rec[(i0 + u) * kJoin + v] : -1;
      w[u] = 0.f;
      if (r < 0) continue;
      w[u] = m[(i0 + u) * kJoin + v];
      const float* src = p.partial + static_cast<int64_t>(r >> 7) * 128 * R + (r & 127) * 8;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float4* g = reinterpret_cast<const float4*>(src + (group + k * 32) * 1024);
        x[u][k][0] = g[0];
        x[u][k][1] = g[1];
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      if (i0 + u >= n || rec[(i0 + u) * kJoin + v] < 0) continue;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        acc[k][0] += w[u] * x[u][k][0].x;
        acc[k][1] += w[u] * x[u][k][0].y;
        acc[k][2] += w[u] * x[u][k][0].z;
        acc[k][3] += w[u] * x[u][k][0].w;
        acc[k][4] += w[u] * x[u][k][1].x;
        acc[k][5] += w[u] * x[u][k][1].y;
        acc[k][6] += w[u] * x[u][k][1].z;
        acc[k][7] += w[u] * x[u][k][1].w;
      }
    }
  }
  const float inv = inverse[v];
  uint16_t* o = p.o + (static_cast<int64_t>(seq) * per + vec0 + v) * R;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    *reinterpret_cast<uint4*>(o + (group + k * 32) * 8) =
        make_uint4(pack_bf16x2(acc[k][0] * inv, acc[k][1] * inv),
                   pack_bf16x2(acc[k][2] * inv, acc[k][3] * inv),
                   pack_bf16x2(acc[k][4] * inv, acc[k][5] * inv),
                   pack_bf16x2(acc[k][6] * inv, acc[k][7] * inv));
}

size_t align_up(size_t x) { return (x + 255) & ~size_t{255}; }

template <int R, bool FP8>
cudaError_t launch_main(const SharedParams& p, const CUtensorMap& tmap, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(decode_shared_kernel<R, FP8>, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  return launch_overlapped(decode_shared_kernel<R, FP8>, dim3(2 * p.pairs), dim3(FP8 ? 512 : 384),
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
  uint8_t* pair_segments = take(pairs * sizeof(int2));
  uint8_t* rows = take(static_cast<size_t>(num_seqs) * sizeof(SharedRow));
  uint8_t* segments = take(slots * sizeof(SharedSegment));
  uint8_t* ml = take(slots * 128 * sizeof(float2));
  uint8_t* partial = take(slots * 128 * sizeof(float) * R);
  if (p) {
    p->pair_segments = reinterpret_cast<int2*>(pair_segments);
    p->rows = reinterpret_cast<SharedRow*>(rows);
    p->segments = reinterpret_cast<SharedSegment*>(segments);
    p->ml = reinterpret_cast<float2*>(ml);
    p->partial = reinterpret_cast<float*>(partial);
  }
  return at;
}

cudaError_t launch_decode_shared(const SharedParams& p_in, const CUtensorMap& tmap, int R, bool fp8,
                                 cudaStream_t stream) {
  SharedParams p = p_in;
  static std::atomic<uint64_t> attr_done{0};
  constexpr int kMostSmem = 200 * 1024;
  cudaError_t e = set_smem_attr_once(shared_schedule_kernel, kMostSmem, attr_done);
  if (e != cudaSuccess) return e;
  static_assert((kMaxSharedGroups + kMaxSharedSeqs + 33) * 8 +
                        (3 * (kMaxSharedGroups + kMaxSharedSeqs) + 2 * kMaxSharedGroups + 1) * 4 <=
                    kMostSmem,
                "the schedule's shared memory");
  const int G = p.num_groups, V = G + p.num_seqs;
  e = launch_overlapped(shared_schedule_kernel, dim3(1), dim3(V <= 512 ? 256 : 1024),
                        schedule_smem(G, V), stream, p);
  if (e != cudaSuccess) return e;
  // A part's chunks and the pairs that each meets: one chunk meets all pairs at
  // most; a part of several blocks has at most pairs / blocks + 1 chunks, each the
  // tiles of a pair long at most, and with those places before meets three at most.
  p.most_items = 2 * (2 * p.pairs + 4);
  if (R == 512)
    e = fp8 ? launch_main<512, true>(p, tmap, stream) : launch_main<512, false>(p, tmap, stream);
  else
    e = fp8 ? launch_main<256, true>(p, tmap, stream) : launch_main<256, false>(p, tmap, stream);
  if (e != cudaSuccess) return e;
  const int64_t per = static_cast<int64_t>(p.rows_per_seq) * p.num_heads;
  const int64_t ctas = (per + kJoin - 1) / kJoin * p.num_seqs;
  const size_t join = static_cast<size_t>(p.most_items) * kJoin * 12;
  const dim3 grid(static_cast<unsigned>(ctas));
  return R == 512
             ? launch_overlapped(shared_join_kernel<512>, grid, dim3(256), join, stream, p)
             : launch_overlapped(shared_join_kernel<256>, grid, dim3(256), join, stream, p);
}

}  // namespace mla
