// The layer's projections: y = act(x W^T + bias) + residual, x [T][K] and W
// [N][K] bf16 as a linear layer stores it, fp32 accumulation in TMEM and fp32
// epilogue, one rounding to bf16.
//
// Three kernels, by an estimate of their times (linear_plan): pairs of CTAs for many
// tokens, which the tensor core bounds, the same with K split where their tiles leave
// SMs without work, and one for few tokens, which W's way into shared memory bounds.
// All bring K in chunks of 64 through a TMA ring (128-byte swizzle; what
// lies past K, N or T is filled with zeros).
//
// Measured on GB300, out of a graph back to back (W mostly in L2) and out of one with a
// flush of L2 before each call, whose time is taken off, and what bounds it (a single call
// between others that wait for it takes 20.6, 7.7, 20.9 and 838 us on the first three and the
// fifth):
//   1 x 8192 -> 7168, bias, residual         19.7 / 27.5 us  memory: 17.3 at 6.8 TB/s
//   64 x 2048 -> 5120, residual               7.2 / 11.1     start, join and end 4.4, then
//                                                            264 KB a CTA at 97 B/ns
//   1001 x 1536 -> 6136, bias, silu          19.8 / 21.7     1.38 MB a CTA at 97 B/ns in two
//                                                            rounds of tiles, 2 of silu
//   1262 x 184 -> 16176, bias, silu, res.    41.4 / 46.1     the tiles' ends: 31 without the
//                                                            residual, 17.5 without silu, too
//   8192 x 16384 -> 5120, bias, residual     768 to 808      1.70 to 1.79 PFLOP/s, by the power
//                                                            limit's clock (732 at best)
//   442 x 9808 -> 3120, bias, relu           30.9 / 38.0     half of K a pair, 2.5 MB a CTA
// What an SM takes in over TMA is 97 B/ns here, however many boxes are under way.  The
// library's product alone: 20.3, 4.2, 12.4, 12.1, 715 to 780, 32.6 us; it shares the sum over
// K out among all SMs whatever the tiles, for which it keeps a workspace.
#include <cuda_bf16.h>
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int TM = 128;  // tokens per tile
constexpr int KC = 64;   // K per ring stage
constexpr int A_BYTES = TM * KC * 2;
constexpr int STORE_ROWS = 32;
constexpr int STORE_BYTES = STORE_ROWS * 128;
// Token blocks side by side in the order of tiles: the tiles of a wave then
// share about as many rows of x as of W, and L2 serves the others.
constexpr int kGroup = 8;

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// Relaxed: what the others see of this CTA, its barriers' initial state, has a fence
// of its own, and what they send it is acquired through its barrier.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0,
                                             int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// 1 / x, results below the normal range 0 (a call of its own: a division's care for
// them was half of silu's instructions).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The normal distribution's share beyond a >= 0, Q(a) = t 2^(P(t) - a^2 log2(e) / 2) with
// t = 1 / (1 + 0.4 a): P is smooth down to t = 0, and the polynomial of degree 8 that
// meets it at the Chebyshev points of a <= 15 is off by 2.2e-7 (1.5e-7 of Q).  Half of the
// exponent is computed, and its power multiplied twice: the exponential gives 0 for what
// lies below the normal range, where Q is from a = 13 on and x Q still is not.  (erfcf took
// 1001 x 1536 -> 6136 with bias and gelu 30.8 us, this 21.8.)
__device__ __forceinline__ float upper_tail(float a) {
  const float t = rcp(fmaf(0.4f, a, 1.f));
  float p = 0.5f * 0.287300513f;
  p = fmaf(p, t, 0.5f * -1.46468399f);
  p = fmaf(p, t, 0.5f * 2.92157221f);
  p = fmaf(p, t, 0.5f * -2.64318639f);
  p = fmaf(p, t, 0.5f * 0.855061624f);
  p = fmaf(p, t, 0.5f * -0.289307705f);
  p = fmaf(p, t, 0.5f * 0.542938226f);
  p = fmaf(p, t, 0.5f * 1.43778876f);
  p = fmaf(p, t, 0.5f * -2.64748304f);
  const float root = ex2(fmaf(0.5f * -0.72134752f * a, a, p));
  return t * root * root;
}

// 1 / (1 + 2^u), as 2^-15 / (2^-15 + 2^(u - 15)): the reciprocal gives 0 for what lies
// below the normal range, and x times a sigmoid of less than that still has bf16 values
// (silu: down to x = -97; as 1 / (1 + 2^u) it was -0 from -87.3 on).
__device__ __forceinline__ float sigmoid2(float u_less_15) {
  constexpr float k = 1.f / 32768;
  return k * rcp(k + ex2(u_less_15));
}

// The activation over a run of values; the choice is made once for all of them.
// gelu takes the tail on x's side, whose small values keep their relative precision
// where 1 + erf cancels; both sigmoid forms go to 0 or x at the ends.
template <int N>
__device__ __forceinline__ void activate(int act, float (&x)[N]) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = x[i] < 0.f ? 0.f : x[i];  // NaN stays
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] *= sigmoid2(fmaf(-1.4426950f, x[i], -15.f));
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float q = upper_tail(fabsf(x[i]));
        x[i] *= x[i] < 0.f ? q : 1.f - q;
      }
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] *= sigmoid2(fmaf(-2.3022082f * x[i], fmaf(0.044715f * x[i], x[i], 1.f), -15.f));
      break;
    default: break;
  }
}

// x += the bf16 values in v.
template <int N>
__device__ __forceinline__ void add_bf16(float (&x)[N], const uint4 (&v)[N / 8]) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {
    const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[8 * q + 2 * e] += lo_f(w[e]);
      x[8 * q + 2 * e + 1] += hi_f(w[e]);
    }
  }
}

// Eight consecutive bf16 of a row, columns past `n` as zeros; one 16-byte load
// where all eight are there.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int n) {
  if (c + 8 <= n) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) w[e >> 1] |= static_cast<uint32_t>(row[c + e]) << ((e & 1) * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One thread's N columns of the residual from column c on (zeros without one).
template <int N>
__device__ __forceinline__ void load_residual(const LinearParams& p, int row, int c,
                                              uint4 (&r)[N / 8]) {
  const bool there = p.residual && row < p.tokens && c < p.n;
  const uint16_t* src = p.residual + (there ? row * p.res_stride : 0);
#pragma unroll
  for (int q = 0; q < N / 8; ++q)
    r[q] = there ? load8(src, c + 8 * q, p.n) : make_uint4(0, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void load_bias(const LinearParams& p, int c, uint4 (&b)[N / 8]) {
#pragma unroll
  for (int q = 0; q < N / 8; ++q) b[q] = load8(p.bias, c + 8 * q, p.n);
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 32)
    tc::ld_32x32b_x32(addr, r);
  else
    tc::ld_32x32b_x16(addr, r);
}

// One epilogue warp's 32 rows x `cols` (a multiple of 64) columns of a tile from
// TMEM column `acc` and y column c0 on: fp32 (a row a lane) through bias,
// activation and residual to bf16 in swizzled boxes of 64 columns (two in turn,
// `nb` counts them) and from there to y.  `before` waits for the accumulator,
// `after` gives it back.  The residual comes 128 bytes of a row at a time, a box ahead,
// and to the lanes of its rows through the box that their results go to (32 bytes of a
// row a lane: 42.1 us for 37.7, 4096 x 512 -> 7168).  The loop is not unrolled, and products without an
// activation have kernels of their own: with all activations in 32 copies of the
// body 1001 x 1536 -> 6136 took 35 us, waiting for instructions, against 22.
// TAIL: N % 8 columns behind those that the map of y has are stored one by one.  A TMA
// store writes the 16 bytes that a row ends in to their end, so the map ends with the
// last whole ones.  (Kernels of their own: the others got 1 to 3 % slower with it.)
template <bool ACT, bool TAIL, typename Before, typename After>
__device__ __forceinline__ bool epilogue(const LinearParams& p, uint32_t acc, int cols, int c0,
                                         int row0, int lane, uint8_t* boxes, int& nb,
                                         const CUtensorMap* map, Before&& before, After&& after) {
  constexpr int N = ACT ? 16 : 32;  // columns of a step
  const int whole = TAIL ? p.n & ~7 : p.n;  // columns that the map has
  // no box follows the one that has y's last column
  if (TAIL && p.n - c0 < cols) cols = max(64, (p.n - c0 + 63) & ~63);
  uint4 res[8], bias[N / 8];  // of the next box: rows 4 k + lane / 8, eight columns
  auto load = [&](int c) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = row0 + 4 * k + (lane >> 3), col = c + (lane & 7) * 8;
      res[k] = row < p.tokens && col < p.n ? load8(p.residual + row * p.res_stride, col, p.n)
                                           : make_uint4(0, 0, 0, 0);
    }
  };
  if (p.residual) load(c0);
  if (p.bias) load_bias<N>(p, c0, bias);
  if (!before()) return false;
  tc::fence_after_sync();
#pragma unroll 1
  for (int j = 0; j < cols; j += N) {
    const int c = c0 + j;
    uint32_t r[N];
    tmem_load<N>(acc + j, r);
    uint8_t* dst = boxes + (nb & 1) * STORE_BYTES;
    if ((j & 63) == 0) {
      // the store that last used this box, the one before the last, has read it
      if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      __syncwarp();
      if (p.residual) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<uint4*>(dst + sw128(4 * k + (lane >> 3), lane & 7)) = res[k];
        __syncwarp();
        if (j + 64 < cols) load(c + 64);
      }
    }
    tc::wait_ld();
    tc::reg_fence(r);
    if (j + N >= cols) {
      tc::fence_before_sync();
      __syncwarp();
      after();
    }
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(r[i]);
    if (p.bias) {
      add_bf16(x, bias);
      if (j + N < cols) load_bias<N>(p, c + N, bias);
    }
    if (ACT) activate(p.act, x);
    if (p.residual) {
      uint4 v[N / 8];
#pragma unroll
      for (int q = 0; q < N / 8; ++q)
        v[q] = *reinterpret_cast<const uint4*>(dst + sw128(lane, (j & 63) / 8 + q));
      add_bf16(x, v);
    }
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1]);
      *reinterpret_cast<uint4*>(dst + sw128(lane, (j & 63) / 8 + q)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    if ((j & 63) == 64 - N) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int cb = c0 + (j & ~63);
        if (row0 < p.tokens && cb < whole) tma_store_3d(map, dst, cb, 0, row0);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
      ++nb;
    }
  }
  if (TAIL && whole >= c0 + cols - 64 && whole < c0 + cols && row0 + lane < p.tokens) {
    // a lane's row of the last box, which a store may still read
    const uint8_t* src = boxes + ((nb - 1) & 1) * STORE_BYTES;
    const uint4 v = *reinterpret_cast<const uint4*>(src + sw128(lane, (whole & 63) / 8));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint16_t* y = p.y + (row0 + lane) * p.y_stride + whole;
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (whole + e < p.n) y[e] = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) * 16));
  }
  return true;
}

// Tile t of `mt` x `nt`, token blocks in groups of kGroup, token blocks of a
// group fastest.
__device__ __forceinline__ void tile_at(int64_t t, int mt, int nt, int& m, int& n) {
  const int64_t per = static_cast<int64_t>(kGroup) * nt;
  const int g = static_cast<int>(t / per);
  const int in = static_cast<int>(t - g * per);
  const int rows = min(kGroup, mt - g * kGroup);
  n = in / rows;
  m = g * kGroup + in % rows;
}

// ---------------------------------------------------------------- CTA pairs
// Two CTAs of a cluster share a tile of 256 tokens x BN columns, each holds its
// 128 tokens of A and half of the columns of B, and cta_group::2 products read both
// halves: at BN = 256 a chunk takes 597 cycles to come in and 553 to multiply.
// One persistent pair per two SMs, two accumulators in TMEM so that one tile's
// epilogue runs under the next one's products.  Rank 0 issues for both; the ring's
// "landed" barrier is rank 0's and counts both CTAs' bytes; "read" and "accumulator
// ready" arrive in both.  Eight epilogue warps own 32 rows and half of the columns
// each: TMEM -> registers, bias, activation and residual there, bf16 in a swizzled
// 4 KiB staging box -> TMA store, which clips the tensor's edges (columns to 16 bytes).
// The next columns' residual and bias are loaded while the current ones are worked on
// (the first before the accumulator is waited for).
constexpr int kPairStages = 5;
constexpr int kPairHalf = A_BYTES;  // A, and room for the half of B, of one stage
constexpr int PP_STORE = kPairStages * 2 * kPairHalf;
constexpr int PP_BAR = PP_STORE + 8 * 2 * STORE_BYTES;
constexpr int PP_TMEM = PP_BAR + (2 * kPairStages + 4) * 8;
constexpr int PP_SMEM = PP_TMEM + 16 + 1024;
static_assert(PP_SMEM <= 227 * 1024, "shared memory");

template <int BN, bool ACT, bool TAIL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
    linear_pair_kernel(const LinearParams p, const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ CUtensorMap mc) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + PP_BAR);  // [stages] rank 0's: both landed
  uint64_t* empty = full + kPairStages;                         // [stages]
  uint64_t* acc_full = empty + kPairStages;                     // [2]
  uint64_t* acc_empty = acc_full + 2;                           // [2] rank 0's: 16 warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PP_TMEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();

  const int nk = (p.k + KC - 1) / KC;
  const int mt = (p.tokens + 2 * TM - 1) / (2 * TM), nt = (p.n + BN - 1) / BN;
  const int64_t total = static_cast<int64_t>(mt) * nt;
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;
  auto request = [&](int st, int m, int n, int kc) {
    uint8_t* dst = smem + st * 2 * kPairHalf;
    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * (A_BYTES + BN / 2 * 128));
    const uint32_t bar = tc::map_peer(smem_u32(&full[st]), 0);
    tc::pair_tma_load_3d(dst, &ma, bar, kc * KC, 0, m * 2 * TM + rank * TM);
    tc::pair_tma_load_3d(dst + kPairHalf, &mb, bar, kc * KC, 0, n * BN + rank * (BN / 2));
  };

  if (threadIdx.x == 128) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    fence_mbar_init();
  }
  if (warp == 4) __syncwarp();
  cluster_arrive();
  if (warp == 5) {
    tc::pair_tmem_alloc(tmem_slot, 512);
    tc::pair_tmem_relinquish();
  }
  cluster_wait();  // both CTAs' barriers are there: the ring is filled at once
  if (threadIdx.x == 128) {
    griddep_wait();
    int m, n;
    tile_at(first, mt, nt, m, n);
    for (int kc = 0; kc < min(nk, kPairStages); ++kc) request(kc, m, n, kc);
  }
  if (warp == 4) __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_arrive();
  if (warp != 4) cluster_wait();  // both have their TMEM
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int64_t t = first; t < total && ok; t += step) {
        int m, n;
        tile_at(t, mt, nt, m, n);
        for (int kc = 0; kc < nk; ++kc, ++it) {
          if (it < kPairStages && t == first) continue;  // asked for above
          const int st = it % kPairStages;
          if (!mbar_wait(&empty[st], ((it / kPairStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          request(st, m, n, kc);
        }
      }
      if (!ok) gave_up(p.err_count);
    }
    __syncwarp();
    cluster_wait();
  } else if (warp == 5) {
    bool ok = true;
    int it = 0, ta = 0;
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_bf16(2 * TM, BN, 0, 0);
      for (int64_t t = first; t < total && ok; t += step, ++ta) {
        const int a = ta & 1;
        const bool free = tc::mbar_wait_cluster(&acc_empty[a], ((ta >> 1) & 1) ^ 1);
        if (!__all_sync(0xffffffffu, free)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        for (int kc = 0; kc < nk; ++kc, ++it) {
          const int st = it % kPairStages;
          if (!warp_wait(&full[st], (it / kPairStages) & 1)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          if (tc::elect_one()) {
            const uint32_t base = smem_u32(smem + st * 2 * kPairHalf);
            const uint64_t da = tc::smem_desc(base, 16, 1024, tc::kLayoutSw128);
            const uint64_t db = tc::smem_desc(base + kPairHalf, 16, 1024, tc::kLayoutSw128);
#pragma unroll
            for (int k = 0; k < KC / 16; ++k)
              tc::pair_mma_ss(tmem + a * 256, da + static_cast<uint64_t>(k * 2),
                              db + static_cast<uint64_t>(k * 2), idesc,
                              (kc > 0 || k > 0) ? 1u : 0u);
            tc::pair_commit(&empty[st], 3);
            if (kc == nk - 1) tc::pair_commit(&acc_full[a], 3);
          }
          __syncwarp();
        }
      }
      for (int j = 0; ok && j < 2 && j < ta; ++j) {
        const int u = ta - 1 - j;
        warp_wait(&acc_full[u & 1], (u >> 1) & 1);
      }
      if (!ok && lane == 0) gave_up(p.err_count);
    }
  } else {
    // warps 0-3 the tile's first half of columns (128 of 192), 6-9 the others; a
    // warp reads the TMEM lanes of its quarter (warp % 4)
    constexpr int kFirst = (BN / 64 + 1) / 2 * 64;
    const int half = warp >= 6, ew = half ? warp - 2 : warp, qd = warp & 3;
    uint8_t* box = smem + PP_STORE + ew * 2 * STORE_BYTES;
    const uint32_t lanes = static_cast<uint32_t>(qd * 32) << 16;
    int ta = 0, nb = 0;
    bool ok = true;
    for (int64_t t = first; t < total && ok; t += step, ++ta) {
      int m, n;
      tile_at(t, mt, nt, m, n);
      const int a = ta & 1;
      ok = epilogue<ACT, TAIL>(
          p, tmem + lanes + a * 256 + half * kFirst, half ? BN - kFirst : kFirst, n * BN + half * kFirst,
          m * 2 * TM + rank * TM + qd * STORE_ROWS, lane, box, nb, &mc,
          [&] { return warp_wait(&acc_full[a], (ta >> 1) & 1); },
          [&] {
            if (lane == 0) tc::arrive_peer(tc::map_peer(smem_u32(&acc_empty[a]), 0));
          });
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) gave_up(p.err_count);
  }

  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // the peer's barriers and operands are used to the end
  if (warp == 5) {
    tc::fence_after_sync();
    tc::pair_tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------- split pairs
// Tiles that do not fill the SMs: 256 tokens x 256 columns, the sum over K split among
// up to four pairs of CTAs of a cluster.  When all products are done a CTA's partial
// sums, 128 rows x 256 columns, go in slabs of 32 columns to the CTA of its rows that
// finishes them, through the ring's place: a warp's 32 rows of a slab are one bulk copy of
// 4 KiB.  That one adds the parts in order and stores 32 bytes of a row a lane.
constexpr int SP_RECV = 6 * 16384;  // what is sent lies before: at most six slabs
constexpr int SP_BAR = SP_RECV + 6 * 16384;  // received: six slabs, too
static_assert(SP_BAR >= kPairStages * 2 * kPairHalf, "the ring");
constexpr int SP_TMEM = SP_BAR + (2 * kPairStages + 2) * 8;
constexpr int SP_SMEM = SP_TMEM + 16 + 1024;
static_assert(SP_SMEM <= 227 * 1024, "shared memory");

template <bool ACT>
__global__ void __launch_bounds__(320, 1)
    linear_split_kernel(const LinearParams p, const __grid_constant__ CUtensorMap ma,
                        const __grid_constant__ CUtensorMap mb) {
  constexpr int BN = 256, N = 16;  // columns of a tile, of a step of the end
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SP_BAR);  // [stages] rank 0's: both landed
  uint64_t* empty = full + kPairStages;                         // [stages]
  uint64_t* acc_full = empty + kPairStages;
  uint64_t* recv_full = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SP_TMEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits;
  const int cta = static_cast<int>(tc::cluster_ctarank());
  const int rank = cta & 1, part = cta >> 1;  // of the pair, of the split
  const int mt = (p.tokens + 2 * TM - 1) / (2 * TM), nt = (p.n + BN - 1) / BN;
  int m, n;
  tile_at(blockIdx.x / (2 * S), mt, nt, m, n);
  const int nk = (p.k + KC - 1) / KC;
  const int k_lo = static_cast<int>(static_cast<int64_t>(nk) * part / S);
  const int k_hi = static_cast<int>(static_cast<int64_t>(nk) * (part + 1) / S);
  const int lo = 8 * part / S, hi = 8 * (part + 1) / S;  // slabs that this CTA finishes
  auto request = [&](int kc) {
    const int st = (kc - k_lo) % kPairStages;
    uint8_t* dst = smem + st * 2 * kPairHalf;
    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * (A_BYTES + BN / 2 * 128));
    const uint32_t bar = tc::map_peer(smem_u32(&full[st]), cta & ~1);
    tc::pair_tma_load_3d(dst, &ma, bar, kc * KC, 0, m * 2 * TM + rank * TM);
    tc::pair_tma_load_3d(dst + kPairHalf, &mb, bar, kc * KC, 0, n * BN + rank * (BN / 2));
  };

  if (threadIdx.x == 128) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(recv_full, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(recv_full, static_cast<uint32_t>((S - 1) * (hi - lo) * 16384));
  }
  if (warp == 4) __syncwarp();
  cluster_arrive();
  if (warp == 5) {
    tc::pair_tmem_alloc(tmem_slot, BN);
    tc::pair_tmem_relinquish();
  }
  cluster_wait();  // all barriers are there: the ring is filled at once
  if (threadIdx.x == 128) {
    griddep_wait();
    for (int kc = k_lo; kc < min(k_hi, k_lo + kPairStages); ++kc) request(kc);
  }
  if (warp == 4) __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_arrive();
  if (warp != 4) cluster_wait();  // all have their TMEM
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 4) {
    if (lane == 0) {
      for (int kc = k_lo + kPairStages; kc < k_hi; ++kc) {
        const int it = kc - k_lo;
        if (!mbar_wait(&empty[it % kPairStages], ((it / kPairStages) & 1) ^ 1)) {
          ok = false;
          break;
        }
        request(kc);
      }
    }
    __syncwarp();
    cluster_wait();
    cluster_arrive();  // (the products' end, for the warps that send)
    cluster_wait();
  } else if (warp == 5) {
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_bf16(2 * TM, BN, 0, 0);
      const uint16_t both = static_cast<uint16_t>(3 << cta);
      for (int kc = k_lo; kc < k_hi; ++kc) {
        const int it = kc - k_lo, st = it % kPairStages;
        if (!warp_wait(&full[st], (it / kPairStages) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (tc::elect_one()) {
          const uint32_t base = smem_u32(smem + st * 2 * kPairHalf);
          const uint64_t da = tc::smem_desc(base, 16, 1024, tc::kLayoutSw128);
          const uint64_t db = tc::smem_desc(base + kPairHalf, 16, 1024, tc::kLayoutSw128);
#pragma unroll
          for (int k = 0; k < KC / 16; ++k)
            tc::pair_mma_ss(tmem, da + static_cast<uint64_t>(k * 2),
                            db + static_cast<uint64_t>(k * 2), idesc, (it > 0 || k > 0) ? 1u : 0u);
          tc::pair_commit(&empty[st], both);
          if (kc == k_hi - 1) tc::pair_commit(acc_full, both);
        }
        __syncwarp();
      }
      if (ok) ok = warp_wait(acc_full, 0);
    }
    cluster_arrive();
    cluster_wait();
  } else {
    const int half = warp >= 6, qd = warp & 3;
    const uint32_t acc = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    const int row = m * 2 * TM + rank * TM + qd * 32 + lane;
    const int first = lo + ((lo ^ half) & 1);  // this warp's slabs: every other one
    auto column = [&](int step) { return n * BN + (first + (step & ~1)) * 32 + (step & 1) * N; };
    const int steps = first < hi ? 2 * ((hi - first + 1) / 2) : 0;
    uint4 res[N / 8];
    if (steps > 0) load_residual<N>(p, row, column(0), res);
    ok = warp_wait(acc_full, 0);
    tc::fence_after_sync();
    // this pair has read its rings to the end
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (ok) {
#pragma unroll 1
      for (int sl = half; sl < 8; sl += 2) {
        if (sl >= lo && sl < hi) continue;
        uint32_t r[32];
        tc::ld_32x32b_x32(acc + sl * 32, r);
        tc::wait_ld();
        tc::reg_fence(r);
        uint8_t* dst = smem + ((sl < lo ? sl : sl - (hi - lo)) * 4 + qd) * 4096 + lane * 16;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(dst + q * 512) =
              make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
      }
      fence_proxy_async_smem();
    }
    __syncwarp();
    cluster_wait();  // so have the others
    if (ok && lane < 4) {
      const int sl = half + 2 * lane;
      if (sl < lo || sl >= hi) {
        const int to = ((sl + 1) * S - 1) / 8;  // the part that finishes it
        const int to_lo = 8 * to / S, to_hi = 8 * (to + 1) / S;
        const int slot = (part - (part > to)) * (to_hi - to_lo) + sl - to_lo;
        tc::bulk_copy_to_peer(
            tc::map_peer(smem_u32(smem + SP_RECV), 2 * to + rank) + (slot * 4 + qd) * 4096,
            smem + ((sl < lo ? sl : sl - (hi - lo)) * 4 + qd) * 4096, 4096,
            tc::map_peer(smem_u32(recv_full), 2 * to + rank));
      }
    }
    __syncwarp();
    const bool got = tc::mbar_wait_cluster(recv_full, 0);
    ok = __all_sync(0xffffffffu, got) && ok;
#pragma unroll 1
    for (int i = 0; ok && i < steps; ++i) {
      const int sl = first + (i & ~1), c = column(i);
      uint32_t r[N];
      tc::ld_32x32b_x16(acc + sl * 32 + (i & 1) * N, r);
      uint4 nxt[N / 8], bias[N / 8];
      if (p.bias) load_bias<N>(p, c, bias);
      if (i + 1 < steps) load_residual<N>(p, row, column(i + 1), nxt);
      tc::wait_ld();
      tc::reg_fence(r);
      float x[N] = {};
      if (p.bias) add_bf16(x, bias);
#pragma unroll 1
      for (int q = 0; q < S; ++q) {
        if (q == part) {
#pragma unroll
          for (int e = 0; e < N; ++e) x[e] += __uint_as_float(r[e]);
        } else {
          const uint8_t* src = smem + SP_RECV +
                               (((q - (q > part)) * (hi - lo) + sl - lo) * 4 + qd) * 4096 +
                               (i & 1) * (N / 4) * 512 + lane * 16;
#pragma unroll
          for (int e = 0; e < N / 4; ++e) {
            const float4 v = *reinterpret_cast<const float4*>(src + e * 512);
            x[4 * e] += v.x;
            x[4 * e + 1] += v.y;
            x[4 * e + 2] += v.z;
            x[4 * e + 3] += v.w;
          }
        }
      }
      if (ACT) activate(p.act, x);
      if (p.residual) add_bf16(x, res);
#pragma unroll
      for (int q = 0; q < N / 8; ++q) {
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = pack_bf16x2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1]);
        if (row < p.tokens) {
          uint16_t* y = p.y + row * p.y_stride;
          const int col = c + 8 * q;
          if (col + 8 <= p.n) {
            *reinterpret_cast<uint4*>(y + col) = make_uint4(o[0], o[1], o[2], o[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e < p.n) y[col + e] = static_cast<uint16_t>(o[e >> 1] >> ((e & 1) * 16));
          }
        }
        res[q] = nxt[q];
      }
    }
    __syncwarp();
  }
  if (!ok && lane == 0) gave_up(p.err_count);

  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();  // what is sent has been received, the peer's TMEM has been read
  if (warp == 5) {
    tc::fence_after_sync();
    tc::pair_tmem_dealloc(tmem, BN);
  }
}

// ---------------------------------------------------------------- few tokens
// The weight is the work, and it has to come in at the rate of memory: the
// operands change places (128 rows of W are A, the tokens B, padded to TN), and the
// sum over K is split over a cluster of up to eight CTAs, so that nearly every SM
// has its part of W under way whatever N is.  The partial sums go from TMEM, in
// groups of four tokens, to the CTA of the cluster that finishes those tokens, which
// adds the parts in rank order.  They are laid out in the ring's place and go as one
// bulk copy a warp and CTA: stores to the peer one vector at a time took 2 us per 32
// KB (64 x 2048 -> 5120: 10.3 us then, 9.3 with the copies, 7.8 with room for two
// CTAs an SM, so that the next kernel starts under this one's end, 7.1 without a wait
// for the cluster at the start).  A lane finishes four columns of four tokens and
// stores 8 bytes of each.
constexpr int kMostSplits = 8;  // a cluster
constexpr int kAhead = 8;  // chunks of W asked for before the kernel before has ended

__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap* map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Four consecutive bf16 of a row from column c, a multiple of 4, on; those past
// `n` are zeros and are not stored.
__device__ __forceinline__ uint2 load4(const uint16_t* row, int c, int n) {
  if (c + 4 <= n) return *reinterpret_cast<const uint2*>(row + c);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < n) w[e >> 1] |= static_cast<uint32_t>(row[c + e]) << ((e & 1) * 16);
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store4(uint16_t* row, int c, int n, uint2 v) {
  if (c + 4 <= n) {
    *reinterpret_cast<uint2*>(row + c) = v;
    return;
  }
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < n) row[c + e] = static_cast<uint16_t>(w[e >> 1] >> ((e & 1) * 16));
}

template <int TN>
struct FewCfg {
  static constexpr int STAGE = A_BYTES + TN * KC * 2;
  static constexpr int CTAS = TN == 128 ? 1 : 2;  // an SM
  // groups of four tokens received from the other ranks, at most
  static constexpr int groups() {
    int most = 0;
    for (int s = 2; s <= kMostSplits; ++s) {
      const int g = (s - 1) * ((TN / 4 + s - 1) / s);
      if (g > most) most = g;
    }
    return most;
  }
  static constexpr int RECV = 2048 * groups();
  static constexpr int STAGES = TN == 16 ? 5 : TN == 64 ? 3 : 4;
  static constexpr int OFF_RECV = STAGES * STAGE;
  static constexpr int OFF_BAR = OFF_RECV + RECV;
  static constexpr int OFF_TMEM = OFF_BAR + (2 * STAGES + 2) * 8;
  static constexpr int SMEM = OFF_TMEM + 16 + 1024;
  static constexpr uint32_t COLS = TN < 32 ? 32 : TN;
  static_assert((SMEM + 1024) * CTAS <= 228 * 1024, "shared memory");
};

template <int TN, bool ACT>
__global__ void __launch_bounds__(192, FewCfg<TN>::CTAS)
    linear_few_kernel(const LinearParams p, const __grid_constant__ CUtensorMap mx,
                      const __grid_constant__ CUtensorMap mw) {
  using C = FewCfg<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [STAGES]
  uint64_t* empty = full + C::STAGES;                               // [STAGES]
  uint64_t* acc_full = empty + C::STAGES;
  uint64_t* recv_full = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits;
  const int rank = static_cast<int>(tc::cluster_ctarank());
  const int n0 = static_cast<int>(blockIdx.x / S) * 128;
  const int t0 = static_cast<int>(blockIdx.y) * TN;
  const int nt = min(TN, p.tokens - t0);  // tokens here
  const int quads = (nt + 3) / 4, per = (quads + S - 1) / S;
  const int q_lo = min(quads, rank * per), q_hi = min(quads, q_lo + per);

  const int nk = (p.k + KC - 1) / KC;
  const int k_lo = static_cast<int>(static_cast<int64_t>(nk) * rank / S);
  const int k_hi = static_cast<int>(static_cast<int64_t>(nk) * (rank + 1) / S);
  auto request = [&](int kc) {
    const int st = (kc - k_lo) % C::STAGES;
    uint8_t* dst = smem + st * C::STAGE;
    mbar_arrive_expect_tx(&full[st], C::STAGE);
    tma_load_3d(dst, &mw, &full[st], kc * KC, 0, n0);
    tma_load_3d(dst + A_BYTES, &mx, &full[st], kc * KC, 0, t0);
  };

  if (threadIdx.x == 128) {
    tma_prefetch_desc(&mw);
    tma_prefetch_desc(&mx);
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(recv_full, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(recv_full, static_cast<uint32_t>((S - 1) * (q_hi - q_lo) * 2048));
    // The first of this CTA's W comes on its way into L2 while the kernel before
    // still runs: L2 holds what that one may write of it, so nothing stale is read.
    for (int kc = k_lo; kc < min(k_hi, k_lo + kAhead); ++kc) tma_prefetch_l2(&mw, kc * KC, 0, n0);
    griddep_wait();
    for (int kc = k_lo; kc < min(k_hi, k_lo + C::STAGES); ++kc) request(kc);
  }
  __syncwarp();
  cluster_arrive();  // waited for before parts are sent
  if (warp == 5) {
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 4) {
    if (lane == 0) {
      for (int kc = k_lo + C::STAGES; kc < k_hi; ++kc) {
        const int it = kc - k_lo;
        if (!mbar_wait(&empty[it % C::STAGES], ((it / C::STAGES) & 1) ^ 1)) {
          ok = false;
          break;
        }
        request(kc);
      }
    }
    __syncwarp();
    cluster_wait();
    cluster_arrive();
  } else if (warp == 5) {
    constexpr uint32_t idesc = tc::idesc_bf16(128, TN, 0, 0);
    for (int kc = k_lo; kc < k_hi; ++kc) {
      const int it = kc - k_lo, st = it % C::STAGES;
      if (!warp_wait(&full[st], (it / C::STAGES) & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (tc::elect_one()) {
        const uint32_t base = smem_u32(smem + st * C::STAGE);
        const uint64_t da = tc::smem_desc(base, 16, 1024, tc::kLayoutSw128);
        const uint64_t db = tc::smem_desc(base + A_BYTES, 16, 1024, tc::kLayoutSw128);
#pragma unroll
        for (int k = 0; k < KC / 16; ++k)
          tc::mma_ss(tmem, da + static_cast<uint64_t>(k * 2), db + static_cast<uint64_t>(k * 2),
                     idesc, (it > 0 || k > 0) ? 1u : 0u);
        tc::commit(&empty[st]);
        if (kc == k_hi - 1) tc::commit(acc_full);
      }
      __syncwarp();
    }
    if (ok) ok = warp_wait(acc_full, 0);  // nothing is in flight when TMEM is freed
    cluster_wait();
    cluster_arrive();
  } else {
    // What this warp finishes: groups of four tokens warp, warp + 4, .. of this
    // CTA's, a lane four columns from n on.  The first residual under the wait.
    const int n = n0 + 4 * lane;
    uint2 res[4];
    auto load = [&](int quad) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = quad * 4 + e;
        res[e] = p.residual && quad < q_hi && t < nt
                     ? load4(p.residual + (t0 + t) * p.res_stride, n, p.n)
                     : make_uint2(0, 0);
      }
    };
    load(q_lo + warp);
    const uint2 bias = p.bias ? load4(p.bias, n, p.n) : make_uint2(0, 0);
    ok = warp_wait(acc_full, 0);
    cluster_wait();  // every CTA's barrier is there
    if (ok) {
      // Parts [warp][group][32 rows][4 tokens] in the ring's place, which nothing
      // reads any more.  Row 4 l + j lies in slot 8 j + (l + 2 j) % 8, so that eight
      // lanes write and read all banks.
      tc::fence_after_sync();
      uint8_t* part = smem + warp * quads * 512;
      const int slot = 8 * (lane & 3) + (((lane >> 2) + 2 * (lane & 3)) & 7);
      const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
#pragma unroll 1
      for (int c = 0; c < nt; c += 16) {
        uint32_t r[16];
        tc::ld_32x32b_x16(tmem + lanes + c, r);
        tc::wait_ld();
        tc::reg_fence(r);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c / 4 + q < quads)
            *reinterpret_cast<uint4*>(part + (c / 4 + q) * 512 + slot * 16) =
                make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      const int lo = min(quads, lane * per), hi = min(quads, lo + per);  // rank `lane`'s
      if (lane < S && lane != rank && hi > lo)
        tc::bulk_copy_to_peer(tc::map_peer(smem_u32(smem + C::OFF_RECV), lane) +
                                  ((rank - (rank > lane)) * 4 + warp) * per * 512,
                              part + lo * 512, (hi - lo) * 512,
                              tc::map_peer(smem_u32(recv_full), lane));
    }
    named_bar_sync(1, 128);  // this CTA's own parts
    if (q_hi > q_lo) {
      const bool got = tc::mbar_wait_cluster(recv_full, 0);
      ok = __all_sync(0xffffffffu, got) && ok;
    }
    cluster_arrive();
    if (ok) {
      const float b[4] = {lo_f(bias.x), hi_f(bias.x), lo_f(bias.y), hi_f(bias.y)};
#pragma unroll 1
      for (int quad = q_lo + warp; quad < q_hi; quad += 4) {
        uint2 r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = res[e];
        load(quad + 4);
        float x[16];  // [column][token]
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[4 * j + e] = b[j];
#pragma unroll 1
        for (int s = 0; s < S; ++s) {
          const uint8_t* src =
              s == rank ? smem + ((lane >> 3) * quads + quad) * 512
                        : smem + C::OFF_RECV +
                              (((s - (s > rank)) * 4 + (lane >> 3)) * per + quad - q_lo) * 512;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v =
                *reinterpret_cast<const float4*>(src + (8 * j + ((lane + 2 * j) & 7)) * 16);
            x[4 * j] += v.x;
            x[4 * j + 1] += v.y;
            x[4 * j + 2] += v.z;
            x[4 * j + 3] += v.w;
          }
        }
        if (ACT) activate(p.act, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = quad * 4 + e;
          if (t >= nt) break;
          if (p.residual) {
            x[e] += lo_f(r[e].x);
            x[4 + e] += hi_f(r[e].x);
            x[8 + e] += lo_f(r[e].y);
            x[12 + e] += hi_f(r[e].y);
          }
          store4(p.y + (t0 + t) * p.y_stride, n, p.n,
                 make_uint2(pack_bf16x2(x[e], x[4 + e]), pack_bf16x2(x[8 + e], x[12 + e])));
        }
      }
    }
    __syncwarp();
  }
  if (!ok && lane == 0) gave_up(p.err_count);

  cluster_wait();  // every CTA has received its parts: this one's are sent
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// Pairs of CTAs at work together (one on a single SM: the launch says that it has no room).
int pairs_of(int sm_count) { return sm_count < 2 ? 1 : sm_count / 2; }

// A launch in clusters of `size` CTAs that may start under the kernel before.
template <typename K, typename... Args>
cudaError_t launch_clusters(K kernel, dim3 grid, int threads, int smem, int size,
                            cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(size);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int BN, bool ACT, bool TAIL>
cudaError_t launch_pair_of(const LinearParams& p, const LinearMaps& m, int sm_count,
                        cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(linear_pair_kernel<BN, ACT, TAIL>, PP_SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.tokens + 255) / 256) * ((p.n + BN - 1) / BN);
  const int most = pairs_of(sm_count), pairs = tiles < most ? static_cast<int>(tiles) : most;
  return launch_overlapped(linear_pair_kernel<BN, ACT, TAIL>, dim3(2 * pairs), dim3(320), PP_SMEM,
                           stream, p, m.a, m.b, m.c);
}
template <int BN, bool ACT>
cudaError_t launch_pair(const LinearParams& p, const LinearMaps& m, int sm_count,
                        cudaStream_t stream) {
  return p.n % 8 ? launch_pair_of<BN, ACT, true>(p, m, sm_count, stream)
                 : launch_pair_of<BN, ACT, false>(p, m, sm_count, stream);
}

template <bool ACT>
cudaError_t launch_split(const LinearParams& p, const LinearMaps& m, cudaStream_t stream) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(linear_split_kernel<ACT>, SP_SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.tokens + 255) / 256) * ((p.n + 255) / 256);
  return launch_clusters(linear_split_kernel<ACT>, dim3(static_cast<unsigned>(tiles * 2 * p.splits)),
                         320, SP_SMEM, 2 * p.splits, stream, p, m.a, m.b);
}

template <int TN, bool ACT>
cudaError_t launch_few(const LinearParams& p, const LinearMaps& m, cudaStream_t stream) {
  using C = FewCfg<TN>;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(linear_few_kernel<TN, ACT>, C::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  return launch_clusters(linear_few_kernel<TN, ACT>,
                         dim3(static_cast<unsigned>((p.n + 127) / 128 * p.splits),
                              static_cast<unsigned>((p.tokens + TN - 1) / TN)),
                         192, C::SMEM, p.splits, stream, p, m.a, m.b);
}

template <bool ACT>
cudaError_t launch_any(const LinearParams& p, const LinearMaps& m, int sm_count,
                       cudaStream_t stream) {
  if (p.form == kLinearFew) {
    switch (p.bn) {
      case 16: return launch_few<16, ACT>(p, m, stream);
      case 32: return launch_few<32, ACT>(p, m, stream);
      case 64: return launch_few<64, ACT>(p, m, stream);
      default: return launch_few<128, ACT>(p, m, stream);
    }
  }
  if (p.splits > 1) return launch_split<ACT>(p, m, stream);
  switch (p.bn) {
    case 256: return launch_pair<256, ACT>(p, m, sm_count, stream);
    case 192: return launch_pair<192, ACT>(p, m, sm_count, stream);
    default: return launch_pair<128, ACT>(p, m, sm_count, stream);
  }
}

int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

// The kernel and tile with the least estimated time, in cycles.  A chunk of K
// takes what its operands' way into shared memory does, about 55 bytes a cycle
// and SM (7/3 cycles for a row of 128 bytes), or its products (2.16 cycles a
// column of 128 rows); a tile's start and end come to about 4000, once for a
// persistent CTA and for every wave of the kernel for few tokens.  Two CTAs of an
// SM share its rate, and clusters leave SMs out: of 152, those of 3, 4 and 8 CTAs
// fill 138, 144 and 120 (6 as many as 3, 7 fewer than 8).  Measured (us, clusters
// of 1, 2, 3, 4, 8, before the last steps): 16 x 2048 -> 5120 10.4, 7.1, 6.1, 6.8, 10.6;
// 64 tokens 12.5, 8.6, 7.8, 8.3, 14.1; 200 x 7168 -> 1536 35.7, 21.3, 16.8, 14.8, 21.1; 1
// x 8192 -> 7168 33, 22, 22, 20.3, 24; 8 x 7168 -> 576 28, 15.8, 11.9, 9.7, 7.0.  Pairs,
// tiles of 128, 192 and 256 columns: 512 x 2048 -> 5120 19.2, 14.3, 16.5; 1024 tokens
// 26.4, 21.9, 25.1; 4096 tokens 76, 60, 58.  Pairs that split K end 3 to 5 us later; 256
// columns and one, two, three, four parts: 442 x 9808 -> 3120 51.7, 30.9, 47.9, 42.4 (128
// columns, one part 43); 1008 x 11512 -> 1224 71, 40.9, 31.7, 50.7 (53); 256 x 18432 ->
// 7168 92, 58, 84, 70 (80); 256 x 2048 -> 5120 15.7, 13.8, 13.6, 24.0 (12.9).
LinearPlan linear_plan(int tokens, int n, int k, int sm_count) {
  const int64_t nk = cdiv64(k, KC);
  LinearPlan best = {};
  int64_t least = 0;
  auto take = [&](int64_t cost, const LinearPlan& plan) {
    if (least == 0 || cost < least) {
      least = cost;
      best = plan;
    }
  };
  auto chunk = [](int rows, int cols) {
    const int64_t loads = int64_t{rows} * 7 / 3, products = int64_t{cols} * 54 / 25;
    return loads > products ? loads : products;
  };
  if (tokens <= 1024) {
    const int tn = tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
    const int64_t ctas = cdiv64(n, 128) * cdiv64(tokens, tn);
    const int slots = tn == 128 ? 1 : 2;
    for (int s : {8, 4, 3, 2, 1}) {
      if (s > nk) continue;
      const int fit = s == 8 ? sm_count * 15 / 19 : s == 4 ? sm_count * 18 / 19
                                                : s == 3   ? sm_count * 10 / 11
                                                           : sm_count;
      if (fit < s) continue;  // (a part of a device with few SMs)
      take(cdiv64(ctas * s, fit) * cdiv64(nk, s) * chunk(128 + tn, 128) +
               cdiv64(ctas * s, slots * fit) * 4000,
           {kLinearFew, tn, s, tn, 128});
    }
  }
  if (tokens > 128) {
    const int most_pairs = pairs_of(sm_count);
    for (int bn = 256; bn >= 128; bn -= 64)
      take(cdiv64(cdiv64(tokens, 256) * cdiv64(n, bn), most_pairs) * nk *
                   chunk(128 + bn / 2, bn) + 4000,
           {kLinearPair, bn, 1, TM, bn / 2});
    const int64_t tiles = cdiv64(tokens, 256) * cdiv64(n, 256);
    for (int s = 2; s <= 4 && s <= nk; ++s) {
      const int fit = (s == 4 ? sm_count * 15 / 19 : s == 3 ? sm_count * 10 / 11
                                                            : sm_count * 18 / 19) / (2 * s);
      if (fit < 1) continue;
      take(cdiv64(tiles, fit) * (cdiv64(nk, s) * chunk(256, 256) + (s == 2 ? 9500 : 12000)),
           {kLinearPair, 256, s, TM, 128});
    }
  }
  return best;
}

cudaError_t launch_linear(const LinearParams& p, const LinearMaps& m, int sm_count,
                          cudaStream_t stream) {
  return p.act == kActNone ? launch_any<false>(p, m, sm_count, stream)
                           : launch_any<true>(p, m, sm_count, stream);
}

}  // namespace mla
