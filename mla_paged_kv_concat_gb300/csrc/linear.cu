// The layer's projections: y = act(x W^T + bias) + residual, x [T][K] and W
// [N][K] bf16 as a linear layer stores it, fp32 accumulation in TMEM and fp32
// epilogue, one rounding to bf16.
//
// One kernel: 128 tokens x BN columns per tile, K in chunks of 64 through a TMA
// ring (128-byte swizzle; what lies past K, N or T is filled with zeros),
// tcgen05 M=128 N=BN K=16, two accumulators in TMEM so that one tile's epilogue
// runs under the next one's products, one persistent CTA per SM.  Epilogue warps
// own 32 rows each: TMEM -> registers, bias, activation and residual there, bf16
// in a swizzled 4 KiB staging box -> TMA store, which clips the tensor's edges.
// The residual's next 64 columns are loaded while the current ones are worked on
// (the first before the accumulator is waited for).  Roles: warps 0-3 epilogue,
// warp 4 TMA producer, warp 5 MMA issuer and TMEM owner.
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

template <int BN>
struct Cfg {
  static constexpr int B_BYTES = BN * KC * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int OFF_STORE = STAGES * STAGE;  // two boxes per epilogue warp
  static constexpr int OFF_BAR = OFF_STORE + 4 * 2 * STORE_BYTES;
  static constexpr int NBARS = 2 * STAGES + 4;
  static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
  static constexpr int SMEM = OFF_TMEM + 16 + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
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

// The activation over a run of values; the choice is made once for all of them.
// gelu is written with erfc, whose small values keep their relative precision
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
      for (int i = 0; i < N; ++i) x[i] = __fdividef(x[i], 1.f + __expf(-x[i]));
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = 0.5f * x[i] * erfcf(x[i] * -0.70710678f);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i)
        x[i] = __fdividef(
            x[i], 1.f + __expf(-1.5957691f * x[i] * fmaf(0.044715f * x[i], x[i], 1.f)));
      break;
    default: break;
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

// One thread's 64 columns of the residual from column c on (zeros without one).
__device__ __forceinline__ void load_residual(const LinearParams& p, int row, int c,
                                              uint4 (&r)[8]) {
  const bool there = p.residual && row < p.tokens;
  const uint16_t* src = p.residual + (there ? row * p.res_stride : 0);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    r[q] = there ? load8(src, c + 8 * q, p.n) : make_uint4(0, 0, 0, 0);
}

// One epilogue warp's 32 rows x 64 columns: the accumulator's fp32 (a row a
// lane) through bias, activation and residual to bf16 in the swizzled box `dst`
// and from there to y (`some`: not all rows are past its end).
__device__ __forceinline__ void finish_box(const LinearParams& p, uint8_t* dst,
                                           const uint32_t (&r)[64], const uint4 (&res)[8], int lane,
                                           bool some, const CUtensorMap* map, int c, int row0) {
  // the store that last used this box, the one before the last, has read it
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r[q * 8 + e]);
    if (p.bias) {
      const uint4 b = load8(p.bias, c + 8 * q, p.n);
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] += lo_f(w[e]);
        x[2 * e + 1] += hi_f(w[e]);
      }
    }
    activate(p.act, x);
    const uint32_t w[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = p.residual ? pack_bf16x2(x[2 * e] + lo_f(w[e]), x[2 * e + 1] + hi_f(w[e]))
                        : pack_bf16x2(x[2 * e], x[2 * e + 1]);
    *reinterpret_cast<uint4*>(dst + sw128(lane, q)) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (some) tma_store_3d(map, dst, c, 0, row0);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
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

template <int BN>
__global__ void __launch_bounds__(192, 1)
    linear_kernel(const LinearParams p, const __grid_constant__ CUtensorMap ma,
                  const __grid_constant__ CUtensorMap mb, const __grid_constant__ CUtensorMap mc) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [STAGES]
  uint64_t* empty = full + C::STAGES;                               // [STAGES]
  uint64_t* acc_full = empty + C::STAGES;                           // [2]
  uint64_t* acc_empty = acc_full + 2;                               // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 128) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    fence_mbar_init();
  }
  if (warp == 5) {
    tc::tmem_alloc(tmem_slot, 2 * BN);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int nk = (p.k + KC - 1) / KC;
  const int mt = (p.tokens + TM - 1) / TM, nt = (p.n + BN - 1) / BN;
  const int64_t total = static_cast<int64_t>(mt) * nt;

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
        int m, n;
        tile_at(t, mt, nt, m, n);
        for (int kc = 0; kc < nk; ++kc, ++it) {
          const int st = it % C::STAGES;
          if (!mbar_wait(&empty[st], ((it / C::STAGES) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + st * C::STAGE;
          // fewer than 128 tokens: the tile's other rows hold what was there; an
          // accumulator's row depends on its own row of A only
          mbar_arrive_expect_tx(&full[st], p.a_rows * 128 + C::B_BYTES);
          tma_load_3d(dst, &ma, &full[st], kc * KC, 0, m * TM);
          tma_load_3d(dst + A_BYTES, &mb, &full[st], kc * KC, 0, n * BN);
        }
      }
      if (!ok) gave_up(p.err_count);
    }
  } else if (warp == 5) {
    constexpr uint32_t idesc = tc::idesc_bf16(TM, BN, 0, 0);
    int it = 0, ta = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x, ++ta) {
      const int a = ta & 1;
      if (!warp_wait(&acc_empty[a], ((ta >> 1) & 1) ^ 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      for (int kc = 0; kc < nk; ++kc, ++it) {
        const int st = it % C::STAGES;
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
            tc::mma_ss(tmem + a * BN, da + static_cast<uint64_t>(k * 2),
                       db + static_cast<uint64_t>(k * 2), idesc, (kc > 0 || k > 0) ? 1u : 0u);
          tc::commit(&empty[st]);
          if (kc == nk - 1) tc::commit(&acc_full[a]);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) gave_up(p.err_count);
    // nothing of this CTA's still runs on the tensor core when TMEM is freed
    for (int j = 0; ok && j < 2 && j < ta; ++j) {
      const int u = ta - 1 - j;
      warp_wait(&acc_full[u & 1], (u >> 1) & 1);
    }
  } else {
    uint8_t* box = smem + C::OFF_STORE + warp * 2 * STORE_BYTES;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    int ta = 0, nb = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x, ++ta) {
      int m, n;
      tile_at(t, mt, nt, m, n);
      const int a = ta & 1;
      const int row0 = m * TM + warp * STORE_ROWS;
      uint4 res[2][8];
      load_residual(p, row0 + lane, n * BN, res[0]);
      if (!warp_wait(&acc_full[a], (ta >> 1) & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
#pragma unroll
      for (int j = 0; j < BN / 64; ++j, ++nb) {
        uint32_t r[64];
        tc::ld_32x32b_x32(tmem + lanes + a * BN + j * 64,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tc::ld_32x32b_x32(tmem + lanes + a * BN + j * 64 + 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        const int c = n * BN + j * 64;
        if (j + 1 < BN / 64) load_residual(p, row0 + lane, c + 64, res[(j + 1) & 1]);
        tc::wait_ld();
        tc::reg_fence(r);
        if (j == BN / 64 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[a]);
        }
        finish_box(p, box + (nb & 1) * STORE_BYTES, r, res[j & 1], lane,
                   row0 < p.tokens && c < p.n, &mc, c, row0);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) gave_up(p.err_count);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 2 * BN);
  }
}

template <int BN>
cudaError_t launch(const LinearParams& p, const LinearMaps& m, int sm_count, cudaStream_t stream) {
  using C = Cfg<BN>;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(linear_kernel<BN>, C::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.tokens + TM - 1) / TM) * ((p.n + BN - 1) / BN);
  const int grid = tiles < sm_count ? static_cast<int>(tiles) : sm_count;
  return launch_overlapped(linear_kernel<BN>, dim3(grid), dim3(192), C::SMEM, stream, p, m.a, m.b,
                           m.c);
}

}  // namespace

// Columns of a tile: those for which the CTA with the most tiles takes in the
// fewest operand rows (tokens and columns; K is the same).
LinearPlan linear_plan(int tokens, int n, int k, int sm_count) {
  LinearPlan plan = {};
  plan.a_rows = tokens < TM ? tokens : TM;
  const int64_t blocks = (tokens + TM - 1) / TM;
  int64_t best = 0;
  for (int bn = 256; bn >= 64; bn /= 2) {
    const int64_t rounds = (blocks * ((n + bn - 1) / bn) + sm_count - 1) / sm_count;
    const int64_t cost = rounds * (plan.a_rows + bn);
    if (plan.bn == 0 || cost < best) {
      plan.bn = bn;
      best = cost;
    }
  }
  plan.b_rows = plan.bn;
  return plan;
}

cudaError_t launch_linear(const LinearParams& p, const LinearMaps& m, int sm_count,
                          cudaStream_t stream) {
  switch (p.bn) {
    case 256: return launch<256>(p, m, sm_count, stream);
    case 128: return launch<128>(p, m, sm_count, stream);
    default: return launch<64>(p, m, sm_count, stream);
  }
}

}  // namespace mla
