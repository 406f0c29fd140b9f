// The products with the kv_b weight W [H * 256][R] (per head h the rows
// [h*256, h*256+128) are W_UK[h], the next 128 are W_UV[h]):
//
//   expand   k_nope[t, h, p] = sum_r c[t, r] W_UK[h][p, r]
//            v[t, h, j]      = sum_r c[t, r] W_UV[h][j, r]
//   absorb   ql[t, h, r]     = sum_p q_nope[t, h, p] W_UK[h][p, r]
//   project  y[t, h, j]      = sum_r o[t, h, r] W_UV[h][j, r]
//
// bf16 in and out, fp32 accumulation in TMEM, one rounding.  All three read
// the weight where the model keeps it: expand and project with r contiguous
// (a K-major B operand), absorb with the output dim contiguous (MN-major).
//
// One kernel: 128 tokens x BN columns of one head per tile, K in chunks of
// 64 through a TMA ring (128-byte swizzle), tcgen05 M=128 N=BN K=16, two
// accumulators in TMEM so that one tile's epilogue runs under the next one's
// products, one persistent CTA per SM.  Epilogue warps own 32 rows each:
// TMEM -> registers -> bf16 in a swizzled 4 KiB staging box -> TMA store,
// which also clips the rows past the last token.  Roles: warps 0-3 epilogue,
// warp 4 TMA producer, warp 5 MMA issuer and TMEM owner.
// Measured: expand, 5001 tokens, 128 heads, R = 256, 77 us (4.28 TB/s written),
// into two buffers or the halves of one; the library's product into one matrix
// takes 70 and a plain fill 82, so neither memory nor the layout is the bound;
// absorb, 2048 tokens, 128 heads, 64 us; project, the same, 56 us (5.9 TB/s);
// absorb, 64 tokens, 16 heads, 3.3 us and project, 128 tokens, 128 heads, 5.7 us
// (11.1 with L2 flushed): launch, first loads and epilogue around short work
// (the library, to a head-major output: 2.2 and 4.2, flushed 10.3).
#include <cuda_bf16.h>
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int TM = 128;   // tokens per tile
constexpr int KC = 64;    // K per ring stage
constexpr int A_BYTES = TM * KC * 2;
constexpr int STORE_ROWS = 32;
constexpr int STORE_BYTES = STORE_ROWS * 128;

template <int BN>
struct ProjCfg {
  static constexpr int B_BYTES = BN * KC * 2;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int OFF_STORE = STAGES * STAGE;  // two boxes per epilogue warp
  static constexpr int OFF_BAR = OFF_STORE + 4 * 2 * STORE_BYTES;
  static constexpr int NBARS = 2 * STAGES + 4;
  static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
  static constexpr int SMEM = OFF_TMEM + 16 + 1024;
  static constexpr uint32_t COLS = 2 * BN;
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

// One epilogue warp's 32 rows x 64 columns: fp32 registers (a row a lane) to
// bf16 in the swizzled box `dst` and from there to the tensor, rows past its
// end left out by the TMA (`some`: not all of them are).
__device__ __forceinline__ void store_box(uint8_t* dst, const uint32_t (&r)[64], int lane, bool some,
                                          const CUtensorMap* map, int c, int h, int row0) {
  // the store that last used this box, the one before the last, has read it
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__uint_as_float(r[q * 8 + 2 * e]), __uint_as_float(r[q * 8 + 2 * e + 1]));
    *reinterpret_cast<uint4*>(dst + sw128(lane, q)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (some) tma_store_3d(map, dst, c, h, row0);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

template <int MODE, int BN>
__global__ void __launch_bounds__(192, 1)
    latent_proj_kernel(const ProjParams p, const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ CUtensorMap mc0,
                       const __grid_constant__ CUtensorMap mc1) {
  using C = ProjCfg<BN>;
  constexpr bool kBMn = MODE == kProjAbsorb;
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
    tc::tmem_alloc(tmem_slot, C::COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int nk = p.k / KC;
  const int ntiles_n = p.cols / BN;
  // columns of a head fastest, then heads, then token blocks: the tiles of a
  // wave write neighbouring columns of the same rows
  auto tile_at = [&](int64_t t, int& m, int& h, int& n) {
    n = static_cast<int>(t % ntiles_n);
    const int64_t u = t / ntiles_n;
    h = static_cast<int>(u % p.heads);
    m = static_cast<int>(u / p.heads);
  };
  const int64_t total =
      static_cast<int64_t>((p.tokens + TM - 1) / TM) * p.heads * ntiles_n;

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
        int m, h, n;
        tile_at(t, m, h, n);
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
          tma_load_3d(dst, &ma, &full[st], kc * KC, MODE == kProjExpand ? 0 : h, m * TM);
          if (kBMn) {
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              tma_load_3d(dst + A_BYTES + j * (KC * 128), &mb, &full[st], n * BN + j * 64,
                          p.w_row0 + kc * KC, h);
          } else {
            tma_load_3d(dst + A_BYTES, &mb, &full[st], kc * KC, p.w_row0 + n * BN, h);
          }
        }
      }
      if (!ok) gave_up(p.err_count);
    }
  } else if (warp == 5) {
    constexpr uint32_t idesc = tc::idesc_bf16(TM, BN, 0, kBMn ? 1 : 0);
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
          // MN-major: the next 64 columns are one box on, 16 rows of K 2 KiB
          const uint64_t db =
              tc::smem_desc(base + A_BYTES, kBMn ? KC * 128 : 16, 1024, tc::kLayoutSw128);
#pragma unroll
          for (int k = 0; k < KC / 16; ++k)
            tc::mma_ss(tmem + a * BN, da + static_cast<uint64_t>(k * 2),
                       db + static_cast<uint64_t>(kBMn ? k * 128 : k * 2), idesc,
                       (kc > 0 || k > 0) ? 1u : 0u);
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
      int m, h, n;
      tile_at(t, m, h, n);
      const int a = ta & 1;
      if (!warp_wait(&acc_full[a], (ta >> 1) & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const int row0 = m * TM + warp * STORE_ROWS;
#pragma unroll
      for (int j = 0; j < BN / 64; ++j, ++nb) {
        uint32_t r[64];
        tc::ld_32x32b_x32(tmem + lanes + a * BN + j * 64,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tc::ld_32x32b_x32(tmem + lanes + a * BN + j * 64 + 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        tc::wait_ld();
        tc::reg_fence(r);
        if (j == BN / 64 - 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[a]);
        }
        const int c = n * BN + j * 64;
        const bool second = MODE == kProjExpand && c >= 128;
        store_box(box + (nb & 1) * STORE_BYTES, r, lane, row0 < p.tokens, second ? &mc1 : &mc0,
                  second ? c - 128 : c, h, row0);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok && lane == 0) gave_up(p.err_count);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::COLS);
  }
}

// ---------------------------------------------------------------- CTA pairs
// expand with a long sum (R = 512) for many tokens, which the tensor core
// bounds.  Two CTAs of a cluster share a tile of 256 tokens x 256 columns (one
// head's W_UK | W_UV): each holds its 128 tokens of A and half of the columns
// of B, and cta_group::2 products read both halves, so a CTA takes in 32 KiB
// per 552 cycles of products instead of 48.  Rank 0 issues for both; the ring's
// "landed" barrier is rank 0's and counts both CTAs' bytes; "read" and
// "accumulator ready" arrive in both.  Eight epilogue warps, four per output.
// 8192 tokens, 16 heads: 25.4 us (1353 TFLOP/s; the library's single matrix
// 21.1) against 27.6 for single CTAs; with four epilogue warps no faster than
// those.  With R = 256 there are half the products to the same bytes written and
// pairs, which drain together, lose: 5001 tokens, 128 heads 100 us against 77.
constexpr int kPairStages = 5;
constexpr int kPairHalf = A_BYTES;  // A, and the half of B, of one stage
constexpr int PP_STORE = kPairStages * 2 * kPairHalf;
constexpr int PP_BAR = PP_STORE + 8 * 2 * STORE_BYTES;
constexpr int PP_TMEM = PP_BAR + (2 * kPairStages + 4) * 8;
constexpr int PP_SMEM = PP_TMEM + 16 + 1024;
static_assert(PP_SMEM <= 227 * 1024, "shared memory");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(320, 1)
    expand_pair_kernel(const ProjParams p, const __grid_constant__ CUtensorMap ma,
                       const __grid_constant__ CUtensorMap mb,
                       const __grid_constant__ CUtensorMap mc0,
                       const __grid_constant__ CUtensorMap mc1) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + PP_BAR);  // [stages] rank 0's: both landed
  uint64_t* empty = full + kPairStages;                         // [stages]
  uint64_t* acc_full = empty + kPairStages;                     // [2]
  uint64_t* acc_empty = acc_full + 2;                           // [2] rank 0's: eight warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + PP_TMEM);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();

  if (threadIdx.x == 128) {
    tma_prefetch_desc(&ma);
    tma_prefetch_desc(&mb);
  }
  if (threadIdx.x == 0) {
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
  if (warp == 5) {
    tc::pair_tmem_alloc(tmem_slot, 512);
    tc::pair_tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  const int nk = p.k / KC;
  // heads fastest, then blocks of 256 tokens
  const int64_t total = static_cast<int64_t>((p.tokens + 2 * TM - 1) / (2 * TM)) * p.heads;
  const int64_t first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 4) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int64_t t = first; t < total && ok; t += step) {
        const int h = static_cast<int>(t % p.heads), m = static_cast<int>(t / p.heads);
        for (int kc = 0; kc < nk; ++kc, ++it) {
          const int st = it % kPairStages;
          if (!mbar_wait(&empty[st], ((it / kPairStages) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* dst = smem + st * 2 * kPairHalf;
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 4 * kPairHalf);
          const uint32_t bar = tc::map_peer(smem_u32(&full[st]), 0);
          tc::pair_tma_load_3d(dst, &ma, bar, kc * KC, 0, m * 2 * TM + rank * TM);
          tc::pair_tma_load_3d(dst + kPairHalf, &mb, bar, kc * KC, rank * 128, h);
        }
      }
      if (!ok) gave_up(p.err_count);
    }
  } else if (warp == 5) {
    bool ok = true;
    int it = 0, ta = 0;
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_bf16(2 * TM, 256, 0, 0);
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
    // warps 0-3 k_nope's columns, 6-9 v's; a warp reads the TMEM lanes of its
    // quarter (warp % 4)
    const int half = warp >= 6, ew = half ? warp - 2 : warp, qd = warp & 3;
    uint8_t* box = smem + PP_STORE + ew * 2 * STORE_BYTES;
    const uint32_t lanes = static_cast<uint32_t>(qd * 32) << 16;
    int ta = 0, nb = 0;
    bool ok = true;
    for (int64_t t = first; t < total; t += step, ++ta) {
      const int h = static_cast<int>(t % p.heads), m = static_cast<int>(t / p.heads);
      const int a = ta & 1;
      if (!warp_wait(&acc_full[a], (ta >> 1) & 1)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const int row0 = m * 2 * TM + rank * TM + qd * STORE_ROWS;
#pragma unroll
      for (int jj = 0; jj < 2; ++jj, ++nb) {
        const int j = half * 2 + jj;
        uint32_t r[64];
        tc::ld_32x32b_x32(tmem + lanes + a * 256 + j * 64,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
        tc::ld_32x32b_x32(tmem + lanes + a * 256 + j * 64 + 32,
                          *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
        tc::wait_ld();
        tc::reg_fence(r);
        if (jj == 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::arrive_peer(tc::map_peer(smem_u32(&acc_empty[a]), 0));
        }
        store_box(box + (nb & 1) * STORE_BYTES, r, lane, row0 < p.tokens, j < 2 ? &mc0 : &mc1,
                  (j & 1) * 64, h, row0);
      }
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

template <int MODE, int BN>
cudaError_t launch(const ProjParams& p, const ProjMaps& m, int sm_count, cudaStream_t stream) {
  using C = ProjCfg<BN>;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(latent_proj_kernel<MODE, BN>, C::SMEM, attr_done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.tokens + TM - 1) / TM) * p.heads * (p.cols / BN);
  const int grid = tiles < sm_count ? static_cast<int>(tiles) : sm_count;
  return launch_overlapped(latent_proj_kernel<MODE, BN>, dim3(grid), dim3(192), C::SMEM, stream, p,
                           m.a, m.b, m.c0, m.c1);
}

template <int MODE>
cudaError_t launch_mode(const ProjParams& p, const ProjMaps& m, int sm_count, cudaStream_t s) {
  switch (p.bn) {
    case 256: return launch<MODE, 256>(p, m, sm_count, s);
    case 128: return launch<MODE, 128>(p, m, sm_count, s);
    default: return launch<MODE, 64>(p, m, sm_count, s);
  }
}

}  // namespace

// Pairs where the products bound the work and their tiles, twice as high,
// still come several to an SM (R = 512: 1000 tokens, 128 heads 27.7 us against
// 30.1; 300 tokens, 128 heads, 256 tiles, 15.1 against 13.8).
bool proj_pairs(int mode, int tokens, int heads, int k, int sm_count) {
  return mode == kProjExpand && k > 256 && tokens > TM &&
         static_cast<int64_t>((tokens + 2 * TM - 1) / (2 * TM)) * heads >= 2 * sm_count;
}

// Columns of a tile: those for which the CTA with the most tiles takes in the
// fewest operand rows (tokens and columns; K is the same).  project, 128 tokens,
// 128 heads: 128 columns, one tile a CTA 6.0 us, 64 columns, two, 7.4; absorb, 64
// tokens, 16 heads: 64 columns 3.6 us, 256 4.8.  Large absorbs, which write
// much for their work (a sum of 128 terms an element), do better with narrower
// tiles once there are many: 2048 tokens, 128 heads, R = 512 64 us at 128 columns,
// 72 at 256; 4096 tokens, 32 heads 32.1 and 33.3; but 500 tokens,
// 128 heads 18.6 and 17.1; expand, R = 256, 5001 tokens, 128 heads 88 and 78.
int proj_tile_cols(int mode, int tokens, int heads, int cols, int sm_count) {
  const int64_t blocks = static_cast<int64_t>((tokens + TM - 1) / TM) * heads;
  if (mode == kProjAbsorb && blocks * (cols / 128) >= 24 * static_cast<int64_t>(sm_count)) return 128;
  const int rows = tokens < TM ? tokens : TM;
  int best = 0;
  int64_t best_cost = 0;
  for (int bn = cols < 256 ? cols : 256; bn >= 64; bn /= 2) {
    const int64_t rounds = (blocks * (cols / bn) + sm_count - 1) / sm_count;
    const int64_t cost = rounds * (rows + bn);
    if (best == 0 || cost < best_cost) {
      best = bn;
      best_cost = cost;
    }
  }
  return best;
}

cudaError_t launch_latent_proj(const ProjParams& p, const ProjMaps& m, int mode, int sm_count,
                               cudaStream_t stream) {
  if (p.pair) {
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = set_smem_attr_once(expand_pair_kernel, PP_SMEM, attr_done);
    if (e != cudaSuccess) return e;
    const int64_t tiles = static_cast<int64_t>((p.tokens + 2 * TM - 1) / (2 * TM)) * p.heads;
    const int pairs = tiles < sm_count / 2 ? static_cast<int>(tiles) : sm_count / 2;
    return launch_overlapped(expand_pair_kernel, dim3(2 * pairs), dim3(320), PP_SMEM, stream, p, m.a,
                             m.b, m.c0, m.c1);
  }
  switch (mode) {
    case kProjExpand: return launch_mode<kProjExpand>(p, m, sm_count, stream);
    case kProjAbsorb: return launch_mode<kProjAbsorb>(p, m, sm_count, stream);
    default: return p.bn == 128 ? launch<kProjProject, 128>(p, m, sm_count, stream)
                                : launch<kProjProject, 64>(p, m, sm_count, stream);
  }
}

}  // namespace mla
