// Prompt attention of the expanded form: every head has its own keys (128
// dims, plus 64 rope dims that all heads share) and values (128 dims), ragged
// sequences, causal or not.
//
//   s_ij  = sm_scale * (q_nope_i . k_nope_j + q_pe_i . k_pe_j),
//           j <= i + Lk - Lq when causal (queries are the last tokens)
//   o_i   = sum_j softmax(s_i)_j v_j,   lse_i = ln sum_j exp(s_ij)
//
// One pass over the keys with the running maximum and sum of the softmax; O
// is rescaled only when a row's maximum has grown by more than 2^8, so the
// unnormalised P stays below 2^8 and fp32 sums lose nothing.  P is rounded to
// bf16 for the second product; the sum adds the fp32 values.
//
// Work.  A unit is 256 query rows of one sequence and head (two tiles of 128)
// and a range of its keys.  The grid has one CTA per unit, longest first; one
// CTA runs on an SM and, instead of ending, takes over the next CTA that has
// not started (cluster launch control), so that the work is shared out as
// it goes, without a counter in memory.  Per 128 keys the tensor core has 2 x
// (888 + 592) cycles of work (M = 128: 192 dims of Q.K at N = 128, then 128 keys
// of P.V at N = 128, 74 cycles an instruction), a tile's softmax takes 1250
// (two cycles an instruction of one warp, four an exponential): with two query
// tiles in turn, one tile's softmax runs under the other's products.  A tile's
// own chain - softmax, barriers, its products - comes to ~3050 and is the
// bound.  Measured: a prompt of 8192 tokens, 16 heads, 217 us, 1580 TFLOP/s of
// the causal half, tensor core 70 % busy (176 us without softmax and loads);
// 17 rows against eight contexts of up to 32768 keys, 218 us, 5.7 TB/s.
//   TMEM (512 columns): S0, S1 (128 each; P as packed bf16 over the first 64
//     of its S), O0, O1 (128 each).
//   Shared memory: Q 2 x 48 KiB, a ring of eight 16 KiB boxes in the order K
//     K K (64 dims x 128 keys each) V V (128 dims x 64 keys each) of every key
//     tile, filled and freed box by box in the order of their use: a box is
//     asked for 1800 to 3000 cycles before its product (K and V waited for
//     together, freed as groups: 770 cycles, less than a load takes).
// The tensor core is kept busy only if its instructions arrive in time: one
// issuing warp spent ~2000 cycles on a step (P.V of a tile, then Q.K of its
// next one: 20 instructions at 25-45 cycles, and ~100 for each wait, vote and
// commit), so each query tile has an issuing warp of its own, with one vote
// and one elected block for P.V and one for Q.K; the commits follow the
// products (between them they cost 3 %).
//
// Roles: warps 0-3 and 4-7 the softmax of query tiles 0 and 1 (thread = TMEM
// lane = query row), warp 8 TMA producer and unit scheduler, warps 9 and 10
// MMA issuers of query tiles 0 and 1, warp 11 value keeper.
//
// Masked keys.  Scores of masked keys are replaced by -inf, whatever K held.
// V of a masked key would still meet a zero of P, and 0 * NaN is NaN: in the
// tiles that a mask cuts, the keeper zeroes the rows past the sequence's end
// and any value that is not finite, and notes the keys these were found in;
// the epilogue adds them back for the rows that do attend to those keys.
#include <cuda_bf16.h>
#include <stdint.h>

#include "kernels.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace mla {

namespace {

constexpr int kDv = 128;               // value dims
constexpr int kTile = 128;             // query rows of a tile, keys of a tile
constexpr int kUnitRows = 2 * kTile;
constexpr int kBox = 16384;            // 64 dims x 128 rows of bf16
constexpr int kRing = 8;               // boxes
constexpr int kUnits = 4;              // unit descriptions in flight
constexpr int kThreads = 384;
constexpr int OFF_Q = 0;
constexpr int OFF_RING = OFF_Q + 6 * kBox;
constexpr int OFF_UNIT = OFF_RING + kRing * kBox;
constexpr int OFF_FLAG = OFF_UNIT + kUnits * 64;
constexpr int kCuCached = 64;          // cumulative lengths kept in shared memory
constexpr int OFF_CU = OFF_FLAG + kUnits * 64;
constexpr int OFF_BAR = OFF_CU + 2 * kCuCached * 4;
constexpr int kBars = 2 * kRing + 2 * kUnits + 15;
constexpr int OFF_NEXT = (OFF_BAR + kBars * 8 + 15) & ~15;
constexpr int OFF_TMEM = OFF_NEXT + 16;
constexpr int kSmem = OFF_TMEM + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t O_COL = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units
// Largest |m c| that is subtracted from s c in one operation: what m c's own
// rounding leaves, 2^-8 here, is a factor of P, and from 2^31 on passes any
// range.  For a row of larger scores m is taken off S in TMEM and the tile read
// again.
constexpr float kLarge = 65536.0f;  // log2 units

struct Unit {
  int q_row;   // first query row (of all tokens); -1: no more units
  int rows;    // query rows, 1 .. 256
  int k_row;   // first key row of the sequence
  int h;
  int split;
  int lk;      // keys of the sequence
  int lim0;    // keys the first row may attend to (lk when not causal)
  int ks, ke;  // this unit's keys [ks, ke)
  int n0, n1;  // key tiles of each query tile
  __device__ __forceinline__ int n(int t) const { return t == 0 ? n0 : n1; }
  __device__ __forceinline__ int most() const { return max(n0, n1); }
};
static_assert(sizeof(Unit) <= 64, "unit slot");

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// Keys that row r (0 .. 255) of the unit may attend to, counted from the
// sequence's first.
__device__ __forceinline__ int row_limit(const Unit& u, int r, bool causal) {
  return causal ? min(u.lk, u.lim0 + r) : u.lk;
}

// First key tile that a mask cuts (for some row of some tile).
__device__ __forceinline__ int first_masked(const Unit& u, int row0, bool causal) {
  const int bound = min(u.ke, row_limit(u, row0, causal));
  return bound <= u.ks ? 0 : (bound - u.ks) / kTile;
}

// Unit `x` of the launch; false when it is empty.  Sequence b owns the block
// slots from cu_q[b] / 256 + b on, at least as many as it has blocks, so
// that a slot is found by one binary search with no sums.  Blocks run from
// the last to the first (with a causal mask the longest come first); the
// heads of a group share a block's turn, so that the CTAs at work together
// read few heads' keys, from L2.
// `cu_q`, `cu_k`: p's, or their copies in shared memory.
__device__ bool unit_at(const PrefillParams& p, const int32_t* cu_q, const int32_t* cu_k,
                        uint32_t x, Unit& u) {
  const uint32_t x1 = x / p.num_splits, x2 = x1 / p.head_group, x3 = x2 / p.slots;
  u.split = static_cast<int>(x - x1 * p.num_splits);
  u.h = static_cast<int>(x3 * p.head_group + (x1 - x2 * p.head_group));
  const int slot = p.slots - 1 - static_cast<int>(x2 - x3 * p.slots);
  if (u.h >= p.heads) return false;
  int a = 0, z = p.num_seqs - 1;
  while (a < z) {
    const int m = (a + z + 1) >> 1;
    const int c = clampi(cu_q[m], 0, p.num_tokens);
    if (c / kUnitRows + m <= slot) a = m; else z = m - 1;
  }
  const int q0 = cu_q[a], q1 = cu_q[a + 1];
  const int k0 = cu_k[a], k1 = cu_k[a + 1];
  const int qa = clampi(q0, 0, p.num_tokens), qz = clampi(q1, qa, p.num_tokens);
  const int ka = clampi(k0, 0, p.num_kv), kz = clampi(k1, ka, p.num_kv);
  const int blk = slot - (qa / kUnitRows + a);
  if (blk == 0 && u.h == 0 && u.split == 0 && p.err_count &&
      (qa != q0 || qz != q1 || ka != k0 || kz != k1))
    atomicAdd(p.err_count, 1);
  const int lq = qz - qa;
  u.lk = kz - ka;
  const int r0 = blk * kUnitRows;
  if (blk < 0 || r0 >= lq) return false;
  u.q_row = qa + r0;
  u.k_row = ka;
  u.rows = min(kUnitRows, lq - r0);
  u.lim0 = p.causal ? r0 + (u.lk - lq) + 1 : u.lk;
  const int per = ((u.lk + p.num_splits - 1) / p.num_splits + kTile - 1) / kTile * kTile;
  const int64_t ks = static_cast<int64_t>(u.split) * per;
  u.ks = ks < u.lk ? static_cast<int>(ks) : u.lk;
  u.ke = ks + per < u.lk ? static_cast<int>(ks + per) : u.lk;
  auto tiles = [&](int t) {
    const int last = min(u.rows, (t + 1) * kTile) - 1;
    const int keys = min(u.ke, row_limit(u, last, p.causal)) - u.ks;
    return u.rows > t * kTile && keys > 0 ? (keys + kTile - 1) / kTile : 0;
  };
  u.n0 = tiles(0);
  u.n1 = tiles(1);
  return true;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Cluster launch control: asks to cancel a CTA of this grid that has not been
// started, to run it here; the answer (16 bytes) arrives in `dst` on `bar`.
__device__ __forceinline__ void next_cta_ask(void* dst, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(smem_u32(dst)),
      "r"(smem_u32(bar))
      : "memory");
}
// The answer: the cancelled CTA's index, or -1 when none was left.
__device__ __forceinline__ int64_t next_cta_answer(const void* src) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(src);
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "mov.b128 h, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "l"(a.x), "l"(a.y)
      : "memory");
  return got ? static_cast<int64_t>(x) : -1;
}

// 32 bytes to a 32-byte aligned address.
__device__ __forceinline__ void store32(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

__device__ __forceinline__ bool finite_bf16(uint32_t h) { return (h & 0x7F80u) != 0x7F80u; }

template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const PrefillParams p, const __grid_constant__ PrefillMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* full = bars;                     // [kRing] box landed
  uint64_t* empty = full + kRing;            // [kRing] read by both query tiles
  uint64_t* unit_full = empty + kRing;       // [kUnits]
  uint64_t* unit_empty = unit_full + kUnits; // [kUnits] 11 reading warps
  uint64_t* q_full = unit_empty + kUnits;    // [2]
  uint64_t* q_empty = q_full + 2;            // [2]
  uint64_t* s_full = q_full + 4;             // [2]
  uint64_t* p_full = q_full + 6;             // [2] P written, O rescaled
  uint64_t* o_full = q_full + 8;             // [2] the unit's last P.V done
  uint64_t* next_full = q_full + 14;         // the next CTA's index arrived
  uint64_t* cut_full = q_full + 12;          // [2] a cut tile's values landed (the keeper does not
                                             // follow the ring box by box)
  uint64_t* v_ok = q_full + 10;              // [2] a cut tile's values are clean (in turn: the
                                             // ring holds two tiles' values)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
  auto unit_slot = [&](int i) { return reinterpret_cast<Unit*>(smem + OFF_UNIT + (i % kUnits) * 64); };
  // keys with values that are not finite: 4 words for each of a unit's cut tiles
  auto flags = [&](int i) { return reinterpret_cast<uint32_t*>(smem + OFF_FLAG + (i % kUnits) * 64); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);  // both query tiles
    }
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(&unit_full[i], 1);
      mbar_init(&unit_empty[i], 11);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cut_full[i], 1);
      mbar_init(&v_ok[i], 32);
    }
    mbar_init(next_full, 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  // One reading warp's walk over the units: f(unit, index) until the end
  // mark or a failed wait.  The softmax warps give the unit's slot back when
  // they are done with it, flags included.
  auto for_each_unit = [&](bool keep, auto&& f) -> bool {
    for (int i = 0;; ++i) {
      if (!warp_wait(&unit_full[i % kUnits], (i / kUnits) & 1)) return false;
      const Unit u = *unit_slot(i);
      __syncwarp();
      if (!keep && lane == 0) mbar_arrive(&unit_empty[i % kUnits]);
      if (u.q_row < 0) return true;
      if (!f(u, i)) return false;
      if (keep) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&unit_empty[i % kUnits]);
      }
    }
  };

  bool ok = true;
  if (warp >= 8) {
    reg_dec<104>();
    if (warp == 8) {
      // ---------------------------------------------------------- producer
      // a few sequences' lengths come in at once, not one search step after
      // the other
      const int32_t *cu_q = p.cu_q, *cu_k = p.cu_k;
      if (p.num_seqs < kCuCached) {
        int32_t* cu = reinterpret_cast<int32_t*>(smem + OFF_CU);
        for (int b = lane; b <= p.num_seqs; b += 32) {
          cu[b] = __ldg(p.cu_q + b);
          cu[kCuCached + b] = __ldg(p.cu_k + b);
        }
        __syncwarp();
        cu_q = cu;
        cu_k = cu + kCuCached;
      }
      if (lane == 0) {
        int i = 0, cut = 0, pos = 0, qn[2] = {0, 0};
        // The next box of the ring, once it is free.
        auto slot = [&]() -> int {
          const int b = pos % kRing;
          if (ok) ok = mbar_wait(&empty[b], ((pos / kRing) & 1) ^ 1);
          ++pos;
          return b;
        };
        auto load_q = [&](const Unit& u, int t) {
          if (u.n(t) == 0) return;
          if (ok) ok = mbar_wait(&q_empty[t], (qn[t] & 1) ^ 1);
          if (!ok) return;
          ++qn[t];
          mbar_arrive_expect_tx(&q_full[t], 3 * kBox);
          uint8_t* dst = smem + OFF_Q + t * 3 * kBox;
          const int row = u.q_row + t * kTile;
          tma_load_3d(dst, &maps.q, &q_full[t], 0, u.h, row);
          tma_load_3d(dst + kBox, &maps.q, &q_full[t], 64, u.h, row);
          if (p.pe_col)
            tma_load_3d(dst + 2 * kBox, &maps.q, &q_full[t], p.pe_col, u.h, row);
          else
            tma_load_3d(dst + 2 * kBox, &maps.q_pe, &q_full[t], 0, u.h, row);
        };
        auto load_k = [&](const Unit& u, int j) {
          const int row = u.k_row + u.ks + j * kTile;
          for (int c = 0; c < 3; ++c) {
            const int b = slot();
            if (!ok) return;
            mbar_arrive_expect_tx(&full[b], kBox);
            tma_load_3d(smem + OFF_RING + b * kBox, c < 2 ? &maps.k : &maps.k_pe, &full[b],
                        c < 2 ? c * 64 : 0, c < 2 ? u.h : 0, row);
          }
        };
        auto load_v = [&](const Unit& u, int j) {
          const int row = u.k_row + u.ks + j * kTile;
          uint64_t* cut_bar = nullptr;
          if (j >= first_masked(u, 0, p.causal)) cut_bar = &cut_full[cut++ & 1];
          for (int c = 0; c < 2; ++c) {
            const int b = slot();
            if (!ok) return;
            uint64_t* bar = &full[b];
            if (cut_bar) {
              mbar_arrive(bar);  // keeps the ring's count; v_ok follows
              bar = cut_bar;
              if (c == 0) mbar_arrive_expect_tx(bar, 2 * kBox);
            } else {
              mbar_arrive_expect_tx(bar, kBox);
            }
            uint8_t* dst = smem + OFF_RING + b * kBox;
            tma_load_3d(dst, &maps.v, bar, 0, u.h, row + c * 64);
            tma_load_3d(dst + kBox / 2, &maps.v, bar, 64, u.h, row + c * 64);
          }
        };
        int64_t x = blockIdx.x;
        for (int asked = 0;; ++asked) {
          // The next unit is asked for when this one's last key tiles are to be
          // loaded: early enough to be there, and no unit waits here while
          // another CTA has nothing to do (asked for at a unit's start, 128
          // units of one sequence's splits took as long as twice as many).
          bool ask = x >= 0;
          Unit u;
          if (x < 0) u.q_row = -1;
          // after a wait that gave up, the CTAs left are taken over and dropped
          if (ok && (x < 0 || unit_at(p, cu_q, cu_k, static_cast<uint32_t>(x), u))) {
            ok = mbar_wait(&unit_empty[i % kUnits], ((i / kUnits) & 1) ^ 1);
            if (ok) {
              *unit_slot(i) = u;
              mbar_arrive(&unit_full[i % kUnits]);
              ++i;
              const int n = x < 0 ? 0 : u.most();
              if (n > 0) {
                load_q(u, 0);
                load_k(u, 0);
                load_q(u, 1);
                load_v(u, 0);
              }
              for (int j = 1; j < n && ok; ++j) {
                if (ask && j >= n - 2) {
                  next_cta_ask(smem + OFF_NEXT, next_full);
                  ask = false;
                }
                load_k(u, j);
                load_v(u, j);
              }
            }
          }
          if (ask) next_cta_ask(smem + OFF_NEXT, next_full);
          if (x < 0 || !mbar_wait(next_full, asked & 1)) break;
          x = next_cta_answer(smem + OFF_NEXT);
          fence_proxy_async_smem();  // read before the next answer is written
        }
      }
    } else if (warp < 11) {
      // ------------------------------------------------------- MMA issuers
      constexpr uint32_t id_qk = tc::idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t id_pv = tc::idesc_bf16(128, 128, 0, 1);
      constexpr uint64_t kBoxStep = kBox >> 4;  // a box, in a descriptor's address field
      const int t = warp - 9;
      const uint32_t s_tm = tmem + t * 128, o_tm = tmem + O_COL + t * 128;
      const uint64_t q_desc =
          tc::smem_desc(smem_u32(smem + OFF_Q + t * 3 * kBox), 16, 1024, tc::kLayoutSw128);
      const uint32_t ring = smem_u32(smem + OFF_RING);
      const uint64_t k_desc = tc::smem_desc(ring, 16, 1024, tc::kLayoutSw128);
      // V is MN-major: the other 64 dims are half a box on, 16 keys 2 KiB
      const uint64_t v_desc = tc::smem_desc(ring, kBox / 2, 1024, tc::kLayoutSw128);
      int pos = 0;                // first box of the unit
      int qn = 0, pn = 0, vn = 0;
      auto ready = [&](int b) { return mbar_try_wait(&full[b % kRing], (b / kRing) & 1); };
      auto await = [&](int b) { return mbar_wait(&full[b % kRing], (b / kRing) & 1); };
      // S = Q K^T, the tile's first box at ring position `b`
      auto qk = [&](int b, bool last) -> bool {
        bool r = ready(b);
        r = ready(b + 1) && r;
        r = ready(b + 2) && r;
        if (!__all_sync(0xffffffffu, r)) {
          r = await(b);
          r = await(b + 1) && r;
          r = await(b + 2) && r;
          if (!__all_sync(0xffffffffu, r)) return false;
        }
        tc::fence_after_sync();
        if (tc::elect_one()) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t db = k_desc + static_cast<uint64_t>((b + c) % kRing) * kBoxStep;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma_ss(s_tm, q_desc + c * kBoxStep + static_cast<uint64_t>(k * 2),
                         db + static_cast<uint64_t>(k * 2), id_qk, (c > 0 || k > 0) ? 1u : 0u);
            if (c == 2) tc::commit(&s_full[t]);
          }
#pragma unroll
          for (int c = 0; c < 3; ++c) tc::commit(&empty[(b + c) % kRing]);
          if (last) tc::commit(&q_empty[t]);
        }
        __syncwarp();
        return true;
      };
      ok = for_each_unit(false, [&](const Unit& u, int) -> bool {
        const int n = u.most(), nt = u.n(t);
        if (n == 0) return true;
        const int im = first_masked(u, 0, p.causal);
        if (nt > 0) {
          if (!warp_wait(&q_full[t], qn & 1)) return false;
          ++qn;
          if (!qk(pos, nt == 1)) return false;
        }
        for (int j = 0; j < nt; ++j, ++pn) {
          // O (+)= P V of key tile j
          int b = pos + 5 * j + 3;
          const bool cut = j >= im;
          bool r = ready(b);
          r = ready(b + 1) && r;
          if (cut) r = mbar_try_wait(&v_ok[vn & 1], (vn >> 1) & 1) && r;
          r = mbar_try_wait(&p_full[t], pn & 1) && r;
          if (!__all_sync(0xffffffffu, r)) {
            r = await(b);
            r = await(b + 1) && r;
            if (cut) r = mbar_wait(&v_ok[vn & 1], (vn >> 1) & 1) && r;
            r = mbar_wait(&p_full[t], pn & 1) && r;
            if (!__all_sync(0xffffffffu, r)) return false;
          }
          if (cut) ++vn;
          tc::fence_after_sync();
          if (tc::elect_one()) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint64_t dv = v_desc + static_cast<uint64_t>((b + c) % kRing) * kBoxStep;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_ts(o_tm, s_tm + (c * 4 + k) * 8, dv + static_cast<uint64_t>(k * 128), id_pv,
                           (c > 0 || k > 0 || j > 0) ? 1u : 0u);
              tc::commit(&empty[(b + c) % kRing]);
            }
            if (j + 1 == nt) tc::commit(&o_full[t]);
          }
          __syncwarp();
          // S of the next one, whose keys may still be on their way
          if (j + 1 < nt && !qk(b + 2, j + 2 == nt)) return false;
        }
        // key tiles that only the other query tile reads
        for (int b = pos + 5 * nt; b < pos + 5 * n; ++b) {
          if ((b - pos) % 5 == 3 && (b - pos) / 5 >= im) ++vn;
          if (!__all_sync(0xffffffffu, await(b))) return false;
          if (lane == 0) mbar_arrive(&empty[b % kRing]);
        }
        pos += 5 * n;
        return true;
      });
    } else {
      // ------------------------------------------------------ value keeper
      int pos = 0, vn = 0;
      ok = for_each_unit(false, [&](const Unit& u, int i) -> bool {
        const int n = u.most(), im = first_masked(u, 0, p.causal);
        for (int j = im; j < n; ++j, ++vn) {
          const int b = pos + 5 * j + 3;
          if (!warp_wait(&cut_full[vn & 1], (vn >> 1) & 1)) return false;
          const int valid = u.lk - (u.ks + j * kTile);  // keys of the sequence in this tile
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int r = q * 32 + lane;  // key of the tile
            uint8_t* box = smem + OFF_RING + ((b + (r >> 6)) % kRing) * kBox;
            auto at = [&](int c) { return box + (c >> 3) * (kBox / 2) + sw128(r & 63, c & 7); };
            const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
            __nv_bfloat162 z[4] = {zero, zero, zero, zero};
            if (r < valid) {
#pragma unroll
              for (int c = 0; c < 16; ++c) {
                // 0 * x stays 0 unless x is not finite
                const uint4 x = *reinterpret_cast<const uint4*>(at(c));
                z[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, z[0]);
                z[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, z[1]);
                z[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, z[2]);
                z[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, z[3]);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                *reinterpret_cast<uint4*>(at(c)) = make_uint4(0, 0, 0, 0);
            }
            z[0] = __hadd2(__hadd2(z[0], z[1]), __hadd2(z[2], z[3]));
            const bool bad = (*reinterpret_cast<uint32_t*>(&z[0]) & 0x7FFF7FFFu) != 0;
            if (bad) {
#pragma unroll 1
              for (int c = 0; c < 64; ++c) {
                uint32_t* a = reinterpret_cast<uint32_t*>(at(c >> 2) + (c & 3) * 4);
                uint32_t x = *a;
                if (!finite_bf16(x)) x &= 0xFFFF0000u;
                if (!finite_bf16(x >> 16)) x &= 0xFFFFu;
                *a = x;
              }
            }
            const uint32_t word = __ballot_sync(0xffffffffu, bad);
            if (lane == 0) flags(i)[(j - im) * 4 + q] = word;
          }
          fence_proxy_async_smem();
          mbar_arrive(&v_ok[vn & 1]);
        }
        pos += 5 * n;
        return true;
      });
    }
  } else {
    // ------------------------------------------------------------- softmax
    reg_inc<200>();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;         // row of the tile, TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + t * 128, o_col = tmem + lanes + O_COL + t * 128;
    const float c = p.sm_scale * kLog2e;
    const uint64_t c2 = pack2(c, c);
    const float large = kLarge / c;
    int sn = 0, on = 0;
    ok = for_each_unit(true, [&](const Unit& u, int i) -> bool {
      const int row = t * kTile + r;         // row of the unit
      const int n = u.n(t);
      const bool live = row < u.rows;
      const int lim = min(u.ke, row_limit(u, row, p.causal)) - u.ks;  // keys of this unit
      const int im = first_masked(u, t * kTile, p.causal);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++sn) {
        if (!warp_wait(&s_full[t], sn & 1)) return false;
        tc::fence_after_sync();
        float off = 0.f;  // taken off this row's scores
      again:
        uint32_t s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tc::ld_32x32b_x32(s_col + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[q * 32]));
        tc::wait_ld();
        tc::reg_fence(s);
        if (j >= im) {
          const int left = lim - j * kTile;
#pragma unroll
          for (int q = 0; q < 128; ++q)
            if (q >= left) s[q] = 0xFF800000u;  // -inf
        }
        const float mo = m - off;
        float mx[4] = {mo, mo, mo, mo};
#pragma unroll
        for (int q = 0; q < 128; q += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[q + 2 * e]), __uint_as_float(s[q + 2 * e + 1])));
        const float m_new = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // O is rescaled only when the maximum has grown by more than 2^8
        // (-inf - -inf is NaN: no)
        const bool grow = (m_new - mo) * c > kRescale;
        if (__any_sync(0xffffffffu, (j > 0 && grow) || fabsf(m_new) > large)) {
          // This tile's S was issued after the last P.V: O is complete.  The loop
          // does O and S alike, so that the rare case adds little code (64
          // instructions more cost short prompts 4 %).
          const float alpha = grow ? ex2((m - m_new) * c) : 1.f;
          l *= alpha;
          if (grow) m = m_new;
          const bool wide = off == 0.f && fabsf(m) > large && m != -INFINITY;
          const bool shift = __any_sync(0xffffffffu, wide);
          if (wide) off = m;
#pragma unroll 1
          for (int q = j > 0 ? 0 : 4; q < (shift ? 8 : 4); ++q) {
            const uint32_t col = q < 4 ? o_col + q * 32 : s_col + (q - 4) * 32;
            const float f = q < 4 ? alpha : 1.f, g = q < 4 ? 0.f : -off;
            uint32_t o[32];
            tc::ld_32x32b_x32(col, o);
            tc::wait_ld();
            tc::reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f + g);
            tc::st_32x32b_x32(col, o);
          }
          if (shift) {
            tc::wait_st();
            goto again;
          }
        }
        if (grow) m = m_new;
        const float mc = m == -INFINITY ? 0.f : (off - m) * c;
        const uint64_t mc2 = pack2(mc, mc);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int q = 0; q < 64; ++q) {
          float a, b;
          unpack2(fma2(pack2(__uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1])), c2, mc2), a,
                  b);
          a = ex2(a);
          b = ex2(b);
          sum[q & 1] = add2(sum[q & 1], pack2(a, b));
          s[q] = pack_bf16x2(a, b);
          if ((q & 31) == 31)
            tc::st_32x32b_x32(s_col + (q - 31), *reinterpret_cast<uint32_t(*)[32]>(&s[q - 31]));
        }
        float a0, a1, b0, b1;
        unpack2(sum[0], a0, a1);
        unpack2(sum[1], b0, b1);
        l += (a0 + a1) + (b0 + b1);
        tc::wait_st();
        tc::fence_before_sync();
        mbar_arrive(&p_full[t]);
      }
      // ---- this row of O, and its lse
      if (n > 0) {
        if (!warp_wait(&o_full[t], on & 1)) return false;
        ++on;
        tc::fence_after_sync();
      }
      const int64_t q_row = u.q_row + row;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // keys of the cut tiles with values that are not finite
      uint32_t any = 0;
      const int um = first_masked(u, 0, p.causal), nm = u.n(t) - um;
      if (n > 0) {
        for (int k = 0; k < nm; ++k) {
          const uint4 x = *reinterpret_cast<const uint4*>(flags(i) + k * 4);
          any |= x.x | x.y | x.z | x.w;
        }
      }
      if (any) {  // the whole tile: those values into O for the rows that attend to their keys
#pragma unroll 1
        for (int q = 0; q < kDv; q += 32) {
          uint32_t o[32];
          tc::ld_32x32b_x32(o_col + q, o);
          tc::wait_ld();
          tc::reg_fence(o);
          for (int k = 0; k < nm * 4; ++k) {
            uint32_t bits = flags(i)[k];
            while (bits) {
              const int key = um * kTile + k * 32 + __ffs(bits) - 1;
              bits &= bits - 1;
              if (key >= lim || !live) continue;
              const uint16_t* v = p.v + (static_cast<int64_t>(u.k_row) + u.ks + key) * p.v_row_stride +
                                  u.h * p.v_head_stride + q;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const uint32_t x = __ldg(v + e);
                if (!finite_bf16(x))
                  o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(x << 16));
              }
            }
          }
          __syncwarp();
          tc::st_32x32b_x32(o_col + q, o);
        }
        tc::wait_st();
      }
      const int64_t part = (static_cast<int64_t>(u.split) * p.num_tokens + q_row) * p.heads + u.h;
      uint32_t o[kDv];
      if (n > 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tc::ld_32x32b_x32(o_col + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&o[q * 32]));
        tc::wait_ld();
        tc::reg_fence(o);
      } else {
#pragma unroll
        for (int e = 0; e < kDv; ++e) o[e] = 0;
      }
      // Rows of different lanes lie far apart, so a store costs a cycle for
      // each lane: 32 bytes at once where the output is aligned for it.
      if (live && p.num_splits == 1) {
        uint16_t* dst = p.o + q_row * p.o_row_stride + u.h * p.o_head_stride;
#pragma unroll
        for (int f = 0; f < kDv / 2; ++f)
          o[f] = pack_bf16x2(__uint_as_float(o[2 * f]) * inv, __uint_as_float(o[2 * f + 1]) * inv);
        if (p.o_aligned32) {
#pragma unroll
          for (int f = 0; f < kDv / 2; f += 8) store32(dst + 2 * f, &o[f]);
        } else {
#pragma unroll
          for (int f = 0; f < kDv / 2; f += 4)
            *reinterpret_cast<uint4*>(dst + 2 * f) = make_uint4(o[f], o[f + 1], o[f + 2], o[f + 3]);
        }
      } else if (live && n > 0) {
        float* dst = p.ws_o + part * kDv;
#pragma unroll
        for (int e = 0; e < kDv; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
        for (int e = 0; e < kDv; e += 8) store32(dst + e, &o[e]);
      }
      if (live) {
        float lg;
        asm("lg2.approx.f32 %0, %1;" : "=f"(lg) : "f"(l));
        const float lse = l == 0.f            ? -INFINITY
                          : fabsf(m) > large ? m * p.sm_scale + lg * kLn2
                                             : (m * c + lg) * kLn2;
        if (p.num_splits == 1)
          p.lse[q_row * p.heads + u.h] = lse;
        else
          p.ws_lse[part] = lse;
      }
      // the reads of O are done before the next unit's first P opens the
      // way for a P.V that overwrites it
      __syncwarp();
      tc::fence_before_sync();
      return true;
    });
  }
  if (!ok && lane == 0) gave_up(p.err_count);

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

// The splits of a row and head joined: M = max lse_s, o = sum e^{lse_s - M}
// o_s / sum e^{lse_s - M}, in split order.  One warp each, four dims a lane.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(kMergeWarps * 32) prefill_merge_kernel(const PrefillParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t rec = static_cast<int64_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int64_t records = static_cast<int64_t>(p.num_tokens) * p.heads;
  if (rec >= records) return;
  const int64_t row = rec / p.heads;
  const int h = static_cast<int>(rec % p.heads);
  // rows of no sequence are left as they were
  if (row < __ldg(p.cu_q) || row >= __ldg(p.cu_q + p.num_seqs)) return;
  const int S = p.num_splits;
  float M = -INFINITY;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, p.ws_lse[s * records + rec]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float den = 0.f;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const float ls = s0 + lane < S ? p.ws_lse[(s0 + lane) * records + rec] : -INFINITY;
    const float w = ls == -INFINITY ? 0.f : ex2((ls - M) * kLog2e);
    uint32_t mask = __ballot_sync(0xffffffffu, ls != -INFINITY);
    while (mask) {
      const int j = __ffs(mask) - 1;
      mask &= mask - 1;
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float4 x = *reinterpret_cast<const float4*>(p.ws_o + ((s0 + j) * records + rec) * kDv +
                                                        lane * 4);
      acc.x += wj * x.x;
      acc.y += wj * x.y;
      acc.z += wj * x.z;
      acc.w += wj * x.w;
      den += wj;
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint2 out;
  out.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  out.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.o + row * p.o_row_stride + h * p.o_head_stride + lane * 4) = out;
  if (lane == 0) p.lse[rec] = den == 0.f ? -INFINITY : M + logf(den);
}

}  // namespace

cudaError_t launch_prefill(const PrefillParams& p_in, const PrefillMaps& maps,
                           cudaStream_t stream) {
  PrefillParams p = p_in;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = set_smem_attr_once(prefill_kernel, kSmem, attr_done);
  if (e != cudaSuccess) return e;
  p.slots = p.num_tokens / kUnitRows + p.num_seqs;
  // heads side by side in the order of units: as many as keep their keys and
  // values (512 bytes a key and head) in half of L2, at least eight
  const int64_t fit = (int64_t{64} << 20) / (512 * static_cast<int64_t>(p.num_kv > 0 ? p.num_kv : 1));
  p.head_group = static_cast<int>(fit < 8 ? 8 : fit > p.heads ? p.heads : fit);
  if (p.head_group > p.heads) p.head_group = p.heads;
  const int groups = (p.heads + p.head_group - 1) / p.head_group;
  const int64_t units = static_cast<int64_t>(groups) * p.slots * p.head_group * p.num_splits;
  if (units > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int grid = static_cast<int>(units);
  e = launch_overlapped(prefill_kernel, dim3(grid), dim3(kThreads), kSmem, stream, p, maps);
  if (e != cudaSuccess || p.num_splits == 1) return e;
  const int64_t records = static_cast<int64_t>(p.num_tokens) * p.heads;
  return launch_overlapped(prefill_merge_kernel,
                           dim3(static_cast<unsigned>((records + kMergeWarps - 1) / kMergeWarps)),
                           dim3(kMergeWarps * 32), 0, stream, p);
}

}  // namespace mla
