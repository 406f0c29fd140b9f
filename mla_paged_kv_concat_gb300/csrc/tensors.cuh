// What the C entry points check of tensors on the host: rows and heads at their
// strides, bytes that two tensors share, and the tensor maps over them.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "abi.cuh"

namespace mla {

// Tensor map over bf16 [d2][d1][d0] at element strides s1, s2, 128-byte
// swizzled, box {64, b1, b2}.
inline mla_status make_map(CUtensorMap* map, const void* base, int64_t d0, int64_t d1, int64_t d2,
                    int64_t s1, int64_t s2, int b1, int b2) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                              static_cast<cuuint64_t>(d2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
  if (encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, dims, strides, box,
                 CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return mla::cuda_fail_text("cuTensorMapEncodeTiled failed");
  return MLA_OK;
}

// A tensor [tokens][heads][cols] of bf16 that a tensor map can describe.
struct Heads {
  const void* p;
  int64_t rs, hs;
  int cols;
};

inline bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t{1} << 38); }

inline bool heads_ok(const Heads& t, int tokens, int heads) {
  return t.p && aligned16(t.p) && stride_ok(t.rs) && (heads == 1 || stride_ok(t.hs)) &&
         (heads == 1 || t.hs >= t.cols) && t.rs >= t.cols &&
         // no buffer is that long, and the products below stay in 64 bits
         t.rs <= (int64_t{1} << 40) / tokens && (heads == 1 || t.hs <= (int64_t{1} << 40) / heads);
}

// Whether no two elements of an output share an address: one of the two
// outer dimensions steps over the whole of the other.
inline bool heads_disjoint(const Heads& t, int tokens, int heads) {
  return heads == 1 || tokens == 1 || t.rs >= (heads - 1) * t.hs + t.cols ||
         t.hs >= (tokens - 1) * t.rs + t.cols;
}

// The bytes of a tensor: runs of `len` at p + i * s[0] + j * s[1], the larger
// stride first, up to `end`.
struct Runs {
  uintptr_t p, end;
  int64_t n[2], s[2], len;
  int64_t inner() const { return (n[1] - 1) * s[1] + len; }
};
// One run; none, which meets nothing, without a pointer or bytes.
inline Runs runs(const void* p, int64_t bytes) {
  const uintptr_t x = bytes > 0 ? reinterpret_cast<uintptr_t>(p) : 0;
  return {x, x ? x + bytes : 0, {1, 1}, {0, 0}, bytes};
}
// Runs that join are one, and a stride that no step takes is 0.
inline Runs runs(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t len) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  const uintptr_t end = x + (n0 - 1) * s0 + (n1 - 1) * s1 + len;
  if (n1 > 1 && s1 == len) {
    len *= n1;
    n1 = 1;
  }
  if (n1 == 1 && n0 > 1 && s0 == len) {
    len *= n0;
    n0 = 1;
  }
  return {x, end, {n0, n1}, {n0 > 1 ? s0 : 0, n1 > 1 ? s1 : 0}, len};
}
inline Runs runs(const Heads& t, int tokens, int heads) {
  const int64_t rs = tokens > 1 ? 2 * t.rs : 0, hs = heads > 1 ? 2 * t.hs : 0;
  return hs > rs ? runs(t.p, heads, hs, tokens, rs, 2 * int64_t{t.cols})
                 : runs(t.p, tokens, rs, heads, hs, 2 * int64_t{t.cols});
}

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// The m of [lo, hi] with -lb < x + m * s < la, from first to last.
struct Steps {
  int64_t first, last;
};
inline Steps steps(int64_t x, int64_t s, int64_t lo, int64_t hi, int64_t la, int64_t lb) {
  if (s == 0) return -lb < x && x < la ? Steps{lo, lo} : Steps{0, -1};
  const int64_t a = floor_div(-lb - x, s) + 1, z = -floor_div(x - la, s) - 1;
  return {a > lo ? a : lo, z < hi ? z : hi};
}

// Whether two tensors share a byte.  Exact but for two that both have rows
// apart from each other, at different distances: those count as sharing one
// only where they start at the same address.
inline bool meet(const Runs& a, const Runs& b) {
  if (a.p == b.p) return true;
  if (a.s[0] && b.s[0] && a.s[0] != b.s[0]) return false;
  const int64_t d = static_cast<int64_t>(b.p - a.p), s0 = a.s[0] ? a.s[0] : b.s[0];
  const Steps k = steps(d, s0, 1 - a.n[0], b.n[0] - 1, a.inner(), b.inner());
  for (int64_t m = k.first; m <= k.last; ++m) {
    const int64_t x = d + m * s0;
    if (!a.s[1] || !b.s[1] || a.s[1] == b.s[1]) {
      const Steps j = steps(x, a.s[1] ? a.s[1] : b.s[1], 1 - a.n[1], b.n[1] - 1, a.len, b.len);
      if (j.first <= j.last) return true;
      continue;
    }
    for (int64_t i = 0; i < a.n[1]; ++i) {
      const Steps j = steps(x - i * a.s[1], b.s[1], 0, b.n[1] - 1, a.len, b.len);
      if (j.first <= j.last) return true;
    }
  }
  return false;
}
inline bool intersect(const Runs& a, const Runs& b) { return a.p < b.end && b.p < a.end && meet(a, b); }

inline mla_status heads_map(CUtensorMap* m, const Heads& t, int tokens, int heads, int box_rows) {
  // the stride of a dimension of size 1 is never used but has to be valid
  return make_map(m, t.p, t.cols, heads, tokens, heads == 1 ? t.cols : t.hs, t.rs, 1, box_rows);
}

}  // namespace mla
