// Host-side helpers the C entry points share: the per-thread error text,
// pointer checks and tensor-map encoding.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

// Records `e` as the calling thread's last CUDA error; returns MLA_ERR_CUDA.
mla_status cuda_fail(cudaError_t e);
// The same with a text of the caller's own.
mla_status cuda_fail_text(const char* text);

// cuTensorMapEncodeTiled, looked up once per process (nullptr when the
// driver has none).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

}  // namespace mla
