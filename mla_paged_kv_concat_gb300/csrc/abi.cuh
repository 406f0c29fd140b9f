// Host-side helpers the C entry points share: the per-thread error text,
// pointer checks and tensor-map encoding.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

// Records `e` as the calling thread's last CUDA error; returns MLA_ERR_CUDA.
mla_status cuda_fail(cudaError_t e);
// The same with a text of the caller's own.
mla_status cuda_fail_text(const char* text);

// cuTensorMapEncodeTiled over three dimensions with unit element strides and
// zeros past the edges.  It needs a current context, which a host thread has
// none of before its first call to the runtime: it gets the device's then.
CUresult encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base,
                    const cuuint64_t (&dims)[3], const cuuint64_t (&strides)[2],
                    const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle,
                    CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

}  // namespace mla
