// What the files of the C ABI share: alignment checks, limits, status codes.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/moe_int4.h"

namespace moe {

// The kernels move activations, outputs, workspace pieces and packed weights
// in 16-byte vectors and everything else in 4-byte words; a misaligned
// pointer is rejected before anything is enqueued (null passes: null checks
// are separate).
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// Row strides of the operators around the layer (elements): in-tile offsets
// of a few hundred rows stay 32-bit in the kernels.
constexpr int64_t kMaxRowStride = int64_t(1) << 20;

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace moe
