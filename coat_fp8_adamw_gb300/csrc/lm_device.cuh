// lm_device.cuh -- what the kernels of the embedding and the cross entropy share on the device.
#pragma once

#include <cstdint>

#include "ckpt_device.cuh"

namespace coat {
namespace lm {

// Indexes of 4 or 8 bytes.  (volatile: the kernels start before the one ahead of them has ended, so no load may move ahead of
// the wait for it; through L1, since many threads read the same ones)
__device__ __forceinline__ int32_t load_index(const int32_t* p) {
    int32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int64_t load_index(const int64_t* p) {
    int64_t v;
    asm volatile("ld.global.b64 %0, [%1];" : "=l"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ int64_t index_at(const void* p, int32_t wide, int64_t i) {
    return wide ? load_index(static_cast<const int64_t*>(p) + i) : (int64_t)load_index(static_cast<const int32_t*>(p) + i);
}

}  // namespace lm
}  // namespace coat
