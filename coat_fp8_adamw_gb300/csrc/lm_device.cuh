// lm_device.cuh -- what the kernels of the embedding and the cross entropy share on the device.
#pragma once

#include <cstdint>

#include "ckpt_device.cuh"

namespace coat {
namespace lm {

// index i of a list of 4- or 8-byte integers (a volatile load: the kernels start before the one ahead of them has ended)
__device__ __forceinline__ int64_t index_at(const void* p, int32_t wide, int64_t i) {
    return wide ? static_cast<const volatile long long*>(p)[i] : (long long)static_cast<const volatile int*>(p)[i];
}

}  // namespace lm
}  // namespace coat
