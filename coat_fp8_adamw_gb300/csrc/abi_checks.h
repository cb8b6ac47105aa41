// abi_checks.h -- argument checks shared by the extern "C" entry points
// (coat_abi.cu, ckpt_abi.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "coat.h"

namespace coat {
namespace abi {

inline bool pow2_group(int32_t G) { return G >= 1 && G <= 256 && (G & (G - 1)) == 0; }
inline bool size_ok(int64_t n) { return n >= 1 && n <= COAT_MAX_N; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

// Device memory of the current device, or managed memory.  Host memory is
// refused even where the GPU could reach it, since the kernels assume HBM,
// and so is another device's memory: the kernels launch on the current one.
inline bool is_device(const void* p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();  // clear the sticky-free error state of this query
        return false;
    }
    if (at.type == cudaMemoryTypeManaged) return true;
    if (at.type != cudaMemoryTypeDevice) return false;
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.device == cur;
}

inline coat_status from_cuda(cudaError_t e) { return e == cudaSuccess ? COAT_OK : COAT_ERR_CUDA; }

inline int64_t num_groups(int64_t n, int32_t G) { return (n + G - 1) / G; }

}  // namespace abi
}  // namespace coat
