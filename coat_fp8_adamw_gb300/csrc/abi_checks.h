// abi_checks.h -- argument checks shared by the extern "C" entry points
// (coat_abi.cu, ckpt_abi.cu, lm_abi.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

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

// A buffer of a call.  A null pointer: not there.
enum Kind { kIn, kOut, kOutRows };
struct Buf {
    const void* p;
    size_t bytes;
    Kind kind;
};

// Alignment, then overlap, then where the memory is.  Outputs overlap nothing,
// except that two outputs of rows (kOutRows) may interleave: rows_apart has
// looked at those.
inline coat_status check_buffers(std::initializer_list<Buf> bufs) {
    for (const Buf& b : bufs)
        if (b.p && !aligned16(b.p)) return COAT_ERR_MISALIGNED;
    for (const Buf* b = bufs.begin(); b != bufs.end(); ++b)
        for (const Buf* c = b + 1; c != bufs.end(); ++c) {
            if (!b->p || !c->p || (b->kind == kIn && c->kind == kIn)) continue;
            if (b->kind == kOutRows && c->kind == kOutRows) continue;
            if (overlaps(b->p, b->bytes, c->p, c->bytes)) return COAT_ERR_INVALID_ARG;
        }
    for (const Buf& b : bufs)
        if (b.p && !is_device(b.p)) return COAT_ERR_NOT_DEVICE;
    return COAT_OK;
}

inline bool shape_ok(int64_t M, int64_t N) { return M >= 1 && N >= 1 && M < (1LL << 31) && N < (1LL << 31); }
inline bool stride_ok(int64_t ld, int64_t N) { return ld >= N && ld % 8 == 0 && ld < (1LL << 31); }
// bytes from the first to the last element of M rows of n elements, ld apart
inline size_t span(int64_t M, int64_t n, int64_t ld, size_t elem) { return ((size_t)(M - 1) * (size_t)ld + (size_t)n) * elem; }

}  // namespace abi
}  // namespace coat
