// divide.h -- n / d for many n below 2^31 and one d, by a multiplication.  Host and device.
//
// With 2^shift < d <= 2^(shift + 1) and mul = ceil(2^(32 + shift) / d), n / d = floor(n mul / 2^(32 + shift)):
// mul d = 2^(32 + shift) + e with 0 <= e < d <= 2^(shift + 1), so n mul / 2^(32 + shift) is n / d plus
// n e / (d 2^(32 + shift)), which is below (2^31 2^(shift + 1)) / (d 2^(32 + shift)) = 1 / d: too little to reach the next
// multiple of 1 / d, and so the next whole number.  mul < 2^32, since d > 2^shift.  (d = 1 is told apart.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define COAT_DIVIDE_FN __host__ __device__ __forceinline__
#else
#define COAT_DIVIDE_FN inline
#endif

namespace coat {

struct Divider {
    uint32_t d, mul;
    int shift;
};
inline Divider divider(uint32_t d) {
    Divider v{d, 0u, 0};
    if (d == 1) return v;
    while ((1ull << (v.shift + 1)) < d) ++v.shift;
    v.mul = (uint32_t)(((1ull << (32 + v.shift)) + d - 1) / d);
    return v;
}
COAT_DIVIDE_FN uint32_t divide(uint32_t n, const Divider& v) {
    return v.d == 1 ? n : (uint32_t)(((uint64_t)n * v.mul) >> 32) >> v.shift;
}

}  // namespace coat
