// ckpt_device.cuh -- what the operators with 8-bit activation checkpoints share
// on the device: sixteen bf16 values per thread in one 256-bit access (two of
// 128 bits where the address is a multiple of 16 bytes alone), a group's scale
// and E4M3 codes, and codes back to values.
//
// A checkpoint of a row is the one coat_act_quantize_fp8 writes: per group of G
// consecutive elements S = RN(max|x| / 448) and q = E4M3(x / S), rounded to
// nearest even of the exact quotient (COAT review page, section 3: FP8
// quantization, 1 x G groups for non-linear layers).
#pragma once

#include <cmath>
#include <cstdint>

#include "coat_device.cuh"

namespace coat {
namespace ckpt {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// ---- memory: N consecutive 32-bit words, streamed past L1 ----
// Ordinary loads, and volatile: the kernels start before the one ahead of them has ended, so that no load of theirs may
// count as one of constant data (ld.global.nc) or be moved ahead of the wait for it.
template <int N>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[N]);
template <>
__device__ __forceinline__ void load_words<4>(const void* p, uint32_t (&w)[4]) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
        : "l"(p));
}
// 32 bytes: one 256-bit access where `wide` (the address is a multiple of 32), else two
__device__ __forceinline__ void load_words8(const void* p, bool wide, uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
            : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
            : "l"(p));
    } else {
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4 + 16];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "l"(p));
    }
}
__device__ __forceinline__ void store_words8(void* p, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ---- programmatic dependent launch ----
// Every kernel here may start while the one before it in the stream ends (launch_next): its launch and what it prepares
// on the SM then cost nothing (2.3 to 2.6 us less per call when calls follow one another, 0.4 in a graph).  Before a thread's
// first access to global memory, reads and writes alike: wait until that kernel has ended and its writes are visible.
// A block of every kernel does so, so that a kernel's end implies the end of all before it.
// In a kernel whose blocks end together: the next one's blocks may be scheduled.
__device__ __forceinline__ void dependents_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_primary() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- bf16 and E4M3 ----
// 2 W bf16 values as float32
template <int W>
__device__ __forceinline__ void unpack(const uint32_t (&w)[W], float (&x)[2 * W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int W>
__device__ __forceinline__ void pack(const float (&x)[2 * W], uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = bf16x2(x[2 * i], x[2 * i + 1]);
}
__device__ __forceinline__ uint16_t bf16_bits(float x) { return (uint16_t)(bf16x2(x, 0.0f) & 0xFFFFu); }

// 4 W E4M3 codes as their values (exact: an E4M3 value is a half value)
template <int W>
__device__ __forceinline__ void decode(const uint32_t (&c)[W], float (&x)[4 * W]) {
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(c[i >> 1] >> (16 * (i & 1)))));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(h));
    }
}

// ---- pairs of float32 (each half rounds like the scalar operation) ----
// 2 W bf16 values as W pairs
template <int W>
__device__ __forceinline__ void unpack2(const uint32_t (&w)[W], uint64_t (&x)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    float a, b;
    upk(v, a, b);
    return a + b;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// max|x| of n pairs from x[from]
template <int from, int n, int L>
__device__ __forceinline__ float max_of(const uint64_t (&x)[L]) {
    float mx = 0.0f;
#pragma unroll
    for (int e = from; e < from + n; ++e) {
        float a, b;
        upk(x[e], a, b);
        mx = max3(mx, fabsf(a), fabsf(b));
    }
    return mx;
}
// the maximum over `lanes` adjacent lanes (a power of two, the same for the whole warp)
__device__ __forceinline__ float lanes_max(float v, int lanes) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

// A group's scale, and what turns its elements into quotients: x / S is taken
// as fma(x, inv, x e), inv + e = 1 / S to about 2^-46 (and a bias, below).  A
// group of zeros has S = 0 and any inv.
struct Scale {
    float S, inv, e;
};
__device__ __forceinline__ void reciprocal(Scale& s) { s.inv = rcp_ftz(s.S > 0.0f ? s.S : 1.0f); }
// Scales whose reciprocal or correction would leave the normal range: by division.
__device__ __forceinline__ bool by_division(const Scale& q) { return q.S > 0.0f && !(q.S > 0x1p-96f && q.S < 0x1p96f); }

// The scale of a group of bf16 values with maximum m: S = RN(m / 448), as the
// product with RN(1/448) and one FMA correction from the exact remainder
// (Markstein's division by a known divisor; right for every bf16 m >= 0).
//
// The codes have to round the EXACT quotient x / S.  With x = X 2^a and
// m = Y 2^b, X, Y < 256, and an E4M3 midpoint Z 2^c, Z < 32, the ratio of
// 448 x / m and the midpoint is 7 X 2^d / (Y Z): it is 1, or at least 1 / 7905
// away from it.  Where it is 1, x / S lies on the side of the midpoint that S's
// own rounding decides, the same for the whole group: above it when S < m / 448,
// below when S > m / 448, on it when S is exact.  So a bias of 2^-18 to that
// side (far below 1 / 7905, far above float32's errors) decides every such
// element, and no element on its own needs a second look; when S is exact
// there is no bias, and the quotient, within 2^-45 of the midpoint, rounds to it
// and then to even.
__device__ __forceinline__ Scale scale_of_bf16_max(float m) {
    constexpr float y = 1.0f / 448.0f;
    const float q = __fmul_rn(m, y);
    Scale s;
    s.S = fmaf(fmaf(-q, 448.0f, m), y, q);
    reciprocal(s);
    const float rem = fmaf(-448.0f, s.S, m);        // 448 (m / 448 - S), exact
    const float bias = rem > 0.0f ? 0x1p-18f : rem < 0.0f ? -0x1p-18f : 0.0f;
    s.e = s.inv * (fmaf(-s.S, s.inv, 1.0f) + bias);
    return s;
}
// The scale of a group of float32 values with maximum m: their quotients are rounded to float32 before they are to E4M3.
__device__ __forceinline__ Scale scale_of_max(float m) {
    Scale s;
    s.S = __fdiv_rn(m, 448.0f);
    reciprocal(s);
    s.e = s.inv * fmaf(-s.S, s.inv, 1.0f);
    return s;
}

// The codes of sixteen elements, as pairs: the first eight with scale lo, the others with hi.
__device__ __forceinline__ void encode16(const uint64_t (&x)[8], const Scale& lo, const Scale& hi, uint32_t (&w)[4]) {
    if (by_division(lo) || by_division(hi)) {
        // one element at a time, in a loop over local memory: nothing of it is held in registers, and no function is
        // called, which would cost every other path registers as well
        float t[16];
        uint32_t c[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) upk(x[i], t[2 * i], t[2 * i + 1]);
#pragma unroll 1
        for (int i = 0; i < 16; ++i) {
            const float S = i < 8 ? lo.S : hi.S;
            c[i] = S > 0.0f ? e4m3x2(__fadd_rn(e4m3_quotient(t[i], S), 0.0f), 0.0f) & 0xFFu : 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = e4m3_canonical_zero(c[4 * i] | c[4 * i + 1] << 8 | c[4 * i + 2] << 16 | c[4 * i + 3] << 24);
        return;
    }
    const uint64_t i0 = pk(lo.inv, lo.inv), e0 = pk(lo.e, lo.e), i1 = pk(hi.inv, hi.inv), e1 = pk(hi.e, hi.e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint64_t xx = x[2 * i + j];
            float y0, y1;
            upk(fma2(xx, i < 2 ? i0 : i1, mul2(xx, i < 2 ? e0 : e1)), y0, y1);
            c[j] = e4m3x2(y0, y1);
        }
        w[i] = e4m3_canonical_zero(c[0] | (c[1] << 16));
    }
}

// Sixteen consecutive elements of a thread: scales and codes.  A group of 8 is
// half of them (two scales), one of 16 all of them, a wider one G / 16 lanes.
struct Scales16 {
    Scale lo, hi;   // equal unless G = 8
};
template <bool kBf16>
__device__ __forceinline__ void quantize16(const uint64_t (&x)[8], int G, Scales16& q, uint32_t (&w)[4]) {
    const float m0 = max_of<0, 4>(x), m1 = max_of<4, 4>(x);
    if (G == 8) {
        q.lo = kBf16 ? scale_of_bf16_max(m0) : scale_of_max(m0);
        q.hi = kBf16 ? scale_of_bf16_max(m1) : scale_of_max(m1);
    } else {
        const float m = lanes_max(fmaxf(m0, m1), G >> 4);
        q.lo = q.hi = kBf16 ? scale_of_bf16_max(m) : scale_of_max(m);
    }
    encode16(x, q.lo, q.hi, w);
}
// Stores the scales of the sixteen elements from flat index `at`.
__device__ __forceinline__ void store_scales16(float* scale, int64_t at, int G, int gshift, const Scales16& q) {
    if (G == 8)
        *reinterpret_cast<float2*>(scale + (at >> 3)) = make_float2(q.lo.S, q.hi.S);
    else if ((at & (G - 1)) == 0)
        scale[at >> gshift] = q.lo.S;
}
__device__ __forceinline__ void load_scales16(const float* scale, int64_t at, int G, int gshift, float& lo, float& hi) {
    if (G == 8) {
        const float2 f = *reinterpret_cast<const float2*>(scale + (at >> 3));
        lo = f.x;
        hi = f.y;
    } else {
        lo = hi = scale[at >> gshift];
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// 1 / sqrt(v), v > 0 (also subnormal: a zero row and an eps below 2^-126): the approximation and one Newton step, within
// 2^-23 relatively for normal v.
__device__ __forceinline__ float rsqrt_newton(float v) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
}

// Where a mean square is past float32 (elements from about 2^57 on, finite ones), it is formed of kFar times the elements:
// the largest sum, 16384 squares of 2^56, and the smallest that comes here, 2^128 kFar^2, are normal numbers.  far_rsqrt:
// what such elements are multiplied with, 1 / sqrt of their mean square; 0 if one is infinite, as 1 / sqrt(inf).  kFar
// times that is 1 / rms itself.
constexpr float kFar = 0x1p-72f;
__device__ __forceinline__ float far_rsqrt(float v) { return v == INFINITY ? 0.0f : rsqrt_newton(v); }

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)); x -> -inf gives 0, +inf gives 1.
__device__ __forceinline__ float sigmoid(float x) { return rcp_ftz(1.0f + ex2_ftz(-1.4426950408889634f * x)); }

}  // namespace ckpt
}  // namespace coat
