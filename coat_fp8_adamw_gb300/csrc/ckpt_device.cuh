// ckpt_device.cuh -- what the operators with 8-bit activation checkpoints share
// on the device: eight bf16 values per 16-byte access, a group's scale and
// E4M3 codes, and codes back to values.
//
// A checkpoint of a row is the one coat_act_quantize_fp8 writes: per group of G
// consecutive elements S = RN(max|x| / 448) and q = E4M3(x / S), rounded to
// nearest even of the exact quotient (COAT review page, section 3: FP8
// quantization, 1 x G groups for non-linear layers).  A thread holds eight
// consecutive elements; a group of G lies in G / 8 adjacent lanes.
#pragma once

#include <cstdint>

#include "coat_device.cuh"

namespace coat {
namespace ckpt {

constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint16_t bf16_bits(float x) { return (uint16_t)(bf16x2(x, 0.0f) & 0xFFFFu); }

// Eight E4M3 codes as their values (exact: an E4M3 value is a half value).
__device__ __forceinline__ void decode8(uint2 c, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)(w[i >> 1] >> (16 * (i & 1)))));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
            : "r"(h));
    }
}

// max|x| over the group: the thread's eight, then the G / 8 lanes that hold the
// group (G a power of two in [8, 128], the same in every lane of the warp).
__device__ __forceinline__ float group_max(const float (&x)[8], int G) {
    float mx = max3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
    mx = max3(mx, fabsf(x[3]), fabsf(x[4]));
    mx = max3(mx, fabsf(x[5]), fabsf(x[6]));
    mx = fmaxf(mx, fabsf(x[7]));
    for (int off = G >> 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
    return mx;
}

// RN(m / 448) of a non-negative bf16 value: the product with RN(1/448) and one
// FMA correction from the exact remainder (Markstein's division by a known
// divisor; right for every non-negative finite bf16 value).
__device__ __forceinline__ float scale_of_bf16_max(float m) {
    constexpr float y = 1.0f / 448.0f;
    const float q = __fmul_rn(m, y);
    return fmaf(fmaf(-q, 448.0f, m), y, q);
}
// RN(m / 448) of any non-negative float32
__device__ __forceinline__ float scale_of_max(float m) { return __fdiv_rn(m, 448.0f); }

// The codes of eight elements of one group with scale S: the codes of
// y (1 - 2^-20) and y (1 + 2^-20), y = x RN(1/S), agree unless an E4M3 midpoint
// lies beside x / S; those few are decided from the exact quotient.  S = 0 (a
// group of zeros) gives zero codes.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float S) {
    const float inv = S > 0.0f ? rcp_approx(S) : 0.0f;
    uint32_t codes[2] = {0u, 0u}, diff[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t yy = fma2(pk(x[e], x[e + 1]), pk(inv, inv), pk(0.0f, 0.0f));   // +0 for a zero of either sign
        float l0, l1, h0, h1;
        upk(mul2(yy, pk(kDn, kDn)), l0, l1);
        upk(mul2(yy, pk(kUp, kUp)), h0, h1);
        const uint32_t clo = e4m3x2(l0, l1), chi = e4m3x2(h0, h1);
        codes[e / 4] |= clo << (16 * ((e >> 1) & 1));
        diff[e / 4] |= (clo ^ chi) << (16 * ((e >> 1) & 1));
    }
    if (!(inv <= 3.40282347e38f)) {   // a subnormal scale: every element by division
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int sh = 8 * (e & 3);
            codes[e / 4] = (codes[e / 4] & ~(0xFFu << sh)) | (e4m3_code_of_quotient_exact(x[e], S) << sh);
        }
    } else if ((diff[0] | diff[1]) != 0u) {   // quotients beside a midpoint: the midpoint decides
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int wd = i >> 1, sh = 16 * (i & 1);
            const uint32_t d = (diff[wd] >> sh) & 0xFFFFu;
            if (d != 0u) {
                const uint32_t lo = (codes[wd] >> sh) & 0xFFFFu;
                const uint32_t c = e4m3x2_resolve(lo, lo ^ d, x[2 * i], x[2 * i + 1], S, S);
                codes[wd] = (codes[wd] & ~(0xFFFFu << sh)) | (c << sh);
            }
        }
    }
    return make_uint2(e4m3_canonical_zero(codes[0]), e4m3_canonical_zero(codes[1]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// sigmoid(x) = 1 / (1 + 2^(-x log2 e)); x -> -inf gives 0, +inf gives 1.
__device__ __forceinline__ float sigmoid(float x) {
    return __fdividef(1.0f, 1.0f + ex2_ftz(-1.4426950408889634f * x));
}

}  // namespace ckpt
}  // namespace coat
