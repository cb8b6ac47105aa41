// ckpt_swiglu.cu -- silu(gate) up with 8-bit checkpoints of both inputs, and its
// backward pass from those checkpoints (COAT review page, section 3: FP8
// activations, 1 x G groups for non-linear layers).
//
//   forward   h = g s(g) u, s(g) = 1 / (1 + e^-g);  checkpoints of g and u
//   backward  from g, u as the checkpoints give them:
//             dg = dh u s (1 + g (1 - s));  du = dh g s;
//             optionally the checkpoint of g s u, which the weight gradient of
//             the projection behind it reads: it is formed here, from values
//             already in registers, instead of being kept since the forward pass
//
// Everything between input and output is float32; h, dg and du are rounded
// once to bf16, and the product's checkpoint is taken from its float32 value.
// A thread holds sixteen consecutive elements (one 256-bit access of a bf16
// tensor, one 128-bit access of codes), so that a group's maximum takes one
// shuffle less than with eight.  Codes and scales are contiguous, so the threads
// walk the flat element range; gate and up (and their gradients) may be column
// ranges of a wider tensor.
//
// Bound by memory: 8192 x 11008, G = 128, halves of one tensor, 107.7 us forward
// and 121.0 us backward with the product's checkpoint, both at the copy rate
// (every tensor is read and written once).  Eight elements per thread took
// 197 and 160 us: what the threads issue per element was the bound then.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"
#include "divide.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kBlock = 256;

// Chunk i of the rows of nc chunks: its first element in a tensor whose rows are ld apart.
__device__ __forceinline__ int64_t strided_at(uint32_t i, const Divider& nc, int64_t ld) {
    const uint32_t r = divide(i, nc);
    return (int64_t)r * ld + (int64_t)(i - r * nc.d) * 16;
}

__global__ void __launch_bounds__(kBlock) swiglu_fwd_kernel(const SwigluFwdArgs a, const Divider nc, bool wide) {
    const uint32_t total = (uint32_t)a.M * nc.d, i = blockIdx.x * kBlock + threadIdx.x;
    const int gshift = 31 - __clz(a.G);
    const bool ok = i < total;       // the lanes past the end take part in the shuffles
    uint32_t gv[8] = {}, uv[8] = {};
    wait_for_primary();
    if (ok) {
        const int64_t at = strided_at(i, nc, a.ld);
        load_words8(a.gate + at, wide, gv);
        load_words8(a.up + at, wide, uv);
    }
    uint64_t g2[8], u2[8];
    uint32_t cg[4], cu[4], hv[8];
    unpack2(gv, g2);
    unpack2(uv, u2);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float ga, gb, ha, hb;
        upk(g2[e], ga, gb);
        upk(mul2(mul2(g2[e], pk(sigmoid(ga), sigmoid(gb))), u2[e]), ha, hb);
        hv[e] = bf16x2(ha, hb);
    }
    Scales16 sg, su;
    quantize16<true>(g2, a.G, sg, cg);
    quantize16<true>(u2, a.G, su, cu);
    if (!ok) return;
    const int64_t at = (int64_t)i * 16;
    store_words8(a.h + at, wide, hv);
    *reinterpret_cast<uint4*>(a.gate_q + at) = make_uint4(cg[0], cg[1], cg[2], cg[3]);
    *reinterpret_cast<uint4*>(a.up_q + at) = make_uint4(cu[0], cu[1], cu[2], cu[3]);
    store_scales16(a.gate_scale, at, a.G, gshift, sg);
    store_scales16(a.up_scale, at, a.G, gshift, su);
}

template <bool kH>
__global__ void __launch_bounds__(kBlock) swiglu_bwd_kernel(const SwigluBwdArgs a, const Divider nc, bool wide) {
    const uint32_t total = (uint32_t)a.M * nc.d, i = blockIdx.x * kBlock + threadIdx.x;
    const int gshift = 31 - __clz(a.G);
    const bool ok = i < total;
    const int64_t at = (int64_t)i * 16;
    uint32_t dv[8] = {}, gq[4] = {}, uq[4] = {};
    float Sg[2] = {0.0f, 0.0f}, Su[2] = {0.0f, 0.0f};
    wait_for_primary();
    if (ok) {
        load_words8(a.dh + at, wide, dv);
        load_words<4>(a.gate_q + at, gq);
        load_words<4>(a.up_q + at, uq);
        load_scales16(a.gate_scale, at, a.G, gshift, Sg[0], Sg[1]);
        load_scales16(a.up_scale, at, a.G, gshift, Su[0], Su[1]);
    }
    uint64_t d[8], h[8];
    float gf[16], uf[16];
    uint32_t wg[8], wu[8];
    unpack2(dv, d);
    decode(gq, gf);
    decode(uq, uf);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint64_t g = mul2(pk(gf[2 * e], gf[2 * e + 1]), pk(Sg[e >> 2], Sg[e >> 2]));
        const uint64_t u = mul2(pk(uf[2 * e], uf[2 * e + 1]), pk(Su[e >> 2], Su[e >> 2]));
        float ga, gb, x, y;
        upk(g, ga, gb);
        const float sa = sigmoid(ga), sb = sigmoid(gb);
        const uint64_t s = pk(sa, sb), gs = mul2(g, s);
        h[e] = mul2(gs, u);
        upk(mul2(d[e], gs), x, y);
        wu[e] = bf16x2(x, y);
        // d u (s + g s (1 - s))
        upk(mul2(mul2(d[e], u), fma2(gs, pk(1.0f - sa, 1.0f - sb), s)), x, y);
        wg[e] = bf16x2(x, y);
    }
    if (ok) {
        const int64_t to = strided_at(i, nc, a.ld);
        store_words8(a.dgate + to, wide, wg);
        store_words8(a.dup + to, wide, wu);
    }
    if constexpr (kH) {
        Scales16 sh;
        uint32_t ch[4];
        quantize16<false>(h, a.G, sh, ch);
        if (ok) {
            *reinterpret_cast<uint4*>(a.h_q + at) = make_uint4(ch[0], ch[1], ch[2], ch[3]);
            store_scales16(a.h_scale, at, a.G, gshift, sh);
        }
    }
}

// rows per launch: its chunks are counted in 31 bits
int64_t slab_rows(int64_t N) {
    const int64_t rows = (((int64_t)1 << 31) - kBlock) / (N / 16);
    return rows;
}
unsigned blocks_of(int64_t M, int64_t N) { return (unsigned)((M * (N / 16) + kBlock - 1) / kBlock); }

}  // namespace

cudaError_t launch_swiglu_fwd(const SwigluFwdArgs& all, cudaStream_t s) {
    const int64_t N = all.N, slab = slab_rows(N);
    const Divider nc = divider((uint32_t)(N / 16));
    const bool wide = aligned32(all.gate) && aligned32(all.up) && aligned32(all.h) && all.ld % 16 == 0;
    for (int64_t r = 0; r < all.M; r += slab) {
        SwigluFwdArgs a = all;
        a.M = all.M - r < slab ? all.M - r : slab;
        a.gate += r * a.ld;
        a.up += r * a.ld;
        a.h += r * N;
        a.gate_q += r * N;
        a.up_q += r * N;
        a.gate_scale += r * (N / a.G);
        a.up_scale += r * (N / a.G);
        const cudaError_t e = launch_next(swiglu_fwd_kernel, blocks_of(a.M, N), kBlock, 0, s, a, nc, wide);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& all, cudaStream_t s) {
    const int64_t N = all.N, slab = slab_rows(N);
    const Divider nc = divider((uint32_t)(N / 16));
    const bool wide = aligned32(all.dgate) && aligned32(all.dup) && aligned32(all.dh) && all.ld % 16 == 0;
    for (int64_t r = 0; r < all.M; r += slab) {
        SwigluBwdArgs a = all;
        a.M = all.M - r < slab ? all.M - r : slab;
        a.dh += r * N;
        a.gate_q += r * N;
        a.up_q += r * N;
        a.gate_scale += r * (N / a.G);
        a.up_scale += r * (N / a.G);
        a.dgate += r * a.ld;
        a.dup += r * a.ld;
        if (a.h_q) {
            a.h_q += r * N;
            a.h_scale += r * (N / a.G);
        }
        const cudaError_t e = launch_next(a.h_q ? swiglu_bwd_kernel<true> : swiglu_bwd_kernel<false>, blocks_of(a.M, N), kBlock,
                                          0, s, a, nc, wide);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace coat
