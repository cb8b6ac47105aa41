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
// A thread holds eight consecutive elements.  Codes and scales are contiguous,
// so the threads walk the flat element range in 16-byte chunks; gate and up
// (and their gradients) may be column ranges of a wider tensor.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kBlock = 256;

// Chunk i of the flat range [M x nc chunks]: its first element in a tensor whose rows are ld apart.
__device__ __forceinline__ int64_t strided_at(int64_t i, int64_t nc, int64_t ld) {
    const int64_t r = i / nc;
    return r * ld + (i - r * nc) * 8;
}

__global__ void __launch_bounds__(kBlock) swiglu_fwd_kernel(const SwigluFwdArgs a) {
    const int64_t nc = a.N >> 3, total = a.M * nc;
    // a warp's lanes run past the end together: the group maximum needs them all
    for (int64_t i0 = (int64_t)blockIdx.x * kBlock; i0 < total; i0 += (int64_t)gridDim.x * kBlock) {
        const int64_t i = i0 + threadIdx.x;
        const bool ok = i < total;
        uint4 gv = make_uint4(0u, 0u, 0u, 0u), uv = gv;
        if (ok) {
            const int64_t at = strided_at(i, nc, a.ld);
            gv = ld_cs(reinterpret_cast<const uint4*>(a.gate + at));
            uv = ld_cs(reinterpret_cast<const uint4*>(a.up + at));
        }
        float g[8], u[8], h[8];
        unpack8(gv, g);
        unpack8(uv, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = g[e] * sigmoid(g[e]) * u[e];
        const float Sg = scale_of_bf16_max(group_max(g, a.G)), Su = scale_of_bf16_max(group_max(u, a.G));
        const uint2 cg = encode8(g, Sg), cu = encode8(u, Su);
        if (ok) {
            const int64_t at = i * 8;
            st_cs(reinterpret_cast<uint4*>(a.h + at), pack8(h));
            __stcs(reinterpret_cast<uint2*>(a.gate_q + at), cg);
            __stcs(reinterpret_cast<uint2*>(a.up_q + at), cu);
            if ((at & (a.G - 1)) == 0) {
                a.gate_scale[at / a.G] = Sg;
                a.up_scale[at / a.G] = Su;
            }
        }
    }
}

template <bool kH>
__global__ void __launch_bounds__(kBlock) swiglu_bwd_kernel(const SwigluBwdArgs a) {
    const int64_t nc = a.N >> 3, total = a.M * nc;
    for (int64_t i0 = (int64_t)blockIdx.x * kBlock; i0 < total; i0 += (int64_t)gridDim.x * kBlock) {
        const int64_t i = i0 + threadIdx.x;
        const bool ok = i < total;
        uint4 dv = make_uint4(0u, 0u, 0u, 0u);
        uint2 gq = make_uint2(0u, 0u), uq = gq;
        float Sg = 0.0f, Su = 0.0f;
        if (ok) {
            const int64_t at = i * 8;
            dv = ld_cs(reinterpret_cast<const uint4*>(a.dh + at));
            gq = __ldcs(reinterpret_cast<const uint2*>(a.gate_q + at));
            uq = __ldcs(reinterpret_cast<const uint2*>(a.up_q + at));
            Sg = __ldg(a.gate_scale + at / a.G);
            Su = __ldg(a.up_scale + at / a.G);
        }
        float d[8], g[8], u[8], h[8], dg[8], du[8];
        unpack8(dv, d);
        decode8(gq, g);
        decode8(uq, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] *= Sg;
            u[e] *= Su;
            const float s = sigmoid(g[e]), gs = g[e] * s;
            h[e] = gs * u[e];
            du[e] = d[e] * gs;
            dg[e] = d[e] * u[e] * fmaf(gs, 1.0f - s, s);
        }
        if (ok) {
            const int64_t at = strided_at(i, nc, a.ld);
            st_cs(reinterpret_cast<uint4*>(a.dgate + at), pack8(dg));
            st_cs(reinterpret_cast<uint4*>(a.dup + at), pack8(du));
        }
        if constexpr (kH) {
            const float Sh = scale_of_max(group_max(h, a.G));
            const uint2 ch = encode8(h, Sh);
            if (ok) {
                const int64_t at = i * 8;
                __stcs(reinterpret_cast<uint2*>(a.h_q + at), ch);
                if ((at & (a.G - 1)) == 0) a.h_scale[at / a.G] = Sh;
            }
        }
    }
}

unsigned swiglu_blocks(int64_t M, int64_t N) {
    const int64_t need = (M * (N >> 3) + kBlock - 1) / kBlock, most = (int64_t)1 << 30;
    return (unsigned)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_swiglu_fwd(const SwigluFwdArgs& a, cudaStream_t s) {
    swiglu_fwd_kernel<<<swiglu_blocks(a.M, a.N), kBlock, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s) {
    if (a.h_q)
        swiglu_bwd_kernel<true><<<swiglu_blocks(a.M, a.N), kBlock, 0, s>>>(a);
    else
        swiglu_bwd_kernel<false><<<swiglu_blocks(a.M, a.N), kBlock, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace coat
