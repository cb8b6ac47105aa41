// ckpt_qk.cu -- RMS norm of every query and key head with the position rotation
// in the same pass, keeping the heads as an 8-bit checkpoint, and its backward
// pass from that checkpoint (COAT review page, section 3: FP8 activations,
// 1 x G groups for non-linear layers).
//
//   forward   per head x of D: r = 1 / sqrt(mean x^2 + eps), y = x r w, then the
//             first rot entries of y are turned in pairs (a, b) by the angle of
//             the token's position: (a c - b s, b c + a s).  Pairs are
//             (i, i + rot/2), or (2i, 2i + 1) when interleaved.
//   backward  dn = the gradient turned back, g = dn w, xh = S E4M3(q) r:
//             dx = r (g - xh mean(g xh));  dw = sum over tokens and heads of dn xh
//
// Everything between input and output is float32, rounded once to bf16.
//
// A head lies in D / 8 lanes, eight elements each (the smallest power of two of
// lanes that holds it; the others idle), so that its sums are a few shuffles,
// and so is a half-split pair, whose partner is rot / 16 lanes away.  A block
// takes one token at a time: the lanes keep their cosines and sines in
// registers over the token's heads.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) { const uint32_t w[4] = {u.x, u.y, u.z, u.w}; unpack(w, x); }
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) { uint32_t w[4]; pack(x, w); return make_uint4(w[0], w[1], w[2], w[3]); }
__device__ __forceinline__ void decode8(uint2 c, float (&x)[8]) { const uint32_t w[2] = {c.x, c.y}; decode(w, x); }
__device__ __forceinline__ float group_max(const float (&x)[8], int G) { return lanes_max(max_of<0, 8>(x), G >> 3); }
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const Scale& S) { uint32_t w[2]; encode<0, 8>(x, S, w); return make_uint2(w[0], w[1]); }

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// A lane's part of the rotation: out[e] = in[e] c[e] + partner(in)[e] s[e], where
// s carries the sign of the lane's side of the pair; lanes behind rot (and a
// position outside the tables: NaN) included.
struct Turn {
    float c[8], s[8];
    int from;          // half-split: the lane that holds the partners
};

// l: lane within the head; base: the head's first lane.
__device__ __forceinline__ void load_turn(const QkArgs& a, int64_t m, int l, int base, bool back, Turn& t) {
    const int half = a.rot >> 1, e0 = l * 8;
    t.from = base + l;
#pragma unroll
    for (int e = 0; e < 8; ++e) { t.c[e] = 1.0f; t.s[e] = 0.0f; }
    if (e0 >= a.rot) return;
    const int64_t pos = a.positions[m];
    const bool ok = pos >= 0 && pos < a.max_pos;
    const float nan = __uint_as_float(0x7FC00000u);
    if (a.interleaved) {
        float4 c = make_float4(nan, nan, nan, nan), s = c;
        if (ok) {
            c = __ldg(reinterpret_cast<const float4*>(a.cos + pos * half + (e0 >> 1)));
            s = __ldg(reinterpret_cast<const float4*>(a.sin + pos * half + (e0 >> 1)));
        }
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t.c[2 * i] = t.c[2 * i + 1] = cc[i];
            t.s[2 * i] = back ? ss[i] : -ss[i];
            t.s[2 * i + 1] = back ? -ss[i] : ss[i];
        }
    } else {
        const bool low = e0 < half;
        t.from = base + (low ? l + (half >> 3) : l - (half >> 3));
        const int i0 = low ? e0 : e0 - half;
        if (ok) {
            load8(a.cos + pos * half + i0, t.c);
            load8(a.sin + pos * half + i0, t.s);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) t.c[e] = t.s[e] = nan;
        }
        if (low != back) {
#pragma unroll
            for (int e = 0; e < 8; ++e) t.s[e] = -t.s[e];
        }
    }
}

// every lane of the warp takes part
__device__ __forceinline__ void turn8(const Turn& t, bool interleaved, float (&x)[8]) {
    float p[8];
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(kFull, x[e], t.from);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = fmaf(p[e], t.s[e], x[e] * t.c[e]);
}

template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

template <int kLanes>
__global__ void __launch_bounds__(kBlock) qk_fwd_kernel(const QkArgs a) {
    constexpr int kHeads = 32 / kLanes;   // heads per warp and pass
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (kLanes - 1), base = lane - l, sub = lane / kLanes;
    const bool in_head = l * 8 < a.D;
    const float inv_d = 1.0f / (float)a.D;
    const int H = a.q.H + a.k.H;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        Turn t;
        load_turn(a, m, l, base, false, t);
        for (int h0 = warp * kHeads; h0 < H; h0 += kWarps * kHeads) {
            const bool ok = h0 + sub < H && in_head;
            const bool is_q = h0 + sub < a.q.H;
            const HeadSide& sd = is_q ? a.q : a.k;
            const int64_t h = is_q ? h0 + sub : h0 + sub - a.q.H;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (ok) {
                u = ld_cs(reinterpret_cast<const uint4*>(sd.in + m * sd.ld + h * a.D + l * 8));
                load8(sd.weight + l * 8, w);
            }
            float x[8], y[8];
            unpack8(u, x);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            ss = head_sum<kLanes>(ss);
            const float r = __frcp_rn(__fsqrt_rn(fmaf(ss, inv_d, a.eps)));
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e] * r * w[e];
            turn8(t, a.interleaved != 0, y);
            const Scale S = scale_of_bf16_max(group_max(x, a.G));
            const uint2 c = encode8(x, S);
            if (ok) {
                const int64_t at = (m * sd.H + h) * a.D + l * 8;
                st_cs(reinterpret_cast<uint4*>(sd.out + at), pack8(y));
                __stcs(reinterpret_cast<uint2*>(sd.codes + at), c);
                if (((l * 8) & (a.G - 1)) == 0) sd.scale[at / a.G] = S.S;
                if (l == 0) sd.rstd[m * sd.H + h] = r;
            }
        }
    }
}

template <int kLanes>
__global__ void __launch_bounds__(kBlock) qk_bwd_kernel(const QkArgs a) {
    constexpr int kHeads = 32 / kLanes;
    __shared__ float part[kBlock / kLanes][2][kLanes * 8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (kLanes - 1), base = lane - l, sub = lane / kLanes;
    const bool in_head = l * 8 < a.D;
    const float inv_d = 1.0f / (float)a.D;
    const int H = a.q.H + a.k.H;
    float dw[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        Turn t;
        load_turn(a, m, l, base, true, t);
        for (int h0 = warp * kHeads; h0 < H; h0 += kWarps * kHeads) {
            const bool ok = h0 + sub < H && in_head;
            const bool is_q = h0 + sub < a.q.H;
            const HeadSide& sd = is_q ? a.q : a.k;
            const int64_t h = is_q ? h0 + sub : h0 + sub - a.q.H;
            const int64_t at = (m * sd.H + h) * a.D + l * 8;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            uint2 q = make_uint2(0u, 0u);
            float S = 0.0f, r = 0.0f;
            float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (ok) {
                u = ld_cs(reinterpret_cast<const uint4*>(sd.in + at));
                q = __ldcs(reinterpret_cast<const uint2*>(sd.codes + at));
                S = __ldg(sd.scale + at / a.G);
                r = __ldg(sd.rstd + m * sd.H + h);
                load8(sd.weight + l * 8, w);
            }
            float g[8], xh[8];
            unpack8(u, g);
            decode8(q, xh);
            turn8(t, a.interleaved != 0, g);
            float c = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[e] = xh[e] * S * r;
                const float d = ok ? g[e] * xh[e] : 0.0f;
                dw[0][e] += is_q ? d : 0.0f;
                dw[1][e] += is_q ? 0.0f : d;
                c = fmaf(d, w[e], c);
                g[e] *= w[e];
            }
            c = head_sum<kLanes>(c) * inv_d;
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-xh[e], c, g[e]);
            if (ok) st_cs(reinterpret_cast<uint4*>(sd.out + m * sd.ld + h * a.D + l * 8), pack8(g));
        }
    }
    const int slot = threadIdx.x / kLanes;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        part[slot][0][l * 8 + e] = dw[0][e];
        part[slot][1][l * 8 + e] = dw[1][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kBlock) {
        const int side = i >= a.D, c = i - side * a.D;
        float s = 0.0f;
        for (int p = 0; p < kBlock / kLanes; ++p) s += part[p][side][c];
        a.partial[((int64_t)side * gridDim.x + blockIdx.x) * a.D + c] = s;
    }
}

template <int kLanes>
cudaError_t launch(const QkArgs& a, bool back, unsigned blocks, cudaStream_t s) {
    if (back)
        qk_bwd_kernel<kLanes><<<blocks, kBlock, 0, s>>>(a);
    else
        qk_fwd_kernel<kLanes><<<blocks, kBlock, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_any(const QkArgs& a, bool back, unsigned blocks, cudaStream_t s) {
    const int lanes = a.D / 8;
    if (lanes <= 2) return launch<2>(a, back, blocks, s);
    if (lanes <= 4) return launch<4>(a, back, blocks, s);
    if (lanes <= 8) return launch<8>(a, back, blocks, s);
    if (lanes <= 16) return launch<16>(a, back, blocks, s);
    return launch<32>(a, back, blocks, s);
}

}  // namespace

int64_t qk_bwd_partials(int64_t M, int sms) {
    const int64_t room = (int64_t)sms * 4;
    return M < room ? M : room;
}

cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t s) {
    return launch_any(a, false, (unsigned)(a.M < (1 << 30) ? a.M : (1 << 30)), s);
}

cudaError_t launch_qk_bwd(const QkArgs& a, cudaStream_t s) {
    const int64_t blocks = qk_bwd_partials(a.M, device_sms());
    cudaError_t e = launch_any(a, true, (unsigned)blocks, s);
    if (e == cudaSuccess && a.q.H > 0) e = launch_column_sum(a.partial, blocks, a.D, a.q.dweight, s);
    if (e == cudaSuccess && a.k.H > 0) e = launch_column_sum(a.partial + blocks * a.D, blocks, a.D, a.k.dweight, s);
    return e;
}

}  // namespace coat
