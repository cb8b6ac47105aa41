// ckpt_norm.cu -- RMS norm that keeps its input as an 8-bit checkpoint, and its
// backward pass from that checkpoint (COAT review page, section 3: FP8
// activations, 1 x G groups for non-linear layers).
//
//   forward   h = x (+ residual, rounded to bf16);  r = 1 / sqrt(mean h^2 + eps)
//             y = h r w;  checkpoint of h: codes and group scales
//   backward  xh = S E4M3(q) r;  g = dy w;  c = mean(g xh)
//             dx = r (g - xh c) (+ dresidual);  dw = sum over rows of dy xh
//
// Sums and every value between input and output are float32; y, h, dx and dw
// are rounded once, to the bf16 tensors that the caller asks for.
//
// A row is held by T = 32 ceil(N / 512) threads, sixteen consecutive elements
// each; a block has as many such row teams as fit 256 threads, and the blocks
// walk the rows.  The weights stay in shared memory and, backward, a thread's
// sums for dw in registers from row to row; the next row's loads are on their
// way while a team works on one.  Across the team's sum a thread keeps its
// elements as they came (bf16 and codes) and unpacks them again behind it: the
// few instructions are cheaper than the registers, which let 1024 threads run
// per SM.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kE = 16;             // elements per thread
constexpr int kMaxTeamWarps = 32;

struct Team {
    int threads;   // per row, a multiple of 32
    int teams;     // per block
};
Team team_of(int64_t N) {
    const int t = 32 * (int)((N + 32 * kE - 1) / (32 * kE));
    return Team{t, t >= 256 ? 1 : 256 / t};
}

// What was unpacked from these words has to be unpacked again: nothing of it is kept in registers.
template <int W>
__device__ __forceinline__ void forget(uint32_t (&w)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) asm volatile("" : "+r"(w[i]));
}

// The team's sum of v.  slots: one float per warp of the team, for this use
// alone until the team's next barrier; `bar` is the team's named barrier.
__device__ __forceinline__ float team_sum(float v, float* slots, int warps, int warp, int lane, int bar) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if (lane == 0) slots[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * warps) : "memory");
    const float s = lane < warps ? slots[lane] : 0.0f;
    return warp_sum(s);
}

// The weights in shared memory: float4 j of thread t's sixteen at [j T + t], so
// that neighbouring lanes read neighbouring float4s.  Zeros behind the row.
__device__ __forceinline__ void stage_weights(const float* w, int64_t N, int T, float4* sw) {
    for (int i = threadIdx.x; i < T * (kE / 4); i += blockDim.x) {
        const int64_t c = (int64_t)i * 4;
        const int t = i / (kE / 4), j = i % (kE / 4);
        sw[j * T + t] = c < N ? __ldg(reinterpret_cast<const float4*>(w + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
}
__device__ __forceinline__ void weights_of(const float4* sw, int T, int t, float (&w)[kE]) {
#pragma unroll
    for (int j = 0; j < kE / 4; ++j) {
        const float4 f = sw[j * T + t];
        w[4 * j] = f.x; w[4 * j + 1] = f.y; w[4 * j + 2] = f.z; w[4 * j + 3] = f.w;
    }
}

template <bool kRes>
__global__ void __launch_bounds__(1024, 1) norm_fwd_kernel(const NormFwdArgs a, int T, int teams, bool wide) {
    __shared__ float slots[2][kMaxTeamWarps];
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const int gshift = 31 - __clz(a.G);
    const float inv_n = 1.0f / (float)a.N;
    const int64_t col = (int64_t)t * kE, step = (int64_t)gridDim.x * teams;
    const bool ok = col < a.N;      // N % 16 == 0: all sixteen or none
    extern __shared__ float4 sw[];
    stage_weights(a.weight, a.N, T, sw);
    uint32_t xn[8] = {}, rn[8] = {};
    int64_t r = (int64_t)blockIdx.x * teams + team;
    if (ok && r < a.M) {
        load_words8(a.x + r * a.N + col, wide, xn);
        if constexpr (kRes) load_words8(a.residual + r * a.N + col, wide, rn);
    }
    for (int par = 0; r < a.M; r += step, par ^= 1) {
        const int64_t at = r * a.N + col;
        uint32_t hv[8];
        float ss = 0.0f;
        if constexpr (kRes) {
            float x[kE], p[kE];
            unpack(xn, x);
            unpack(rn, p);
#pragma unroll
            for (int e = 0; e < kE; ++e) x[e] += p[e];
            pack(x, hv);
            if (ok) store_words8(a.h + at, wide, hv);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) hv[i] = xn[i];
        }
        if (ok && r + step < a.M) {
            load_words8(a.x + at + step * a.N, wide, xn);
            if constexpr (kRes) load_words8(a.residual + at + step * a.N, wide, rn);
        }
        {
            float x[kE];
            unpack(hv, x);
#pragma unroll
            for (int e = 0; e < kE; ++e) ss = fmaf(x[e], x[e], ss);
            Scales16 q;
            uint32_t c[4];
            quantize16<true>(x, a.G, q, c);
            if (ok) {
                *reinterpret_cast<uint4*>(a.q + at) = make_uint4(c[0], c[1], c[2], c[3]);
                store_scales16(a.scale, at, a.G, gshift, q);
            }
        }
        ss = team_sum(ss, slots[par] + team * warps, warps, warp, lane, 1 + team);
        const float rstd = __frcp_rn(__fsqrt_rn(fmaf(ss, inv_n, a.eps)));
        if (t == 0) a.rstd[r] = rstd;
        forget(hv);
        float x[kE], w[kE];
        unpack(hv, x);
        weights_of(sw, T, t, w);
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = x[e] * rstd * w[e];
        pack(x, hv);
        if (ok) store_words8(a.y + at, wide, hv);
    }
}

template <bool kRes>
__global__ void __launch_bounds__(1024, 1) norm_bwd_kernel(const NormBwdArgs a, int T, int teams, bool wide) {
    __shared__ float slots[2][kMaxTeamWarps];
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const int gshift = 31 - __clz(a.G);
    const float inv_n = 1.0f / (float)a.N;
    const int64_t col = (int64_t)t * kE, step = (int64_t)gridDim.x * teams;
    const bool ok = col < a.N;
    extern __shared__ float4 sw[];
    stage_weights(a.weight, a.N, T, sw);
    float dw[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) dw[e] = 0.0f;
    uint32_t dn[8] = {}, qn[4] = {};
    int64_t r = (int64_t)blockIdx.x * teams + team;
    if (ok && r < a.M) {
        load_words8(a.dy + r * a.N + col, wide, dn);
        load_words<4>(a.q + r * a.N + col, qn);
    }
    for (int par = 0; r < a.M; r += step, par ^= 1) {
        const int64_t at = r * a.N + col;
        const float rstd = __ldg(a.rstd + r);
        float S[2] = {0.0f, 0.0f};
        if (ok) load_scales16(a.scale, at, a.G, gshift, S[0], S[1]);
        S[0] *= rstd;
        S[1] *= rstd;
        uint32_t dv[8], qv[4], rv[8] = {};
#pragma unroll
        for (int i = 0; i < 8; ++i) dv[i] = dn[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = qn[i];
        if (ok) {
            if constexpr (kRes) load_words8(a.dresidual + at, wide, rv);
            if (r + step < a.M) {
                load_words8(a.dy + at + step * a.N, wide, dn);
                load_words<4>(a.q + at + step * a.N, qn);
            }
        }
        float c = 0.0f;
        {
            float g[kE], xh[kE], w[kE];
            unpack(dv, g);
            decode(qv, xh);
            weights_of(sw, T, t, w);
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                const float p = g[e] * (xh[e] * S[e >> 3]);
                dw[e] += p;
                c = fmaf(p, w[e], c);
            }
        }
        c = team_sum(c, slots[par] + team * warps, warps, warp, lane, 1 + team) * inv_n;
        forget(dv);
        forget(qv);
        float g[kE], xh[kE], w[kE];
        unpack(dv, g);
        decode(qv, xh);
        weights_of(sw, T, t, w);
        const float k0 = -c * S[0], k1 = -c * S[1];
#pragma unroll
        for (int e = 0; e < kE; ++e) g[e] = rstd * fmaf(xh[e], e < 8 ? k0 : k1, g[e] * w[e]);
        if constexpr (kRes) {
            unpack(rv, w);
#pragma unroll
            for (int e = 0; e < kE; ++e) g[e] += w[e];
        }
        pack(g, dv);
        if (ok) store_words8(a.dx + at, wide, dv);
    }
    if (ok) {
        float4* part = reinterpret_cast<float4*>(a.partial + ((int64_t)blockIdx.x * teams + team) * a.N + col);
#pragma unroll
        for (int i = 0; i < kE / 4; ++i) part[i] = make_float4(dw[4 * i], dw[4 * i + 1], dw[4 * i + 2], dw[4 * i + 3]);
    }
}

// 32 columns per block; its 32 warps take every 32nd row of the partial sums, four loads on their way each
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partial, int64_t P, int64_t N, uint16_t* out) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < N) {
        int64_t p = row;
        for (; p + 96 < P; p += 128) {
            const float v0 = partial[p * N + c], v1 = partial[(p + 32) * N + c];
            const float v2 = partial[(p + 64) * N + c], v3 = partial[(p + 96) * N + c];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; p < P; p += 32) s += partial[p * N + c];
    }
    part[row][lane] = s;
    __syncthreads();
    s = warp_sum(part[lane][row]);   // this warp's column `row` of the block
    if (lane == 0 && (int64_t)blockIdx.x * 32 + row < N) out[(int64_t)blockIdx.x * 32 + row] = bf16_bits(s);
}

// blocks that run at once: 64 registers a thread leave room for 1024 threads per SM
int64_t norm_blocks(int64_t M, const Team& tm, int sms) {
    const int64_t need = (M + tm.teams - 1) / tm.teams, room = (int64_t)sms * (1024 / (tm.threads * tm.teams));
    return need < room ? need : room;
}

size_t smem_of(const Team& tm) { return sizeof(float) * kE * (size_t)tm.threads; }   // 64 KB at most

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// more than the 48 KB that every kernel may have (N > 12288)
template <typename F>
cudaError_t allow_smem(F* kernel, size_t bytes) {
    return bytes <= (48u << 10) ? cudaSuccess
                                : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

int device_sms() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

int64_t norm_bwd_partials(int64_t M, int64_t N, int sms) {
    const Team tm = team_of(N);
    return norm_blocks(M, tm, sms) * tm.teams;
}

cudaError_t launch_column_sum(const float* partial, int64_t P, int64_t N, uint16_t* out, cudaStream_t s) {
    column_sum_kernel<<<(unsigned)((N + 31) / 32), 1024, 0, s>>>(partial, P, N, out);
    return cudaGetLastError();
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
    const Team tm = team_of(a.N);
    const unsigned blocks = (unsigned)norm_blocks(a.M, tm, device_sms());
    const bool wide = aligned32(a.x) && aligned32(a.residual) && aligned32(a.h) && aligned32(a.y);
    const cudaError_t e = allow_smem(a.residual ? norm_fwd_kernel<true> : norm_fwd_kernel<false>, smem_of(tm));
    if (e != cudaSuccess) return e;
    if (a.residual)
        norm_fwd_kernel<true><<<blocks, tm.threads * tm.teams, smem_of(tm), s>>>(a, tm.threads, tm.teams, wide);
    else
        norm_fwd_kernel<false><<<blocks, tm.threads * tm.teams, smem_of(tm), s>>>(a, tm.threads, tm.teams, wide);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    const Team tm = team_of(a.N);
    const int64_t blocks = norm_blocks(a.M, tm, device_sms());
    const bool wide = aligned32(a.dy) && aligned32(a.dresidual) && aligned32(a.dx);
    cudaError_t e = allow_smem(a.dresidual ? norm_bwd_kernel<true> : norm_bwd_kernel<false>, smem_of(tm));
    if (e != cudaSuccess) return e;
    if (a.dresidual)
        norm_bwd_kernel<true><<<(unsigned)blocks, tm.threads * tm.teams, smem_of(tm), s>>>(a, tm.threads, tm.teams, wide);
    else
        norm_bwd_kernel<false><<<(unsigned)blocks, tm.threads * tm.teams, smem_of(tm), s>>>(a, tm.threads, tm.teams, wide);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_column_sum(a.partial, blocks * tm.teams, a.N, a.dweight, s);
}

}  // namespace coat
