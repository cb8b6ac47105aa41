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
// A row is held by T = 32 ceil(N / 512) threads, 16 elements each (two 16-byte
// chunks, T chunks apart); a block has as many such row teams as fit 256
// threads, and the blocks walk the rows.  A team keeps its columns' weights
// (and, backward, its columns' sums for dw) in registers from row to row.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kV = 2;              // 8-element chunks per thread
constexpr int kMaxTeamWarps = 32;

struct Team {
    int threads;   // per row, a multiple of 32
    int teams;     // per block
};
Team team_of(int64_t N) {
    const int t = 32 * (int)((N + 32 * 8 * kV - 1) / (32 * 8 * kV));
    return Team{t, t >= 256 ? 1 : 256 / t};
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

__device__ __forceinline__ void load_weights(const float* w, int64_t c, bool ok, float (&out)[8]) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (ok) {
        a = __ldg(reinterpret_cast<const float4*>(w + c));
        b = __ldg(reinterpret_cast<const float4*>(w + c) + 1);
    }
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
}

template <bool kRes>
__global__ void __launch_bounds__(1024, 1) norm_fwd_kernel(const NormFwdArgs a, int T, int teams) {
    __shared__ float slots[2][kMaxTeamWarps];
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const float inv_n = 1.0f / (float)a.N;
    float w[kV][8];
    bool ok[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int64_t c = (int64_t)(j * T + t) * 8;
        ok[j] = c < a.N;
        load_weights(a.weight, c, ok[j], w[j]);
    }
    int par = 0;
    for (int64_t r = (int64_t)blockIdx.x * teams + team; r < a.M; r += (int64_t)gridDim.x * teams, par ^= 1) {
        float x[kV][8];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int64_t at = r * a.N + (int64_t)(j * T + t) * 8;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (ok[j]) u = ld_cs(reinterpret_cast<const uint4*>(a.x + at));
            unpack8(u, x[j]);
            if constexpr (kRes) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (ok[j]) v = ld_cs(reinterpret_cast<const uint4*>(a.residual + at));
                float p[8];
                unpack8(v, p);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[j][e] += p[e];
                u = pack8(x[j]);
                unpack8(u, x[j]);
                if (ok[j]) st_cs(reinterpret_cast<uint4*>(a.h + at), u);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[j][e], x[j][e], ss);
        }
        ss = team_sum(ss, slots[par] + team * warps, warps, warp, lane, 1 + team);
        const float rstd = __frcp_rn(__fsqrt_rn(fmaf(ss, inv_n, a.eps)));
        if (t == 0) a.rstd[r] = rstd;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int64_t at = r * a.N + (int64_t)(j * T + t) * 8;
            const float S = scale_of_bf16_max(group_max(x[j], a.G));
            const uint2 c = encode8(x[j], S);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[j][e] * rstd * w[j][e];
            if (ok[j]) {
                st_cs(reinterpret_cast<uint4*>(a.y + at), pack8(y));
                __stcs(reinterpret_cast<uint2*>(a.q + at), c);
                if ((at & (a.G - 1)) == 0) a.scale[at / a.G] = S;
            }
        }
    }
}

template <bool kRes>
__global__ void __launch_bounds__(1024, 1) norm_bwd_kernel(const NormBwdArgs a, int T, int teams) {
    __shared__ float slots[2][kMaxTeamWarps];
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const float inv_n = 1.0f / (float)a.N;
    float w[kV][8], dw[kV][8];
    bool ok[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int64_t c = (int64_t)(j * T + t) * 8;
        ok[j] = c < a.N;
        load_weights(a.weight, c, ok[j], w[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    int par = 0;
    for (int64_t r = (int64_t)blockIdx.x * teams + team; r < a.M; r += (int64_t)gridDim.x * teams, par ^= 1) {
        const float rstd = __ldg(a.rstd + r);
        float g[kV][8], xh[kV][8];
        float c = 0.0f;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int64_t at = r * a.N + (int64_t)(j * T + t) * 8;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            uint2 q = make_uint2(0u, 0u);
            float S = 0.0f;
            if (ok[j]) {
                u = ld_cs(reinterpret_cast<const uint4*>(a.dy + at));
                q = __ldcs(reinterpret_cast<const uint2*>(a.q + at));
                S = __ldg(a.scale + at / a.G);
            }
            unpack8(u, g[j]);
            decode8(q, xh[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xh[j][e] = xh[j][e] * S * rstd;
                dw[j][e] = fmaf(g[j][e], xh[j][e], dw[j][e]);
                g[j][e] *= w[j][e];
                c = fmaf(g[j][e], xh[j][e], c);
            }
        }
        c = team_sum(c, slots[par] + team * warps, warps, warp, lane, 1 + team) * inv_n;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const int64_t at = r * a.N + (int64_t)(j * T + t) * 8;
            float d[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = rstd * fmaf(-xh[j][e], c, g[j][e]);
            if (ok[j]) {
                if constexpr (kRes) {
                    float p[8];
                    unpack8(ld_cs(reinterpret_cast<const uint4*>(a.dresidual + at)), p);
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] += p[e];
                }
                st_cs(reinterpret_cast<uint4*>(a.dx + at), pack8(d));
            }
        }
    }
    float* part = a.partial + ((int64_t)blockIdx.x * teams + team) * a.N;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        const int64_t c = (int64_t)(j * T + t) * 8;
        if (ok[j]) {
            reinterpret_cast<float4*>(part + c)[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            reinterpret_cast<float4*>(part + c)[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
        }
    }
}

// 32 columns per block, 8 rows of the partial sums at a time
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partial, int64_t P, int64_t N, uint16_t* out) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < N)
        for (int64_t p = row; p < P; p += 8) s += partial[p * N + c];
    part[row][lane] = s;
    __syncthreads();
    if (row != 0 || c >= N) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) s += part[i][lane];
    out[c] = bf16_bits(s);
}

// blocks that run at once: two per SM while a block is at most 512 threads
int64_t norm_blocks(int64_t M, const Team& tm, int sms) {
    const int64_t need = (M + tm.teams - 1) / tm.teams, room = (int64_t)sms * (tm.threads * tm.teams <= 512 ? 2 : 1);
    return need < room ? need : room;
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
    column_sum_kernel<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(partial, P, N, out);
    return cudaGetLastError();
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
    const Team tm = team_of(a.N);
    const unsigned blocks = (unsigned)norm_blocks(a.M, tm, device_sms());
    if (a.residual)
        norm_fwd_kernel<true><<<blocks, tm.threads * tm.teams, 0, s>>>(a, tm.threads, tm.teams);
    else
        norm_fwd_kernel<false><<<blocks, tm.threads * tm.teams, 0, s>>>(a, tm.threads, tm.teams);
    return cudaGetLastError();
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    const Team tm = team_of(a.N);
    const int64_t blocks = norm_blocks(a.M, tm, device_sms());
    if (a.dresidual)
        norm_bwd_kernel<true><<<(unsigned)blocks, tm.threads * tm.teams, 0, s>>>(a, tm.threads, tm.teams);
    else
        norm_bwd_kernel<false><<<(unsigned)blocks, tm.threads * tm.teams, 0, s>>>(a, tm.threads, tm.teams);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_column_sum(a.partial, blocks * tm.teams, a.N, a.dweight, s);
}

}  // namespace coat
