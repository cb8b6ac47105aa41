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
#include "tc_pipeline.cuh"

#ifndef DEPTH
#define DEPTH 3
#endif
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

// The same for a block whose teams keep step: a barrier of the whole block.
__device__ __forceinline__ float block_sum(float v, float* slots, int warps, int warp, int lane) {
    v = warp_sum(v);
    if (lane == 0) slots[warp] = v;
    __syncthreads();
    if (warps == 1) return v;
    const float s = lane < warps ? slots[lane] : 0.0f;
    return warp_sum(s);
}

// Chunk c of a row in shared memory: eight gradients, code values and weights.
__device__ __forceinline__ void read_chunk(const uint4* dy, const uint2* q, const float4* sw, int c, int T, float (&g)[8],
                                           float (&x)[8], float (&w)[8]) {
    const uint4 d = dy[c];
    const uint2 v = q[c];
    const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, vw[2] = {v.x, v.y};
    unpack(dw, g);
    decode(vw, x);
    const float4 f0 = sw[c], f1 = sw[2 * T + c];
    w[0] = f0.x; w[1] = f0.y; w[2] = f0.z; w[3] = f0.w;
    w[4] = f1.x; w[5] = f1.y; w[6] = f1.z; w[7] = f1.w;
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

// Backward: the rows come through a ring in shared memory, two to four iterations
// of a block deep (dy, codes and dresidual of its teams' rows, each one bulk copy:
// the rows of a block lie together), because loads kept on their way in registers
// beside the sums for dw left too few threads.  A thread has two chunks of eight
// columns, T chunks apart: neighbouring lanes read neighbouring 16 bytes.
constexpr int kMaxDepth = 4;

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

struct BwdShape {
    int T, teams;          // team of a row, rows per block and iteration
    int N, depth;
    uint32_t stage;        // bytes of a stage: teams rows of dy, codes, dresidual
    uint32_t q_off, r_off; // of the codes and of dresidual in it
};

template <bool kRes>
__global__ void __launch_bounds__(1024, 1) norm_bwd_kernel(const NormBwdArgs a, const BwdShape sh) {
    __shared__ float slots[2][kMaxTeamWarps];
    __shared__ uint64_t bars[kMaxDepth];
    extern __shared__ __align__(16) unsigned char dyn[];
    float4* sw = reinterpret_cast<float4*>(dyn);                       // float4 i of chunk c at [i 2T + c]
    unsigned char* ring = dyn + (size_t)sh.T * kE * 4;
    const int T = sh.T, teams = sh.teams, N = sh.N, depth = sh.depth;
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const int gshift = 31 - __clz(a.G);
    const float inv_n = 1.0f / (float)N;
    const int64_t ngr = N >> gshift;
    const uint32_t bar0 = smem_u32(bars), ring0 = smem_u32(ring);
    const int64_t rows_per = teams, step = (int64_t)gridDim.x * teams, first = (int64_t)blockIdx.x * teams;
    auto issue = [&](int64_t r0, int s) {                              // rows r0 .. of this block's next iteration
        const int64_t left = a.M - r0;
        const uint32_t rows = (uint32_t)(left < rows_per ? left : rows_per), n = rows * (uint32_t)N;
        const uint32_t d = ring0 + (uint32_t)s * sh.stage, bar = bar0 + 8u * (uint32_t)s;
        mbar_expect_tx(bar, n * (kRes ? 5u : 3u));
        bulk_load(d, a.dy + r0 * N, 2 * n, bar);
        bulk_load(d + sh.q_off, a.q + r0 * N, n, bar);
        if constexpr (kRes) bulk_load(d + sh.r_off, a.dresidual + r0 * N, 2 * n, bar);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < depth; ++s) mbar_init(bar0 + 8u * (uint32_t)s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int s = 0; s < depth; ++s)
            if (first + s * step < a.M) issue(first + s * step, s);
    }
    for (int i = threadIdx.x; i < 2 * T * 2; i += blockDim.x) {        // 2 T chunks of two float4s
        const int c = i >> 1, j = i & 1;
        sw[j * 2 * T + c] = 8 * c < N ? __ldg(reinterpret_cast<const float4*>(a.weight) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    bool ok[2];
    int col[2];
    float dw[2][8], Sn[2] = {0.0f, 0.0f}, rn = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        col[j] = (j * T + t) * 8;
        ok[j] = col[j] < N;
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    auto fetch_scales = [&](int64_t r) {                               // one iteration ahead
        if (r < a.M) {
            rn = __ldg(a.rstd + r);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (ok[j]) Sn[j] = __ldg(a.scale + r * ngr + (col[j] >> gshift));
        }
    };
    fetch_scales(first + team);
    int s = 0;
    uint32_t ph = 0;
    for (int64_t r0 = first, it = 0; r0 < a.M; r0 += step, ++it) {
        const int64_t r = r0 + team;
        const bool live = r < a.M;                                     // a team past the last row only keeps step
        const float rstd = rn, S[2] = {Sn[0] * rn, Sn[1] * rn};
        fetch_scales(r + step);
        if (!mbar_wait_fast(bar0 + 8u * (uint32_t)s, ph, nullptr)) break;
        const unsigned char* st = ring + (size_t)s * sh.stage;
        const uint4* dyp = reinterpret_cast<const uint4*>(st + (size_t)team * N * 2);
        const uint2* qp = reinterpret_cast<const uint2*>(st + sh.q_off + (size_t)team * N);
        const uint4* rp = reinterpret_cast<const uint4*>(st + sh.r_off + (size_t)team * N * 2);
        float c = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!live || !ok[j]) continue;
            float g[8], xh[8], w[8];
            read_chunk(dyp, qp, sw, col[j] >> 3, T, g, xh, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = g[e] * (xh[e] * S[j]);
                dw[j][e] += p;
                c = fmaf(p, w[e], c);
            }
        }
        c = block_sum(c, slots[it & 1] + team * warps, warps, warp, lane) * inv_n;
        // behind that barrier every thread is done with the iteration before this one: its stage is free
        if (threadIdx.x == 0 && it > 0) {
            const int64_t rr = r0 + (depth - 1) * step;
            if (rr < a.M) issue(rr, s == 0 ? depth - 1 : s - 1);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!live || !ok[j]) continue;
            float g[8], xh[8], w[8];
            read_chunk(dyp, qp, sw, col[j] >> 3, T, g, xh, w);
            const float k = -c * S[j];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rstd * fmaf(xh[e], k, g[e] * w[e]);
            if constexpr (kRes) {
                const uint4 v = rp[col[j] >> 3];
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
                unpack(vw, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[e] += w[e];
            }
            uint32_t o[4];
            pack(g, o);
            *reinterpret_cast<uint4*>(a.dx + r * N + col[j]) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (++s == depth) { s = 0; ph ^= 1u; }
    }
    float* part = a.partial + (first + team) * N;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (ok[j]) {
            reinterpret_cast<float4*>(part + col[j])[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
            reinterpret_cast<float4*>(part + col[j])[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
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

constexpr size_t kSmem = 227u << 10;   // per SM and at most per block; 1 KB of the SM's per block is the system's
BwdShape bwd_shape(const Team& tm, int64_t N, bool res) {
    const uint32_t n = (uint32_t)(tm.teams * N);
    BwdShape sh{tm.threads, tm.teams, (int)N, DEPTH, res ? 5 * n : 3 * n, 2 * n, 3 * n};
    while (sh.depth > 2 && smem_of(tm) + sh.depth * (size_t)(5 * n) + 2048 > kSmem) --sh.depth;
    return sh;
}
size_t bwd_smem(const Team& tm, const BwdShape& sh) { return smem_of(tm) + (size_t)sh.depth * sh.stage; }
// blocks that run at once: by threads (64 registers each) and shared memory (227 KB per SM, 1 KB of it per block)
int64_t bwd_blocks(int64_t M, const Team& tm, size_t smem, int sms) {
    int64_t per = 1024 / (tm.threads * tm.teams);
    const int64_t fit = (int64_t)(kSmem / (smem + 2048));
    if (per > fit) per = fit;
    if (per < 1) per = 1;
    const int64_t need = (M + tm.teams - 1) / tm.teams;
    return need < sms * per ? need : sms * per;
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
    return bwd_blocks(M, tm, bwd_smem(tm, bwd_shape(tm, N, true)), sms) * tm.teams;
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
    const bool res = a.dresidual != nullptr;
    const BwdShape sh = bwd_shape(tm, a.N, res);
    const size_t smem = bwd_smem(tm, sh);
    // as many blocks as norm_bwd_partials counts, whatever the gradient past the norm
    const int64_t blocks = bwd_blocks(a.M, tm, bwd_smem(tm, bwd_shape(tm, a.N, true)), device_sms());
    cudaError_t e = allow_smem(res ? norm_bwd_kernel<true> : norm_bwd_kernel<false>, smem);
    if (e != cudaSuccess) return e;
    if (res)
        norm_bwd_kernel<true><<<(unsigned)blocks, tm.threads * tm.teams, smem, s>>>(a, sh);
    else
        norm_bwd_kernel<false><<<(unsigned)blocks, tm.threads * tm.teams, smem, s>>>(a, sh);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_column_sum(a.partial, blocks * tm.teams, a.N, a.dweight, s);
}

cudaError_t read_norm_wait_timeouts(unsigned long long* out, bool reset) { return read_own_wait_timeouts(out, reset); }

}  // namespace coat
