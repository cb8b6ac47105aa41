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
// A row is held by a team of T = 32 ceil(N / 512) threads, sixteen elements each;
// a block has as many teams as fit 256 threads.  Sixteen elements are one 256-bit
// access of a bf16 tensor and one 128-bit access of codes; every tensor is read
// and written once.
//
// Bound by memory.  8192 x 4096, G = 128, with a residual: forward 46.1 us, 98 %
// of the copy rate (without a residual 31.4 us, 80 %); backward 43.5 us, 81 %, of
// which about 10 do not grow with the rows once there are some thousands (two
// kernels, the ring's first rows, the sum over the blocks' dw; a single row takes
// 5): 4099 x 5120 takes 26.7 us, 60 %.  Forward a block has its rows (one team
// each) once, without a loop, so that blocks in different phases keep loads on
// their way; backward persistent blocks, since each keeps its sums for dw in
// registers, fed by a ring of rows in shared memory.
#include <cstdint>
#include <type_traits>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"
#include "ring.h"
#include "tc_pipeline.cuh"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kE = 16;             // elements per thread
constexpr int kMaxWarps = 32;
constexpr int kMaxDepth = 4;

struct Shape {
    int T, teams;          // threads of a row, rows per block and iteration
    int N, depth;          // iterations in the ring
    uint32_t stage;        // bytes of one
    uint32_t b_off, c_off; // of its second and third tensor
    int span;              // the power of two that a team's warps are rounded up to
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// Each team's sum of v over its threads; a barrier of the whole block.
// slots: one float per warp, for this use alone until the next one's barrier;
// `span`: the power of two that the team's warps are rounded up to.
// `stop`, where it is given: set to what `flag` holds behind the barrier.
__device__ __forceinline__ float team_sum(float v, float* slots, int warps, int span, int warp, int lane,
                                          const volatile uint32_t* flag = nullptr, uint32_t* stop = nullptr) {
    v = warp_sum(v);
    if (lane == 0) slots[warp] = v;
    __syncthreads();
    if (flag) *stop = *flag;
    if (warps == 1) return v;
    const int i = lane & (span - 1);
    float s = i < warps ? slots[i] : 0.0f;
    for (int off = span >> 1; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
    return s;
}

// The weights in shared memory: float4 j of the n / 4 of item i at [j items + i], so that
// neighbouring threads read neighbouring float4s.  Zeros behind the row.
template <int n>
__device__ __forceinline__ void stage_weights(const float* w, int N, int items, float4* sw) {
    for (int i = threadIdx.x; i < items * (n / 4); i += blockDim.x)
        sw[(i % (n / 4)) * items + i / (n / 4)] =
            4 * i < N ? reinterpret_cast<const float4*>(w)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
}
template <int n>
__device__ __forceinline__ void weights_of(const float4* sw, int items, int i, float (&w)[n]) {
#pragma unroll
    for (int j = 0; j < n / 4; ++j) {
        const float4 f = sw[j * items + i];
        w[4 * j] = f.x; w[4 * j + 1] = f.y; w[4 * j + 2] = f.z; w[4 * j + 3] = f.w;
    }
}

// Eight weights, in pairs: one 256-bit access where `wide`, which L1 serves in half the passes of two (a lane's sixteen
// lie 64 bytes from the next lane's; 8192 x 4096 without a residual 35.4 us with 128-bit accesses, 31.4 so)
__device__ __forceinline__ void load_weights8(const float* p, bool wide, uint64_t (&w)[4]) {
    if (wide) {
        asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(w[0]), "=l"(w[1]), "=l"(w[2]), "=l"(w[3]) : "l"(p));
    } else {
        const ulonglong2 lo = reinterpret_cast<const ulonglong2*>(p)[0], hi = reinterpret_cast<const ulonglong2*>(p)[1];
        w[0] = lo.x; w[1] = lo.y; w[2] = hi.x; w[3] = hi.y;
    }
}

// y and 1 / rms of a row whose mean square leaves float32's range, again: the sum is formed of kFar times the elements.
// All threads of the team come here, behind everything else, and each warp forms the sum by itself, from memory, so that
// the usual path keeps neither a register nor a barrier for it: 8192 x 4096 without a residual takes 31 us as without
// this function; 39 with the sum formed of the elements in registers and barriers of the team (one whose number is known
// at run time only reserves all sixteen of the block, and fewer blocks fit the SM), 32.6 with this inlined.
template <bool kRes>
__device__ __noinline__ void far_row(const NormFwdArgs& a, const Shape& sh) {
    uint32_t tid;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid) : : "memory");
    const int team = (int)tid / sh.T, t = (int)tid - team * sh.T;
    const int64_t r = (int64_t)blockIdx.x * sh.teams + team, at = r * a.N;
    auto input = [&](int64_t c) {              // not read back from h, which other warps write
        const float v = __uint_as_float((uint32_t)a.x[at + c] << 16);
        if constexpr (!kRes) return v;
        return __uint_as_float(bf16x2(0.0f, v + __uint_as_float((uint32_t)a.residual[at + c] << 16)));
    };
    float ss = 0.0f;
#pragma unroll 1
    for (int c = t & 31; c < sh.N; c += 32) {
        const float v = input(c) * kFar;
        ss = fmaf(v, v, ss);
    }
    const float rstd = kFar * far_rsqrt(fmaf(warp_sum(ss), 1.0f / (float)sh.N, a.eps * kFar * kFar));
#pragma unroll 1
    for (int c = t * kE; c < t * kE + kE && c < sh.N; ++c) a.y[at + c] = bf16_bits(input(c) * rstd * a.weight[c]);
    if (t == 0) a.rstd[r] = rstd;
}

// Forward: a block has its rows once, a thread sixteen consecutive elements (so that a
// group of G >= 16 is G / 16 lanes).  What keeps the memory busy are many small
// blocks per SM in different phases: at 8192 x 4096 with a residual 46.1 us with
// 40 registers (six blocks of 256 threads per SM), 51.0 with 50 (four); blocks
// that walk the rows through a ring of bulk copies, as backward, took 53.3.
template <bool kRes, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) norm_fwd_kernel(const __grid_constant__ NormFwdArgs a, const __grid_constant__ Shape sh, bool wide, bool wide_w) {
    __shared__ float slots[kMaxWarps];
    const int T = sh.T, teams = sh.teams, N = sh.N;
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const int gshift = 31 - __clz(a.G);
    const float inv_n = 1.0f / (float)N;
    const int col = t * kE;
    const int64_t r = (int64_t)blockIdx.x * teams + team, at = r * N + col;
    const bool ok = col < N && r < a.M;
    uint64_t x[kE / 2] = {}, ss2 = 0ull;
    wait_for_primary();
    if (ok) {
        uint32_t u[8];
        load_words8(a.x + at, wide, u);
        if constexpr (kRes) {
            uint32_t v[8];
            uint64_t p[kE / 2];
            load_words8(a.residual + at, wide, v);
            unpack2(u, x);
            unpack2(v, p);
#pragma unroll
            for (int e = 0; e < kE / 2; ++e) {
                float lo, hi;
                upk(add2(x[e], p[e]), lo, hi);
                u[e] = bf16x2(lo, hi);
            }
            store_words8(a.h + at, wide, u);
        }
        unpack2(u, x);
    }
#pragma unroll
    for (int e = 0; e < kE / 2; ++e) ss2 = fma2(x[e], x[e], ss2);
    Scales16 q;
    uint32_t c[4];
    quantize16<true>(x, a.G, q, c);
    if (ok) {
        *reinterpret_cast<uint4*>(a.q + at) = make_uint4(c[0], c[1], c[2], c[3]);
        store_scales16(a.scale, at, a.G, gshift, q);
    }
    const float ss = team_sum(sum2(ss2), slots + team * warps, warps, sh.span, warp, lane);
    const float v = fmaf(ss, inv_n, a.eps), rstd = rsqrt_newton(v);
    const bool far = !(v < INFINITY);
    if (ok) {
        uint32_t u[8];
        const uint64_t r2 = pk(rstd, rstd);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint64_t w[4];
            load_weights8(a.weight + col + 8 * h, wide_w, w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo, hi;
                upk(mul2(mul2(x[4 * h + e], r2), w[e]), lo, hi);
                u[4 * h + e] = bf16x2(lo, hi);
            }
        }
        store_words8(a.y + at, wide, u);
        if (t == 0) a.rstd[r] = rstd;
    }
    if (far) far_row<kRes>(a, sh);   // NaN of an infinite mean square, which the whole team has
}

// Backward: the blocks walk the rows, so many consecutive ones at a time as they
// have teams, with the sums for dw in registers.  The rows come through a ring in
// shared memory, each tensor's one bulk copy: the copies stay ahead without
// registers.  A thread has two chunks of eight columns, T chunks apart, so that
// neighbouring lanes read neighbouring 16 bytes of shared memory.  kThreads: most
// threads of a block.  512: the compiler takes 96 registers, or 99 with a residual,
// which is too many for the 20 warps of two blocks of 320 threads (8192 x 5120
// 67 us, a second wave); 320, bound to 96, is for them (52 us; where both fit, 2 %
// slower).  1024 (N > 8192): 64 registers, so a row's elements are formed again
// from shared memory after its sum instead of being held over it (8192 x 12288
// and 16384 99 and 123 us; held, in local memory, 164 and 222; at N <= 5120 forming
// them again for three or more blocks per SM costs 4 to 8 us).
template <bool kRes, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 320 ? 2 : 1) norm_bwd_kernel(const NormBwdArgs a, const Shape sh) {
    __shared__ float slots[2][kMaxWarps];
    __shared__ uint64_t bars[kMaxDepth];
    __shared__ uint32_t lost[2];       // a wait gave up in an even, in an odd iteration
    extern __shared__ __align__(16) unsigned char dyn[];
    const int T = sh.T, teams = sh.teams, N = sh.N, depth = sh.depth;
    float4* sw = reinterpret_cast<float4*>(dyn);
    unsigned char* ring = dyn + (size_t)T * kE * 4;
    const int team = threadIdx.x / T, t = threadIdx.x - team * T;
    const int lane = threadIdx.x & 31, warps = T >> 5, warp = t >> 5;
    const int gshift = 31 - __clz(a.G);
    const float inv_n = 1.0f / (float)N;
    const int64_t ngr = N >> gshift;
    const uint32_t bar0 = smem_u32(bars), ring0 = smem_u32(ring);
    // Rows as 32-bit numbers (M < 2^31, and a ring's rows beyond the last one stay far below 2^32): 64-bit ones take 98
    // registers where 96 are there for two blocks (8192 x 5120 58.6 us instead of 43.0), and are slower without a residual
    // (8192 x 12288 and 16384 104 and 130 us instead of 99 and 123).  But with one, in the widest rows, they are not:
    // 152 and 181 us instead of 156 and 182.
    using Row = typename std::conditional<kRes && kThreads == 1024, int64_t, uint32_t>::type;
    const Row M = (Row)a.M, step = (Row)gridDim.x * (Row)teams, first = (Row)blockIdx.x * (Row)teams;
    auto issue = [&](Row r0, int s) {
        const uint32_t n = (uint32_t)min(M - r0, (Row)teams) * (uint32_t)N;
        const uint32_t d = ring0 + (uint32_t)s * sh.stage, bar = bar0 + 8u * (uint32_t)s;
        mbar_expect_tx(bar, n * (kRes ? 5u : 3u));
        const int64_t at = (int64_t)r0 * N;
        bulk_load(d, a.dy + at, 2 * n, bar);
        bulk_load(d + sh.b_off, a.q + at, n, bar);
        if constexpr (kRes) bulk_load(d + sh.c_off, a.dresidual + at, 2 * n, bar);
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < depth; ++s) mbar_init(bar0 + 8u * (uint32_t)s, 1);
        lost[0] = lost[1] = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    wait_for_primary();
    if (threadIdx.x == 0) {
        for (int s = 0; s < depth; ++s)
            if (first + s * step < M) issue(first + s * step, s);
    }
    stage_weights<8>(a.weight, N, 2 * T, sw);
    __syncthreads();
    bool in_row[2];
    int col[2];
    uint64_t dw[2][4];
    float Sn[2] = {0.0f, 0.0f}, rn = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        col[j] = (j * T + t) * 8;
        in_row[j] = col[j] < N;
#pragma unroll
        for (int e = 0; e < 4; ++e) dw[j][e] = 0ull;
    }
    auto fetch_scales = [&](Row r) {   // one iteration ahead
        if (r < M) {
            rn = a.rstd[r];
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (in_row[j]) Sn[j] = a.scale[(int64_t)r * ngr + (col[j] >> gshift)];
        }
    };
    fetch_scales(first + team);
    int s = 0;
    uint32_t ph = 0;
    Row r0 = first;
    uint32_t it = 0;
    for (; r0 < M; r0 += step, ++it) {
        const Row r = r0 + team;
        bool live = r < M;                 // a team past the last row only keeps step
        const float rstd = rn, S[2] = {Sn[0] * rn, Sn[1] * rn};
        fetch_scales(r + step);
        mbar_wait_fast(bar0 + 8u * (uint32_t)s, ph, &lost[it & 1]);   // what it says is asked behind the barrier
        const unsigned char* st = ring + (size_t)s * sh.stage;
        uint64_t g[2][4], xh[2][4], c2 = 0ull;
        auto values = [&](int j, uint64_t (&dy)[4]) {   // of eight elements: dy, g and xh
            const uint4 d = *reinterpret_cast<const uint4*>(st + ((size_t)team * N + col[j]) * 2);
            const uint2 q = *reinterpret_cast<const uint2*>(st + sh.b_off + (size_t)team * N + col[j]);
            const uint32_t dw4[4] = {d.x, d.y, d.z, d.w}, qw[2] = {q.x, q.y};
            float gf[8], xf[8], w[8];
            unpack(dw4, gf);
            decode(qw, xf);
            weights_of(sw, 2 * T, j * T + t, w);
            const uint64_t SS = pk(S[j], S[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dy[e] = pk(gf[2 * e], gf[2 * e + 1]);
                xh[j][e] = mul2(pk(xf[2 * e], xf[2 * e + 1]), SS);
                g[j][e] = mul2(dy[e], pk(w[2 * e], w[2 * e + 1]));
            }
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!live || !in_row[j]) continue;
            uint64_t dy[4];
            values(j, dy);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dw[j][e] = fma2(dy[e], xh[j][e], dw[j][e]);
                c2 = fma2(g[j][e], xh[j][e], c2);
            }
        }
        float c0, c1;
        upk(c2, c0, c1);
        uint32_t stop;
        const float c = team_sum(c0 + c1, slots[it & 1] + team * warps, warps, sh.span, warp, lane, &lost[it & 1], &stop) * inv_n;
        // a wait that gave up ends the loop for the whole block (below): the flag is read between this iteration's barrier
        // and the next one, and written before the one or behind the other
        live = live && stop == 0u;
        // behind that barrier every thread is done with the iteration before this one: its stage is free
        if (threadIdx.x == 0 && it > 0 && stop == 0u) {
            const Row rr = r0 + (depth - 1) * step;
            if (rr < M) issue(rr, s == 0 ? depth - 1 : s - 1);
        }
        const uint64_t nc = pk(-c, -c), rr2 = pk(rstd, rstd);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!live || !in_row[j]) continue;
            if constexpr (kThreads > 512) {   // formed again: 64 registers do not hold them over the barrier
                uint64_t dy[4];
                values(j, dy);
            }
            uint32_t o[4];
            uint32_t p[4] = {};
            if constexpr (kRes) {
                const uint4 v = *reinterpret_cast<const uint4*>(st + sh.c_off + ((size_t)team * N + col[j]) * 2);
                p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t d = fma2(xh[j][e], nc, g[j][e]);
                const uint64_t res = kRes ? pk(__uint_as_float(p[e] << 16), __uint_as_float(p[e] & 0xFFFF0000u)) : 0ull;
                float lo, hi;
                upk(kRes ? fma2(d, rr2, res) : mul2(d, rr2), lo, hi);
                o[e] = bf16x2(lo, hi);
            }
            *reinterpret_cast<uint4*>(a.dx + (int64_t)r * N + col[j]) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (stop != 0u) break;
        if (++s == depth) { s = 0; ph ^= 1u; }
    }
    dependents_may_start();
    float* part = a.partial + (int64_t)(first + team) * N;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (in_row[j]) {
            ulonglong2* p = reinterpret_cast<ulonglong2*>(part + col[j]);   // pairs of floats, as they lie
            p[0] = make_ulonglong2(dw[j][0], dw[j][1]);
            p[1] = make_ulonglong2(dw[j][2], dw[j][3]);
        }
    // stopped early: the copies on their way have to land before the block may leave its shared memory
    if (r0 < M && threadIdx.x == 0)
        ring_drain(it, (M - first + step - 1) / step, depth,
                   [&](int stage, uint32_t parity) { mbar_wait(bar0 + 8u * (uint32_t)stage, parity, nullptr); });
}

// kCols columns of one of two sums per block, 1024 / kCols rows of the partial sums side by side and four more on their
// way in each thread.  32 columns read whole lines; 8 give four times the blocks, which is what few columns need.
template <int kCols>
__global__ void __launch_bounds__(1024) column_sum_kernel(const ColumnSum first, const ColumnSum second, int64_t N) {
    constexpr int kRows = 1024 / kCols;
    __shared__ float part[kCols][kRows + 1];
    const ColumnSum cs = blockIdx.y == 0 ? first : second;
    const int col = threadIdx.x % kCols, row = threadIdx.x / kCols;
    const int64_t c = (int64_t)blockIdx.x * kCols + col;
    if (cs.P == 0) return;
    wait_for_primary();
    float s = 0.0f;
    if (c < N) {
        int64_t p = row;
        for (; p + 3 * kRows < cs.P; p += 4 * kRows) {
            const float v0 = cs.partial[p * N + c], v1 = cs.partial[(p + kRows) * N + c];
            const float v2 = cs.partial[(p + 2 * kRows) * N + c], v3 = cs.partial[(p + 3 * kRows) * N + c];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; p < cs.P; p += kRows) s += cs.partial[p * N + c];
    }
    part[col][row] = s;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= kCols) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kRows; i += 32) s += part[warp][lane + i];
    s = warp_sum(s);
    if (lane == 0 && (int64_t)blockIdx.x * kCols + warp < N) cs.out[(int64_t)blockIdx.x * kCols + warp] = bf16_bits(s);
}

constexpr size_t kSmem = 227u << 10;   // shared memory per SM, and at most per block
constexpr size_t kMostDynamic = kSmem - 2048;

Shape team_shape(int64_t N) {
    const int T = 32 * (int)((N + 32 * kE - 1) / (32 * kE)), teams = T >= 256 ? 1 : 256 / T;
    Shape sh{T, teams, (int)N, 0, 0, 0, 0, 1};
    while (32 * sh.span < T) sh.span *= 2;
    return sh;
}
size_t smem_of(const Shape& sh) { return (size_t)sh.T * kE * 4 + (size_t)sh.depth * sh.stage; }
Shape bwd_shape(int64_t N, bool res) {
    Shape sh = team_shape(N);
    const uint32_t n = (uint32_t)(sh.teams * N);
    sh.stage = res ? 5 * n : 3 * n;
    sh.b_off = 2 * n;
    sh.c_off = 3 * n;
    // iterations in the ring: 8192 x 4096 takes 58 us with two, 44 with three or four; one block per SM (T > 320) wants
    // four: 8192 x 8192 69 us with three, 66 with four; fewer where a row is too wide
    sh.depth = sh.T > 320 ? 4 : 3;
    while (sh.depth > 2 && smem_of(sh) > kMostDynamic) --sh.depth;
    return sh;
}
// Blocks that run at once, so that the grid is one wave: by registers (`regs` per thread, a multiple of eight; each of the
// SM's four parts has 16384 of them for whole warps) and by shared memory (2 KB more per block: the static part, and the
// system's).
int64_t blocks_of(int64_t M, const Shape& sh, int regs, int sms) {
    int64_t per = 4 * (16384 / (32 * regs)) / (sh.T * sh.teams / 32);
    const int64_t fit = (int64_t)(kSmem / (smem_of(sh) + 2048));
    if (per > fit) per = fit;
    if (per < 1) per = 1;
    const int64_t need = (M + sh.teams - 1) / sh.teams;
    return need < sms * per ? need : sms * per;
}
int64_t bwd_blocks(int64_t M, int64_t N, bool res, int sms) {
    const Shape sh = bwd_shape(N, res);
    return blocks_of(M, sh, sh.T <= 320 ? 96 : sh.T <= 512 ? 128 : 64, sms);
}

// More than the 48 KB that every kernel may have, its static part (under 1 KB) included.  The most of any width, not this
// call's: another thread, whose rows are narrower, may set it before this one launches.
template <typename F>
cudaError_t allow_smem(F* kernel, size_t bytes) {
    return bytes <= (47u << 10) ? cudaSuccess
                                : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostDynamic);
}

template <bool kRes>
cudaError_t launch_fwd(const NormFwdArgs& a, cudaStream_t s) {
    const Shape sh = team_shape(a.N);
    const bool wide = aligned32(a.x) && aligned32(a.residual) && aligned32(a.h) && aligned32(a.y);
    const bool wide_w = aligned32(a.weight);
    const unsigned blocks = (unsigned)((a.M + sh.teams - 1) / sh.teams);
    const int threads = sh.T * sh.teams;
    if (threads <= 256)
        return launch_next(norm_fwd_kernel<kRes, 256, 6>, blocks, threads, 0, s, a, sh, wide, wide_w);
    if (threads <= 512)
        return launch_next(norm_fwd_kernel<kRes, 512, 3>, blocks, threads, 0, s, a, sh, wide, wide_w);
    // two blocks per SM up to N = 12288 (8192 x 12288 without a residual: 169 us with one, 117 with two; 102 now)
    if (threads <= 768) return launch_next(norm_fwd_kernel<kRes, 768, 2>, blocks, threads, 0, s, a, sh, wide, wide_w);
    return launch_next(norm_fwd_kernel<kRes, 1024, 1>, blocks, threads, 0, s, a, sh, wide, wide_w);
}

template <bool kRes, int kThreads>
cudaError_t launch_bwd(const NormBwdArgs& a, int64_t blocks, const Shape& sh, cudaStream_t s) {
    const cudaError_t e = allow_smem(norm_bwd_kernel<kRes, kThreads>, smem_of(sh));
    if (e != cudaSuccess) return e;
    return launch_next(norm_bwd_kernel<kRes, kThreads>, (unsigned)blocks, sh.T * sh.teams, smem_of(sh), s, a, sh);
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
    const int64_t with = bwd_blocks(M, N, true, sms), without = bwd_blocks(M, N, false, sms);
    return (with > without ? with : without) * bwd_shape(N, false).teams;
}

cudaError_t launch_column_sums(const ColumnSum& first, const ColumnSum& second, int64_t N, cudaStream_t s) {
    const int cols = N <= 512 ? 8 : 32;
    const dim3 grid((unsigned)((N + cols - 1) / cols), second.P > 0 ? 2 : 1);
    return launch_next(cols == 8 ? column_sum_kernel<8> : column_sum_kernel<32>, grid, 1024, 0, s, first, second, N);
}

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s) {
    return a.residual ? launch_fwd<true>(a, s) : launch_fwd<false>(a, s);
}

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) {
    const bool res = a.dresidual != nullptr;
    const Shape sh = bwd_shape(a.N, res);
    const int64_t blocks = bwd_blocks(a.M, a.N, res, device_sms());
    cudaError_t e;
    if (res && sh.T <= 320 && sh.T * sh.teams != 256)   // 256 threads: two blocks with 104 registers as with 96
        e = launch_bwd<true, 320>(a, blocks, sh, s);
    else if (sh.T <= 512)
        e = res ? launch_bwd<true, 512>(a, blocks, sh, s) : launch_bwd<false, 512>(a, blocks, sh, s);
    else
        e = res ? launch_bwd<true, 1024>(a, blocks, sh, s) : launch_bwd<false, 1024>(a, blocks, sh, s);
    if (e != cudaSuccess) return e;
    return launch_column_sums(ColumnSum{a.partial, blocks * sh.teams, a.dweight}, ColumnSum{nullptr, 0, nullptr}, a.N, s);
}

cudaError_t read_norm_wait_timeouts(unsigned long long* out, bool reset) { return read_own_wait_timeouts(out, reset); }

}  // namespace coat
