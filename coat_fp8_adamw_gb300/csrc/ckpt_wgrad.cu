// ckpt_wgrad.cu -- the weight gradient of a linear layer from the 8-bit checkpoint
// of its input (COAT review page, section 3: FP8 activations kept for the
// backward pass).
//
//   dW[n, k] = c[k] sum_m dY[m, n] X[m, k],  X[m, k] = r[m] S[m, k / G] E4M3(q[m, k])
//
// r (per token) and c (per input column) are optional factors: with r = 1 / rms
// and c = the norm's weight, the checkpoint of a norm's input serves the
// linear layer behind the norm too.
//
// The sum runs over tokens, and a scale belongs to one token and G columns, so
// it cannot be taken out of the sum: X is formed in shared memory as a bf16
// operand, RN((S r) E4M3(q)), one rounding of a relative 2^-9 at most (dY is
// bf16 already), and the products are summed in float32 by the tensor cores.
// Both operands lie in memory with the output index along the row, which
// the tensor cores read as "MN-major" operands: nothing is transposed.
//
// Persistent CTA pairs (clusters of two, one CTA per SM) walk 256 x 256 tiles of
// dW, 64 tokens per step.  Per step a CTA holds dY for its 128 rows of the tile
// and X for its 128 columns:
//   TMA warp       dY (two 64-column boxes, 128-byte swizzle; both CTAs' bytes
//                  counted on the even CTA's barrier) and the raw codes;
//   scale warp     the stage's group scales and token factors (cp.async);
//   8 warps        codes -> bf16 operand in the swizzled layout;
//   MMA thread     (even CTA) four tcgen05.mma.cta_group::2 kind::f16, M = N = 256,
//                  K = 16, into one of two 256-column accumulators;
//   4 warps        the finished accumulator: times c, to bf16, stored.
// Tiles left over after the last full round of the pairs are split along the
// tokens, so that they too keep every pair busy: each part leaves a float32
// tile in the workspace, and a second kernel adds the parts in order.
//
// Every wait on an mbarrier is bounded, as in linear_fp8.cu.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"
#include "tc_pipeline.cuh"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kTile = 256;                     // rows (n) and columns (k) of a pair's tile of dW
constexpr int kHalf = kTile / 2;               // a CTA's rows of it, and its columns of X
constexpr int kTok = 64;                       // tokens per stage
constexpr int kMmaTok = 16;                    // tokens of one kind::f16 MMA
constexpr int kStages = 5;
constexpr int kBoxBytes = kTok * 128;          // 64 tokens x 64 bf16 columns
constexpr int kYBytes = 2 * kBoxBytes;         // dY: 64 tokens x 128 columns
constexpr int kXBytes = 2 * kBoxBytes;         // X in bf16
constexpr int kQBytes = kTok * kHalf;          // the codes
constexpr int kStageBytes = kYBytes + kXBytes + kQBytes;
constexpr int kEpiWarps = 4;
constexpr int kDeqWarps = 8;
constexpr int kWgThreads = 32 * (4 + kEpiWarps + kDeqWarps);
constexpr uint32_t kTmemCols = 2 * kTile;      // two accumulators of 256 f32 columns
constexpr int kMaxGroups = kHalf / 8;           // scale groups of a CTA's 128 columns
constexpr int kSPitch = kTok + 4;              // floats between two groups' scales: banks 4 apart
constexpr int kScaleBytes = (kMaxGroups * kSPitch + kTok) * 4;   // a stage's scales, and its tokens' r
constexpr int kScaleOff = kStages * kStageBytes;
constexpr int kBarOff = kScaleOff + kStages * kScaleBytes;
constexpr int kNumBars = 4 * kStages + 5;      // dY full, codes full, X full, empty; acc full x2, acc empty x2, done
constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 16 + 1024;   // + slack for 1024-B alignment
constexpr int kMinSteps = 8;                   // fewest steps of a split's part

// Instruction descriptor: D in f32 (bits 4-5 = 1), A and B bf16 (bits 7-9 and
// 10-12 = 1), both MN-major (bits 15, 16), N / 8 in bits 17-22, M / 16 in bits
// 24-28 (M = 256 over the two CTAs).
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                            ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);

// Shared-memory matrix descriptor of an MN-major operand in the 128-byte
// swizzled layout: rows (tokens) of 128 bytes = 64 columns, 8-row (1024-byte)
// swizzle atoms.  Start address / 16 in bits 0-13; the distance between two
// blocks of 64 columns / 16 in bits 16-29; the distance between two groups of
// 8 tokens / 16 in bits 32-45; version 1 in bits 46-47; swizzle mode 2 (128
// bytes) in bits 61-63.
__device__ __forceinline__ uint64_t mn_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kBoxBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
        : "memory");
}
// 4 bytes global -> shared, asynchronously; zero where `ok` is not set
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
// one arrival on `bar` once every cp.async that this thread issued before has landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// a 2-D tile into this CTA's shared memory, counted on this CTA's own barrier
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// How the tiles of dW go to the pairs: the first `whole` tiles one by one, the
// other `tail` ones in `parts` parts along the tokens each.
struct Plan {
    int64_t tn, tk;          // tiles along n and k
    int64_t whole, tail;
    int32_t parts, steps;    // steps: 64-token steps in all
};
Plan make_plan(int64_t M, int64_t N, int64_t K, int64_t pairs) {
    Plan p;
    p.tn = (N + kTile - 1) / kTile;
    p.tk = (K + kTile - 1) / kTile;
    p.steps = (int32_t)((M + kTok - 1) / kTok);
    const int64_t tiles = p.tn * p.tk, rest = tiles % pairs;
    int64_t parts = rest > 0 ? pairs / rest : 1;
    if (parts > p.steps / kMinSteps) parts = p.steps / kMinSteps;
    p.parts = parts > 1 ? (int32_t)parts : 1;
    p.tail = parts > 1 ? rest : 0;
    p.whole = tiles - p.tail;
    return p;
}

// Tile order: bands of kBand tiles along n, k-major inside a band, so that the
// pairs that run at once share rows of dY and of X in L2.
constexpr int64_t kBand = 8;
__device__ __forceinline__ void tile_at(int64_t t, const Plan& p, int64_t& n, int64_t& k) {
    const int64_t band = t / (kBand * p.tk), first = band * kBand;
    const int64_t rows = p.tn - first < kBand ? p.tn - first : kBand;
    const int64_t r = t - band * kBand * p.tk;
    n = first + r % rows;
    k = r / rows;
}
struct Item {
    int64_t n, k;        // tile
    int32_t from, to;    // steps
    int64_t part;        // index of its float32 tile, or -1: the whole sum
};
__device__ __forceinline__ Item item_at(int64_t i, const Plan& p) {
    Item it;
    if (i < p.whole) {
        tile_at(i, p, it.n, it.k);
        it.from = 0;
        it.to = p.steps;
        it.part = -1;
    } else {
        const int64_t j = i - p.whole;
        const int32_t s = (int32_t)(j % p.parts);
        tile_at(p.whole + j / p.parts, p, it.n, it.k);
        it.from = (int32_t)((int64_t)p.steps * s / p.parts);
        it.to = (int32_t)((int64_t)p.steps * (s + 1) / p.parts);
        it.part = j;
    }
    return it;
}

// Two codes as bf16(value * s), packed
__device__ __forceinline__ uint32_t deq2(uint32_t codes, float s) {
    uint32_t h;
    float lo, hi;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return bf16x2(lo * s, hi * s);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ float lds32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__global__ void __launch_bounds__(kWgThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap tmy, const __grid_constant__ CUtensorMap tmq, const WgradArgs a,
             const Plan plan) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // the same offset in both CTAs
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar0 = sb + kBarOff;
    auto bar = [&](int kind, int s) { return bar0 + 8u * (uint32_t)(kind * kStages + s); };
    auto y_full = [&](int s) { return bar(0, s); };
    auto q_full = [&](int s) { return bar(1, s); };
    auto x_full = [&](int s) { return bar(2, s); };
    auto empty = [&](int s) { return bar(3, s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (uint32_t)(4 * kStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (uint32_t)(4 * kStages + 2 + b); };
    const uint32_t done = bar0 + 8u * (uint32_t)(4 * kStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kNumBars);
    volatile uint32_t* abort = tmem_slot + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();   // 0: the CTA that issues the pair's MMAs
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(y_full(s), 1);
            mbar_init(q_full(s), 1 + 32);   // the codes' copy, and every lane's scales
            mbar_init(x_full(s), 2 * kDeqWarps);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) { mbar_init(acc_full(b), 1); mbar_init(acc_empty(b), 2 * kEpiWarps); }
        mbar_init(done, 1);
        *abort = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmy)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmq)) : "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();   // barriers initialised and tensor memory allocated in both CTAs
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int64_t items = plan.whole + plan.tail * plan.parts;
    const int64_t cid = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        // ---- TMA producer (both CTAs) ----
        int s = 0;
        uint32_t ph = 0, issued = 0, last_ph = 0;   // per stage: issued at all, parity of the last issue
        bool ok = true;
        const uint32_t yb0 = map_to_rank(y_full(0), 0);
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            const int32_t n0 = (int32_t)(it.n * kTile + rank * kHalf), k0 = (int32_t)(it.k * kTile + rank * kHalf);
            for (int32_t st = it.from; st < it.to; ++st) {
                if (!mbar_wait_fast(empty(s), ph ^ 1u, abort)) { ok = false; break; }
                if (leader) mbar_expect_tx(y_full(s), (uint32_t)(2 * kYBytes));
                mbar_expect_tx(q_full(s), (uint32_t)kQBytes);
                const uint32_t sa = sb + (uint32_t)(s * kStageBytes), yb = yb0 + 8u * (uint32_t)s;
                tma_load_2d(sa + kYBytes + kXBytes, &tmq, k0, st * kTok, q_full(s));
                tma_load_2d_pair(sa, &tmy, n0, st * kTok, yb);
                tma_load_2d_pair(sa + kBoxBytes, &tmy, n0 + 64, st * kTok, yb);
                issued |= 1u << s;
                last_ph = (last_ph & ~(1u << s)) | (ph << s);
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        // every stage issued has been read by the MMAs before the CTA may exit
        for (int i = 0; i < kStages; ++i)
            if (issued & (1u << i)) mbar_wait(empty(i), (last_ph >> i) & 1u, nullptr);
    } else if (warp == 1 && lane == 0) {
        if (leader) {
            // ---- MMA issuer ----
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            const uint64_t ydesc0 = mn_desc(sb), xdesc0 = mn_desc(sb + kYBytes);
            for (int64_t i = cid; ok && i < items; i += nclusters) {
                const Item it = item_at(i, plan);
                if (!mbar_wait_fast(acc_empty(acc), aph ^ 1u, abort)) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * kTile);
                for (int32_t st = it.from; st < it.to; ++st) {
                    if (!mbar_wait_fast(y_full(s), ph, abort) || !mbar_wait_fast(x_full(s), ph, abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)(s * (kStageBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kTok / kMmaTok; ++kk) {
                        const uint64_t off = so + (uint64_t)(kk * ((kMmaTok * 128) >> 4));
                        mma_bf16_pair(d, ydesc0 + off, xdesc0 + off, st != it.from || kk != 0);
                    }
                    mma_commit_pair(empty(s), 0x3);   // both CTAs' stage s is free once read
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                }
                if (!ok) break;
                mma_commit_pair(acc_full(acc), 0x3);
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            mma_commit_pair(done, 0x3);   // every MMA issued has completed before either CTA frees tensor memory
        }
        mbar_wait(done, 0u, nullptr);
    } else if (warp == 3) {
        // ---- scale loader (both CTAs): two tokens per lane, every group of this CTA's columns ----
        const int64_t ngr = a.K / a.G;
        const int groups = kHalf / a.G;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            const int64_t g0 = (it.k * kTile + rank * kHalf) / a.G;
            for (int32_t st = it.from; st < it.to; ++st) {
                if (!mbar_wait_fast(empty(s), ph ^ 1u, abort)) { ok = false; break; }
                const uint32_t dst = sb + kScaleOff + (uint32_t)(s * kScaleBytes);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t m = (int64_t)st * kTok + lane + 32 * h;
                    const bool row_ok = m < a.M;
                    const float* src = a.scale + (row_ok ? m * ngr : 0);
                    const uint32_t d = dst + 4u * (uint32_t)(lane + 32 * h);
                    for (int j = 0; j < groups; ++j) {
                        const bool in = row_ok && g0 + j < ngr;
                        cp_async4(d + 4u * (uint32_t)(j * kSPitch), in ? src + g0 + j : a.scale, in);
                    }
                    if (a.row_scale)
                        cp_async4(d + 4u * (uint32_t)(kMaxGroups * kSPitch), a.row_scale + (row_ok ? m : 0), row_ok);
                }
                cp_async_arrive(q_full(s));
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4 && warp < 4 + kEpiWarps) {
        // ---- epilogue: lane = one row n of the tile ----
        const int q4 = warp & 3;
        int acc = 0;
        uint32_t aph = 0;
        for (int64_t i = cid; i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            if (!mbar_wait_fast(acc_full(acc), aph, abort)) break;
            tc_fence_after();
            const int row = (int)rank * kHalf + 32 * q4 + lane;
            const int64_t n = it.n * kTile + row, k0 = it.k * kTile;
            const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(acc * kTile);
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
                if (k0 + c >= a.K) break;   // the same for the whole warp
                uint32_t v[32];
                __syncwarp();
                tmem_ld<32>(taddr + (uint32_t)c, v);
                if (it.part >= 0) {
                    float4* p = reinterpret_cast<float4*>(a.partial + (it.part * kTile + row) * kTile + c);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                           __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                } else if (n < a.N) {
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        const int64_t k = k0 + c + j;
                        if (k >= a.K) break;
                        float x[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(v[j + e]);
                        if (a.col_scale) {
                            const float4 f0 = __ldg(reinterpret_cast<const float4*>(a.col_scale + k));
                            const float4 f1 = __ldg(reinterpret_cast<const float4*>(a.col_scale + k) + 1);
                            x[0] *= f0.x; x[1] *= f0.y; x[2] *= f0.z; x[3] *= f0.w;
                            x[4] *= f1.x; x[5] *= f1.y; x[6] *= f1.z; x[7] *= f1.w;
                        }
                        *reinterpret_cast<uint4*>(a.dw + n * a.K + k) = pack8(x);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_to_rank(acc_empty(acc), 0));
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    } else if (warp >= 4 + kEpiWarps) {
        // ---- codes -> bf16 operand: a thread takes 16 columns of two tokens per stage ----
        const int t = threadIdx.x - 32 * (4 + kEpiWarps);
        const int r0 = t >> 3, c = t & 7;              // token of the stage (and r0 + 32), 16-column chunk
        const uint32_t xb0 = map_to_rank(x_full(0), 0);
        // the scales of the chunk's first and last eight columns, and the tokens' factors
        const uint32_t s0 = 4u * (uint32_t)(((16 * c) / a.G) * kSPitch + r0);
        const uint32_t s1 = 4u * (uint32_t)(((16 * c + 8) / a.G) * kSPitch + r0);
        const uint32_t sr = 4u * (uint32_t)(kMaxGroups * kSPitch + r0);
        const int u = 2 * (c & 3);         // 16-byte unit of the row; the swizzle XORs it with row % 8
        const bool swap = c >= 4;          // the order of a chunk's halves that keeps a quarter-warp's eight stores on different banks
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            for (int32_t st = it.from; st < it.to; ++st) {
                if (!mbar_wait_fast(q_full(s), ph, abort)) { ok = false; break; }
                const uint32_t sa = sb + (uint32_t)(s * kStageBytes), ss = sb + kScaleOff + (uint32_t)(s * kScaleBytes);
                uint4 v[2];
                float f0[2], f1[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[h] = lds128(sa + kYBytes + kXBytes + (uint32_t)((r0 + 32 * h) * kHalf + 16 * c));
                    f0[h] = lds32(ss + s0 + 128u * h);
                    f1[h] = lds32(ss + s1 + 128u * h);
                }
                if (a.row_scale) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float r = lds32(ss + sr + 128u * h);
                        f0[h] *= r;
                        f1[h] *= r;
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = r0 + 32 * h;
                    const uint4 lo = make_uint4(deq2(v[h].x & 0xFFFFu, f0[h]), deq2(v[h].x >> 16, f0[h]),
                                                deq2(v[h].y & 0xFFFFu, f0[h]), deq2(v[h].y >> 16, f0[h]));
                    const uint4 hi = make_uint4(deq2(v[h].z & 0xFFFFu, f1[h]), deq2(v[h].z >> 16, f1[h]),
                                                deq2(v[h].w & 0xFFFFu, f1[h]), deq2(v[h].w >> 16, f1[h]));
                    const uint32_t base = sa + kYBytes + (uint32_t)((c >> 2) * kBoxBytes + row * 128);
                    const uint32_t a0 = base + (uint32_t)((u ^ (row & 7)) * 16), a1 = base + (uint32_t)(((u + 1) ^ (row & 7)) * 16);
                    sts128(swap ? a1 : a0, swap ? hi : lo);
                    sts128(swap ? a0 : a1, swap ? lo : hi);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_at(xb0 + 8u * (uint32_t)s);
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
    }
    tc_fence_before();
    cluster_sync();   // no arrival or copy is still on its way to either CTA
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
}

// The tiles that were split: parts added in order, times c, to bf16.  A block takes 8 rows of a tile.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const WgradArgs a, const Plan plan) {
    const int64_t j = blockIdx.x >> 5;                // tail tile
    const int row = (int)(blockIdx.x & 31) * 8 + (threadIdx.x >> 5), c = (threadIdx.x & 31) * 8;
    int64_t tn, tk;
    tile_at(plan.whole + j, plan, tn, tk);
    const int64_t n = tn * kTile + row, k = tk * kTile + c;
    if (n >= a.N || k >= a.K) return;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < plan.parts; ++p) {
        const float4* src = reinterpret_cast<const float4*>(a.partial + ((j * plan.parts + p) * kTile + row) * kTile + c);
        const float4 f0 = src[0], f1 = src[1];
        x[0] += f0.x; x[1] += f0.y; x[2] += f0.z; x[3] += f0.w;
        x[4] += f1.x; x[5] += f1.y; x[6] += f1.z; x[7] += f1.w;
    }
    if (a.col_scale) {
        const float4 f0 = __ldg(reinterpret_cast<const float4*>(a.col_scale + k));
        const float4 f1 = __ldg(reinterpret_cast<const float4*>(a.col_scale + k) + 1);
        x[0] *= f0.x; x[1] *= f0.y; x[2] *= f0.z; x[3] *= f0.w;
        x[4] *= f1.x; x[5] *= f1.y; x[6] *= f1.z; x[7] *= f1.w;
    }
    *reinterpret_cast<uint4*>(a.dw + n * a.K + k) = pack8(x);
}

// rows x cols elements, row-major, ld elements apart; boxes of box_cols x 64 rows, zeros outside the tensor
bool encode(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, bool bf16) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(bf16 ? 2 * ld : ld)};
    const cuuint32_t box[2] = {(cuuint32_t)(bf16 ? 64 : kHalf), (cuuint32_t)kTok};
    const cuuint32_t elem[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
              strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
              bf16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs: the plan (and with it the workspace and the order of the sums) goes by the SM count alone
int64_t pairs_of(int sms) { return sms / 2; }

}  // namespace

size_t wgrad_workspace(int64_t M, int64_t N, int64_t K, int sms) {
    const Plan p = make_plan(M, N, K, pairs_of(sms));
    return (size_t)(p.tail * p.parts) * (size_t)(kTile * kTile) * sizeof(float);
}

cudaError_t launch_wgrad(const WgradArgs& a, cudaStream_t s) {
    const int64_t pairs = pairs_of(device_sms());
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    const Plan p = make_plan(a.M, a.N, a.K, pairs);
    alignas(64) CUtensorMap tmy, tmq;
    if (!encode(&tmy, a.dy, a.M, a.N, a.dy_ld, true) || !encode(&tmq, a.q, a.M, a.K, a.K, false)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWgThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int64_t items = p.whole + p.tail * p.parts;
    cfg.gridDim = dim3(2u * (unsigned)(items < pairs ? items : pairs));
    if ((e = cudaLaunchKernelEx(&cfg, wgrad_kernel, tmy, tmq, a, p)) != cudaSuccess) return e;
    if (p.tail > 0) wgrad_join_kernel<<<(unsigned)(p.tail * 32), 256, 0, s>>>(a, p);
    return cudaGetLastError();
}

cudaError_t read_wgrad_wait_timeouts(unsigned long long* out, bool reset) {
    const unsigned long long zero = 0ull;
    const cudaError_t e = cudaMemcpyFromSymbol(out, g_wait_timeouts, sizeof(*out));
    return e == cudaSuccess && reset ? cudaMemcpyToSymbol(g_wait_timeouts, &zero, sizeof(zero)) : e;
}

}  // namespace coat
