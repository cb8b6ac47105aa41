// lm_lce.cu -- softmax cross entropy of a linear layer over a large vocabulary, and its gradient, without the logits
// being kept.
//
//   z = x W^T;  lse[m] = log sum_v e^z[m, v];  loss[m] = lse[m] - z[m, t[m]]
//   dz[m, v] = e^(z[m, v] - lse[m]) (g[m] + h[m]) - [v = t[m]] g[m];  dx = dz W;  dW = dz^T x
//
// Four matrix products of 2 M V C operations, one forward and three backward (z is formed again), on the tensor cores:
//   forward   a tile's logits stay in tensor memory; each of its rows leaves its maximum and sum of exponentials per
//             half a tile (and the target's logit), which a second kernel joins: loss and lse;
//   backward  in pieces of the vocabulary: a piece's logits again, whose epilogue leaves dz (bf16, in the workspace); then
//             dx (added up over the pieces in float32) and the piece's rows of dW in one launch.
// dz is rounded to bf16, since it is an operand of the tensor cores, like a layer's gradient that a step keeps as bf16.
//
// One kernel for all four: persistent CTA pairs (clusters of two, one CTA per SM) walk tiles of 256 rows x BN columns,
// 64 of the summed index per stage, as in linear_fp8.cu: each CTA has its 128 rows of A and half of the columns of B in
// a ring of stages filled by TMA (128-byte swizzle), one thread of the even CTA issues tcgen05.mma.cta_group::2
// kind::f16, and eight epilogue warps per CTA read one of two accumulators in tensor memory while the other one fills.
// An operand lies as it is in memory, with its summed index along the row (K-major: x and W for z, dz for dx) or across
// it (MN-major: W for dx, dz and x for dW): the MMA takes both, and nothing is transposed.
// Every wait on an mbarrier is bounded, as in linear_fp8.cu.
#include <cstdint>

#include "ckpt_kernels.h"
#include "lm_device.cuh"
#include "lm_kernels.h"
#include "tc_pipeline.cuh"

namespace coat {

namespace {

using namespace ckpt;
using lm::index_at;

constexpr int kBM = 128;                       // rows per CTA (the pair's MMA has M = 256)
constexpr int kBK = 64;                        // of the summed index per stage: 128 bytes
constexpr int kMmaK = 16;
constexpr int kABytes = kBM * kBK * 2;         // 16 KB
constexpr int kBoxBytes = kBK * 128;           // MN-major: 64 of the summed index x 64 of the other one
constexpr int kEpiWarps = 8;                   // two per SM sub-partition, each half the columns
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kChunk = 32;                     // columns that an epilogue thread holds at once
constexpr float kLog2e = 1.4426950408889634f;

template <int BN>
struct Shape {
    static constexpr int kBBytes = (BN / 2) * kBK * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = BN == 256 ? 7 : 9;
    static constexpr int kBarOff = kStages * kStageBytes;
    static constexpr int kNumBars = 2 * kStages + 5;   // full, empty, acc full x2, acc empty x2, done
    static constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 16 + 1024;   // + slack for 1024-B alignment
    static_assert(kSmemBytes <= 232448, "shared memory of an SM");
};

// What a launch does with a tile's sums.
enum Mode : int32_t { kStats, kDz, kDx, kDw };

struct Job {
    int32_t mode;
    int32_t a_mn, b_mn;      // the operands are MN-major
    int32_t steps;           // 64 of the summed index each
    int64_t tm, tn;          // tiles
    int64_t rows, cols;      // of the product
    uint16_t* out;           // kDz, kDx (last piece), kDw: bf16, ld apart
    int64_t ld;
    float* sums;             // kDx in several pieces: the float32 sums so far, rows x cols
    int32_t first, last;     // kDx: the first and last piece
};
struct Work {
    Job job[2];
    int32_t jobs;
    // rows of the logits
    const void* targets;
    int32_t wide, V;
    int64_t v0;              // first row of the weight of this piece
    const float* lse;
    const float* dloss;
    const float* dlse;
    float2* stats;           // kStats: [column half tile][row], rows padded
    int64_t stats_ld;
    float* target_logit;
};

// Shared-memory matrix descriptors, 128-byte swizzle: see linear_fp8.cu (K-major) and ckpt_wgrad.cu (MN-major).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn ? kBoxBytes >> 4 : 1) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D in f32 (bits 4-5 = 1), A and B bf16 (bits 7-9 and 10-12 = 1), MN-major operands (bits 15, 16), N / 8 in bits 17-22,
// M / 16 in bits 24-28 (M = 256 over the two CTAs).
template <int BN>
__device__ __forceinline__ uint32_t instr_desc(const Job& j) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)j.a_mn << 15) | ((uint32_t)j.b_mn << 16) | ((uint32_t)(BN >> 3) << 17) |
           ((uint32_t)((2 * kBM) >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Tile order: bands of kBand tiles of rows, column-major inside a band, so that the pairs that run at once share a band of
// A and walk B together.
constexpr int64_t kBand = 16;
struct Item {
    int32_t job;
    int64_t m, n;
};
__device__ __forceinline__ Item item_at(int64_t t, const Work& w) {
    Item it;
    const int64_t first = w.job[0].tm * w.job[0].tn;
    it.job = t >= first;
    if (it.job) t -= first;
    const int64_t tm = w.job[it.job].tm, tn = w.job[it.job].tn;
    const int64_t band = t / (kBand * tn), top = band * kBand;
    const int64_t rows = tm - top < kBand ? tm - top : kBand;
    const int64_t r = t - band * kBand * tn;
    it.m = top + r % rows;
    it.n = r / rows;
    return it;
}

// ---- epilogues: one row of the tile, BN / 2 columns from n0, per thread ----
template <int BN>
__device__ __forceinline__ void stats_of_row(const Work& w, const Job& j, uint32_t taddr, int64_t row, int64_t n0, int64_t part) {
    float top = -INFINITY, sum = 0.0f;
    const int64_t target = row < j.rows ? index_at(w.targets, w.wide, row) : -1;
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += kChunk) {
        const int64_t col = n0 + c;
        if (col >= j.cols) break;   // the same for the whole warp
        uint32_t v[kChunk];
        __syncwarp();   // tcgen05.ld is warp-collective
        tmem_ld<kChunk>(taddr + (uint32_t)c, v);
        if (col + kChunk > j.cols) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (col + e >= j.cols) v[e] = 0xFF800000u;   // -inf: not a column
        }
        const bool has = target >= col && target < col + kChunk;
        if (__any_sync(kFull, has)) {
            float z = 0.0f;
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (col + e == target) z = __uint_as_float(v[e]);
            if (has && target < j.cols) w.target_logit[row] = z;
        }
        float mx = top;
#pragma unroll
        for (int e = 0; e < kChunk; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
        const float ref = mx == -INFINITY ? 0.0f : mx;   // a row of -inf so far
        sum *= ex2_ftz((top - ref) * kLog2e);
        top = mx;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < kChunk; ++e) s[e & 3] += ex2_ftz((__uint_as_float(v[e]) - ref) * kLog2e);
        sum += (s[0] + s[1]) + (s[2] + s[3]);
    }
    if (row < j.rows && n0 < j.cols) w.stats[part * w.stats_ld + row] = make_float2(top, sum);
}

// 32 bf16 columns of a row; n of them (a multiple of 16) are there
__device__ __forceinline__ void store_row(uint16_t* p, int64_t n, bool wide, const uint32_t (&o)[kChunk / 2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (16 * h >= n) return;
        const uint32_t w8[8] = {o[8 * h], o[8 * h + 1], o[8 * h + 2], o[8 * h + 3], o[8 * h + 4], o[8 * h + 5], o[8 * h + 6], o[8 * h + 7]};
        store_words8(p + 16 * h, wide, w8);
    }
}

template <int BN>
__device__ __forceinline__ void dz_of_row(const Work& w, const Job& j, uint32_t taddr, int64_t row, int64_t n0, bool wide) {
    const bool ok = row < j.rows;
    float lse = 0.0f, g = 0.0f, p = 0.0f;   // dz = p e^(z - lse) - [v = t] g
    int64_t target = -1;
    if (ok) {
        target = index_at(w.targets, w.wide, row);
        lse = static_cast<const volatile float*>(w.lse)[row];
        if (target >= 0) g = target < w.V ? static_cast<const volatile float*>(w.dloss)[row] : NAN;
        p = w.dlse ? g + static_cast<const volatile float*>(w.dlse)[row] : g;
    }
    target -= w.v0;
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += kChunk) {
        const int64_t col = n0 + c;
        if (col >= j.cols) break;
        uint32_t v[kChunk], o[kChunk / 2];
        __syncwarp();
        tmem_ld<kChunk>(taddr + (uint32_t)c, v);
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[e] = __float_as_uint(p * ex2_ftz((__uint_as_float(v[e]) - lse) * kLog2e));
        if (__any_sync(kFull, target >= col && target < col + kChunk)) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (col + e == target) v[e] = __float_as_uint(__uint_as_float(v[e]) - g);
        }
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) o[e / 2] = bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        // the buffer's rows are whole tiles, and what lies behind the piece's columns is not read
        if (ok) store_row(j.out + row * j.ld + col, kChunk, wide, o);
    }
}

template <int BN>
__device__ __forceinline__ void sums_of_row(const Job& j, uint32_t taddr, int64_t row, int64_t n0, bool wide) {
    const bool ok = row < j.rows;
#pragma unroll 1
    for (int c = 0; c < BN / 2; c += kChunk) {
        const int64_t col = n0 + c, left = j.cols - col;
        if (left <= 0) break;
        uint32_t v[kChunk];
        __syncwarp();   // tcgen05.ld is warp-collective
        tmem_ld<kChunk>(taddr + (uint32_t)c, v);
        if (!ok) continue;
        if (j.sums) {
            float4* p = reinterpret_cast<float4*>(j.sums + row * j.cols + col);
            if (!j.first) {
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q) {
                    if (4 * q >= left) break;
                    const float4 f = p[q];
                    v[4 * q] = __float_as_uint(__uint_as_float(v[4 * q]) + f.x);
                    v[4 * q + 1] = __float_as_uint(__uint_as_float(v[4 * q + 1]) + f.y);
                    v[4 * q + 2] = __float_as_uint(__uint_as_float(v[4 * q + 2]) + f.z);
                    v[4 * q + 3] = __float_as_uint(__uint_as_float(v[4 * q + 3]) + f.w);
                }
            }
            if (!j.last) {
#pragma unroll
                for (int q = 0; q < kChunk / 4; ++q)
                    if (4 * q < left)
                        p[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), __uint_as_float(v[4 * q + 2]),
                                           __uint_as_float(v[4 * q + 3]));
                continue;
            }
        }
        uint32_t o[kChunk / 2];
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) o[e / 2] = bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        store_row(j.out + row * j.ld + col, left, wide, o);
    }
}

// The maps: A and B of the two jobs.
struct Maps {
    CUtensorMap a[2], b[2];
};

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) lce_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Work w, const bool wide) {
    using S = Shape<BN>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // the same offset in both CTAs
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar0 = sb + S::kBarOff;
    auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(kStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kStages + 2 + b); };
    const uint32_t done = bar0 + 8u * (uint32_t)(2 * kStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kBarOff + 8 * S::kNumBars);
    volatile uint32_t* abort = tmem_slot + 1;

    const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();   // 0: the CTA that issues the pair's MMAs
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int b = 0; b < 2; ++b) { mbar_init(acc_full(b), 1); mbar_init(acc_empty(b), 2 * kEpiWarps); }
        mbar_init(done, 1);
        *abort = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < w.jobs; ++i) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.a[i])) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.b[i])) : "memory");
        }
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(2 * BN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();   // barriers initialised and tensor memory allocated in both CTAs
    tc_fence_after();
    wait_for_primary();
    const uint32_t tmem = *tmem_slot;

    const int64_t items = w.job[0].tm * w.job[0].tn + (w.jobs > 1 ? w.job[1].tm * w.job[1].tn : 0);
    const int64_t cid = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (warp == 0 && lane == 0) {
        // ---- TMA producer (both CTAs): this CTA's 128 rows of A and BN / 2 columns of B ----
        int s = 0;
        uint32_t ph = 0, issued = 0, last_ph = 0;   // per stage: issued at all, parity of the last issue
        bool ok = true;
        const uint32_t fb0 = map_to_rank(full(0), 0);   // the leader's barriers, contiguous like ours
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, w);
            const Job& j = w.job[it.job];
            const CUtensorMap *ma = &maps.a[it.job], *mb = &maps.b[it.job];
            const int32_t m0 = (int32_t)(it.m * (2 * kBM) + rank * kBM), n0 = (int32_t)(it.n * BN + rank * (BN / 2));
            const int steps = j.steps;
            const bool a_mn = j.a_mn, b_mn = j.b_mn;
            for (int k = 0; k < steps; ++k) {
                if (!mbar_wait_fast(empty(s), ph ^ 1u, abort)) { ok = false; break; }
                if (leader) mbar_expect_tx(full(s), (uint32_t)(2 * S::kStageBytes));   // the bytes of both CTAs
                const uint32_t fb = fb0 + 8u * (uint32_t)s, sa = sb + (uint32_t)(s * S::kStageBytes), sbb = sa + kABytes;
                const int32_t k0 = k * kBK;
                if (a_mn) {
                    tma_load_2d_pair(sa, ma, m0, k0, fb);
                    tma_load_2d_pair(sa + kBoxBytes, ma, m0 + 64, k0, fb);
                } else {
                    tma_load_2d_pair(sa, ma, k0, m0, fb);
                }
                if (b_mn) {
#pragma unroll
                    for (int q = 0; q < BN / 128; ++q) tma_load_2d_pair(sbb + (uint32_t)(q * kBoxBytes), mb, n0 + 64 * q, k0, fb);
                } else {
                    tma_load_2d_pair(sbb, mb, k0, n0, fb);
                }
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
            // ---- MMA issuer (even CTA) ----
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int64_t i = cid; ok && i < items; i += nclusters) {
                const Job& j = w.job[item_at(i, w).job];
                const uint32_t idesc = instr_desc<BN>(j);
                const uint64_t adesc0 = smem_desc(sb, j.a_mn), bdesc0 = smem_desc(sb + kABytes, j.b_mn);
                // 16 of the summed index: 32 bytes along a row, or 16 rows of 128 bytes
                const uint64_t ka = j.a_mn ? (kMmaK * 128) >> 4 : (kMmaK * 2) >> 4, kb = j.b_mn ? (kMmaK * 128) >> 4 : (kMmaK * 2) >> 4;
                const int steps = j.steps;
                if (!mbar_wait_relaxed(acc_empty(acc), aph ^ 1u, abort)) break;   // see mbar_arrive_relaxed
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * BN);
                for (int k = 0; k < steps; ++k) {
                    if (!mbar_wait_fast(full(s), ph, abort)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)(s * (S::kStageBytes >> 4));
#pragma unroll
                    for (int kk = 0; kk < kBK / kMmaK; ++kk)
                        mma_bf16_pair(d, adesc0 + so + kk * ka, bdesc0 + so + kk * kb, idesc, (k | kk) != 0);
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
    } else if (warp >= 4) {
        // ---- epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31, columns BN / 2 ((w - 4) / 4) onwards ----
        const int q4 = warp & 3, half = (warp - 4) >> 2;
        int acc = 0;
        uint32_t aph = 0;
        for (int64_t i = cid; i < items; i += nclusters) {
            if (!__all_sync(kFull, mbar_wait_fast(acc_full(acc), aph, abort))) break;
            tc_fence_after();
            const Item it = item_at(i, w);
            const Job& j = w.job[it.job];
            const int64_t row = it.m * (2 * kBM) + rank * kBM + 32 * q4 + lane, n0 = it.n * BN + half * (BN / 2);
            const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(acc * BN + half * (BN / 2));
            if (j.mode == kStats)
                stats_of_row<BN>(w, j, taddr, row, n0, 2 * it.n + half);
            else if (j.mode == kDz)
                dz_of_row<BN>(w, j, taddr, row, n0, wide);
            else
                sums_of_row<BN>(j, taddr, row, n0, wide);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(map_to_rank(acc_empty(acc), 0));
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    }
    dependents_may_start();
    tc_fence_before();
    cluster_sync();   // no arrival or copy is still on its way to either CTA
    tc_fence_after();
    __syncwarp();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * BN) : "memory");
}

// loss and lse from the tiles' maxima and sums: 32 rows per block, a warp for every eighth part
__global__ void __launch_bounds__(256) lce_join_kernel(const float2* stats, int64_t ld, int64_t parts, const void* targets, int32_t wide,
                                                       int64_t M, int64_t V, float* loss, float* lse) {
    __shared__ float2 part[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 32 + lane;
    wait_for_primary();
    float top = -INFINITY, sum = 0.0f;
    auto join = [&](float2 f) {
        const float mx = fmaxf(top, f.x), ref = mx == -INFINITY ? 0.0f : mx;
        sum = sum * ex2_ftz((top - ref) * kLog2e) + f.y * ex2_ftz((f.x - ref) * kLog2e);
        top = mx;
    };
    if (row < M)
        for (int64_t p = warp; p < parts; p += 8) join(stats[p * ld + row]);
    part[warp][lane] = make_float2(top, sum);
    __syncthreads();
    if (warp != 0 || row >= M) return;
    for (int k = 1; k < 8; ++k) join(part[k][lane]);
    const float low = logf(sum);
    const int64_t t = index_at(targets, wide, row);
    lse[row] = top + low;
    // (top - z) + log(sum): nothing cancels where the target's logit is the largest
    loss[row] = t < 0 ? 0.0f : t >= V ? NAN : (top - loss[row]) + low;
}

// rows x cols bf16, row-major, ld elements apart; boxes of 64 columns x box_rows rows, zeros outside
bool encode(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    const EncodeTiled fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(2 * ld)};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t elem[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A matrix as an operand: along its rows or across them.  The box of a K-major one is all of a CTA's rows.
struct Operand {
    const uint16_t* p;
    int64_t rows, cols, ld;
    bool mn;
};
int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

template <int BN>
bool add_job(Work& w, Maps& maps, int32_t mode, const Operand& a, const Operand& b, uint16_t* out, int64_t ld) {
    Job& j = w.job[w.jobs];
    const int64_t K = a.mn ? a.rows : a.cols;
    j.mode = mode;
    j.a_mn = a.mn;
    j.b_mn = b.mn;
    j.rows = a.mn ? a.cols : a.rows;
    j.cols = b.mn ? b.cols : b.rows;
    j.steps = (int32_t)up(K, kBK);
    j.tm = up(j.rows, 2 * kBM);
    j.tn = up(j.cols, BN);
    j.out = out;
    j.ld = ld;
    j.sums = nullptr;
    j.first = j.last = 1;
    if (!encode(&maps.a[w.jobs], a.p, a.rows, a.cols, a.ld, a.mn ? kBK : kBM) ||
        !encode(&maps.b[w.jobs], b.p, b.rows, b.cols, b.ld, b.mn ? kBK : BN / 2))
        return false;
    ++w.jobs;
    return true;
}

template <int BN>
cudaError_t launch_work(const Work& w, const Maps& maps, bool wide, cudaStream_t s) {
    const int64_t pairs = device_sms() / 2;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(lce_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<BN>::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Shape<BN>::kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    int64_t items = 0;
    for (int i = 0; i < w.jobs; ++i) items += w.job[i].tm * w.job[i].tn;
    cfg.gridDim = dim3(2u * (unsigned)(items < pairs ? items : pairs));
    return cudaLaunchKernelEx(&cfg, lce_kernel<BN>, maps, w, wide);
}

template <int BN>
cudaError_t forward(const LceFwdArgs& a, cudaStream_t s) {
    Work w = {};
    alignas(64) Maps maps;
    if (!add_job<BN>(w, maps, kStats, Operand{a.x, a.M, a.C, a.x_ld, false}, Operand{a.weight, a.V, a.C, a.C, false}, nullptr, 0))
        return cudaErrorInvalidValue;
    w.targets = a.targets;
    w.wide = a.wide;
    w.V = (int32_t)a.V;
    w.stats = reinterpret_cast<float2*>(a.stats);
    w.stats_ld = up(a.M, 32) * 32;
    w.target_logit = a.loss;
    cudaError_t e = launch_work<BN>(w, maps, true, s);
    if (e != cudaSuccess) return e;
    return launch_next(lce_join_kernel, (unsigned)up(a.M, 32), 256, 0, s, (const float2*)w.stats, w.stats_ld, up(a.V, BN / 2),
                       a.targets, a.wide, a.M, a.V, a.loss, a.lse);
}

template <int BN>
cudaError_t backward(const LceBwdArgs& a, cudaStream_t s) {
    const bool wide = aligned32(a.dx) && aligned32(a.dweight);
    const int64_t ld = lce_piece_ld(a.piece, a.V);
    for (int64_t v0 = 0; v0 < a.V; v0 += a.piece) {
        const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
        const uint16_t* W = a.weight + v0 * a.C;
        Work w = {};
        alignas(64) Maps maps;
        if (!add_job<BN>(w, maps, kDz, Operand{a.x, a.M, a.C, a.x_ld, false}, Operand{W, n, a.C, a.C, false}, a.dz, ld))
            return cudaErrorInvalidValue;
        w.targets = a.targets;
        w.wide = a.wide;
        w.V = (int32_t)a.V;
        w.v0 = v0;
        w.lse = a.lse;
        w.dloss = a.dloss;
        w.dlse = a.dlse;
        cudaError_t e = launch_work<BN>(w, maps, aligned32(a.dz), s);
        if (e != cudaSuccess) return e;
        w.jobs = 0;
        if (!add_job<BN>(w, maps, kDw, Operand{a.dz, a.M, n, ld, true}, Operand{a.x, a.M, a.C, a.x_ld, true}, a.dweight + v0 * a.C, a.C) ||
            !add_job<BN>(w, maps, kDx, Operand{a.dz, a.M, n, ld, false}, Operand{W, n, a.C, a.C, true}, a.dx, a.C))
            return cudaErrorInvalidValue;
        w.job[1].sums = a.piece < a.V ? a.sums : nullptr;
        w.job[1].first = v0 == 0;
        w.job[1].last = v0 + n == a.V;
        e = launch_work<BN>(w, maps, wide, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

int64_t lce_piece(int64_t M, int64_t V, int64_t piece) {
    if (piece < 1) {   // as few pieces, of about the same width, as leave dz within kLceDzBytes
        int64_t most = kLceDzBytes / (2 * M) / 256 * 256;
        if (most < 256) most = 256;
        piece = up(V, up(V, most));
    }
    return piece < V ? up(piece, 256) * 256 < V ? up(piece, 256) * 256 : V : V;
}
int64_t lce_piece_ld(int64_t piece, int64_t V) { return up(piece < V ? piece : V, 256) * 256; }
size_t lce_stats_bytes(int64_t M, int64_t V) { return 8 * (size_t)(up(M, 32) * 32) * (size_t)up(V, 64); }

cudaError_t launch_lce_fwd(const LceFwdArgs& a, cudaStream_t s) { return forward<256>(a, s); }
cudaError_t launch_lce_bwd(const LceBwdArgs& a, cudaStream_t s) { return backward<256>(a, s); }

cudaError_t read_lce_wait_timeouts(unsigned long long* out, bool reset) { return read_own_wait_timeouts(out, reset); }

}  // namespace coat
