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
// it cannot be taken out of the sum: X is formed on the way as a bf16 operand,
// RN((S r) E4M3(q)), one rounding of a relative 2^-8 at most (dY is bf16
// already), and the products are summed in float32 by the tensor cores.
//
// Persistent CTA pairs (clusters of two, one CTA per SM) walk 256 x 256 tiles of
// dW, 64 tokens per step, and compute dW^T: M = 256 columns k (128 per CTA),
// N = 256 rows n.  X is the MMA's first operand and lies in TENSOR memory, dY the
// second one in shared memory as it comes ("MN-major": the output index along the
// row; nothing is transposed).  Per step:
//   TMA warp        dY (64 tokens x this CTA's 128 rows n, two 128-byte-swizzled
//                   boxes; both CTAs' bytes counted on the even CTA's barrier)
//                   and the codes (64 tokens x this CTA's 128 columns k);
//   scale warp      S of the 64 tokens and the columns' groups, and r (cp.async);
//   8 warps         codes -> X: a 16 x 16 block of codes is read transposed
//                   (ldmatrix .b8), so that a thread has four tokens of one
//                   column, and goes to tensor memory as 16 lanes x 16 bf16;
//   MMA warp        (even CTA) four tcgen05.mma.cta_group::2 kind::f16, K = 16;
//   8 warps         the finished accumulator into registers, times c, to bf16, stored.
// X in tensor memory is what makes the tensor cores the bound: with X written to
// and read from shared memory its traffic (copies in, codes out, X in, both
// operands out: 5 KB for each of the 128 B per clock that 512 clocks of MMA
// leave) held the 8192 x 11008 x 4096 product at 0.54 ms.  The price is half of
// tensor memory, so there is one accumulator, and the MMAs of a tile wait until
// the last one's is read.
//
// Measured (8192 tokens, G = 128): N x K = 11008 x 4096 0.41 to 0.44 ms alone (1.68 to 1.79 PFLOP/s) and 0.48 to 0.51 ms when
// repeated for seconds, where the GPU stands at its power limit; 4096 x 4096
// 0.157 ms, 2048 x 2048 0.046 ms; the smallest calls 8 us (launch, tensor
// memory, first tiles, join).  11008 x 4096 at G = 16 0.46 ms, at G = 8 0.63 ms.
//
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
constexpr int kHalf = kTile / 2;               // a CTA's columns k of it, and its rows n of dY
constexpr int kTok = 64;                       // tokens per stage
constexpr int kMmaTok = 16;                    // tokens of one kind::f16 MMA
constexpr int kBoxBytes = kTok * 128;          // 64 tokens x 64 bf16 columns
constexpr int kYBytes = 2 * kBoxBytes;         // dY: 64 tokens x 128 columns
constexpr int kQBytes = kTok * kHalf;          // the codes
constexpr int kStageBytes = kYBytes + kQBytes;
constexpr int kEpiWarps = 8;                   // two per SM sub-partition, each half the rows n
constexpr int kEpiRows = kTile / (kEpiWarps / 4);
constexpr int kDeqWarps = 8;
constexpr int kFirstEpi = 3;                    // TMA, MMA and tensor-memory warp; then the epilogue, then the conversion
constexpr int kFirstDeq = kFirstEpi + kEpiWarps;
constexpr int kWgThreads = 32 * (kFirstDeq + kDeqWarps);
constexpr uint32_t kXCols = kTok / 2;          // tensor-memory columns of a stage of X
constexpr uint32_t kTmemCols = 512;            // the accumulator (256) and the stages of X
constexpr int kMinSteps = 8;                   // fewest steps of a split's part
// By group size: stages (the scales of G = 8 leave room for seven), floats between two groups' scales (four more than
// the tokens, so that lanes that write 32 / groups tokens of every group meet different banks), and what follows.
constexpr int stages(int G) { return G == 8 ? 7 : 8; }
constexpr int scale_pitch(int G) { return G == kHalf ? kTok : kTok + 4; }
constexpr int scale_bytes(int G) { return ((kHalf / G) * scale_pitch(G) + kTok) * 4; }   // of a stage, with the tokens' factors
constexpr int num_bars(int G) { return 4 * stages(G) + 3; }   // dY full, codes full, X full, empty; acc full, acc empty, done
constexpr int bar_off(int G) { return stages(G) * (kStageBytes + scale_bytes(G)); }
constexpr int smem_bytes(int G) { return bar_off(G) + 8 * num_bars(G) + 16 + 1024; }   // + slack for 1024-B alignment
static_assert(kTile + stages(128) * kXCols <= kTmemCols && smem_bytes(8) <= 232448 && smem_bytes(16) <= 232448, "SM");

// Instruction descriptor: D in f32 (bits 4-5 = 1), A and B bf16 (bits 7-9 and
// 10-12 = 1), A as tensor memory holds it, B MN-major (bit 16), N / 8 in bits
// 17-22, M / 16 in bits 24-28 (M = 256 over the two CTAs).
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(kTile >> 3) << 17) |
                            ((uint32_t)(kTile >> 4) << 24);

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
// a_tmem: lane = row of A, K consecutive bf16 values, two per column
__device__ __forceinline__ void mma_bf16_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(kIdesc), "r"(accumulate)
        : "memory");
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

__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p;
}

// whether the phase is over, without a wait (a try may hold the warp until its phase ends)
template <bool kRelaxed = false>
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (kRelaxed)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0u;
}

// Two 16 x 16 blocks of bytes, transposed: lane's address = row `lane` of the two
// blocks (16 bytes each); r[2 b + h] = bytes 4 (lane % 4) .. + 3 of the
// transposed block b's row lane / 4 + 8 h.
__device__ __forceinline__ void ldmatrix_bytes(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// 16 lanes x 16 columns: registers 4 b + 2 h + i of a thread are columns
// 8 b + 2 (lane % 4) + i of tensor-memory lane taddr's + lane / 4 + 8 h.
__device__ __forceinline__ void tmem_st_16x256x2(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// Four codes as bf16(value * s), two to a register; s: the scales as two pairs
__device__ __forceinline__ void deq4(uint32_t codes, const ulonglong2& s, uint32_t& r0, uint32_t& r1) {
    uint32_t h0, h1;
    float x0, x1, x2, x3;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"((unsigned short)(codes & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"((unsigned short)(codes >> 16)));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x0), "=f"(x1)
        : "r"(h0));
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(x2), "=f"(x3)
        : "r"(h1));
    upk(mul2(pk(x0, x1), s.x), x0, x1);
    upk(mul2(pk(x2, x3), s.y), x2, x3);
    r0 = bf16x2(x0, x1);
    r1 = bf16x2(x2, x3);
}
__device__ __forceinline__ ulonglong2 lds128(uint32_t a) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(a));
    return v;
}
// 4 bytes global -> shared, asynchronously; zero where `in` is not set
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// one arrival on `bar` once every cp.async that this thread issued before has landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

template <int G>
__global__ void __launch_bounds__(kWgThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap tmy, const __grid_constant__ CUtensorMap tmq, const WgradArgs a,
             const Plan plan) {
    constexpr int kStages = stages(G);
    constexpr int kGroups = kHalf / G;             // scale groups of this CTA's columns
    constexpr int kPitch = scale_pitch(G);
    constexpr uint32_t kFactors = 4u * kGroups * kPitch;   // the tokens' factors, behind the scales
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // the same offset in both CTAs
    const uint32_t sb = smem_u32(smem);
    const uint32_t scales0 = sb + kStages * kStageBytes;   // per stage [group][token]
    const uint32_t bar0 = sb + bar_off(G);
    auto bar = [&](int kind, int s) { return bar0 + 8u * (uint32_t)(kind * kStages + s); };
    auto y_full = [&](int s) { return bar(0, s); };
    auto q_full = [&](int s) { return bar(1, s); };
    auto x_full = [&](int s) { return bar(2, s); };
    auto empty = [&](int s) { return bar(3, s); };
    const uint32_t acc_full = bar0 + 8u * (uint32_t)(4 * kStages);
    const uint32_t acc_empty = acc_full + 8u, done = acc_full + 16u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + bar_off(G) + 8 * num_bars(G));
    volatile uint32_t* abort = tmem_slot + 1;

    const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();   // 0: the CTA that issues the pair's MMAs
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(y_full(s), 1);
            mbar_init(q_full(s), 1 + 32);          // the codes' copy, and every lane's scales
            mbar_init(x_full(s), 2 * kDeqWarps);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 2 * kEpiWarps);
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
    wait_for_primary();
    const uint32_t tmem = *tmem_slot, xmem = tmem + (uint32_t)kTile;

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
                tma_load_2d(sa + kYBytes, &tmq, k0, st * kTok, q_full(s));
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
    } else if (warp == 1) {
        if (leader) {
            // ---- MMA issuer: the whole warp walks, so that addresses and descriptors stay in uniform registers, and one
            // elected lane issues.  The tensor cores queue only a few MMAs, so what lies between two steps' MMAs has to
            // be short: the next stage's barriers are asked before this one's MMAs are issued, and the answers come
            // while they run.  (4096 x 4096, 8192 tokens: 181 us with one thread that waits, issues and turns, and two
            // scale warps that read into registers; 167 us so.) ----
            int s = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            const uint32_t elected = elect_one();
            const uint64_t ydesc0 = mn_desc(sb);
            bool ready = false;
            for (int64_t i = cid; ok && i < items; i += nclusters, aph ^= 1u) {
                const Item it = item_at(i, plan);
                ok = __all_sync(kFull, mbar_wait_relaxed(acc_empty, aph ^ 1u, abort));
                if (!ok) break;
                tc_fence_after();
                for (int32_t st = it.from; st < it.to; ++st) {
                    if (!ready) {
                        ok = __all_sync(kFull, mbar_wait_fast(y_full(s), ph, abort) && mbar_wait_relaxed(x_full(s), ph, abort));
                        if (!ok) break;
                    }
                    tc_fence_after();
                    const uint64_t yd = ydesc0 + (uint64_t)(s * (kStageBytes >> 4));
                    const uint32_t xd = xmem + (uint32_t)s * kXCols, freed = empty(s);
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                    const bool y_in = mbar_test(y_full(s), ph), x_in = mbar_test<true>(x_full(s), ph);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < kTok / kMmaTok; ++kk)
                            mma_bf16_pair(tmem, xd + (uint32_t)(kk * (kMmaTok / 2)), yd + (uint64_t)(kk * ((kMmaTok * 128) >> 4)),
                                          st != it.from || kk != 0);
                        mma_commit_pair(freed, 0x3);   // both CTAs' stage is free once read
                        if (st + 1 == it.to) mma_commit_pair(acc_full, 0x3);
                    }
                    ready = __all_sync(kFull, y_in && x_in);
                }
            }
            if (elected) mma_commit_pair(done, 0x3);   // every MMA issued has completed before either CTA frees tensor memory
        }
        if (lane == 0) mbar_wait(done, 0u, nullptr);
        __syncwarp();
    } else if (warp == 2) {
        // ---- scales: a lane has one group of every 32 / groups-th token, so that an access reads the groups of a token
        // together; and two tokens' factors ----
        constexpr int kVals = 2 * kGroups, kRows = 32 / kGroups;   // scales per lane; tokens between two of them
        const int64_t ngr = a.K / G, step = kRows * ngr;
        const int grp = lane % kGroups, tok = lane / kGroups;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            const int64_t g = (it.k * kTile + rank * kHalf) / G + grp;
            const bool in = g < ngr;
            const float* p0 = a.scale + ((int64_t)it.from * kTok + tok) * ngr + (in ? g : 0);
            for (int32_t st = it.from; st < it.to; ++st, p0 += kTok * ngr) {
                ok = __all_sync(kFull, mbar_wait_fast(empty(s), ph ^ 1u, abort));
                if (!ok) break;
                const uint32_t d = scales0 + (uint32_t)(s * scale_bytes(G));
                const int64_t m0 = (int64_t)st * kTok;
                const int rest = a.M - m0 < kTok ? (int)(a.M - m0) : kTok;   // tokens of this step
                const float* p = p0;
#pragma unroll
                for (int v = 0; v < kVals; ++v, p += step) {
                    const bool here = in && tok + v * kRows < rest;
                    cp_async4(d + (uint32_t)(4 * (grp * kPitch + tok + v * kRows)), here ? p : a.scale, here);
                }
                if (a.row_scale) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool here = lane + 32 * h < rest;
                        cp_async4(d + kFactors + 4u * (uint32_t)(lane + 32 * h), a.row_scale + (here ? m0 + lane + 32 * h : 0), here);
                    }
                }
                cp_async_arrive(q_full(s));
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= kFirstEpi && warp < kFirstDeq) {
        // ---- epilogue: lane = one column k of the tile; tensor-memory columns = rows n ----
        const int q4 = warp & 3, nh = ((warp - kFirstEpi) >> 2) * kEpiRows;
        const uint32_t ae = map_to_rank(acc_empty, 0);
        auto release = [&]() {                     // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(ae);
        };
        uint32_t aph = 0;
        for (int64_t i = cid; i < items; i += nclusters, aph ^= 1u) {
            const Item it = item_at(i, plan);
            // the column's factor on its way: it is read when the MMAs have ended, between them and the next tile's (in a
            // register it would be one too many: 112 bytes of this kernel's registers then lie in local memory, and
            // every call takes 3 us longer)
            if (a.col_scale) {
                const int64_t kp = it.k * kTile + (int64_t)rank * kHalf + 32 * q4 + lane;
                if (kp < a.K) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.col_scale + kp));
            }
            if (!__all_sync(kFull, mbar_wait_fast(acc_full, aph, abort))) break;
            tc_fence_after();
            const int kl = (int)rank * kHalf + 32 * q4 + lane;
            const int64_t k = it.k * kTile + kl, n0 = it.n * kTile + nh;
            const uint32_t taddr = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)nh;
            if (it.part >= 0) {
                // the parts' tiles are [n][k]
                float* p = a.partial + (it.part * kTile + nh) * kTile + kl;
#pragma unroll 1
                for (int c = 0; c < kEpiRows; c += 32) {
                    if (n0 + c >= a.N) break;   // the same for the whole warp
                    uint32_t v[32];
                    tmem_ld<32>(taddr + (uint32_t)c, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) p[(c + e) * kTile] = __uint_as_float(v[e]);
                }
                release();
            } else {
                // all of it into registers, as pairs of rows, so that the next tile's MMAs may start; 8 columns at a
                // time, which leaves nothing in local memory (16: 0.3 us more per call)
                const float cs = a.col_scale && k < a.K ? a.col_scale[k] : 1.0f;
                uint32_t w[kEpiRows / 2];
#pragma unroll
                for (int c = 0; c < kEpiRows; c += 8) {
                    uint32_t v[8];
                    tmem_ld<8>(taddr + (uint32_t)c, v);
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        w[(c + e) / 2] = bf16x2(__uint_as_float(v[e]) * cs, __uint_as_float(v[e + 1]) * cs);
                }
                release();
                // two lanes exchange, so that each has two neighbours k of one row: the even lane of row n + e, the
                // odd one of row n + e + 1
                const int odd = lane & 1;
                uint16_t* p = a.dw + (n0 + odd) * a.K + (k - odd);
                const int rows = k < a.K ? (int)(a.N - n0 - odd < kEpiRows ? a.N - n0 - odd : kEpiRows) : 0;
#pragma unroll
                for (int e = 0; e < kEpiRows; e += 2) {
                    const uint32_t got = __shfl_xor_sync(kFull, w[e / 2], 1);
                    const uint32_t out = odd ? __byte_perm(got, w[e / 2], 0x7632) : __byte_perm(w[e / 2], got, 0x5410);
                    if (e < rows) *reinterpret_cast<uint32_t*>(p + (int64_t)e * a.K) = out;
                }
            }
        }
    } else if (warp >= kFirstDeq) {
        // ---- codes -> X: a warp takes the 32 columns k of its tensor-memory lanes, and 32 of the 64 tokens ----
        const int q4 = warp & 3, th = (warp - kFirstDeq) >> 2;
        const uint32_t xb0 = map_to_rank(x_full(0), 0);
        const int row = 32 * th + lane;                            // token of this lane's ldmatrix address
        uint32_t q_at[2];                                          // 16-byte unit of the row, as the 128-byte swizzle puts it
#pragma unroll
        for (int kh = 0; kh < 2; ++kh)
            q_at[kh] = (uint32_t)(kYBytes + row * 128 + (((2 * q4 + kh) ^ (row & 7)) * 16));
        const uint32_t s_at = (uint32_t)(4 * (32 * th + 4 * (lane & 3)));
        const uint32_t x_at = xmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(16 * th);
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t i = cid; ok && i < items; i += nclusters) {
            const Item it = item_at(i, plan);
            for (int32_t st = it.from; st < it.to; ++st) {
                if (!__all_sync(kFull, mbar_wait_fast(q_full(s), ph, abort))) { ok = false; break; }
                const uint32_t sa = sb + (uint32_t)(s * kStageBytes), ss = scales0 + (uint32_t)(s * scale_bytes(G)) + s_at;
                uint32_t q[2][4];
                ldmatrix_bytes(sa + q_at[0], q[0]);
                ldmatrix_bytes(sa + q_at[1], q[1]);
                // the scales of its tokens (four of each block) for the groups of its 32 columns: one, two or four
                constexpr int kSets = G >= 32 ? 1 : 32 / G;
                ulonglong2 f[kSets][2];
#pragma unroll
                for (int j = 0; j < kSets; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) f[j][b] = lds128(ss + (uint32_t)(4 * ((32 * q4 / G + j) * kPitch + 16 * b)));
                if (a.row_scale) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const ulonglong2 r = lds128(ss + kFactors + (uint32_t)(64 * b));
#pragma unroll
                        for (int j = 0; j < kSets; ++j) f[j][b] = make_ulonglong2(mul2(f[j][b].x, r.x), mul2(f[j][b].y, r.y));
                    }
                }
#pragma unroll
                for (int kh = 0; kh < 2; ++kh) {
                    uint32_t x[8];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            deq4(q[kh][2 * b + h], f[(16 * kh + 8 * h) * kSets / 32][b], x[4 * b + 2 * h], x[4 * b + 2 * h + 1]);
                    tmem_st_16x256x2(x_at + (uint32_t)s * kXCols + ((uint32_t)(16 * kh) << 16), x);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(xb0 + 8u * (uint32_t)s);
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
    }
    dependents_may_start();
    tc_fence_before();
    cluster_sync();   // no arrival or copy is still on its way to either CTA
    tc_fence_after();
    __syncwarp();
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
    wait_for_primary();
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < plan.parts; ++p) {
        const float4* src = reinterpret_cast<const float4*>(a.partial + ((j * plan.parts + p) * kTile + row) * kTile + c);
        const float4 f0 = src[0], f1 = src[1];
        x[0] += f0.x; x[1] += f0.y; x[2] += f0.z; x[3] += f0.w;
        x[4] += f1.x; x[5] += f1.y; x[6] += f1.z; x[7] += f1.w;
    }
    if (a.col_scale) {
        const float4 f0 = *reinterpret_cast<const float4*>(a.col_scale + k);
        const float4 f1 = reinterpret_cast<const float4*>(a.col_scale + k)[1];
        x[0] *= f0.x; x[1] *= f0.y; x[2] *= f0.z; x[3] *= f0.w;
        x[4] *= f1.x; x[5] *= f1.y; x[6] *= f1.z; x[7] *= f1.w;
    }
    uint32_t w[4];
    pack(x, w);
    *reinterpret_cast<uint4*>(a.dw + n * a.K + k) = make_uint4(w[0], w[1], w[2], w[3]);
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
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs: the plan (and with it the workspace and the order of the sums) goes by the SM count alone
int64_t pairs_of(int sms) { return sms / 2; }

template <int G>
cudaError_t launch_pairs(const WgradArgs& a, const Plan& p, int64_t pairs, cudaStream_t s) {
    alignas(64) CUtensorMap tmy, tmq;
    if (!encode(&tmy, a.dy, a.M, a.N, a.dy_ld, true) || !encode(&tmq, a.q, a.M, a.K, a.K, false)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(wgrad_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(G));
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWgThreads);
    cfg.dynamicSmemBytes = smem_bytes(G);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int64_t items = p.whole + p.tail * p.parts;
    cfg.gridDim = dim3(2u * (unsigned)(items < pairs ? items : pairs));
    return cudaLaunchKernelEx(&cfg, wgrad_kernel<G>, tmy, tmq, a, p);
}

}  // namespace

size_t wgrad_workspace(int64_t M, int64_t N, int64_t K, int sms) {
    const Plan p = make_plan(M, N, K, pairs_of(sms));
    return (size_t)(p.tail * p.parts) * (size_t)(kTile * kTile) * sizeof(float);
}

cudaError_t launch_wgrad(const WgradArgs& a, cudaStream_t s) {
    const int64_t pairs = pairs_of(device_sms());
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    const Plan p = make_plan(a.M, a.N, a.K, pairs);
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.G) {
        case 8: e = launch_pairs<8>(a, p, pairs, s); break;
        case 16: e = launch_pairs<16>(a, p, pairs, s); break;
        case 32: e = launch_pairs<32>(a, p, pairs, s); break;
        case 64: e = launch_pairs<64>(a, p, pairs, s); break;
        case 128: e = launch_pairs<128>(a, p, pairs, s); break;
    }
    if (e != cudaSuccess) return e;
    if (p.tail == 0) return cudaSuccess;
    return launch_next(wgrad_join_kernel, (unsigned)(p.tail * 32), 256, 0, s, a, p);
}

cudaError_t read_wgrad_wait_timeouts(unsigned long long* out, bool reset) { return read_own_wait_timeouts(out, reset); }

}  // namespace coat
