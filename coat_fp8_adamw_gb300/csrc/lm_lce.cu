// lm_lce.cu -- softmax cross entropy of a linear layer over a large vocabulary, and its gradient, without the logits
// being kept.
//
//   z = x W^T;  lse[m] = log sum_v e^z[m, v];  loss[m] = lse[m] - z[m, t[m]]
//   dz[m, v] = e^(z[m, v] - lse[m]) (g[m] + h[m]) - [v = t[m]] g[m];  dx = dz W;  dW = dz^T x
//
// Four matrix products of 2 M V C operations, one forward and three backward (z is formed again), on the tensor cores:
//   forward   a tile's logits stay in tensor memory; each of its rows leaves its maximum and sum of exponentials per
//             half a tile (and the target's logit), which a second kernel joins: loss and lse (of few tokens with the
//             largest and the target's logit formed by itself);
//   backward  in pieces of the vocabulary: a piece's logits again, whose epilogue leaves dz (bf16, in the workspace); then
//             dx (added up over the pieces in float32) and the piece's rows of dW in one launch.
// dz is rounded to bf16, since it is an operand of the tensor cores, like a layer's gradient that a step keeps as bf16.
//
// One kernel for all four: persistent CTA pairs (clusters of two, one CTA per SM) walk tiles of 256 rows x up to 256 columns,
// 64 of the summed index per stage, as in linear_fp8.cu: each CTA has its 128 rows of A and half of the columns of B in
// a ring of stages filled by TMA (128-byte swizzle), one thread of the even CTA issues tcgen05.mma.cta_group::2
// kind::f16, and eight epilogue warps per CTA read one of several accumulators in tensor memory while another one fills.
// B has its summed index along the row (K-major); A has it so too (x for z) or across the row (MN-major), which the MMA
// takes at the same rate (8192^3: 1.79 PFLOP/s both; with B MN-major 1.46).  So dx is formed as its transpose, of W
// (MN-major) and dz, and dW of dz (MN-major) and x's transpose, which a kernel lays out before.
// Every wait on an mbarrier is bounded, as in linear_fp8.cu.
#include <cstdint>

#include "ckpt_kernels.h"
#include "divide.h"
#include "lm_device.cuh"
#include "lm_kernels.h"
#include "tc_pipeline.cuh"

namespace coat {

namespace {

using namespace ckpt;
using lm::index_at;
using lm::load_index;

constexpr int kBM = 128;                       // rows per CTA (the pair's MMA has M = 256)
constexpr int kBK = 64;                        // of the summed index per stage: 128 bytes
constexpr int kMmaK = 16;
constexpr int kABytes = kBM * kBK * 2;         // 16 KB
constexpr int kBoxBytes = kBK * 128;           // MN-major: 64 of the summed index x 64 of the other one
constexpr int kEpiWarps = 8;                   // two per SM sub-partition, each half the columns
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kChunk = 32;                     // columns that an epilogue thread holds at once
constexpr int64_t kPairs = 76;                  // that the division of the work goes by, on every device
constexpr float kLog2e = 1.4426950408889634f;
// The tensor cores truncate when they add to an accumulator, so that a sum falls short by up to 2^-24 of its size at every
// addition.  Logits are therefore added up by them over 512 of the summed index at a time, and the epilogue adds those sums
// in its registers, with float32's rounding (lse of C = 4096: 4.6e-6 off in one go, 5.2e-7 so; the plain float32 form 8.6e-7).
constexpr int kSegment = 8;                    // steps
// of few tokens, whose time goes to the weight's bytes, 128 (33 x 50304 x 2048 forward in tiles of 256 rows, of 64 / 128 / 256 / 512: 50.4 / 43.6 / 42.5 / 42.3 us)
constexpr int kFewSegment = 2;
// Registers: the epilogue warps hold their logits, 128 a thread, and take what the other four warps give up.  Every one of
// 384 threads is launched with kLaunchRegs.
constexpr int kLaunchRegs = 168, kOtherRegs = 72, kEpiRegs = 216;
static_assert(128 * kOtherRegs + 256 * kEpiRegs <= 384 * kLaunchRegs, "setmaxnreg.inc would wait for ever");

constexpr int kBN = 256;                       // most columns of a tile
// Shared memory: the ring of stages (A's 16 KB and B's columns each, as many as fit), then 4 KB for every epilogue warp
// (which kFewStats uses as 32 rows of 33 floats), then the barriers.
constexpr int kStageArea = 6 * 32768;
constexpr int kMaxStages = 10;
constexpr int kMaxAccs = 4;
constexpr int kStagingBytes = 32 * 33 * 4;
constexpr int kBarOff = kStageArea + 8 * kStagingBytes;
constexpr int kNumBars = 2 * kMaxStages + 2 * kMaxAccs + 1;   // full, empty, acc full, acc empty, done
constexpr int kSmemBytes = kBarOff + 8 * kNumBars + 16 + 1024;   // + slack for 1024-B alignment
constexpr int slot_bytes(int bn) { return kABytes + bn / 2 * kBK * 2; }
constexpr int stages_of(int bn) { return kStageArea / slot_bytes(bn) < kMaxStages ? kStageArea / slot_bytes(bn) : kMaxStages; }
static_assert(kSmemBytes <= 232448 && stages_of(256) == 6 && stages_of(32) == 10, "shared memory of an SM");
// Up to so many tokens, the logits are formed with the tokens as the only tile's columns, so that the product has no rows
// without a token (50304 x 2048 forward, 1 / 33 / 100 tokens: 37 / 38 / 39 us, with the tokens as rows 62 / 46 / 46; with 200 / 256
// tokens 46 / 48 in segments of 512, as rows 46 / 47).
constexpr int64_t kFewTokens = 128;
constexpr int kFewChunks = (int)kFewTokens / 2 / kChunk;   // of an epilogue warp

// What a launch does with a tile's sums.
// Of few tokens, the logits' rows are those of the weight and their columns the tokens (kFewStats, kFewDz).
enum Mode : int32_t { kStats, kDz, kFewStats, kFewDz, kDx, kDw };
// The kernels: by what their epilogue warps hold.
enum Kind { kLogits, kFewLogits, kProducts };
constexpr Kind kind_of(int32_t mode) { return mode <= kDz ? kLogits : mode <= kFewDz ? kFewLogits : kProducts; }
// Accumulators in tensor memory, of at most 512 / accs_of columns each.  Few tokens leave room for four: segments are short, and
// while the epilogue works on a tile's logits the next one's are formed.
constexpr int accs_of(Kind kind) { return kind == kFewLogits ? 4 : 2; }
static_assert(kFewTokens <= 512 / accs_of(kFewLogits) && kBN <= 512 / accs_of(kLogits) && accs_of(kFewLogits) <= kMaxAccs, "tensor memory");

// A product: its tiles, each summed in `parts` parts of the summed index.
struct Job {
    int32_t mode;
    int32_t a_mn;            // A is MN-major
    int32_t steps;           // 64 of the summed index each
    int32_t segment;         // steps that the tensor cores add up by themselves
    int32_t bm;              // rows of a tile: 2 kBM, or, of few tokens, a multiple of 32 up to it
    int32_t bn;              // columns of a tile: a multiple of 32
    int32_t parts;
    int64_t tm, tn;          // tiles
    int64_t rows, cols;      // of the product
    uint16_t* out;           // kFewDz, kDx (last piece): bf16, rows ld apart (kDz and kDw store by their tensor map)
    int64_t ld;
    float* sums;             // [parts][out's shape] float32: of parts, or of the pieces so far
    Divider by_tiles, by_band, by_last, by_parts;   // tm tn; kBand tn; the last band's rows; parts
    int32_t first, last;     // sums: the first piece, which writes them; the last one of a product in one part, which ends in out
};
// The jobs of a launch, the one with the longer items first.  Of its items every pair has one in turn; `ahead` pairs have one
// more of them than the others, and those have `extra` items of the second job for it.  Everything else goes in turn again.
struct Work {
    Job job[2];
    int32_t jobs;
    int32_t slot, stages;    // bytes of a stage, and their number
    int32_t pairs, ahead;
    int64_t items[2], extra;
    Divider by_pairs, by_lot;   // pairs; those that are not ahead
    // rows of the logits
    const void* targets;
    int32_t wide, V;
    int64_t v0;              // first row of the weight of this piece
    const float* lse;
    const float* dloss;
    const float* dlse;
    const float* unit;       // backward: what dz is stored times, and its reciprocal (see unit_of)
    const float* share;      // backward, of few tokens: e^(z - lse) - 1 of the target's logit (see exact_parts), share_ld apart
    int64_t share_ld;
    float2* stats;           // {maximum, rest} (see kNoRest), [half of a tile's columns, or, of few tokens, CTA][token], tokens padded
    int64_t stats_ld;
    int32_t* tops;           // of few tokens: the maximum's row of the weight, likewise (-1: of no logits, or of -inf alone)
    float* target_logit;
};

// Shared-memory matrix descriptors, 128-byte swizzle: see linear_fp8.cu (K-major) and ckpt_wgrad.cu (MN-major).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(mn ? kBoxBytes >> 4 : 1) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// D in f32 (bits 4-5 = 1), A and B bf16 (bits 7-9 and 10-12 = 1), A MN-major (bit 15) or not, N / 8 in bits 17-22, M / 16 in
// bits 24-28 (M = 256 over the two CTAs).
__device__ __forceinline__ uint32_t instr_desc(const Job& j) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)j.a_mn << 15) | ((uint32_t)(j.bn >> 3) << 17) | ((uint32_t)((2 * kBM) >> 4) << 24);
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
constexpr uint32_t kBand = 16;
struct Item {
    int32_t job, part;
    int32_t from, to;        // steps
    int64_t m, n;            // tile
};
// A pair's way through the items: the first job's in turn, those that make up for one less of them, and the rest.  Every role
// reckons its own, so without a division (8192 x 32000 x 4096 with 64-bit divisions: 1500 clocks an item; 1000 x 100000 x 128 with
// 32-bit ones: 730).
struct Walk {
    uint32_t pair, own, behind, mine;
    __device__ __forceinline__ Walk(const Work& w, uint32_t p) {
        const uint32_t P = (uint32_t)w.pairs, ahead = (uint32_t)w.ahead;
        pair = p;
        own = divide((uint32_t)w.items[0] + P - 1u - p, w.by_pairs);   // of the first job
        behind = p - ahead;
        mine = p >= ahead && behind < (uint32_t)w.extra ? divide((uint32_t)w.extra - behind + P - ahead - 1u, w.by_lot) : 0u;
    }
    // the k-th item; false: there is none
    __device__ __forceinline__ bool item(uint32_t k, const Work& w, Item& it) const {
        const uint32_t P = (uint32_t)w.pairs;
        uint32_t t;
        it.job = k >= own;
        if (it.job == 0) {
            t = pair + k * P;
        } else {
            k -= own;
            t = k < mine ? behind + k * (P - (uint32_t)w.ahead) : (uint32_t)w.extra + (k - mine) * P + pair;
            if (t >= (uint32_t)w.items[1]) return false;
        }
        const Job& j = w.job[it.job];
        it.part = 0;
        it.from = 0;
        it.to = j.steps;
        if (j.parts > 1) {
            it.part = (int32_t)divide(t, j.by_tiles);
            t -= (uint32_t)it.part * j.by_tiles.d;
            it.from = (int32_t)divide((uint32_t)(j.steps * it.part), j.by_parts);   // (steps < 2^25, parts <= 32)
            it.to = (int32_t)divide((uint32_t)(j.steps * (it.part + 1)), j.by_parts);
        }
        const uint32_t band = divide(t, j.by_band), top = band * kBand, r = t - band * j.by_band.d;
        const bool whole = (uint32_t)j.tm - top >= kBand;
        const uint32_t rows = whole ? kBand : j.by_last.d, n = whole ? r / kBand : divide(r, j.by_last);
        it.m = top + (r - n * rows);
        it.n = n;
        return true;
    }
};

// ---- epilogues: one row of the tile, columns n0 .. end - 1 (at most 128, a multiple of 16 but for the matrix's end), per
// thread; where a chunk of 32 goes past them, it reads columns of the other half, which do not count ----
// What is needed of a token (a lane's row of the logits, or its column of 32), loaded while the tile's MMAs still run.
struct RowValues {
    int32_t target;          // -1: none; V: past the vocabulary
    float lse, g, p;         // dz = p e^(z - lse) - [v = target] g; of few tokens, g is the target's dz itself
};
__device__ __forceinline__ RowValues row_values(const Work& w, const Job& j, int64_t token, int64_t tokens, float unit) {
    RowValues r{-1, 0.0f, 0.0f, 0.0f};
    if (j.mode > kFewDz || token >= tokens) return r;
    const int64_t t = index_at(w.targets, w.wide, token);
    r.target = t < 0 ? -1 : t < w.V ? (int32_t)t : w.V;
    if (j.mode == kStats || j.mode == kFewStats) return r;
    const float g = static_cast<const volatile float*>(w.dloss)[token], h = w.dlse ? static_cast<const volatile float*>(w.dlse)[token] : 0.0f;
    r.lse = static_cast<const volatile float*>(w.lse)[token];
    r.g = r.target < 0 ? 0.0f : r.target < w.V ? g : NAN;
    r.p = (r.g + h) * unit;
    r.g *= unit;
    if (j.mode == kFewDz) {   // (g + h) e^(z - lse) - g, without a difference of e^(z - lse) and 1
        r.g = h * unit;
        if (r.target >= 0 && r.target < w.V && r.p != 0.0f)
            r.g = fmaf(r.p, static_cast<const volatile float*>(w.share)[token * w.share_ld], r.g);
    }
    return r;
}

// e^(z - ref) of two logits (the difference first: with one fused multiply-add of z log2(e) and ref's, the largest logit's
// share would be 1 to float32's last bits only, and so would the loss of a certain token)
__device__ __forceinline__ void exp2_of(uint32_t z0, uint32_t z1, uint64_t minus_ref, float& a, float& b) {
    upk(mul2(add2(pk(__uint_as_float(z0), __uint_as_float(z1)), minus_ref), pk(kLog2e, kLog2e)), a, b);
    a = ex2_ftz(a);
    b = ex2_ftz(b);
}

// The logits that an epilogue thread holds: four times 32 columns of its row, or, of few tokens, of which there are two times
// 32, a row of the weight's.  Columns 32 c .. + 31 begin at column off(c) of the tile: every second 64 columns, so that a
// store by TMA has 64 neighbours.
constexpr int kChunks = 4;
template <int kN>
struct Logits {
    uint32_t z[kN][kChunk];
};
__device__ __forceinline__ int chunk_off(int half, int c) { return 64 * half + 128 * (c >> 1) + kChunk * (c & 1); }
// one segment's sums of them; the chunks that have columns below `cols` of the tile, the same for the whole warp
template <bool kFirst, int kN>
__device__ __forceinline__ void add_segment(uint32_t acc0, int half, int bn, int cols, Logits<kN>& l) {
    constexpr int kLoad = kN == kFewChunks ? 32 : 16;   // columns: with 32 beside 128 logits, a thread's registers do not suffice
#pragma unroll
    for (int c = 0; c < kN; ++c) {
        const int off = kN == kFewChunks ? half * (bn / 2) + kChunk * c : chunk_off(half, c);
        if (off >= cols) continue;
        __syncwarp();   // tcgen05.ld is warp-collective
        if constexpr (kFirst) {
            tmem_ld<kChunk>(acc0 + (uint32_t)off, l.z[c]);
        } else {
#pragma unroll
            for (int h = 0; h < kChunk; h += kLoad) {
                uint32_t v[kLoad];
                tmem_ld<kLoad>(acc0 + (uint32_t)(off + h), v);
#pragma unroll
                for (int e = 0; e < kLoad; e += 2) {
                    float x, y;
                    upk(add2(pk(__uint_as_float(l.z[c][h + e]), __uint_as_float(l.z[c][h + e + 1])),
                             pk(__uint_as_float(v[e]), __uint_as_float(v[e + 1]))), x, y);
                    l.z[c][h + e] = __float_as_uint(x);
                    l.z[c][h + e + 1] = __float_as_uint(y);
                }
            }
        }
    }
}

// Of a sum of e^(z - top), with top the largest z, a float32 keeps the terms but the largest only in units of 2^-23 of it, and the
// loss of a certain token is the sum of those.  So what is kept of a sum is the rest: what it is beside the largest one's 1 (of
// no logits, or of -inf alone, -1).  Of many tokens, the 1 is summed with the up to 31 terms of its own chunk of columns and then
// taken off, so that those terms alone are still in units of 2^-23; of few, it is left out.
constexpr float kNoRest = -1.0f;
// joined with the rest of others
__device__ __forceinline__ void join_rest(float& top, float& rest, float top1, float rest1) {
    const float mx = fmaxf(top, top1), ref = mx == -INFINITY ? 0.0f : mx;
    const float f = ex2_ftz((fminf(top, top1) - ref) * kLog2e);
    rest = top1 > top ? rest1 + (1.0f + rest) * f : rest + (1.0f + rest1) * f;
    top = mx;
}
// joined with a sum of e^(z - mx) of more logits, mx the largest of all; before: e^(top - mx)
__device__ __forceinline__ void add_to_rest(float& top, float& rest, float mx, float before, float sum) {
    rest = mx > top ? (sum - 1.0f) + (1.0f + rest) * before : rest + sum;
    top = mx;
}

// Of a tile with all its columns, the largest of the chunks and the rest of the sum.  Maxima first, then exponentials, the chunks side
// by side and without a branch: with only two warps of a scheduler their chains of additions are what takes time (1000 x 100000 x
// 128: 47 us, chunk by chunk 52; other tiles, whose chunks may not be there, go chunk by chunk: 2048 x 512 x 1024 8.6 us, side by
// side 8.9).
__device__ __forceinline__ float2 stats_of_all(const Logits<kChunks>& l) {
    float most[kChunks];
    uint64_t sums[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        most[c] = -INFINITY;
        sums[c] = pk(0.0f, 0.0f);
    }
#pragma unroll
    for (int e = 0; e < kChunk; e += 2)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) most[c] = max3(most[c], __uint_as_float(l.z[c][e]), __uint_as_float(l.z[c][e + 1]));
    float top = most[0];
#pragma unroll
    for (int c = 1; c < kChunks; ++c) top = fmaxf(top, most[c]);
    const float ref = top == -INFINITY ? 0.0f : top;   // a row of -inf
#pragma unroll
    for (int e = 0; e < kChunk; e += 2)
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            float x, y;
            exp2_of(l.z[c][e], l.z[c][e + 1], pk(-ref, -ref), x, y);
            sums[c] = add2(sums[c], pk(x, y));
        }
    float rest = 0.0f;
    bool one = false;   // the largest one's 1 has been left out, of its chunk's sum
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const bool here = !one && most[c] == top;
        rest += here ? sum2(sums[c]) - 1.0f : sum2(sums[c]);
        one |= here;
    }
    return make_float2(top, rest);
}

// columns col0 .. end - 1 of the tile are logits
__device__ __forceinline__ void stats_of_row(const Work& w, const Job& j, const RowValues& r, Logits<kChunks>& l, int64_t row, int64_t col0, int64_t end,
                                             int half, int64_t part) {
    const int cols = (int)(end - col0), target = r.target - (int)col0;   // in the tile
    auto say_target = [&](int c, int off) {
        const bool has = target >= off && target < off + kChunk;
        if (!__any_sync(kFull, has)) return;
        float z = 0.0f;
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (off + e == target) z = __uint_as_float(l.z[c][e]);
        if (has && target < cols && row < j.rows) w.target_logit[row] = z;
    };
    float top = -INFINITY, rest = kNoRest;
    if (cols == kBN) {
        if (__any_sync(kFull, target >= 0 && target < kBN && (target >> 6 & 1) == half)) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) say_target(c, chunk_off(half, c));
        }
        const float2 f = stats_of_all(l);
        if (row < j.rows) w.stats[part * w.stats_ld + row] = f;
        return;
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int off = chunk_off(half, c);
        if (off >= cols) continue;
        uint32_t (&v)[kChunk] = l.z[c];
        if (off + kChunk > cols) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (off + e >= cols) v[e] = 0xFF800000u;   // -inf: not a column
        }
        say_target(c, off);
        float mx = top;
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) mx = max3(mx, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        const float ref = mx == -INFINITY ? 0.0f : mx;   // a row of -inf so far
        uint64_t sums = pk(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
            float x, y;
            exp2_of(v[e], v[e + 1], pk(-ref, -ref), x, y);
            sums = add2(sums, pk(x, y));
        }
        add_to_rest(top, rest, mx, ex2_ftz((top - ref) * kLog2e), sum2(sums));
    }
    if (row < j.rows) w.stats[part * w.stats_ld + row] = make_float2(top, rest);
}

// What an epilogue warp keeps of its few tokens from tile to tile: the lane's one of every 32.
struct FewTokens {
    RowValues r[kFewChunks];
    float top[kFewChunks], rest[kFewChunks];
    int32_t at[kFewChunks];          // top's row of the weight
};
__device__ __forceinline__ void few_tokens(const Work& w, const Job& j, int64_t n0, int64_t end, int lane, float unit, FewTokens& f) {
#pragma unroll
    for (int c = 0; c < kFewChunks; ++c) {
        f.r[c] = row_values(w, j, n0 + kChunk * c + lane, end, unit);
        f.top[c] = -INFINITY;
        f.rest[c] = kNoRest;
        f.at[c] = -1;
    }
}

// The statistics of few tokens: a warp has 32 rows of the weight and its tokens n0 .. end - 1, 32 of which at a time it turns
// over in shared memory, so that a lane has one token.
__device__ __forceinline__ void few_stats(const Work& w, const Logits<kFewChunks>& l, uint32_t buf, int64_t row0, int64_t rows, int lane, int64_t n0,
                                          int64_t end, FewTokens& f) {
    const bool in = row0 + lane < rows;
#pragma unroll
    for (int c = 0; c < kFewChunks; ++c) {
        if (n0 + kChunk * c >= end) break;   // the same for the whole warp
        __syncwarp();   // the chunk before has been read
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(buf + (uint32_t)(4 * (33 * lane + e))), "r"(in ? l.z[c][e] : 0xFF800000u) : "memory");
        __syncwarp();
        uint32_t v[kChunk];
        float mx = f.top[c];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[k]) : "r"(buf + (uint32_t)(4 * (33 * k + lane))));
            mx = fmaxf(mx, __uint_as_float(v[k]));
        }
        const int64_t token = n0 + kChunk * c + lane;
        const int at = f.r[c].target - (int)row0;
        if (at >= 0 && at < kChunk && f.r[c].target < rows && token < end) {
            float z;
            asm volatile("ld.shared.b32 %0, [%1];" : "=f"(z) : "r"(buf + (uint32_t)(4 * (33 * at + lane))));
            w.target_logit[token] = z;
        }
        const bool more = mx > f.top[c];   // seldom behind the first tiles
        int32_t at_k = -1;
        if (__any_sync(kFull, more)) {
#pragma unroll
            for (int k = 0; k < kChunk; ++k)
                if (more && __uint_as_float(v[k]) == mx) at_k = k;
            if (more) f.at[c] = (int32_t)row0 + at_k;
        }
        const float ref = mx == -INFINITY ? 0.0f : mx;
        uint64_t sums = pk(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kChunk; k += 2) {
            float x, y;
            exp2_of(k == at_k ? 0xFF800000u : v[k], k + 1 == at_k ? 0xFF800000u : v[k + 1], pk(-ref, -ref), x, y);
            sums = add2(sums, pk(x, y));
        }
        // the largest one's 1 is not in the sum, or, where an earlier chunk has it, its whole sum is beside that
        f.rest[c] = sum2(sums) + (more ? (1.0f + f.rest[c]) * ex2_ftz((f.top[c] - ref) * kLog2e) : f.rest[c]);
        f.top[c] = mx;
    }
}

// ---- stores of bf16 by TMA: 64 columns of a warp's 32 rows through its 4 KB of shared memory, 128-byte swizzle ----
__device__ __forceinline__ void staging_free(int lane) {   // the copy before has read its values
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}
// columns 32 h .. + 31 of the lane's row
__device__ __forceinline__ void stage_row(uint32_t buf, int lane, int h, const uint32_t (&o)[kChunk / 2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + (uint32_t)(128 * lane + (((4 * h + i) ^ (lane & 7)) << 4))),
                     "r"(o[4 * i]), "r"(o[4 * i + 1]), "r"(o[4 * i + 2]), "r"(o[4 * i + 3])
                     : "memory");
}
// (columns and rows that the tensor does not have are left out)
__device__ __forceinline__ void store_staged(const CUtensorMap* map, uint32_t buf, int64_t col, int64_t row0, int64_t rows, int lane) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0 && row0 < rows) {
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(reinterpret_cast<uint64_t>(map)),
                     "r"((int32_t)col), "r"((int32_t)row0), "r"(buf)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// kDz: boxes of 64 columns
__device__ __forceinline__ void dz_of_row(const Work& w, const Job& j, const RowValues& r, Logits<kChunks>& l, uint32_t buf, const CUtensorMap* map,
                                          int64_t row0, int64_t col0, int half, int lane) {
    const uint64_t minus_lse = pk(-r.lse, -r.lse), p2 = pk(r.p, r.p);
    const int target = r.target - (int)w.v0 - (int)col0;         // in the tile
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int off = chunk_off(half, c & ~1), at = chunk_off(half, c);   // of the box, and of its columns
        if (off >= j.bn || col0 + off >= j.cols) continue;      // the same for the whole warp
        if ((c & 1) == 0) staging_free(lane);
        uint32_t (&v)[kChunk] = l.z[c];
        uint32_t o[kChunk / 2];
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
            float x, y;
            exp2_of(v[e], v[e + 1], minus_lse, x, y);
            upk(mul2(pk(x, y), p2), x, y);
            v[e] = r.p == 0.0f ? 0u : __float_as_uint(x);   // without a gradient, whatever the logits are
            v[e + 1] = r.p == 0.0f ? 0u : __float_as_uint(y);
        }
        if (__any_sync(kFull, target >= at && target < at + kChunk)) {
#pragma unroll
            for (int e = 0; e < kChunk; ++e)
                if (at + e == target) v[e] = __float_as_uint(__uint_as_float(v[e]) - r.g);
        }
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) o[e / 2] = bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        stage_row(buf, lane, c & 1, o);
        if ((c & 1) == 1) store_staged(map, buf, col0 + off, row0, j.rows, lane);
    }
}

// kDw in one part: likewise
__device__ __forceinline__ void dw_of_row(const Job& j, uint32_t taddr, uint32_t buf, const CUtensorMap* map, int64_t row0, int64_t col0,
                                          int half, int lane, float unit) {
#pragma unroll 1
    for (int b = 64 * half; b < j.bn && col0 + b < j.cols; b += 128) {
        staging_free(lane);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[kChunk], o[kChunk / 2];
            tmem_ld<kChunk>(taddr + (uint32_t)(b + 32 * h), v);
#pragma unroll
            for (int e = 0; e < kChunk; e += 2) o[e / 2] = bf16x2(__uint_as_float(v[e]) * unit, __uint_as_float(v[e + 1]) * unit);
            stage_row(buf, lane, h, o);
        }
        store_staged(map, buf, col0 + b, row0, j.rows, lane);
    }
}

// 32 columns of the product, rows of `out`, whose columns `row` are the lanes' (the first `left` of them; 0: not a row):
// two lanes exchange, so that each has two neighbours of one of them: the even lane of column e, the odd one of e + 1
__device__ __forceinline__ void store_columns(uint16_t* out, int64_t ld, int64_t row, int64_t col, int64_t left, int lane,
                                              const uint32_t (&v)[kChunk]) {
    const int odd = lane & 1;
    uint16_t* p = out + (col + odd) * ld + (row - odd);
#pragma unroll
    for (int e = 0; e < kChunk; e += 2) {
        const uint32_t own = bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), got = __shfl_xor_sync(kFull, own, 1);
        const uint32_t x = odd ? __byte_perm(got, own, 0x7632) : __byte_perm(own, got, 0x5410);
        if (e + odd < left) *reinterpret_cast<uint32_t*>(p + e * ld) = x;
    }
}

// kFewDz.  (A last column without a neighbour takes one of the row's padding with it.)
__device__ __forceinline__ void few_dz(const Work& w, const Job& j, Logits<kFewChunks>& l, int64_t row0, int64_t rows, int lane, int64_t n0,
                                       int64_t end, const FewTokens& f) {
    const int64_t row = row0 + lane;
    const bool ok = row - (lane & 1) < rows;
#pragma unroll
    for (int c = 0; c < kFewChunks; ++c) {
        const int64_t col = n0 + kChunk * c;
        if (col >= end) break;
        const RowValues& r = f.r[c];
        uint32_t (&v)[kChunk] = l.z[c];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kChunk; e += 2) {
            const float s0 = __shfl_sync(kFull, r.lse, e), s1 = __shfl_sync(kFull, r.lse, e + 1);
            const float p0 = __shfl_sync(kFull, r.p, e), p1 = __shfl_sync(kFull, r.p, e + 1);
            float x, y;
            exp2_of(v[e], v[e + 1], pk(-s0, -s1), x, y);
            upk(mul2(pk(x, y), pk(p0, p1)), x, y);
            v[e] = p0 == 0.0f ? 0u : __float_as_uint(x);
            v[e + 1] = p1 == 0.0f ? 0u : __float_as_uint(y);
        }
        const int at = r.target - (int)w.v0 - (int)row0;
        if (__any_sync(kFull, at >= 0 && at < 32)) {
            const int mine = at >= 0 && at < 32 ? at : -1;
#pragma unroll
            for (int e = 0; e < kChunk; ++e) {
                const int t = __shfl_sync(kFull, mine, e);
                const float g = __shfl_sync(kFull, r.g, e);
                if (t == lane) v[e] = __float_as_uint(g);
            }
        }
        store_columns(j.out, j.ld, row, col, ok ? end - col : 0, lane, v);
    }
}

// `left` of 32 sums of a row (a multiple of 16)
__device__ __forceinline__ void store_sums(float* p, int64_t left, const uint32_t (&v)[kChunk]) {
    float4* q = reinterpret_cast<float4*>(p);
#pragma unroll
    for (int i = 0; i < kChunk / 4; ++i)
        if (4 * i < left)
            q[i] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]), __uint_as_float(v[4 * i + 2]),
                               __uint_as_float(v[4 * i + 3]));
}
// Where there are sums of other parts or pieces: those of the pieces before are added; true: more will be added to these, here
// or behind the last piece, and they are stored, so nothing else is to do.  `left` of the 32 sums are there, `stride` apart.
__device__ __forceinline__ bool with_sums_of_column(const Job& j, float* p, int64_t stride, int64_t left, uint32_t (&v)[kChunk]) {
    if (!j.first) {
#pragma unroll
        for (int e = 0; e < kChunk; ++e)
            if (e < left) v[e] = __float_as_uint(__uint_as_float(v[e]) + p[e * stride]);
    }
    if (j.last) return false;
#pragma unroll
    for (int e = 0; e < kChunk; ++e)
        if (e < left) p[e * stride] = __uint_as_float(v[e]);
    return true;
}

// kDw in several parts
__device__ __forceinline__ void dw_sums_of_row(const Job& j, uint32_t taddr, int64_t row, int64_t n0, int64_t end, int part) {
#pragma unroll 1
    for (int64_t col = n0; col < end; col += kChunk) {
        uint32_t v[kChunk];
        __syncwarp();
        tmem_ld<kChunk>(taddr + (uint32_t)(col - n0), v);
        if (row < j.rows) store_sums(j.sums + (part * j.rows + row) * j.cols + col, end - col, v);
    }
}

// kDx: the product's rows are the columns of dx, its columns the tokens, so the lanes of a warp have neighbours of one token
__device__ __forceinline__ void dx_of_column(const Job& j, uint32_t taddr, int64_t row, int64_t n0, int64_t end, int part, int lane,
                                             float unit) {
    const bool ok = row < j.rows;
#pragma unroll 1
    for (int64_t col = n0; col < end; col += kChunk) {
        uint32_t v[kChunk];
        __syncwarp();
        tmem_ld<kChunk>(taddr + (uint32_t)(col - n0), v);
        const int64_t left = ok ? end - col : 0;
        if (j.sums && with_sums_of_column(j, j.sums + (part * j.cols + col) * j.rows + row, j.rows, left, v)) continue;   // not j.last: all lanes
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kChunk; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * unit);
        store_columns(j.out, j.ld, row, col, left, lane, v);
    }
}

// The maps of the two jobs: A, B, and the output of kDz and kDw.
struct Maps {
    CUtensorMap a[2], b[2], o[2];
};

template <Kind kKind>
__global__ void __launch_bounds__(kThreads, 1) lce_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Work w) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);   // the same offset in both CTAs
    const uint32_t sb = smem_u32(smem);
    const uint32_t bar0 = sb + kBarOff;
    auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(kMaxStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (uint32_t)(2 * kMaxStages + kMaxAccs + b); };
    const uint32_t done = bar0 + 8u * (uint32_t)(2 * kMaxStages + 2 * kMaxAccs);
    constexpr int kAccs = accs_of(kKind), kAccStride = 2 * kBN / kAccs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kBarOff + 8 * kNumBars);
    volatile uint32_t* abort = tmem_slot + 1;

    const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();   // 0: the CTA that issues the pair's MMAs
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int b = 0; b < kAccs; ++b) { mbar_init(acc_full(b), 1); mbar_init(acc_empty(b), 2 * kEpiWarps); }
        mbar_init(done, 1);
        *abort = 0u;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < w.jobs; ++i) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.a[i])) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.b[i])) : "memory");
        }
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(2 * kBN)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync();   // barriers initialised and tensor memory allocated in both CTAs
    tc_fence_after();
    wait_for_primary();
    dependents_may_start();   // their launch costs nothing then (2048 x 512 x 1024 forward: 8.6 us, at the end or never 9.3)
    const uint32_t tmem = *tmem_slot;

    const int64_t pair = blockIdx.x >> 1;
    const Walk walk(w, blockIdx.x >> 1);
    const int stages = w.stages, slot = w.slot;
    Item it;

    // The producer's and the issuer's warps walk together and one elected lane issues, so that addresses and descriptors stay
    // in uniform registers, and ask for the next stage's barrier before they issue for this one: a single thread that waits,
    // issues and turns takes 550 clocks a step, more than the 512 of a 256 x 256 tile's MMAs.
    if constexpr (kKind == kLogits) {
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    }
    if (warp == 0) {
        // ---- TMA producer (both CTAs): this CTA's 128 rows of A and half of the columns of B ----
        int s = 0;
        uint32_t ph = 0, issued = 0, last_ph = 0;   // per stage: issued at all, parity of the last issue
        bool ok = true, ready = false;
        const uint32_t elected = elect_one();
        const uint32_t fb0 = map_to_rank(full(0), 0);   // the leader's barriers, contiguous like ours
        for (uint32_t i = 0; ok && walk.item(i, w, it); ++i) {
            const Job& j = w.job[it.job];
            const CUtensorMap *ma = &maps.a[it.job], *mb = &maps.b[it.job];
            const int32_t bm = kKind == kFewLogits ? j.bm : 2 * kBM;
            const int32_t m0 = (int32_t)(it.m * bm + rank * (bm / 2)), n0 = (int32_t)(it.n * j.bn + rank * (j.bn / 2));
            const uint32_t bytes = 2u * (uint32_t)((bm / 2 + j.bn / 2) * kBK * 2);   // of both CTAs
            const bool a_mn = j.a_mn;
            for (int k = it.from; k < it.to; ++k) {
                if (!ready) ok = __all_sync(kFull, mbar_wait_fast(empty(s), ph ^ 1u, abort));
                if (!ok) break;
                const uint32_t fb = fb0 + 8u * (uint32_t)s, own = full(s), sa = sb + (uint32_t)(s * slot), sbb = sa + kABytes;
                issued |= 1u << s;
                last_ph = (last_ph & ~(1u << s)) | (ph << s);
                if (++s == stages) { s = 0; ph ^= 1u; }
                const bool next = mbar_test(empty(s), ph ^ 1u);
                const int32_t k0 = k * kBK;
                if (elected) {
                    if (leader) mbar_expect_tx(own, bytes);
                    if (a_mn) {
                        tma_load_2d_pair(sa, ma, m0, k0, fb);
                        tma_load_2d_pair(sa + kBoxBytes, ma, m0 + 64, k0, fb);
                    } else {
                        tma_load_2d_pair(sa, ma, k0, m0, fb);
                    }
                    tma_load_2d_pair(sbb, mb, k0, n0, fb);
                }
                ready = __all_sync(kFull, next);
            }
        }
        // every stage issued has been read by the MMAs before the CTA may exit
        for (int i = 0; i < kMaxStages; ++i)
            if (issued & (1u << i)) mbar_wait(empty(i), (last_ph >> i) & 1u, nullptr);
        __syncwarp();
    } else if (warp == 1) {
        if (leader) {
            // ---- MMA issuer (even CTA) ----
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, ready = false;
            const uint32_t elected = elect_one();
            const uint64_t bdesc0 = smem_desc(sb + kABytes, false);
            for (uint32_t i = 0; ok && walk.item(i, w, it); ++i) {
                const Job& j = w.job[it.job];
                const uint32_t idesc = instr_desc(j);
                const uint64_t adesc0 = smem_desc(sb, j.a_mn);
                // 16 of the summed index: 32 bytes along a row, or 16 rows of 128 bytes
                const uint64_t ka = j.a_mn ? (kMmaK * 128) >> 4 : (kMmaK * 2) >> 4;
                for (int from = it.from; ok && from < it.to; from += j.segment) {
                    const int to = it.to - from < j.segment ? it.to : from + j.segment;
                    ok = __all_sync(kFull, mbar_wait_relaxed(acc_empty(acc), aph ^ 1u, abort));   // see mbar_arrive_relaxed
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + (uint32_t)(acc * kAccStride), af = acc_full(acc);
                    for (int k = from; k < to; ++k) {
                        if (!ready) ok = __all_sync(kFull, mbar_wait_fast(full(s), ph, abort));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t so = (uint64_t)(s * (slot >> 4)), ad = adesc0 + so, bd = bdesc0 + so;
                        const uint32_t freed = empty(s);
                        if (++s == stages) { s = 0; ph ^= 1u; }
                        const bool next = mbar_test(full(s), ph);
                        if (elected) {
#pragma unroll
                            for (int kk = 0; kk < kBK / kMmaK; ++kk)
                                mma_bf16_pair(d, ad + kk * ka, bd + (uint64_t)(kk * ((kMmaK * 2) >> 4)), idesc, k != from || kk != 0);
                            mma_commit_pair(freed, 0x3);   // both CTAs' stage is free once read
                            if (k + 1 == to) mma_commit_pair(af, 0x3);
                        }
                        ready = __all_sync(kFull, next);
                    }
                    if (++acc == kAccs) { acc = 0; aph ^= 1u; }
                }
            }
            if (elected) mma_commit_pair(done, 0x3);   // every MMA issued has completed before either CTA frees tensor memory
        }
        if (lane == 0) mbar_wait(done, 0u, nullptr);
        __syncwarp();
    } else if (warp >= 4) {
        if constexpr (kKind == kLogits) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        // ---- epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31, half (w - 4) / 4 of the columns ----
        const int q4 = warp & 3, half = (warp - 4) >> 2;
        const uint32_t staging = sb + kStageArea + (uint32_t)((warp - 4) * kStagingBytes);   // of kFewStats
        const uint32_t box = sb + kStageArea + (uint32_t)((warp - 4) * 4096);                // of TMA stores: 1024-byte aligned
        const int64_t few_n0 = half * (w.job[0].bn / 2), few_end = few_n0 + w.job[0].bn / 2 < w.job[0].cols ? few_n0 + w.job[0].bn / 2 : w.job[0].cols;
        const float unit = w.unit ? static_cast<const volatile float*>(w.unit)[kKind == kProducts] : 1.0f;
        FewTokens tokens;
        if constexpr (kKind == kFewLogits) few_tokens(w, w.job[0], few_n0, few_end, lane, unit, tokens);
        int acc = 0;
        uint32_t aph = 0;
        auto release = [&] {   // the accumulator has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(map_to_rank(acc_empty(acc), 0));
            if (++acc == kAccs) { acc = 0; aph ^= 1u; }
        };
        for (uint32_t i = 0; walk.item(i, w, it); ++i) {
            if (it.from == it.to) continue;
            const Job& j = w.job[it.job];
            const int bm = kKind == kFewLogits ? j.bm : 2 * kBM;
            const int64_t top = it.m * bm + rank * (bm / 2), row0 = top + 32 * q4, row = row0 + lane, col0 = it.n * j.bn;
            if constexpr (kKind != kProducts) {
                constexpr bool few = kKind == kFewLogits;
                const RowValues r = row_values(w, j, row, few ? 0 : j.rows, unit);
                const int64_t end = col0 + j.bn < j.cols ? col0 + j.bn : j.cols;
                Logits<few ? kFewChunks : kChunks> l;
                bool ok = true;
                for (int from = it.from; from < it.to; from += j.segment) {
                    ok = __all_sync(kFull, mbar_wait_inline(acc_full(acc), aph, abort));   // the sums so far stay in registers
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t acc0 = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(acc * kAccStride);
                    if (from == it.from)
                        add_segment<true>(acc0, half, j.bn, (int)(end - col0), l);
                    else
                        add_segment<false>(acc0, half, j.bn, (int)(end - col0), l);
                    release();
                }
                if (!ok) break;
                if constexpr (few) {
                    const int64_t rows = top + bm / 2 < j.rows ? top + bm / 2 : j.rows;   // up to this CTA's last one
                    if (j.mode == kFewStats) few_stats(w, l, staging, row0, rows, lane, few_n0, few_end, tokens);
                    else few_dz(w, j, l, row0, rows, lane, few_n0, few_end, tokens);
                } else {
                    if (j.mode == kStats) stats_of_row(w, j, r, l, row, col0, end, half, 2 * it.n + half);
                    else dz_of_row(w, j, r, l, box, &maps.o[it.job], row0, col0, half, lane);
                }
            } else {
                if (!__all_sync(kFull, mbar_wait_fast(acc_full(acc), aph, abort))) break;
                tc_fence_after();
                const int64_t n0 = col0 + half * (j.bn / 2), end = n0 + j.bn / 2 < j.cols ? n0 + j.bn / 2 : j.cols;
                const uint32_t acc0 = tmem + ((uint32_t)(32 * q4) << 16) + (uint32_t)(acc * kAccStride), taddr = acc0 + (uint32_t)(half * (j.bn / 2));
                if (j.mode == kDx)
                    dx_of_column(j, taddr, row, n0, end, it.part, lane, unit);
                else if (j.sums)
                    dw_sums_of_row(j, taddr, row, n0, end, it.part);
                else
                    dw_of_row(j, acc0, box, &maps.o[it.job], row0, col0, half, lane, unit);
                release();
            }
        }
        if (kKind == kFewLogits && w.job[0].mode == kFewStats) {   // the four warps of a half, which have the same tokens
            auto at = [&](int q, int c) { return staging + (uint32_t)((q - q4) * kStagingBytes + 16 * (kChunk * c + lane)); };
            __syncwarp();
#pragma unroll
            for (int c = 0; c < kFewChunks; ++c)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %3};" ::"r"(at(q4, c)), "r"(__float_as_uint(tokens.top[c])),
                             "r"(__float_as_uint(tokens.rest[c])), "r"(tokens.at[c])
                             : "memory");
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
#pragma unroll
            for (int c = 0; c < kFewChunks; ++c) {
                const int64_t token = few_n0 + kChunk * c + lane;
                if (q4 != 0 || token >= few_end) continue;
#pragma unroll
                for (int q = 1; q < 4; ++q) {
                    uint32_t top1, rest1, at1, same;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(top1), "=r"(rest1), "=r"(at1), "=r"(same) : "r"(at(q, c)) : "memory");
                    if (__uint_as_float(top1) > tokens.top[c]) tokens.at[c] = (int32_t)at1;
                    join_rest(tokens.top[c], tokens.rest[c], __uint_as_float(top1), __uint_as_float(rest1));
                }
                const int64_t i = (2 * pair + rank) * w.stats_ld + token;
                w.stats[i] = make_float2(tokens.top[c], tokens.rest[c]);
                w.tops[i] = tokens.at[c];
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the stores by TMA are done
        __syncwarp();
    }
    tc_fence_before();
    cluster_sync();   // no arrival or copy is still on its way to either CTA
    tc_fence_after();
    __syncwarp();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kBN) : "memory");
}

// loss and lse from the half tiles' maxima and rests: 32 rows per block, each warp every 32nd of them
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) lce_join_kernel(const float2* stats, int64_t ld, int64_t parts, const void* targets,
                                                                   int32_t wide, int64_t M, int64_t V, float* loss, float* lse) {
    __shared__ float2 part[kJoinWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row0 = (int64_t)blockIdx.x * 32, row = row0 + warp;
    wait_for_primary();
    dependents_may_start();
    int64_t t = -1;
    float z = 0.0f;
    if (row < M) {   // what the end needs, with the first loads
        t = index_at(targets, wide, row);
        z = static_cast<const volatile float*>(loss)[row];
    }
    float top = -INFINITY, rest = kNoRest;
    // stats_ld is a multiple of 32: the rows behind the last one are there, whatever they hold
    const float2* p = stats + row0 + lane;
#pragma unroll 8
    for (int64_t i = warp; i < parts; i += kJoinWarps) {
        const float2 f = p[i * ld];
        join_rest(top, rest, f.x, f.y);
    }
    part[warp][lane] = make_float2(top, rest);
    __syncthreads();
    // a warp for each row: its 32 lanes hold the warps' results
    if (row >= M) return;
    top = part[lane][warp].x;
    rest = part[lane][warp].y;
    for (int off = 16; off > 0; off >>= 1) {
        const float top1 = __shfl_xor_sync(kFull, top, off), rest1 = __shfl_xor_sync(kFull, rest, off);
        join_rest(top, rest, top1, rest1);
    }
    if (lane != 0) return;
    const float low = log1pf(rest);
    lse[row] = top + low;
    // (top - z) + log(sum): nothing cancels where the target's logit is the largest
    loss[row] = t < 0 ? 0.0f : t >= V ? NAN : (top - z) + low;
}

// Of few tokens, logits by themselves: four warps have one token and kN rows of the weight, every fourth 256 columns each, products
// added in float32 with its rounding, C / 512 of them in a chain.  What the tensor cores make of a logit falls short by about
// 2e-7 of its size (lse of logits of 64: 1.2e-5, in all tokens alike), and the gradient of a token that is all but certain is a
// difference with its logit: 6 % off with a probability of 1 - 2e-4, and with fewer than ten tokens all results may be one
// such token's.  So few tokens' loss and gradient are formed with these, for the largest and the target's logit (33 x 50304 x
// 2048 forward 39.3 us for 38.4, 33 x 512 x 2048 14.5 for 12.5; backward of 33 x 512 x 256 12.3 for 12.0).
constexpr int kSplit = 4;
template <int kN>
__device__ __forceinline__ void exact_parts(const uint16_t* x, const uint16_t* const (&w)[kN], int64_t C, int lane, int quarter, float (&z)[kN]) {
    constexpr int kDot = 2, kStep = 256 * kSplit;   // chunks of 256 columns on their way at once
    float sum[kN][4] = {};
#pragma unroll 1
    for (int64_t c0 = 256 * quarter + 8 * lane; c0 < C; c0 += kStep * kDot) {
        uint32_t xv[kDot][4], wv[kN][kDot][4];
#pragma unroll
        for (int k = 0; k < kDot; ++k) {   // (no load behind a branch: behind the end the ones before again, which do not count)
            const int64_t c = c0 + kStep * k < C ? c0 + kStep * k : c0;
            load_words<4>(x + c, xv[k]);
#pragma unroll
            for (int n = 0; n < kN; ++n) load_words<4>(w[n] + c, wv[n][k]);
        }
#pragma unroll
        for (int k = 0; k < kDot; ++k) {
            if (c0 + kStep * k >= C) continue;
            float a[8], b[8];
            unpack(xv[k], a);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                unpack(wv[n][k], b);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[n][e & 3] = fmaf(a[e], b[e], sum[n][e & 3]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        z[n] = (sum[n][0] + sum[n][1]) + (sum[n][2] + sum[n][3]);
        for (int off = 16; off > 0; off >>= 1) z[n] += __shfl_xor_sync(kFull, z[n], off);
    }
}
__device__ __forceinline__ float exact_logit(const float (&parts)[kSplit]) { return (parts[0] + parts[1]) + (parts[2] + parts[3]); }

// loss and lse of few tokens from the CTAs' maxima and rests: kFewRows rows per block, with kSplit warps each in the end.  lse is
// the same whatever the targets are.
constexpr int kFewRows = 8;
static_assert(kFewRows * kSplit == 32, "a block's warps");
__global__ void __launch_bounds__(1024) lce_join_few_kernel(const LceFwdArgs a, const float2* stats, const int32_t* tops, int64_t ld, int64_t parts) {
    __shared__ float2 part[32][kFewRows];
    __shared__ int32_t part_at[32][kFewRows];
    __shared__ float exact[2][kFewRows][kSplit];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / kSplit, quarter = warp % kSplit;
    const int64_t row0 = (int64_t)blockIdx.x * kFewRows, row = row0 + mine;
    wait_for_primary();
    dependents_may_start();
    int64_t t = -1;
    float z = 0.0f;
    if (row < a.M) {   // what the end needs, with the first loads
        t = index_at(a.targets, a.wide, row);
        z = static_cast<const volatile float*>(a.loss)[row];
    }
    float top = -INFINITY, rest = kNoRest;
    int32_t at = -1;
    auto join = [&](float top1, float rest1, int32_t at1) {   // (of two that are the largest alike, the lower row: all lanes hold the same)
        if (top1 > top || (top1 == top && (uint32_t)at1 < (uint32_t)at)) at = at1;
        join_rest(top, rest, top1, rest1);
    };
    auto join_lanes = [&](int least) {
        for (int off = 16; off >= least; off >>= 1)
            join(__shfl_xor_sync(kFull, top, off), __shfl_xor_sync(kFull, rest, off), __shfl_xor_sync(kFull, at, off));
    };
    // stats_ld is a multiple of 32: the rows behind the last one are there, whatever they hold
    const int64_t from = row0 + lane % kFewRows;
#pragma unroll 2
    for (int64_t i = kSplit * warp + lane / kFewRows; i < parts; i += 32 * kSplit) {
        const float2 f = stats[i * ld + from];
        join(f.x, f.y, tops[i * ld + from]);
    }
    join_lanes(kFewRows);
    if (lane < kFewRows) {
        part[warp][lane] = make_float2(top, rest);
        part_at[warp][lane] = at;
    }
    __syncthreads();
    top = part[lane][mine].x;
    rest = part[lane][mine].y;
    at = part_at[lane][mine];
    join_lanes(1);
    if (at >= a.V) at = -1;   // a row of the weight, whatever another call has done to the workspace
    if (row < a.M && at >= 0) {
        const uint16_t* const w[2] = {a.weight + at * a.C, a.weight + (t >= 0 && t < a.V ? t : at) * a.C};
        float e[2];
        exact_parts(a.x + row * a.x_ld, w, a.C, lane, quarter, e);
        if (lane < 2) exact[lane][mine][quarter] = lane == 0 ? e[0] : e[1];
    }
    __syncthreads();
    if (row >= a.M || quarter != 0 || lane != 0) return;
    if (at >= 0) {
        const float e = exact_logit(exact[0][mine]);
        if (fabsf(e) < INFINITY) {   // the rest is of the others, against the largest one
            rest *= expf(top - e);
            top = e;
            z = exact_logit(exact[1][mine]);
        }
    }
    const float low = log1pf(rest);
    a.lse[row] = top + low;
    // (top - z) + log(sum): nothing cancels where the target's logit is the largest
    a.loss[row] = t < 0 ? 0.0f : t >= a.V ? NAN : (top - z) + low;
}

// The gradient of a target's logit is -g (1 - e^(z - lse)), which is -g for most tokens, and with a mean over the tokens g is
// the same for all of them: rounded to bf16, they would all be off by the same share of themselves, up to 2^-8, and dx and dW
// with them (8192 x 32000 x 4096, a mean over the tokens: 2.0e-3 to 2.9e-3 off by the number of tokens, so 2.0e-3).  So dz is
// stored times a factor within 1 +- 2^-8, with which the g of the first token that has a target and a g between 2^-100 and 2^100
// in size is a bf16 value, and the products are multiplied by its reciprocal.  (Without such a token, 1.)  A block of its own
// looks for that token, kUnitAhead a thread at once, since a long prompt without targets may come first (2^20 tokens, none with
// a target: 0.8 us for 1024 of them).
constexpr int kUnitAhead = 4;   // 8: 40 registers and six blocks per SM instead of eight, 8192 x 4096 22.7 us for 21.2
__device__ __forceinline__ void unit_of(const void* targets, int32_t wide, const float* dloss, int64_t M, float* unit) {
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    __shared__ uint32_t first;
    if (threadIdx.x == 0) first = kNone;
    __syncthreads();
    uint32_t mine = kNone;
    float own = 1.0f;
    for (int64_t m0 = 0; m0 < M; m0 += kUnitAhead * blockDim.x) {
        int64_t at[kUnitAhead], t[kUnitAhead];
        float g[kUnitAhead];
#pragma unroll
        for (int k = 0; k < kUnitAhead; ++k) {   // (the last token again: no load behind a branch, see lm_embed.cu)
            const int64_t m = m0 + k * blockDim.x + threadIdx.x;
            at[k] = m < M ? m : M - 1;
            g[k] = static_cast<const volatile float*>(dloss)[at[k]];
        }
        if (wide) {
#pragma unroll
            for (int k = 0; k < kUnitAhead; ++k) t[k] = load_index(static_cast<const int64_t*>(targets) + at[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kUnitAhead; ++k) t[k] = load_index(static_cast<const int32_t*>(targets) + at[k]);
        }
#pragma unroll
        for (int k = kUnitAhead - 1; k >= 0; --k)
            if (t[k] >= 0 && fabsf(g[k]) > 0x1p-100f && fabsf(g[k]) < 0x1p100f) {
                mine = (uint32_t)at[k];
                own = g[k];
            }
        const uint32_t lowest = __reduce_min_sync(kFull, mine);
        if ((threadIdx.x & 31) == 0) atomicMin(&first, lowest);
        if (__syncthreads_or(mine != kNone)) break;
    }
    if (first == kNone ? threadIdx.x == 0 : mine == first) {
        const float f = first == kNone ? 1.0f : __uint_as_float(bf16x2(own, 0.0f) << 16) / own;
        unit[0] = f;
        unit[1] = 1.0f / f;
    }
}

// Where few tokens' shares are kept until dx is written: in dx itself, at the beginning of the token's row.
__host__ __device__ __forceinline__ float* share_of(const LceBwdArgs& a) { return reinterpret_cast<float*>(a.dx); }

// xt[c][m] = x[m][c]: tiles of 64 x 64 through shared memory, behind a block that finds the unit and, of few tokens, in front of
// those that find their shares.  (xt's rows are whole 16-byte units; what lies behind their M elements is not read.)
template <bool kFew>
__global__ void __launch_bounds__(256) lce_transpose_kernel(const LceBwdArgs a) {
    __shared__ uint16_t tile[64][66];
    const int64_t M = a.M, C = a.C, ld = (M + 7) / 8 * 8, across = (M + 63) / 64;
    const int64_t i0 = (int64_t)blockIdx.x - 1, m0 = i0 % across * 64, c0 = i0 / across * 64;
    wait_for_primary();
    dependents_may_start();
    if (i0 < 0) {
        unit_of(a.targets, a.wide, a.dloss, M, a.unit);
        return;
    }
    if (kFew && c0 >= C) {
        __shared__ float exact[8 / kSplit][kSplit];
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp / kSplit, quarter = warp % kSplit;
        const int64_t m = (i0 - across * ((C + 63) / 64)) * (8 / kSplit) + mine, t = m < M ? index_at(a.targets, a.wide, m) : -1;
        const bool has = t >= 0 && t < a.V;
        if (has) {
            const uint16_t* const w[1] = {a.weight + t * C};
            float z[1];
            exact_parts(a.x + m * a.x_ld, w, C, lane, quarter, z);
            if (lane == 0) exact[mine][quarter] = z[0];
        }
        __syncthreads();
        if (has && quarter == 0 && lane == 0)
            share_of(a)[m * (C / 2)] = expm1f(exact_logit(exact[mine]) - static_cast<const volatile float*>(a.lse)[m]);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = threadIdx.x + 256 * h, r = i >> 3, c = (i & 7) * 8;
        uint32_t w[4] = {};
        if (m0 + r < M && c0 + c < C) load_words<4>(a.x + (m0 + r) * a.x_ld + c0 + c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t*>(&tile[r][c + 2 * k]) = w[k];
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = threadIdx.x + 256 * h, c = i >> 3, r = (i & 7) * 8;
        if (c0 + c >= C || m0 + r >= M) continue;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = (uint32_t)tile[r + 2 * k][c] | (uint32_t)tile[r + 2 * k + 1][c] << 16;
        *reinterpret_cast<uint4*>(a.xt + (c0 + c) * ld + m0 + r) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// out[i] = bf16(unit[1] sum over parts of sums[part][i]): products summed in parts.  A warp has 256 elements, and where there are
// several parts several warps of the block share them, every one some of the parts (200 x 30000 x 256, 32 parts: 4.5 us; all
// parts in one thread 11 us).
constexpr int kPartWarps = 8;
__global__ void __launch_bounds__(32 * kPartWarps) lce_parts_kernel(const float* sums, int parts, int teams, int64_t n, const float* unit, uint16_t* out) {
    __shared__ __align__(16) float part[kPartWarps][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp % teams;
    const int64_t at = ((int64_t)blockIdx.x * (kPartWarps / teams) + warp / teams) * 256 + 8 * lane;
    wait_for_primary();
    dependents_may_start();
    float x[8] = {};
    auto add = [&](const float* p) {
        const float4 f = *reinterpret_cast<const float4*>(p), g = *reinterpret_cast<const float4*>(p + 4);
        x[0] += f.x; x[1] += f.y; x[2] += f.z; x[3] += f.w;
        x[4] += g.x; x[5] += g.y; x[6] += g.z; x[7] += g.w;
    };
    if (at < n) {
#pragma unroll 4
        for (int p = team; p < parts; p += teams) add(sums + p * n + at);
    }
    if (teams > 1) {
        float4* mine = reinterpret_cast<float4*>(&part[warp][8 * lane]);
        mine[0] = make_float4(x[0], x[1], x[2], x[3]);
        mine[1] = make_float4(x[4], x[5], x[6], x[7]);
        __syncthreads();
        if (team > 0) return;
        for (int t = 1; t < teams; ++t) add(&part[warp + t][8 * lane]);
    }
    if (at >= n) return;
    const float u = static_cast<const volatile float*>(unit)[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= u;
    uint32_t w[4];
    pack(x, w);
    *reinterpret_cast<uint4*>(out + at) = make_uint4(w[0], w[1], w[2], w[3]);
}
cudaError_t launch_parts(const float* sums, int parts, int64_t n, const float* unit, uint16_t* out, cudaStream_t s) {
    const int teams = parts >= 8 ? 8 : parts >= 4 ? 4 : parts >= 2 ? 2 : 1;
    const int64_t per = 256 * (kPartWarps / teams);
    return launch_next(lce_parts_kernel, (unsigned)((n + per - 1) / per), 32 * kPartWarps, 0, s, sums, parts, teams, n, unit,
                       out);
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

// A matrix as an operand: with the summed index along its rows, or (A alone) across them.
struct Operand {
    const uint16_t* p;
    int64_t rows, cols, ld;
    bool mn;
};
int64_t up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// What a step of a tile of n columns takes, as the columns that its MMAs alone would take: they and the rows of A are loaded
// in 64 columns' time more, and the steps' barriers take as long as 208 (8192 rows, 64 x 64 of the summed index: 309 ns a
// step with 256 columns, 276 with 224, 245 with 192, 220 with 160, 207 with 128, 198 with 64).
int64_t step_cost(int64_t n) { return n + 64 > 208 ? n + 64 : 208; }
constexpr int64_t kWholeStep = kBN + 64;

// Columns of a tile, of the multiples of 32.  Of a product alone: those with which the pairs that have most tiles take least
// time (33 x 50304 x 2048 forward: 225 tiles of 224 for 76 pairs, instead of 197 of 256).  Of one of two products, which make up
// for each other's last tiles: those that cover it in the least time.
int tile_columns(int64_t rows, int64_t cols, int32_t mode) {
    const bool alone = mode < kDx;
    const int step = mode == kDz || mode == kDw ? 64 : 32;   // a store by TMA has 64 columns
    int64_t best = 0;
    int bn = kBN;
    for (int n = kBN; n >= step; n -= step) {
        const int64_t tiles = up(rows, 2 * kBM) * up(cols, n), cost = (alone ? up(tiles, kPairs) : tiles) * step_cost(n);
        if (best == 0 || cost < best) {
            best = cost;
            bn = n;
        }
    }
    if (mode == kFewStats || mode == kFewDz) bn = (int)up(cols, 32) * 32;   // all tokens
    return bn;
}

// Rows of a tile of few tokens' logits, which are the weight's, of the multiples of 32: where there are more tiles than pairs,
// those with which the pairs that have most have fewest rows (50304 rows: 225 tiles of 224 for 76 pairs, three each, instead of
// 197 of 256: 33 x 50304 x 2048 38.1 us for 39.2, 20 x 24000 x 2048 25.0 for 27.9; otherwise more pairs with fewer rows each
// only take longer, 20 x 9000 x 2048 15.9 for 15.0 us).  The MMA's other rows hold what was there before: no element of the
// product but theirs depends on them.
int tile_rows(int64_t rows, int32_t mode) {
    int64_t best = 0;
    int bm = 2 * kBM;
    if (kind_of(mode) != kFewLogits || up(rows, bm) <= kPairs) return bm;
    for (int m = 2 * kBM; m >= 128; m -= 32) {
        const int64_t cost = up(up(rows, m), kPairs) * m;
        if (best == 0 || cost < best) {
            best = cost;
            bm = m;
        }
    }
    return bm;
}

bool add_job(Work& w, Maps& maps, int32_t mode, const Operand& a, const Operand& b, uint16_t* out, int64_t ld) {
    Job& j = w.job[w.jobs];
    const int64_t K = a.mn ? a.rows : a.cols;
    j.mode = mode;
    j.a_mn = a.mn;
    j.rows = a.mn ? a.cols : a.rows;
    j.cols = b.rows;
    j.steps = (int32_t)up(K, kBK);
    j.segment = kind_of(mode) == kLogits ? kSegment : kind_of(mode) == kFewLogits ? kFewSegment : j.steps;
    j.bn = tile_columns(j.rows, j.cols, mode);
    j.bm = tile_rows(j.rows, mode);
    j.parts = 1;
    j.tm = up(j.rows, j.bm);
    j.tn = up(j.cols, j.bn);
    j.out = out;
    j.ld = ld;
    j.sums = nullptr;
    j.first = j.last = 1;
    if (!encode(&maps.a[w.jobs], a.p, a.rows, a.cols, a.ld, a.mn ? kBK : j.bm / 2) ||
        !encode(&maps.b[w.jobs], b.p, b.rows, b.cols, b.ld, j.bn / 2) ||
        ((mode == kDz || mode == kDw) && !encode(&maps.o[w.jobs], out, j.rows, j.cols, ld, 32)))
        return false;
    ++w.jobs;
    return true;
}

// What an item takes, in the unit of step_cost: its steps, or its epilogue where that is longer (a tile's 128 KB of bf16 at a
// pair's share of the memory take as long as five steps), and one for its ends.
int64_t item_cost(int64_t steps, int64_t parts, int bn) {
    const int64_t n = up(steps, parts);
    return (n > 5 ? n : 5) * step_cost(bn) + step_cost(bn);
}

// How the items of a launch go to the pairs: see Work.
struct Split {
    int64_t pairs, ahead, extra;
};
Split split_of(int64_t first, int64_t first_cost, int64_t second, int64_t second_cost, int64_t pairs) {
    Split s;
    s.pairs = first + second < pairs ? first + second : pairs;
    s.ahead = first % s.pairs;
    s.extra = 0;
    if (s.ahead > 0 && second > 0) {
        s.extra = (s.pairs - s.ahead) * ((first_cost + second_cost / 2) / second_cost);
        if (s.extra > second) s.extra = second;
    }
    return s;
}

cudaError_t launch_work(Work& w, const Maps& maps, cudaStream_t s) {
    const int64_t sms = device_sms(), pairs = sms / 2 < kPairs ? sms / 2 : kPairs;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    int64_t cost[2] = {0, 0};
    for (int i = 0; i < w.jobs; ++i) {
        Job& j = w.job[i];
        w.items[i] = j.tm * j.tn * j.parts;
        j.by_tiles = divider((uint32_t)(j.tm * j.tn));
        j.by_band = divider((uint32_t)(kBand * j.tn));
        j.by_last = divider(j.tm % kBand ? (uint32_t)(j.tm % kBand) : kBand);
        j.by_parts = divider((uint32_t)j.parts);
        cost[i] = item_cost(w.job[i].steps, w.job[i].parts, w.job[i].bn);
    }
    if (w.jobs < 2) w.items[1] = 0;
    if (w.items[0] + w.items[1] >= ((int64_t)1 << 31) - 2 * kPairs) return cudaErrorInvalidValue;   // (2^40 logits are 2^27 tiles)
    const Split sp = split_of(w.items[0], cost[0], w.items[1], cost[1], pairs);
    w.pairs = (int32_t)sp.pairs;
    w.ahead = (int32_t)sp.ahead;
    w.extra = sp.extra;
    w.by_pairs = divider((uint32_t)sp.pairs);
    w.by_lot = divider((uint32_t)(sp.pairs - sp.ahead));
    int bn = 0;
    for (int i = 0; i < w.jobs; ++i) bn = w.job[i].bn > bn ? w.job[i].bn : bn;
    w.slot = slot_bytes(bn);
    w.stages = stages_of(bn);
    const Kind kind = kind_of(w.job[0].mode);
    auto* const kernel = kind == kLogits ? lce_kernel<kLogits> : kind == kFewLogits ? lce_kernel<kFewLogits> : lce_kernel<kProducts>;
    cudaError_t e = cudaSuccess;
    if (kind == kLogits) {
        // with fewer registers than the roles divide among them setmaxnreg would wait for ever: such a build is not launched
        cudaFuncAttributes built;
        if ((e = cudaFuncGetAttributes(&built, kernel)) != cudaSuccess) return e;
        if (built.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    }
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
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
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(2u * (unsigned)w.pairs);
    return cudaLaunchKernelEx(&cfg, kernel, maps, (const Work&)w);
}

// The two products behind a piece of n columns: their parts, and which has the longer items.  Few tiles with many steps leave
// pairs idle; parts of them cost float32 sums that are written, read and added by a kernel of their own.  The parts with which
// the busiest pair and that together take least (a whole tile's step is 0.31 us or 2 MB of memory traffic; the kernel 8).
struct Parts {
    int dx, dw;
    bool dx_first;
};
int64_t busiest(int64_t first, int64_t first_cost, int64_t second, int64_t second_cost) {
    const Split s = split_of(first, first_cost, second, second_cost, kPairs);
    const int64_t whole = first / s.pairs * first_cost, with = s.ahead > 0 ? first_cost : 0;
    const int64_t lot = s.pairs - s.ahead, without = s.extra > 0 ? up(s.extra, lot) * second_cost : 0;
    return whole + (with > without ? with : without) + up(second - s.extra, s.pairs) * second_cost;
}
Parts parts_of(int64_t M, int64_t n, int64_t C) {
    const int64_t dx = up(n, kBK), dw = up(M, kBK);   // steps
    const int dx_bn = tile_columns(C, M, kDx), dw_bn = tile_columns(n, C, kDw);
    const int64_t dx_tiles = up(C, 2 * kBM) * up(M, dx_bn), dw_tiles = up(n, 2 * kBM) * up(C, dw_bn);
    constexpr int kTry[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
    Parts best{1, 1, true};
    int64_t least = -1;
    for (const int px : kTry)
        for (const int pw : kTry) {
            if (px > dx || pw > dw) continue;
            const int64_t lx = item_cost(dx, px, dx_bn), lw = item_cost(dw, pw, dw_bn);
            const bool dx_first = lx >= lw;
            int64_t cost = dx_first ? busiest(dx_tiles * px, lx, dw_tiles * pw, lw) : busiest(dw_tiles * pw, lw, dx_tiles * px, lx);
            if (px > 1) cost += (8 + (px * M * C * 8 >> 21)) * kWholeStep;
            if (pw > 1) cost += (8 + (pw * n * C * 8 >> 21)) * kWholeStep;
            if (least < 0 || cost < least) {
                least = cost;
                best = Parts{px, pw, dx_first};
            }
        }
    return best;
}

}  // namespace

cudaError_t launch_lce_fwd(const LceFwdArgs& a, cudaStream_t s) {
    Work w = {};
    alignas(64) Maps maps;
    const Operand x{a.x, a.M, a.C, a.x_ld, false}, W{a.weight, a.V, a.C, a.C, false};
    const bool few = a.M <= kFewTokens;
    if (!(few ? add_job(w, maps, kFewStats, W, x, nullptr, 0) : add_job(w, maps, kStats, x, W, nullptr, 0))) return cudaErrorInvalidValue;
    w.targets = a.targets;
    w.wide = a.wide;
    w.V = (int32_t)a.V;
    w.stats = reinterpret_cast<float2*>(a.stats);
    w.stats_ld = up(a.M, 32) * 32;
    w.tops = reinterpret_cast<int32_t*>(w.stats + w.stats_ld * 2 * kPairs);
    w.target_logit = a.loss;
    cudaError_t e = launch_work(w, maps, s);
    if (e != cudaSuccess) return e;
    const int64_t parts = few ? 2 * (int64_t)w.pairs : 2 * w.job[0].tn;   // the CTAs, or two of each tile
    if (few)
        return launch_next(lce_join_few_kernel, (unsigned)up(a.M, kFewRows), 1024, 0, s, a, (const float2*)w.stats, (const int32_t*)w.tops,
                           w.stats_ld, parts);
    return launch_next(lce_join_kernel, (unsigned)up(a.M, 32), 32 * kJoinWarps, 0, s, (const float2*)w.stats, w.stats_ld,
                       parts, a.targets, a.wide, a.M, a.V, a.loss, a.lse);
}

cudaError_t launch_lce_bwd(const LceBwdArgs& a, cudaStream_t s) {
    const int64_t ld = lce_piece_ld(a.piece, a.V);
    const Parts parts = parts_of(a.M, a.piece, a.C);
    float* const dw_sums = a.sums + lce_dx_sums(a.M, a.V, a.C, a.piece);
    const bool dx_sums = parts.dx > 1 || a.piece < a.V;
    const bool few = a.M <= kFewTokens;
    cudaError_t e = launch_next(few ? lce_transpose_kernel<true> : lce_transpose_kernel<false>,
                                (unsigned)(1 + up(a.M, 64) * up(a.C, 64) + (few ? up(a.M * kSplit, 8) : 0)), 256, 0, s, a);
    if (e != cudaSuccess) return e;
    for (int64_t v0 = 0; v0 < a.V; v0 += a.piece) {
        const int64_t n = a.V - v0 < a.piece ? a.V - v0 : a.piece;
        const uint16_t* W = a.weight + v0 * a.C;
        Work w = {};
        alignas(64) Maps maps;
        const Operand x{a.x, a.M, a.C, a.x_ld, false}, Wz{W, n, a.C, a.C, false};
        if (!(few ? add_job(w, maps, kFewDz, Wz, x, a.dz, ld) : add_job(w, maps, kDz, x, Wz, a.dz, ld)))
            return cudaErrorInvalidValue;
        w.targets = a.targets;
        w.wide = a.wide;
        w.V = (int32_t)a.V;
        w.v0 = v0;
        w.lse = a.lse;
        w.dloss = a.dloss;
        w.dlse = a.dlse;
        w.unit = a.unit;
        w.share = share_of(a);
        w.share_ld = a.C / 2;
        e = launch_work(w, maps, s);
        if (e != cudaSuccess) return e;
        w.jobs = 0;
        for (int i = 0; i < 2; ++i) {
            Job& j = w.job[i];
            if (parts.dx_first == (i == 0)) {   // the product with the longer items first
                if (!add_job(w, maps, kDx, Operand{W, n, a.C, a.C, true}, Operand{a.dz, a.M, n, ld, false}, a.dx, a.C))
                    return cudaErrorInvalidValue;
                j.parts = parts.dx;
                j.sums = dx_sums ? a.sums : nullptr;
                j.first = v0 == 0;
                j.last = parts.dx == 1 && v0 + n == a.V;
            } else {
                if (!add_job(w, maps, kDw, Operand{a.dz, a.M, n, ld, true}, Operand{a.xt, a.C, a.M, lce_xt_ld(a.M), false},
                             a.dweight + v0 * a.C, a.C))
                    return cudaErrorInvalidValue;
                j.parts = parts.dw;
                j.sums = parts.dw > 1 ? dw_sums : nullptr;
                j.last = parts.dw == 1;
            }
        }
        e = launch_work(w, maps, s);
        if (e == cudaSuccess && parts.dw > 1)
            e = launch_parts(dw_sums, parts.dw, n * a.C, a.unit, a.dweight + v0 * a.C, s);
        if (e != cudaSuccess) return e;
    }
    if (parts.dx == 1) return cudaSuccess;
    return launch_parts(a.sums, parts.dx, a.M * a.C, a.unit, a.dx, s);
}

int64_t lce_piece(int64_t M, int64_t V, int64_t piece) {
    if (piece < 1) {   // as few pieces, of about the same width, as leave dz within kLceDzBytes
        int64_t most = kLceDzBytes / (2 * M) / 256 * 256;
        if (most < 256) most = 256;
        piece = up(V, up(V, most));
    }
    return piece < V ? up(piece, 256) * 256 < V ? up(piece, 256) * 256 : V : V;
}
int64_t lce_piece_ld(int64_t piece, int64_t V) { return up(piece < V ? piece : V, 256) * 256; }
int64_t lce_xt_ld(int64_t M) { return up(M, 8) * 8; }
int64_t lce_dx_sums(int64_t M, int64_t V, int64_t C, int64_t piece) {
    const Parts p = parts_of(M, piece, C);
    return p.dx > 1 || piece < V ? p.dx * M * C : 0;
}
int64_t lce_sums(int64_t M, int64_t V, int64_t C, int64_t piece) {
    const Parts p = parts_of(M, piece, C);
    return lce_dx_sums(M, V, C, piece) + (p.dw > 1 ? p.dw * piece * C : 0);
}
size_t lce_stats_bytes(int64_t M, int64_t V) {
    const size_t tokens = (size_t)(up(M, 32) * 32);
    return M <= kFewTokens ? 12 * tokens * (size_t)(2 * kPairs) : 8 * tokens * (size_t)(2 * up(V, tile_columns(M, V, kStats)));
}

cudaError_t read_lce_wait_timeouts(unsigned long long* out, bool reset) { return read_own_wait_timeouts(out, reset); }

}  // namespace coat
