// lm_embed.cu -- embedding lookup with a scale, and the gradient of the table from sorted tokens.
//
//   forward   out[m] = RN(scale table[ids[m]]); a negative id gives zeros, one past the table NaN
//   backward  dtable[v] = RN(scale sum over m with ids[m] = v of dout[m] (+ dtable[v]))
//
// Backward in three kernels, sums in float32 and in an order that the ids alone decide (within a chunk that of the tokens; then
// the chunks' shares, which teams_of warps take in turn; then those warps' sums):
//   sort    the tokens by their row of the table, stably: block b has rows of its own (every B-th), walks all M ids (they
//           are few bytes) and counts those of the blocks before it, which is where its part of the sorted order begins, so
//           that no block waits for another;
//   chunks  the sorted order in chunks of 32 tokens, a warp for each and 256 columns: rows that begin and end in the chunk
//           are finished; of one that goes on the chunk's share goes to the workspace, so that the work of a row with
//           many tokens (text has some that are a tenth of all) goes to many warps;
//   join    the rows that go on: their shares are added up, by 4 warps, or 2 where the gradient is added to what is there (so
//           that a long row written, and the same one added to zeros, may differ in float32's last bits); and rows without
//           a token become zeros, unless the gradient is added.
#include <cstdint>

#include "ckpt_kernels.h"
#include "divide.h"
#include "lm_device.cuh"
#include "lm_kernels.h"

namespace coat {

namespace {

using namespace ckpt;
using lm::index_at;
using lm::load_index;

constexpr int kBlock = 256;
constexpr int kChunk = 32;            // tokens of a chunk, one of a warp's lanes each
constexpr int kSlice = 256;           // columns of a warp: 8 per lane
// Tokens whose loads are on their way at once.  Many chunks: 4, and registers for 32 warps per SM (16411 x 2048, added / 8192 x
// 4096, all three kernels: 35.7 / 59.4 us; 8 and 20 warps 37.3 / 61.9; 16 and 10 warps 38.4 / 61.3).  Up to kFewUnits warps: 16
// (300 x 4096, added: 12.2 us; 4 18.3 in blocks of eight warps; 32 13.2: more code to fetch).
constexpr int kDeep = 4, kDeepest = 16;
constexpr int kResident = 32, kResidentFew = 8;
constexpr int64_t kFewUnits = 152 * 8;
constexpr int kSortBlock = 1024;
constexpr int kSortWarps = kSortBlock / 32;
// Ids on their way at once; of a warp's last ones, fewer than 32 kIds, which cost more in code to fetch than in waiting, kLastIds
// (300 / 4099 / 16411 / 40000 tokens, all three kernels, 8 / 4 / 2 / 1: 12.1 / 11.3 / 11.1 / 10.7, 13.7 / 13.9 / 13.7 / 13.6, 35.4 /
// 34.8 / 34.8 / 35.9, 49.1 / 50.1 / 50.8 / 52.0 us).
constexpr int kIds = 8, kLastIds = 2;
constexpr int kMaxRange = 768;        // rows of a sorting block: they take 256 bytes of shared memory each
// Warps that add up a row's shares.  Most blocks find that their chunk begins no such row; with zeros to fill there are more blocks,
// and what they take counts less (16411 x 2048 / 8192 x 4096, added, 1 / 2 / 4: 34.9 / 33.8 / 34.8, 30.1 / 30.1 / 32.1 us; 8192 x
// 4096 written, 2 / 4 / 8: 62.4 / 59.7 / 62.0).
constexpr int teams_of(bool add) { return add ? 2 : 4; }
// Rows of a filling block.  More copies at once per SM are slower: 8192 tokens, 32000 x 4096, all three kernels: 60 us with 4
// and 8, 62 with 16 and 32, 66 with 64, 67 with 128.
constexpr int kFill = 8;
constexpr int kZeroBytes = 8192;

// ---- forward ----
// A thread has kPer times 16 columns of a row, whose ids and then rows are on their way together.  Two where there are more of them
// than threads of one each on the device at once (8192 x 4096 / 40000 x 800 / 4099 x 4096: 16.0 / 14.0 / 6.5 us, one each 16.3 /
// 15.0 / 7.0, four 15.9 / 13.9 / 7.0; 1000 x 4096 / 17 x 2048: 2.6 / 1.3, one each 2.5 / 1.1).
constexpr int64_t kOneEach = 152 * 2048;
template <int kPer>
__global__ void __launch_bounds__(kBlock) embed_fwd_kernel(const EmbedFwdArgs a, const Divider nc, bool wide) {
    const uint32_t total = (uint32_t)a.M * nc.d, i0 = blockIdx.x * (kPer * kBlock) + threadIdx.x;
    wait_for_primary();
    uint32_t w[kPer][8];
    int64_t id[kPer];
    uint32_t col[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t i = i0 + k * kBlock < total ? i0 + k * kBlock : total - 1, m = divide(i, nc);   // (the last one again: not stored)
        col[k] = (i - m * nc.d) * 16;
        id[k] = index_at(a.ids, a.wide, m);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const bool in = id[k] >= 0 && id[k] < a.V;
        load_words8(a.table + (in ? id[k] : 0) * a.C + col[k], wide, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const uint32_t i = i0 + k * kBlock;
        float x[16];
        unpack(w[k], x);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= a.scale;
        pack(x, w[k]);
        if (id[k] < 0 || id[k] >= a.V) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[k][e] = id[k] < 0 ? 0u : 0x7FFF7FFFu;
        }
        if (i < total) store_words8(a.out + (int64_t)i * 16, wide, w[k]);
    }
}

// ---- backward: sort ----
// An id as a row of the table: itself, or -1 where it is none's.
__device__ __forceinline__ int row_of(int32_t id) { return id; }
__device__ __forceinline__ int row_of(int64_t id) { return id < 0 || id > 0x7FFFFFFF ? -1 : (int)id; }
// f(token, id's row) for the tokens m0 + lane, m0 + lane + 32, ... below m1; the whole warp calls f together, with a row of -1
// behind the last token.
template <typename T, typename F>
__device__ __forceinline__ void for_ids(const void* ids, int64_t m0, int64_t m1, int lane, F f) {
    int64_t m = m0;
    for (; m + 32 * kIds <= m1; m += 32 * kIds) {
        const T* p = static_cast<const T*>(ids) + m + lane;
        T v[kIds];
#pragma unroll
        for (int k = 0; k < kIds; ++k) v[k] = load_index(p + 32 * k);
#pragma unroll
        for (int k = 0; k < kIds; ++k) f((int)m + 32 * k + lane, row_of(v[k]));
    }
#pragma unroll 1
    for (; m < m1; m += 32 * kLastIds) {
        T v[kLastIds];
#pragma unroll
        for (int k = 0; k < kLastIds; ++k) {   // (a load without a condition: behind a branch every load would wait for the one before it)
            const int64_t at = m + 32 * k + lane;
            v[k] = load_index(static_cast<const T*>(ids) + (at < m1 ? at : m1 - 1));
        }
#pragma unroll
        for (int k = 0; k < kLastIds; ++k)
            if (m + 32 * k < m1) f((int)m + 32 * k + lane, m + 32 * k + lane < m1 ? row_of(v[k]) : -1);
    }
}

// A block's rows are every B-th row of the table (B a power of two), so that rows that lie together, as frequent tokens' rows
// do, go to different blocks; the sorted order is that of (row mod B, row / B).
struct Ranges {
    int32_t shift;     // B = 1 << shift blocks
    int32_t R;         // most rows of a block
};
struct Slot {
    int32_t next;      // where the warp's next token of the row goes
    uint32_t lanes;    // of this step: those with a token of the row
};
// dynamic shared memory: slots[kSortWarps][R]
template <typename T>
__global__ void __launch_bounds__(kSortBlock) embed_sort_kernel(const EmbedBwdArgs a, const Ranges by) {
    extern __shared__ __align__(8) Slot slots[];
    __shared__ int scan[kSortWarps];
    __shared__ int below_all;
    const int R = by.R, t = threadIdx.x, lane = t & 31, warp = __shfl_sync(kFull, t >> 5, 0);   // (the same for the warp, for the compiler)
    const unsigned b = blockIdx.x, mask = (1u << by.shift) - 1u, V = (unsigned)a.V;
    for (int i = t; i < kSortWarps * R; i += kSortBlock) slots[i] = Slot{0, 0u};
    if (t == 0) below_all = 0;
    __syncthreads();
    wait_for_primary();
    // a warp has tokens m0 .. m1 - 1, so that the order of the warps is the order of the tokens
    const int64_t per = (a.M + kSortWarps - 1) / kSortWarps, m0 = per * warp, m1 = m0 + per < a.M ? m0 + per : a.M;
    Slot* mine = slots + warp * R;
    int below = 0;
    for_ids<T>(a.ids, m0, m1, lane, [&](int, int id) {
        const unsigned at = (unsigned)id & mask;
        if ((unsigned)id < V) {
            below += at < b;
            if (at == b) atomicAdd(&mine[id >> by.shift].next, 1);
        }
    });
    below = __reduce_add_sync(kFull, below);
    if (lane == 0) atomicAdd(&below_all, below);   // whole numbers: any order gives the same sum
    __syncthreads();
    // counts -> places in the sorted order; a row per thread (R <= kSortBlock)
    int own = 0;
    if (t < R) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) own += slots[w * R + t].next;
    }
    int incl = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    const int all = scan[lane];
    int next = below_all + incl - own + __reduce_add_sync(kFull, lane < warp ? all : 0);
    if (t < R) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = slots[w * R + t].next;
            slots[w * R + t].next = next;
            next += n;
        }
        if (!a.accumulate) a.empty[(int64_t)b * R + t] = own == 0;
    }
    if (b == gridDim.x - 1) {   // behind the last row: the tokens without one
        const int64_t end = (int64_t)below_all + __reduce_add_sync(kFull, all);
        for (int64_t j = end + t; j < a.M; j += kSortBlock) a.sorted[j] = Entry{-1, -1};
    }
    __syncthreads();
    for_ids<T>(a.ids, m0, m1, lane, [&](int m, int id) {
        const bool in = (unsigned)id < V && ((unsigned)id & mask) == b;
        if (!__any_sync(kFull, in)) return;
        // the lanes with the same row, in a word of the row (__match_any_sync takes longer the more rows there are)
        Slot* s = mine + (in ? id >> by.shift : 0);
        if (in) atomicOr(&s->lanes, 1u << lane);
        __syncwarp();
        const Slot v = *s;
        const uint32_t before = v.lanes & ((1u << lane) - 1u);
        __syncwarp();
        if (in) {
            if (before == 0u) *s = Slot{v.next + __popc(v.lanes), 0u};
            a.sorted[v.next + __popc(before)] = Entry{m, id};
        }
        __syncwarp();
    });
}

// ---- backward: sums ----
__device__ __forceinline__ Entry entry_at(const EmbedBwdArgs& a, int64_t j) {
    if (j < 0 || j >= a.M) return Entry{-1, -1};
    const int2 e = *reinterpret_cast<const int2*>(a.sorted + j);
    return Entry{e.x, e.y};
}
// a chunk's float32 row in the workspace: 0 of the row that the chunk before it has begun, 1 of one that goes on behind it
__device__ __forceinline__ float* partial_at(const EmbedBwdArgs& a, int64_t chunk, int which) {
    return a.partial + (2 * chunk + which) * a.C;
}
__device__ __forceinline__ void add_row(const float* p, float (&sum)[8]) {
    const float4 f = reinterpret_cast<const float4*>(p)[0], g = reinterpret_cast<const float4*>(p)[1];
    sum[0] += f.x; sum[1] += f.y; sum[2] += f.z; sum[3] += f.w;
    sum[4] += g.x; sum[5] += g.y; sum[6] += g.z; sum[7] += g.w;
}
__device__ __forceinline__ void store_row(float* p, const float (&sum)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
}
// 16 bytes, or zeros where not `there`.  A predicated load, not a load in a branch: behind a branch the compiler copies the
// loaded words, and every load of a batch waits for the one before it.
__device__ __forceinline__ void load_words_if(uint32_t there, const void* p, uint32_t (&w)[4]) {
    w[0] = w[1] = w[2] = w[3] = 0u;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "@p ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3])
        : "l"(p), "r"(there));
}
// the table's row from the sum of its tokens; old: what it held
template <bool kAdd>
__device__ __forceinline__ void store_table(const EmbedBwdArgs& a, int row, int64_t col, const float (&sum)[8], const uint32_t (&old)[4]) {
    float x[8];
    uint32_t w[4];
    if constexpr (kAdd) unpack(old, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kAdd ? fmaf(sum[i], a.scale, x[i]) : sum[i] * a.scale;
    pack(x, w);
    *reinterpret_cast<uint4*>(a.dtable + (int64_t)row * a.C + col) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A block is one warp, so that all that its lanes have in common is so for the compiler too: addresses of entries, counts and
// branches stay in uniform registers (16411 x 2048, added: 35.6 us; in blocks of two, four and eight warps 39.4, 39.3 and 40.0).
template <bool kAdd, int kDeep>
__global__ void __launch_bounds__(32, kDeep == kDeepest ? kResidentFew : kResident) embed_chunks_kernel(const EmbedBwdArgs a, int slices) {
    const int64_t unit = blockIdx.x, chunk = unit / slices;
    const int lane = threadIdx.x;
    wait_for_primary();
    const Entry e = entry_at(a, chunk * kChunk + lane);
    const int before = entry_at(a, chunk * kChunk - 1).row, behind = entry_at(a, (chunk + 1) * kChunk).row;
    int next = __shfl_down_sync(kFull, e.row, 1);
    if (lane == 31) next = behind;
    const uint32_t here = __ballot_sync(kFull, e.row >= 0), ends = __ballot_sync(kFull, e.row >= 0 && e.row != next);
    const int64_t col = (unit - chunk * slices) * kSlice + 8 * lane;
    const bool ok = col < a.C;
    const int64_t from = ok ? col : 0;
    const bool begun = before >= 0 && before == __shfl_sync(kFull, e.row, 0);
    uint32_t mine = ends;                      // the tokens whose rows begin and end in this chunk
    if (begun) mine &= mine - 1u;
    float sum[8] = {};
#pragma unroll 1
    for (int k0 = 0; k0 < kChunk; k0 += kDeep) {
        if ((here >> k0 & 1u) == 0u) break;    // behind the last token
        uint32_t w[kDeep][4], old[kAdd ? kDeep : 1][4];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int m = __shfl_sync(kFull, e.token, k0 + k);
            load_words_if(here >> (k0 + k) & 1u, a.dout + (int64_t)m * a.C + from, w[k]);
        }
        if constexpr (kAdd) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                const int row = __shfl_sync(kFull, e.row, k0 + k);
                load_words_if(mine >> (k0 + k) & 1u, a.dtable + (int64_t)row * a.C + from, old[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int row = __shfl_sync(kFull, e.row, k0 + k);
            if ((here >> (k0 + k) & 1u) == 0u) break;
            float x[8];
            unpack(w[k], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += x[i];
            if (ends >> (k0 + k) & 1u) {
                if (ok) {
                    if (mine >> (k0 + k) & 1u) store_table<kAdd>(a, row, col, sum, old[kAdd ? k : 0]);
                    else store_row(partial_at(a, chunk, 0) + col, sum);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
            }
        }
    }
    // a row that goes on: the whole chunk of one that the chunk before has begun, or the beginning of one
    if (here == kFull && (ends >> 31) == 0u && ok) store_row(partial_at(a, chunk, begun && ends == 0u ? 0 : 1) + col, sum);
}

// Of the chunks behind `chunk`, how many begin with a token of `row` (they are consecutive), if the first 64 do; the whole
// warp.
__device__ __noinline__ int64_t chunks_of_row(const EmbedBwdArgs& a, int row, int64_t chunk, int lane) {
    int64_t n = 64, step = 1;
    uint32_t in;
    auto probe = [&] { return __ballot_sync(kFull, entry_at(a, (chunk + n + step * (lane + 1)) * kChunk).row == row); };
    // in steps that grow 32 times each, as far as all 32 probes are in the row
    while ((in = probe()) == kFull) {
        n += 32 * step;
        step *= 32;
    }
    n += step * (__ffs(~in) - 1);
    while (step > 1) {   // the first chunk that is not lies within `step` of chunk + n
        step /= 32;
        in = probe();
        n += step * (in == kFull ? 32 : __ffs(~in) - 1);
    }
    return n;
}

// Zeros over the rows without a token: kFill rows per block, one thread for each, whose copies read
// the same zeros in shared memory.
__device__ __forceinline__ void fill_rows(const EmbedBwdArgs& a, const Ranges& by, int64_t block, float* zeros) {
    for (int i = threadIdx.x; i < kZeroBytes / 4; i += blockDim.x) zeros[i] = 0.0f;
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the copies read them
    __syncthreads();
    const int64_t row = block * kFill + threadIdx.x;
    if (threadIdx.x >= kFill || row >= a.V || a.empty[(row & ((1 << by.shift) - 1)) * by.R + (row >> by.shift)] == 0) return;
    char* p = reinterpret_cast<char*>(a.dtable + row * a.C);
    for (int64_t n = 2 * a.C; n > 0; n -= kZeroBytes, p += kZeroBytes)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(p),
                     "r"((uint32_t)__cvta_generic_to_shared(zeros)), "r"((uint32_t)(n < kZeroBytes ? n : kZeroBytes))
                     : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// The first `fills` blocks fill.  Of the others each has a chunk and 256 columns, and its warps add up a row's shares.
template <bool kAdd>
__global__ void __launch_bounds__(32 * teams_of(kAdd)) embed_join_kernel(const EmbedBwdArgs a, int slices, const Ranges by, unsigned fills) {
    constexpr int kTeams = teams_of(kAdd);
    __shared__ __align__(16) float part[kAdd ? (kTeams - 1) * kSlice : kZeroBytes / 4];
    wait_for_primary();
    if (!kAdd && blockIdx.x < fills) {
        fill_rows(a, by, blockIdx.x, part);
        return;
    }
    const int64_t block = blockIdx.x - fills, chunk = block / slices;
    const int lane = threadIdx.x & 31, team = threadIdx.x >> 5;
    // a row that begins in this chunk and goes on behind it: in n chunks (all of these loads at once)
    const int64_t last = chunk * kChunk + kChunk - 1;
    const int near = entry_at(a, last + 1 + kChunk * lane).row, far = entry_at(a, last + 1 + kChunk * (32 + lane)).row;
    const int row = entry_at(a, last).row, first = entry_at(a, last - kChunk + 1).row, before = entry_at(a, last - kChunk).row;
    if (row < 0 || (first == row && before == row)) return;   // the same for the whole block
    const uint32_t in = __ballot_sync(kFull, near == row), more = __ballot_sync(kFull, far == row);
    if (in == 0u) return;
    const int64_t n = in != kFull ? __popc(in) : more != kFull ? 32 + __popc(more) : chunks_of_row(a, row, chunk, lane);
    const int64_t col = (block - chunk * slices) * kSlice + 8 * lane;
    const bool ok = col < a.C;
    uint32_t old[4];
    load_words_if(kAdd && ok && team == 0, a.dtable + (int64_t)row * a.C + (ok ? col : 0), old);
    float sum[8] = {};
    if (ok) {
        if (team == 0) add_row(partial_at(a, chunk, 1) + col, sum);
#pragma unroll 8
        for (int64_t i = 1 + team; i <= n; i += kTeams) add_row(partial_at(a, chunk + i, 0) + col, sum);
    }
    if (team > 0) store_row(part + (team - 1) * kSlice + 8 * lane, sum);
    __syncthreads();
    if (team > 0 || !ok) return;
#pragma unroll
    for (int t = 0; t < kTeams - 1; ++t) add_row(part + t * kSlice + 8 * lane, sum);
    store_table<kAdd>(a, row, col, sum, old);
}

}  // namespace

int64_t embed_chunks(int64_t M) { return (M + kChunk - 1) / kChunk; }

cudaError_t launch_embed_fwd(const EmbedFwdArgs& all, cudaStream_t s) {
    const int64_t nc = all.C / 16, slab = (((int64_t)1 << 31) - 2 * kBlock) / nc;   // a launch's pieces are counted in 31 bits
    const int per = all.M * nc > kOneEach ? 2 : 1;
    const Divider by = divider((uint32_t)nc);
    const bool wide = aligned32(all.table) && aligned32(all.out);
    for (int64_t m = 0; m < all.M; m += slab) {
        EmbedFwdArgs a = all;
        a.M = all.M - m < slab ? all.M - m : slab;
        a.ids = static_cast<const char*>(all.ids) + m * (all.wide ? 8 : 4);
        a.out += m * a.C;
        const cudaError_t e = launch_next(per == 2 ? embed_fwd_kernel<2> : embed_fwd_kernel<1>,
                                          (unsigned)((a.M * nc + per * kBlock - 1) / (per * kBlock)), kBlock, 0, s, a, by, wide);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

namespace {
Ranges ranges_of(int64_t V) {
    Ranges by{7, 0};
    while (((V - 1) >> by.shift) + 1 > kMaxRange) ++by.shift;
    by.R = (int32_t)(((V - 1) >> by.shift) + 1);
    return by;
}
}  // namespace

int64_t embed_flags(int64_t V) {
    const Ranges by = ranges_of(V);
    return (int64_t)by.R << by.shift;
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, cudaStream_t s) {
    const Ranges by = ranges_of(a.V);
    const size_t smem = (size_t)kSortWarps * (size_t)by.R * sizeof(Slot);
    auto* const sort = a.wide ? embed_sort_kernel<int64_t> : embed_sort_kernel<int32_t>;
    // the most of any table, not this one's: another thread, whose table is another one, may set it before this one launches
    cudaError_t e = cudaFuncSetAttribute(sort, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortWarps * kMaxRange * (int)sizeof(Slot));
    if (e != cudaSuccess) return e;
    e = launch_next(sort, 1u << by.shift, kSortBlock, smem, s, a, by);
    if (e != cudaSuccess) return e;
    const int slices = (int)((a.C + kSlice - 1) / kSlice);
    const int64_t chunks = embed_chunks(a.M);
    auto* const sums = chunks * slices <= kFewUnits
                           ? (a.accumulate ? embed_chunks_kernel<true, kDeepest> : embed_chunks_kernel<false, kDeepest>)
                           : (a.accumulate ? embed_chunks_kernel<true, kDeep> : embed_chunks_kernel<false, kDeep>);
    e = launch_next(sums, (unsigned)(chunks * slices), 32, 0, s, a, slices);
    if (e != cudaSuccess) return e;
    const unsigned fills = a.accumulate ? 0u : (unsigned)((a.V + kFill - 1) / kFill);
    const int64_t joins = chunks > 1 ? chunks * slices : 0;   // one chunk: no row goes on behind it
    if (fills + joins == 0) return cudaSuccess;
    return launch_next(a.accumulate ? embed_join_kernel<true> : embed_join_kernel<false>, (unsigned)(fills + joins),
                       32 * teams_of(a.accumulate), 0, s, a, slices, by, fills);
}

}  // namespace coat
