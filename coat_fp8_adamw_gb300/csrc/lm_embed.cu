// lm_embed.cu -- embedding lookup with a scale, and the gradient of the table from sorted tokens.
//
//   forward   out[m] = RN(scale table[ids[m]]); a negative id gives zeros, one past the table NaN
//   backward  dtable[v] = RN(scale sum over m with ids[m] = v of dout[m] (+ dtable[v]))
//
// Backward in three kernels, sums in float32 and in a fixed order (that of the tokens, chunk by chunk):
//   sort    the tokens by their row of the table, stably: block b has a range of rows of its own, walks all M ids (they
//           are few bytes) and counts what lies below its range, which is where its part of the sorted order begins, so
//           that no block waits for another.  Rows without a token are written as zeros here, unless the gradient is
//           added to what is there.
//   chunks  the sorted order in chunks of 32 tokens: those of one row alone are summed into the workspace, so that the
//           work of a row with many tokens (text has some that are a tenth of all) goes to many warps;
//   rows    a warp for each sorted token and 512 columns: the first token of a row adds up the row's tokens and chunks.
#include <cstdint>

#include "ckpt_kernels.h"
#include "divide.h"
#include "lm_device.cuh"
#include "lm_kernels.h"

namespace coat {

namespace {

using namespace ckpt;
using lm::index_at;

constexpr int kBlock = 256;
constexpr int kWarps = kBlock / 32;
constexpr int kChunk = 32;            // tokens of a chunk: a warp's lanes hold one's entries
constexpr int kSlice = 512;           // columns of a warp: 16 per lane
constexpr int kSortBlock = 1024;
constexpr int kSortWarps = kSortBlock / 32;
constexpr int kMaxRange = 1024;       // rows of a sorting block: their counts take 128 KB of shared memory

// ---- forward ----
__global__ void __launch_bounds__(kBlock) embed_fwd_kernel(const EmbedFwdArgs a, const Divider nc, bool wide) {
    const uint32_t total = (uint32_t)a.M * nc.d, i = blockIdx.x * kBlock + threadIdx.x;
    wait_for_primary();
    if (i >= total) return;
    const uint32_t m = divide(i, nc);
    const int64_t col = (int64_t)(i - m * nc.d) * 16, id = index_at(a.ids, a.wide, m);
    uint32_t w[8] = {};
    if (id >= 0 && id < a.V) {
        float x[16];
        load_words8(a.table + id * a.C + col, wide, w);
        unpack(w, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= a.scale;
        pack(x, w);
    } else if (id >= a.V) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 0x7FFF7FFFu;
    }
    store_words8(a.out + (int64_t)i * 16, wide, w);
}

// ---- backward: sort ----
// dynamic shared memory: counts[kSortWarps][R], then totals[R]
__global__ void __launch_bounds__(kSortBlock) embed_sort_kernel(const EmbedBwdArgs a, int R, bool wide) {
    extern __shared__ int counts[];
    __shared__ int scan[kSortWarps];
    __shared__ int below_all;
    int* totals = counts + kSortWarps * R;
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int64_t v0 = (int64_t)blockIdx.x * R, v1 = v0 + R < a.V ? v0 + R : a.V;
    const int rows = (int)(v1 - v0);
    for (int i = t; i < kSortWarps * R; i += kSortBlock) counts[i] = 0;
    if (t == 0) below_all = 0;
    __syncthreads();
    wait_for_primary();
    // a warp has tokens m0 .. m1 - 1, so that the order of the warps is the order of the tokens
    const int64_t per = (a.M + kSortWarps - 1) / kSortWarps, m0 = per * warp, m1 = m0 + per < a.M ? m0 + per : a.M;
    int* mine = counts + warp * R;
    int below = 0;
    for (int64_t m = m0 + lane; m < m1; m += 32) {
        const int64_t id = index_at(a.ids, a.wide, m);
        below += id >= 0 && id < v0;
        if (id >= v0 && id < v1) atomicAdd(mine + (id - v0), 1);
    }
    for (int off = 16; off > 0; off >>= 1) below += __shfl_xor_sync(kFull, below, off);
    if (lane == 0) atomicAdd(&below_all, below);   // whole numbers: any order gives the same sum
    __syncthreads();
    // counts -> where the warp's first token of the row goes, from the row's start; totals: tokens of the row
    for (int r = t; r < rows; r += kSortBlock) {
        int sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = counts[w * R + r];
            counts[w * R + r] = sum;
            sum += n;
        }
        totals[r] = sum;
    }
    __syncthreads();
    // rows' starts: R <= kSortBlock, a row per thread
    const int own = t < rows ? totals[t] : 0;
    int incl = own;
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int start = below_all + incl - own;
    for (int w = 0; w < warp; ++w) start += scan[w];
    if (t < rows) {
        for (int w = 0; w < kSortWarps; ++w) counts[w * R + t] += start;
    }
    if (blockIdx.x == gridDim.x - 1) {   // behind the last row: the tokens without one
        int64_t end = below_all;
        for (int w = 0; w < kSortWarps; ++w) end += scan[w];
        for (int64_t j = end + t; j < a.M; j += kSortBlock) a.sorted[j] = Entry{-1, -1};
    }
    __syncthreads();
    for (int64_t m = m0; m < m1; m += 32) {
        const int64_t id = m + lane < m1 ? index_at(a.ids, a.wide, m + lane) : -1;
        const bool in = id >= v0 && id < v1;
        const uint32_t some = __ballot_sync(kFull, in);
        if (in) {
            const int r = (int)(id - v0);
            const uint32_t same = __match_any_sync(some, r), before = same & ((1u << lane) - 1u);
            const int at = mine[r] + __popc(before);
            __syncwarp(some);
            if (before == 0) mine[r] += __popc(same);
            a.sorted[at] = Entry{(int32_t)(m + lane), (int32_t)id};
        }
        __syncwarp();
    }
    if (!a.accumulate) {
        const uint32_t zero[8] = {};
        for (int r = warp; r < rows; r += kSortWarps) {
            if (totals[r] != 0) continue;
            uint16_t* p = a.dtable + (v0 + r) * a.C;
            for (int64_t c = 16 * lane; c < a.C; c += kSlice) store_words8(p + c, wide, zero);
        }
    }
}

// ---- backward: sums ----
__device__ __forceinline__ Entry entry_at(const EmbedBwdArgs& a, int64_t j) {
    if (j < 0 || j >= a.M) return Entry{-1, -1};
    const int2 e = *reinterpret_cast<const int2*>(a.sorted + j);
    return Entry{e.x, e.y};
}
// adds 16 columns from col of the tokens that the first n lanes hold
__device__ __forceinline__ void add_tokens(const EmbedBwdArgs& a, int token, int n, int64_t col, bool wide, float (&sum)[16]) {
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const int m = __shfl_sync(kFull, token, k);
        uint32_t w[8];
        float x[16];
        load_words8(a.dout + (int64_t)m * a.C + col, wide, w);
        unpack(w, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] += x[e];
    }
}
__device__ __forceinline__ void add_partial(const float* p, float (&sum)[16]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 f = reinterpret_cast<const float4*>(p)[q];
        sum[4 * q] += f.x;
        sum[4 * q + 1] += f.y;
        sum[4 * q + 2] += f.z;
        sum[4 * q + 3] += f.w;
    }
}

__global__ void __launch_bounds__(kBlock) embed_chunks_kernel(const EmbedBwdArgs a, int slices, bool wide) {
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), chunk = unit / slices;
    const int lane = threadIdx.x & 31;
    wait_for_primary();
    if ((chunk + 1) * kChunk > a.M) return;
    const Entry e = entry_at(a, chunk * kChunk + lane);
    if (__shfl_sync(kFull, e.row, 0) != __shfl_sync(kFull, e.row, 31) || __shfl_sync(kFull, e.row, 31) < 0) return;
    const int64_t col = (unit - chunk * slices) * kSlice + 16 * lane;
    const bool ok = col < a.C;
    float sum[16] = {};
    add_tokens(a, e.token, kChunk, ok ? col : 0, wide, sum);
    if (!ok) return;
    float4* p = reinterpret_cast<float4*>(a.partial + chunk * a.C + col);
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]);
}

__global__ void __launch_bounds__(kBlock) embed_rows_kernel(const EmbedBwdArgs a, int slices, bool wide) {
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), j = unit / slices;
    const int lane = threadIdx.x & 31;
    wait_for_primary();
    if (j >= a.M) return;
    Entry e = entry_at(a, j + lane);
    const int row = __shfl_sync(kFull, e.row, 0);
    if (row < 0 || entry_at(a, j - 1).row == row) return;   // the same for the whole warp
    const int64_t col = (unit - j * slices) * kSlice + 16 * lane;
    const bool ok = col < a.C;
    float sum[16] = {};
    // the tokens up to the end of the chunk that the row begins in, unless it begins with the chunk and fills it
    int64_t at = j;
    const int rest = kChunk - (int)(j % kChunk);
    int run = __ffs(~__ballot_sync(kFull, e.row == row));   // 1 + the tokens of the row from j on, 0: all 32
    run = run == 0 ? 32 : run - 1;
    bool more = run >= rest;
    if (rest < kChunk || run < kChunk) {
        add_tokens(a, e.token, run < rest ? run : rest, ok ? col : 0, wide, sum);
        at = j + rest;
    }
    // whole chunks
    while (more) {
        const int64_t chunk = at / kChunk;
        const uint32_t whole = __ballot_sync(kFull, entry_at(a, at + (int64_t)kChunk * lane + kChunk - 1).row == row);
        int n = __ffs(~whole);
        n = n == 0 ? 32 : n - 1;
        if (ok)
            for (int k = 0; k < n; ++k) add_partial(a.partial + (chunk + k) * a.C + col, sum);
        at += (int64_t)n * kChunk;
        more = n == 32;
        if (!more) {   // the tokens of the chunk that the row ends in
            e = entry_at(a, at + lane);
            const uint32_t here = __ballot_sync(kFull, e.row == row);
            add_tokens(a, e.token, __popc(here), ok ? col : 0, wide, sum);
        }
    }
    if (!ok) return;
    uint16_t* p = a.dtable + (int64_t)row * a.C + col;
    uint32_t w[8];
    if (a.accumulate) {
        float x[16];
        load_words8(p, wide, w);
        unpack(w, x);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = fmaf(sum[i], a.scale, x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] *= a.scale;
    }
    pack(sum, w);
    store_words8(p, wide, w);
}

}  // namespace

int64_t embed_chunks(int64_t M) { return M / kChunk; }

cudaError_t launch_embed_fwd(const EmbedFwdArgs& all, cudaStream_t s) {
    const int64_t nc = all.C / 16, slab = (((int64_t)1 << 31) - kBlock) / nc;   // a launch's chunks are counted in 31 bits
    const Divider by = divider((uint32_t)nc);
    const bool wide = aligned32(all.table) && aligned32(all.out);
    for (int64_t m = 0; m < all.M; m += slab) {
        EmbedFwdArgs a = all;
        a.M = all.M - m < slab ? all.M - m : slab;
        a.ids = static_cast<const char*>(all.ids) + m * (all.wide ? 8 : 4);
        a.out += m * a.C;
        const cudaError_t e = launch_next(embed_fwd_kernel, (unsigned)((a.M * nc + kBlock - 1) / kBlock), kBlock, 0, s, a, by, wide);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, cudaStream_t s) {
    const int sms = device_sms();
    if (sms < 1) return cudaErrorInvalidConfiguration;
    const bool wide = aligned32(a.dout) && aligned32(a.dtable);
    int64_t R = (a.V + sms - 1) / sms;
    R = R > kMaxRange ? kMaxRange : R;
    const size_t smem = (size_t)(kSortWarps + 1) * (size_t)R * sizeof(int);
    cudaError_t e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_next(embed_sort_kernel, (unsigned)((a.V + R - 1) / R), kSortBlock, smem, s, a, (int)R, wide);
    if (e != cudaSuccess) return e;
    const int slices = (int)((a.C + kSlice - 1) / kSlice);
    if (embed_chunks(a.M) > 0) {
        e = launch_next(embed_chunks_kernel, (unsigned)((embed_chunks(a.M) * slices + kWarps - 1) / kWarps), kBlock, 0, s, a, slices, wide);
        if (e != cudaSuccess) return e;
    }
    return launch_next(embed_rows_kernel, (unsigned)((a.M * slices + kWarps - 1) / kWarps), kBlock, 0, s, a, slices, wide);
}

}  // namespace coat
