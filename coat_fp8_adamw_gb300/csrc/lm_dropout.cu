// lm_dropout.cu -- dropout whose mask is drawn where it is needed and stored nowhere (forward and backward), with an
// optional residual addition.
//
//   y[i] = keep[i] x[i] 65536 / (65536 - T) (+ residual[i]),  keep[i] = draw[i] >= T,  T = round(65536 p), halves up
//
// draw[i] is 16 bits of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011): counter (i / 8, rng[1]), key rng[0]; the four words hold eight draws, the low half of each word first.  The
// backward pass draws the same bits again.  Sixteen bits, not 32, of a word per element: the generator's ten rounds take
// two wide products each, and with a word per element they would take as long as the memory accesses do; the price is
// that p goes in steps of 2^-16, and the scale is the exact one for the step.
// rng lies in device memory, so that a captured graph draws other bits whenever what is there has changed.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"
#include "lm_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

// threads: 33 x 2048 1.2 us, 1000 x 4096 with a residual 3.7 (256: 1.4, 3.9; 512: 1.9, 4.5); larger tensors take the same
constexpr int kBlock = 128;

struct Draws {
    uint32_t w[4];
};
__device__ __forceinline__ Draws philox(uint64_t index, uint64_t offset, uint64_t key) {
    uint32_t c0 = (uint32_t)index, c1 = (uint32_t)(index >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)q;
        c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Draws{{c0, c1, c2, c3}};
}

// an element: dropped ones do not count, whatever they hold; draw in the upper half of the word, whatever the lower one holds
__device__ __forceinline__ float kept(float x, uint32_t draw, const DropoutArgs& a) {
    return draw >= a.drop << 16 ? x * a.scale : 0.0f;
}

template <bool kResidual>
__global__ void __launch_bounds__(kBlock) dropout_kernel(const DropoutArgs a, bool wide) {
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x, at = 16 * i;
    wait_for_primary();
    if (at >= a.n) return;
    // through L1: all threads read the same 16 bytes (a load of each thread from L2 alone, 8192 x 4096 with a residual: 45 us)
    uint64_t key, offset;
    asm volatile("ld.global.v2.u64 {%0, %1}, [%2];" : "=l"(key), "=l"(offset) : "l"(a.rng));
    if (at + 16 <= a.n) {
        uint32_t xv[8], rv[8], yv[8];
        load_words8(a.x + at, wide, xv);
        if constexpr (kResidual) load_words8(a.residual + at, wide, rv);
        const Draws d[2] = {philox(2 * (uint64_t)i, offset, key), philox(2 * (uint64_t)i + 1, offset, key)};
        float x[16], r[16];
        unpack(xv, x);
        if constexpr (kResidual) unpack(rv, r);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const uint32_t w = d[e >> 3].w[(e & 7) >> 1];
            x[e] = kept(x[e], w << 16, a);
            x[e + 1] = kept(x[e + 1], w, a);
            if constexpr (kResidual) {
                x[e] += r[e];
                x[e + 1] += r[e + 1];
            }
        }
        pack(x, yv);
        store_words8(a.y + at, wide, yv);
        return;
    }
    for (int64_t j = at; j < a.n; ++j) {   // the last elements, fewer than sixteen
        const Draws d = philox((uint64_t)j >> 3, offset, key);
        float y = kept(__uint_as_float((uint32_t)a.x[j] << 16), d.w[(j & 7) >> 1] << (16 * (~j & 1)), a);
        if constexpr (kResidual) y += __uint_as_float((uint32_t)a.residual[j] << 16);
        a.y[j] = bf16_bits(y);
    }
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s) {
    const bool wide = aligned32(a.x) && aligned32(a.y) && (!a.residual || aligned32(a.residual));
    const int64_t blocks = (a.n + 16 * kBlock - 1) / (16 * kBlock);
    return launch_next(a.residual ? dropout_kernel<true> : dropout_kernel<false>, (unsigned)blocks, kBlock, 0, s, a, wide);
}

}  // namespace coat
