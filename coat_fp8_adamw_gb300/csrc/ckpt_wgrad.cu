// ckpt_wgrad.cu -- the weight gradient of a linear layer from the 8-bit checkpoint
// of its input (COAT review page, section 3: FP8 activations kept for the
// backward pass).
//
//   dW[n, k] = c[k] sum_m dY[m, n] r[m] S[m, k / G] E4M3(q[m, k])
//
// r (per token) and c (per input column) are optional factors: with r = 1 / rms
// and c = the norm's weight, the checkpoint of a norm's input serves the
// linear layer behind the norm too.
#include <cstdint>

#include "ckpt_device.cuh"
#include "ckpt_kernels.h"

namespace coat {

namespace {

using namespace ckpt;

constexpr int kT = 64;    // tile of dW, both ways
constexpr int kR = 16;    // tokens per step

// 256 threads, 4 x 4 outputs each
__global__ void __launch_bounds__(256) wgrad_kernel(const WgradArgs a) {
    __shared__ float sy[kR][kT], sx[kR][kT];
    const int64_t n0 = (int64_t)blockIdx.y * kT, k0 = (int64_t)blockIdx.x * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t m0 = 0; m0 < a.M; m0 += kR) {
        for (int i = threadIdx.x; i < kR * kT; i += 256) {
            const int64_t m = m0 + i / kT, n = n0 + i % kT, k = k0 + i % kT;
            sy[i / kT][i % kT] = m < a.M && n < a.N ? __uint_as_float((uint32_t)a.dy[m * a.dy_ld + n] << 16) : 0.0f;
            float x = 0.0f;
            if (m < a.M && k < a.K) {
                float v[8];
                decode8(make_uint2(a.q[m * a.K + k], 0u), v);
                x = v[0] * a.scale[m * (a.K / a.G) + k / a.G];
                if (a.row_scale) x *= a.row_scale[m];
            }
            sx[i / kT][i % kT] = x;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sy[r][ty * 4 + i], sx[r][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
            if (n < a.N && k < a.K) a.dw[n * a.K + k] = bf16_bits(a.col_scale ? acc[i][j] * a.col_scale[k] : acc[i][j]);
        }
}

}  // namespace

size_t wgrad_workspace(int64_t, int64_t, int64_t, int) { return 0; }

cudaError_t launch_wgrad(const WgradArgs& a, cudaStream_t s) {
    wgrad_kernel<<<dim3((unsigned)((a.K + kT - 1) / kT), (unsigned)((a.N + kT - 1) / kT)), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace coat
