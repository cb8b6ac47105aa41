// ckpt_kernels.h -- internal launch interface between the C ABI (ckpt_abi.cu)
// and the kernels of the operators with 8-bit activation checkpoints.  Not part
// of the public header.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace coat {

// Launch a kernel that may start when the one before it in the stream has no block left to run, or allows it earlier;
// every thread waits for that kernel's end (wait_for_primary) before its first access to global memory.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 blocks, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = blocks;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// whether a 256-bit access may start there
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

struct NormFwdArgs {
    const uint16_t* x;         // M x N bf16
    const uint16_t* residual;  // M x N bf16, or null
    const float* weight;       // N
    float eps;
    int64_t M, N;
    int32_t G;
    uint16_t* h;               // M x N bf16: x + residual (null without a residual)
    uint16_t* y;               // M x N bf16
    uint8_t* q;                // M x N codes of the norm's input
    float* scale;              // M x N/G
    float* rstd;               // M
};

struct NormBwdArgs {
    const uint16_t* dy;        // M x N bf16
    const uint8_t* q;          // M x N codes
    const float* scale;        // M x N/G
    const float* rstd;         // M
    const float* weight;       // N
    const uint16_t* dresidual; // M x N bf16, or null
    int64_t M, N;
    int32_t G;
    uint16_t* dx;              // M x N bf16
    uint16_t* dweight;         // N bf16
    float* partial;            // norm_bwd_partials(...) x N
};

struct SwigluFwdArgs {
    const uint16_t* gate;      // M rows of N bf16, ld apart
    const uint16_t* up;
    int64_t ld;
    int64_t M, N;
    int32_t G;
    uint16_t* h;               // M x N bf16
    uint8_t* gate_q;           // M x N codes
    float* gate_scale;         // M x N/G
    uint8_t* up_q;
    float* up_scale;
};

struct SwigluBwdArgs {
    const uint16_t* dh;        // M x N bf16
    const uint8_t* gate_q;
    const float* gate_scale;
    const uint8_t* up_q;
    const float* up_scale;
    int64_t M, N;
    int32_t G;
    uint16_t* dgate;           // M rows of N bf16, ld apart
    uint16_t* dup;
    int64_t ld;
    uint8_t* h_q;              // M x N codes of silu(gate) up, or null
    float* h_scale;            // M x N/G, or null
};

// One of the two sides (queries, keys) of the head norm; H = 0: no such side.
struct HeadSide {
    const uint16_t* in;        // forward: x (rows ld apart); backward: dy, contiguous
    uint16_t* out;             // forward: y, contiguous; backward: dx (rows ld apart)
    int64_t ld;
    int32_t H;
    const float* weight;       // D
    uint8_t* codes;            // M x H x D (read in the backward pass)
    float* scale;              // M x H x D/G
    float* rstd;               // M x H
    uint16_t* dweight;         // D bf16 (backward only)
};
struct QkArgs {
    HeadSide q, k;
    const float* cos;          // max_pos x rot/2
    const float* sin;
    const int32_t* positions;  // M
    int64_t M, max_pos;
    int32_t D, rot, G;
    int32_t interleaved;
    float eps;
    float* partial;            // backward only
};

struct WgradArgs {
    const uint16_t* dy;        // M rows of N bf16, dy_ld apart
    int64_t dy_ld;
    const uint8_t* q;          // M x K codes
    const float* scale;        // M x K/G
    const float* row_scale;    // M, or null
    const float* col_scale;    // K, or null
    int64_t M, N, K;
    int32_t G;
    uint16_t* dw;              // N x K bf16
    float* partial;
};

constexpr int64_t kNormMaxN = 16384;   // columns of a normalised row

int device_sms();
int64_t norm_bwd_partials(int64_t M, int64_t N, int sms);
int64_t qk_bwd_partials(int sms);
size_t wgrad_workspace(int64_t M, int64_t N, int64_t K, int sms);

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s);
cudaError_t launch_swiglu_fwd(const SwigluFwdArgs& a, cudaStream_t s);
cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s);
cudaError_t launch_qk_fwd(const QkArgs& a, cudaStream_t s);
cudaError_t launch_qk_bwd(const QkArgs& a, cudaStream_t s);
cudaError_t launch_wgrad(const WgradArgs& a, cudaStream_t s);
// bounded waits that gave up in the kernels of ckpt_wgrad.cu and ckpt_norm.cu, on the current device
cudaError_t read_wgrad_wait_timeouts(unsigned long long* out, bool reset);
cudaError_t read_norm_wait_timeouts(unsigned long long* out, bool reset);
// out[c] = bf16(sum over p of partial[p * N + c]), for one or two sums (out null or P = 0: none); launched as a
// dependent of the kernel before it in the stream, which writes the partial sums
struct ColumnSum {
    const float* partial;
    int64_t P;
    uint16_t* out;
};
cudaError_t launch_column_sums(const ColumnSum& first, const ColumnSum& second, int64_t N, cudaStream_t s);

}  // namespace coat
