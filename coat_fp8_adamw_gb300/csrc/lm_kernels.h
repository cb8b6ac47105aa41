// lm_kernels.h -- internal launch interface between the C ABI (lm_abi.cu) and the kernels of the operators at the two ends
// of a language model (cross entropy of a linear layer, embedding) and of dropout.  Not part of the public header.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace coat {

struct EmbedFwdArgs {
    const uint16_t* table;     // V x C bf16
    const void* ids;           // M indexes of 4 or 8 bytes
    int32_t wide;              // 8 bytes
    float scale;
    int64_t M, V, C;
    uint16_t* out;             // M x C bf16
};

// A token of the sorted order: its place among the M tokens and its row of the table (-1: none).
struct Entry {
    int32_t token, row;
};
struct EmbedBwdArgs {
    const uint16_t* dout;      // M x C bf16
    const void* ids;
    int32_t wide;
    float scale;
    int64_t M, V, C;
    int32_t accumulate;
    uint16_t* dtable;          // V x C bf16
    Entry* sorted;             // M
    float* partial;            // embed_chunks(M) x C
};
int64_t embed_chunks(int64_t M);

struct DropoutArgs {
    const uint16_t* x;         // n bf16
    const uint16_t* residual;  // n bf16, or null
    const uint64_t* rng;       // key, and the upper half of the counter
    uint32_t drop;             // of 65536 draws, those that drop an element
    float scale;               // 65536 / (65536 - drop)
    int64_t n;
    uint16_t* y;               // n bf16
};

cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, cudaStream_t s);
cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, cudaStream_t s);
cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s);

}  // namespace coat
