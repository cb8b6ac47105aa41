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
    float* partial;            // embed_chunks(M) x 2 x C
    uint8_t* empty;            // embed_flags(V): rows without a token
};
int64_t embed_chunks(int64_t M);
int64_t embed_flags(int64_t V);

struct DropoutArgs {
    const uint16_t* x;         // n bf16
    const uint16_t* residual;  // n bf16, or null
    const uint64_t* rng;       // key, and the upper half of the counter
    uint32_t drop;             // of 65536 draws, those that drop an element
    float scale;               // 65536 / (65536 - drop)
    int64_t n;
    uint16_t* y;               // n bf16
};

struct LceFwdArgs {
    const uint16_t* x;         // M rows of C bf16, x_ld apart
    int64_t x_ld;
    const uint16_t* weight;    // V x C bf16
    const void* targets;       // M indexes of 4 or 8 bytes
    int32_t wide;              // 8 bytes
    int64_t M, V, C;
    float* loss;               // M
    float* lse;                // M
    void* stats;               // lce_stats_bytes(M, V)
};
struct LceBwdArgs {
    const uint16_t* x;
    int64_t x_ld;
    const uint16_t* weight;
    const void* targets;
    int32_t wide;
    const float* lse;          // M
    const float* dloss;        // M
    const float* dlse;         // M, or null
    int64_t M, V, C;
    int64_t piece;             // rows of the weight at once
    uint16_t* dx;              // M x C bf16
    uint16_t* dweight;         // V x C bf16
    uint16_t* dz;              // M x lce_piece_ld(piece, V) bf16
    uint16_t* xt;              // C x lce_xt_ld(M) bf16: x transposed
    float* unit;               // 4 floats
    float* sums;               // lce_sums(...): of products in several parts or pieces
};
// Of a piece's gradient of the logits, unless the caller says how wide a piece is: the fewest pieces within it, since every one
// more costs time and saves workspace (8192 x 32000 x 4096 in 1 / 2 / 3 / 4 / 8 pieces: 3.59 / 3.65 / 3.74 / 3.92 / 4.07 ms with 564 /
// 444 / 360 / 320 / 256 MiB; 1000 x 100000 x 128 in 1 / 2 / 4: 138 / 154 / 188 us with 197 / 102 / 56 MiB).
constexpr int64_t kLceDzBytes = 512 << 20;
int64_t lce_piece(int64_t M, int64_t V, int64_t piece);
int64_t lce_piece_ld(int64_t piece, int64_t V);
int64_t lce_xt_ld(int64_t M);
int64_t lce_dx_sums(int64_t M, int64_t V, int64_t C, int64_t piece);
int64_t lce_sums(int64_t M, int64_t V, int64_t C, int64_t piece);
size_t lce_stats_bytes(int64_t M, int64_t V);

cudaError_t launch_lce_fwd(const LceFwdArgs& a, cudaStream_t s);
cudaError_t launch_lce_bwd(const LceBwdArgs& a, cudaStream_t s);
// bounded waits that gave up in the kernels of lm_lce.cu, on the current device
cudaError_t read_lce_wait_timeouts(unsigned long long* out, bool reset);
cudaError_t launch_embed_fwd(const EmbedFwdArgs& a, cudaStream_t s);
cudaError_t launch_embed_bwd(const EmbedBwdArgs& a, cudaStream_t s);
cudaError_t launch_dropout(const DropoutArgs& a, cudaStream_t s);

}  // namespace coat
