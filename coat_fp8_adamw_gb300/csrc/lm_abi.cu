// lm_abi.cu -- the extern "C" entry points of the operators at the two ends of a language model (cross entropy of a linear
// layer, embedding) and of dropout (declared in include/coat.h): argument validation and dispatch.  No allocation, no
// state, no host sync.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "abi_checks.h"
#include "coat.h"
#include "lm_kernels.h"

namespace {

using namespace coat::abi;

// rows x C elements: C a multiple of 16, and no more elements than any entry point takes
bool rows_ok(int64_t rows, int64_t C) { return shape_ok(rows, C) && C % 16 == 0 && rows * C <= COAT_MAX_N; }
size_t index_bytes(int64_t M, int32_t wide) { return (size_t)M * (wide ? 8 : 4); }

coat_status dropout(const uint16_t* x, const uint16_t* residual, float p, const uint64_t* rng, int64_t n, uint16_t* y, void* stream) {
    if (!x || !rng || !y || !size_ok(n)) return COAT_ERR_INVALID_ARG;
    if (!(p >= 0.0f) || !(p < 1.0f)) return COAT_ERR_INVALID_ARG;
    const long drop = std::lround((double)p * 65536.0);
    if (drop > 65535) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{x, 2 * (size_t)n, kIn}, {residual, 2 * (size_t)n, kIn}, {rng, 16, kIn},
                                          {y, 2 * (size_t)n, kOut}});
    if (st != COAT_OK) return st;
    const coat::DropoutArgs a{x, residual, rng, (uint32_t)drop, (float)(65536.0 / (65536.0 - (double)drop)), n, y};
    return from_cuda(coat::launch_dropout(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

coat_status coat_embedding(const uint16_t* table, const void* ids, int32_t wide_ids, float scale, int64_t M, int64_t V, int64_t C,
                           uint16_t* out, void* stream) {
    if (!table || !ids || !out || !std::isfinite(scale)) return COAT_ERR_INVALID_ARG;
    if (!rows_ok(M, C) || !rows_ok(V, C)) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{table, 2 * (size_t)V * (size_t)C, kIn}, {ids, index_bytes(M, wide_ids), kIn},
                                          {out, 2 * (size_t)M * (size_t)C, kOut}});
    if (st != COAT_OK) return st;
    const coat::EmbedFwdArgs a{table, ids, wide_ids, scale, M, V, C, out};
    return from_cuda(coat::launch_embed_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_embedding_backward_workspace_bytes(int64_t M, int64_t C) {
    if (!rows_ok(M, C)) return 0;
    return (sizeof(coat::Entry) * (size_t)M + 15) / 16 * 16 + 4 * (size_t)coat::embed_chunks(M) * (size_t)C;
}

coat_status coat_embedding_backward(const uint16_t* dout, const void* ids, int32_t wide_ids, float scale, int64_t M, int64_t V,
                                    int64_t C, int32_t accumulate, uint16_t* dtable, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    if (!dout || !ids || !dtable || !workspace || !std::isfinite(scale)) return COAT_ERR_INVALID_ARG;
    if (!rows_ok(M, C) || !rows_ok(V, C)) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{dout, 2 * (size_t)M * (size_t)C, kIn}, {ids, index_bytes(M, wide_ids), kIn},
                                          {dtable, 2 * (size_t)V * (size_t)C, kOut}, {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    if (workspace_bytes < coat_embedding_backward_workspace_bytes(M, C)) return COAT_ERR_INVALID_ARG;
    char* partial = static_cast<char*>(workspace) + (sizeof(coat::Entry) * (size_t)M + 15) / 16 * 16;
    const coat::EmbedBwdArgs a{dout, ids, wide_ids, scale, M, V, C, accumulate, dtable, static_cast<coat::Entry*>(workspace),
                               reinterpret_cast<float*>(partial)};
    return from_cuda(coat::launch_embed_bwd(a, static_cast<cudaStream_t>(stream)));
}

coat_status coat_dropout(const uint16_t* x, const uint16_t* residual, float p, const uint64_t* rng, int64_t n, uint16_t* y,
                         void* stream) {
    return dropout(x, residual, p, rng, n, y, stream);
}

coat_status coat_dropout_backward(const uint16_t* dy, float p, const uint64_t* rng, int64_t n, uint16_t* dx, void* stream) {
    return dropout(dy, nullptr, p, rng, n, dx, stream);
}

}  // extern "C"
