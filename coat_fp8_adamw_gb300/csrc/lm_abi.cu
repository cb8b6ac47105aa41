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
// the parts of the embedding gradient's workspace: the sorted tokens, the chunks' shares, and a flag per row of the table
size_t sorted_bytes(int64_t M) { return (sizeof(coat::Entry) * (size_t)M + 15) / 16 * 16; }
size_t partial_bytes(int64_t M, int64_t C) { return 8 * (size_t)coat::embed_chunks(M) * (size_t)C; }
bool lce_ok(int64_t M, int64_t V, int64_t C, int64_t x_ld) {
    return rows_ok(M, C) && rows_ok(V, C) && stride_ok(x_ld, C) && M * V <= COAT_MAX_N;
}
size_t dz_bytes(int64_t M, int64_t V, int64_t piece) { return 2 * (size_t)M * (size_t)coat::lce_piece_ld(piece, V); }
size_t xt_bytes(int64_t M, int64_t C) { return 2 * (size_t)C * (size_t)coat::lce_xt_ld(M); }
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

size_t coat_embedding_backward_workspace_bytes(int64_t M, int64_t V, int64_t C) {
    if (!rows_ok(M, C) || !rows_ok(V, C)) return 0;
    return sorted_bytes(M) + partial_bytes(M, C) + (size_t)coat::embed_flags(V);
}

coat_status coat_embedding_backward(const uint16_t* dout, const void* ids, int32_t wide_ids, float scale, int64_t M, int64_t V,
                                    int64_t C, int32_t accumulate, uint16_t* dtable, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    if (!dout || !ids || !dtable || !workspace || !std::isfinite(scale)) return COAT_ERR_INVALID_ARG;
    if (!rows_ok(M, C) || !rows_ok(V, C)) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{dout, 2 * (size_t)M * (size_t)C, kIn}, {ids, index_bytes(M, wide_ids), kIn},
                                          {dtable, 2 * (size_t)V * (size_t)C, kOut}, {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    if (workspace_bytes < coat_embedding_backward_workspace_bytes(M, V, C)) return COAT_ERR_INVALID_ARG;
    char* partial = static_cast<char*>(workspace) + sorted_bytes(M);
    const coat::EmbedBwdArgs a{dout, ids, wide_ids, scale, M, V, C, accumulate, dtable, static_cast<coat::Entry*>(workspace),
                               reinterpret_cast<float*>(partial), reinterpret_cast<uint8_t*>(partial) + partial_bytes(M, C)};
    return from_cuda(coat::launch_embed_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_linear_cross_entropy_workspace_bytes(int64_t M, int64_t V) {
    return shape_ok(M, V) && M * V <= COAT_MAX_N ? coat::lce_stats_bytes(M, V) : 0;
}

coat_status coat_linear_cross_entropy(const uint16_t* x, int64_t x_ld, const uint16_t* weight, const void* targets,
                                      int32_t wide_targets, int64_t M, int64_t V, int64_t C, float* loss, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!x || !weight || !targets || !loss || !lse || !workspace) return COAT_ERR_INVALID_ARG;
    if (!lce_ok(M, V, C, x_ld)) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{x, span(M, C, x_ld, 2), kIn}, {weight, 2 * (size_t)V * (size_t)C, kIn},
                                          {targets, index_bytes(M, wide_targets), kIn}, {loss, 4 * (size_t)M, kOut},
                                          {lse, 4 * (size_t)M, kOut}, {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    if (workspace_bytes < coat_linear_cross_entropy_workspace_bytes(M, V)) return COAT_ERR_INVALID_ARG;
    const coat::LceFwdArgs a{x, x_ld, weight, targets, wide_targets, M, V, C, loss, lse, workspace};
    return from_cuda(coat::launch_lce_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_linear_cross_entropy_backward_workspace_bytes(int64_t M, int64_t V, int64_t C, int64_t piece) {
    if (!lce_ok(M, V, C, C) || piece < 0) return 0;
    const int64_t p = coat::lce_piece(M, V, piece);
    return dz_bytes(M, V, p) + xt_bytes(M, C) + 16 + 4 * (size_t)coat::lce_sums(M, V, C, p);
}

coat_status coat_linear_cross_entropy_backward(const uint16_t* x, int64_t x_ld, const uint16_t* weight, const void* targets,
                                               int32_t wide_targets, const float* lse, const float* dloss, const float* dlse,
                                               int64_t M, int64_t V, int64_t C, int64_t piece, uint16_t* dx, uint16_t* dweight,
                                               void* workspace, size_t workspace_bytes, void* stream) {
    if (!x || !weight || !targets || !lse || !dloss || !dx || !dweight || !workspace) return COAT_ERR_INVALID_ARG;
    if (!lce_ok(M, V, C, x_ld) || piece < 0) return COAT_ERR_INVALID_ARG;
    const coat_status st = check_buffers({{x, span(M, C, x_ld, 2), kIn}, {weight, 2 * (size_t)V * (size_t)C, kIn},
                                          {targets, index_bytes(M, wide_targets), kIn}, {lse, 4 * (size_t)M, kIn},
                                          {dloss, 4 * (size_t)M, kIn}, {dlse, 4 * (size_t)M, kIn},
                                          {dx, 2 * (size_t)M * (size_t)C, kOut}, {dweight, 2 * (size_t)V * (size_t)C, kOut},
                                          {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    if (workspace_bytes < coat_linear_cross_entropy_backward_workspace_bytes(M, V, C, piece)) return COAT_ERR_INVALID_ARG;
    const int64_t p = coat::lce_piece(M, V, piece);
    char* xt = static_cast<char*>(workspace) + dz_bytes(M, V, p);
    const coat::LceBwdArgs a{x, x_ld, weight, targets, wide_targets, lse, dloss, dlse, M, V, C, p, dx, dweight,
                             static_cast<uint16_t*>(workspace), reinterpret_cast<uint16_t*>(xt),
                             reinterpret_cast<float*>(xt + xt_bytes(M, C)), reinterpret_cast<float*>(xt + xt_bytes(M, C) + 16)};
    return from_cuda(coat::launch_lce_bwd(a, static_cast<cudaStream_t>(stream)));
}

coat_status coat_dropout(const uint16_t* x, const uint16_t* residual, float p, const uint64_t* rng, int64_t n, uint16_t* y,
                         void* stream) {
    return dropout(x, residual, p, rng, n, y, stream);
}

coat_status coat_dropout_backward(const uint16_t* dy, float p, const uint64_t* rng, int64_t n, uint16_t* dx, void* stream) {
    return dropout(dy, nullptr, p, rng, n, dx, stream);
}

}  // extern "C"
