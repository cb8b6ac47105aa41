// ckpt_abi.cu -- the extern "C" entry points of the operators with 8-bit
// activation checkpoints (declared in include/coat.h): argument validation and
// dispatch.  No allocation, no state, no host sync.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>
#include <initializer_list>

#include "abi_checks.h"
#include "ckpt_kernels.h"
#include "coat.h"

namespace {

using namespace coat::abi;

// A buffer of a call.  A null pointer: not there.
enum Kind { kIn, kOut, kOutRows };
struct Buf {
    const void* p;
    size_t bytes;
    Kind kind;
};

// Alignment, then overlap, then where the memory is.  Outputs overlap nothing,
// except that two outputs of rows (kOutRows) may interleave: rows_apart has
// looked at those.
coat_status check_buffers(std::initializer_list<Buf> bufs) {
    for (const Buf& b : bufs)
        if (b.p && !aligned16(b.p)) return COAT_ERR_MISALIGNED;
    for (const Buf* b = bufs.begin(); b != bufs.end(); ++b)
        for (const Buf* c = b + 1; c != bufs.end(); ++c) {
            if (!b->p || !c->p || (b->kind == kIn && c->kind == kIn)) continue;
            if (b->kind == kOutRows && c->kind == kOutRows) continue;
            if (overlaps(b->p, b->bytes, c->p, c->bytes)) return COAT_ERR_INVALID_ARG;
        }
    for (const Buf& b : bufs)
        if (b.p && !is_device(b.p)) return COAT_ERR_NOT_DEVICE;
    return COAT_OK;
}

// 1 x G groups of rows of N: G a power of two in [8, 128], N a multiple of it and of 16
bool group_ok(int32_t G) { return G >= 8 && G <= 128 && (G & (G - 1)) == 0; }
bool shape_ok(int64_t M, int64_t N) { return M >= 1 && N >= 1 && M < (1LL << 31) && N < (1LL << 31); }
bool width_ok(int64_t N, int32_t G) { return N % 16 == 0 && N % G == 0; }
bool stride_ok(int64_t ld, int64_t N) { return ld >= N && ld % 8 == 0 && ld < (1LL << 31); }
// bytes from the first to the last element of M rows of n elements, ld apart
size_t span(int64_t M, int64_t n, int64_t ld, size_t elem) { return ((size_t)(M - 1) * (size_t)ld + (size_t)n) * elem; }

// Two sets of M rows of n elements with row stride ld that share no element:
// apart in memory, or column ranges of one tensor.
bool rows_apart(const uint16_t* a, int64_t na, const uint16_t* b, int64_t nb, int64_t M, int64_t ld) {
    if (!overlaps(a, span(M, na, ld, 2), b, span(M, nb, ld, 2))) return true;
    const intptr_t bytes = (intptr_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    int64_t d = (int64_t)(bytes / 2) % ld;
    if (d < 0) d += ld;
    return d >= na && d + nb <= ld;
}

bool head_ok(int32_t H, int32_t D, int64_t ld) { return H >= 0 && H <= 65536 && (H == 0 || stride_ok(ld, (int64_t)H * D)); }

coat_status check_qk_shape(int64_t M, int32_t Hq, int64_t q_ld, int32_t Hk, int64_t k_ld, int32_t D, int32_t rot,
                           int64_t max_pos, int32_t G) {
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (M < 1 || M >= (1LL << 31) || D < 16 || D > 256 || D % 16 != 0 || D % G != 0) return COAT_ERR_INVALID_ARG;
    if (rot < 16 || rot > D || rot % 16 != 0 || max_pos < 1 || max_pos >= (1LL << 31)) return COAT_ERR_INVALID_ARG;
    if (!head_ok(Hq, D, q_ld) || !head_ok(Hk, D, k_ld) || Hq + Hk < 1) return COAT_ERR_INVALID_ARG;
    return COAT_OK;
}

}  // namespace

extern "C" {

coat_status coat_rmsnorm_ckpt(const uint16_t* x, const uint16_t* residual, const float* weight, float eps, int64_t M,
                              int64_t N, int32_t G, uint16_t* h, uint16_t* y, uint8_t* q, float* scale, float* rstd,
                              void* stream) {
    if (!x || !weight || !y || !q || !scale || !rstd || (residual != nullptr) != (h != nullptr)) return COAT_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return COAT_ERR_INVALID_ARG;
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (!shape_ok(M, N) || !width_ok(N, G) || N > coat::kNormMaxN) return COAT_ERR_INVALID_ARG;
    const size_t n = (size_t)M * (size_t)N;
    const coat_status st = check_buffers({{x, 2 * n, kIn}, {residual, 2 * n, kIn}, {weight, 4 * (size_t)N, kIn},
                                          {h, 2 * n, kOut}, {y, 2 * n, kOut}, {q, n, kOut}, {scale, 4 * n / (size_t)G, kOut},
                                          {rstd, 4 * (size_t)M, kOut}});
    if (st != COAT_OK) return st;
    const coat::NormFwdArgs a{x, residual, weight, eps, M, N, G, h, y, q, scale, rstd};
    return from_cuda(coat::launch_norm_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_rmsnorm_ckpt_backward_workspace_bytes(int64_t M, int64_t N) {
    if (!shape_ok(M, N) || N > coat::kNormMaxN) return 0;
    const int sms = coat::device_sms();
    return sms > 0 ? 4 * (size_t)coat::norm_bwd_partials(M, N, sms) * (size_t)N : 0;
}

coat_status coat_rmsnorm_ckpt_backward(const uint16_t* dy, const uint8_t* q, const float* scale, const float* rstd,
                                       const float* weight, const uint16_t* dresidual, int64_t M, int64_t N, int32_t G,
                                       uint16_t* dx, uint16_t* dweight, void* workspace, size_t workspace_bytes,
                                       void* stream) {
    if (!dy || !q || !scale || !rstd || !weight || !dx || !dweight || !workspace) return COAT_ERR_INVALID_ARG;
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (!shape_ok(M, N) || !width_ok(N, G) || N > coat::kNormMaxN) return COAT_ERR_INVALID_ARG;
    const size_t n = (size_t)M * (size_t)N;
    const coat_status st = check_buffers({{dy, 2 * n, kIn}, {q, n, kIn}, {scale, 4 * n / (size_t)G, kIn},
                                          {rstd, 4 * (size_t)M, kIn}, {weight, 4 * (size_t)N, kIn},
                                          {dresidual, 2 * n, kIn}, {dx, 2 * n, kOut}, {dweight, 2 * (size_t)N, kOut},
                                          {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    const size_t need = coat_rmsnorm_ckpt_backward_workspace_bytes(M, N);
    if (need == 0) return COAT_ERR_CUDA;
    if (workspace_bytes < need) return COAT_ERR_INVALID_ARG;
    const coat::NormBwdArgs a{dy, q, scale, rstd, weight, dresidual, M, N, G, dx, dweight, static_cast<float*>(workspace)};
    return from_cuda(coat::launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

coat_status coat_swiglu_ckpt(const uint16_t* gate, const uint16_t* up, int64_t ld, int64_t M, int64_t N, int32_t G,
                             uint16_t* h, uint8_t* gate_q, float* gate_scale, uint8_t* up_q, float* up_scale,
                             void* stream) {
    if (!gate || !up || !h || !gate_q || !gate_scale || !up_q || !up_scale) return COAT_ERR_INVALID_ARG;
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (!shape_ok(M, N) || !width_ok(N, G) || !stride_ok(ld, N)) return COAT_ERR_INVALID_ARG;
    const size_t n = (size_t)M * (size_t)N, in = span(M, N, ld, 2), ns = 4 * n / (size_t)G;
    const coat_status st = check_buffers({{gate, in, kIn}, {up, in, kIn}, {h, 2 * n, kOut}, {gate_q, n, kOut},
                                          {gate_scale, ns, kOut}, {up_q, n, kOut}, {up_scale, ns, kOut}});
    if (st != COAT_OK) return st;
    const coat::SwigluFwdArgs a{gate, up, ld, M, N, G, h, gate_q, gate_scale, up_q, up_scale};
    return from_cuda(coat::launch_swiglu_fwd(a, static_cast<cudaStream_t>(stream)));
}

coat_status coat_swiglu_ckpt_backward(const uint16_t* dh, const uint8_t* gate_q, const float* gate_scale,
                                      const uint8_t* up_q, const float* up_scale, int64_t M, int64_t N, int32_t G,
                                      uint16_t* dgate, uint16_t* dup, int64_t ld, uint8_t* h_q, float* h_scale,
                                      void* stream) {
    if (!dh || !gate_q || !gate_scale || !up_q || !up_scale || !dgate || !dup || (h_q != nullptr) != (h_scale != nullptr))
        return COAT_ERR_INVALID_ARG;
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (!shape_ok(M, N) || !width_ok(N, G) || !stride_ok(ld, N)) return COAT_ERR_INVALID_ARG;
    if (!aligned16(dgate) || !aligned16(dup)) return COAT_ERR_MISALIGNED;
    if (!rows_apart(dgate, N, dup, N, M, ld)) return COAT_ERR_INVALID_ARG;
    const size_t n = (size_t)M * (size_t)N, out = span(M, N, ld, 2), ns = 4 * n / (size_t)G;
    const coat_status st = check_buffers({{dh, 2 * n, kIn}, {gate_q, n, kIn}, {gate_scale, ns, kIn}, {up_q, n, kIn},
                                          {up_scale, ns, kIn}, {dgate, out, kOutRows}, {dup, out, kOutRows},
                                          {h_q, n, kOut}, {h_scale, ns, kOut}});
    if (st != COAT_OK) return st;
    const coat::SwigluBwdArgs a{dh, gate_q, gate_scale, up_q, up_scale, M, N, G, dgate, dup, ld, h_q, h_scale};
    return from_cuda(coat::launch_swiglu_bwd(a, static_cast<cudaStream_t>(stream)));
}

coat_status coat_qk_norm_rope_ckpt(const uint16_t* q, int64_t q_ld, int32_t Hq, const uint16_t* k, int64_t k_ld,
                                   int32_t Hk, int32_t D, const float* q_weight, const float* k_weight, float eps,
                                   const float* cos, const float* sin, int64_t max_pos, int32_t rot,
                                   const int32_t* positions, int32_t interleaved, int64_t M, int32_t G, uint16_t* q_out,
                                   uint8_t* q_codes, float* q_scale, float* q_rstd, uint16_t* k_out, uint8_t* k_codes,
                                   float* k_scale, float* k_rstd, void* stream) {
    if (!cos || !sin || !positions) return COAT_ERR_INVALID_ARG;
    if (Hq > 0 && (!q || !q_weight || !q_out || !q_codes || !q_scale || !q_rstd)) return COAT_ERR_INVALID_ARG;
    if (Hk > 0 && (!k || !k_weight || !k_out || !k_codes || !k_scale || !k_rstd)) return COAT_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return COAT_ERR_INVALID_ARG;
    coat_status st = check_qk_shape(M, Hq, q_ld, Hk, k_ld, D, rot, max_pos, G);
    if (st != COAT_OK) return st;
    const size_t nq = (size_t)M * (size_t)Hq * (size_t)D, nk = (size_t)M * (size_t)Hk * (size_t)D;
    const size_t table = 2 * (size_t)max_pos * (size_t)rot, hd = 4 * (size_t)D, g = (size_t)G;
    // a side without heads has no buffers
    const bool Q = Hq > 0, K = Hk > 0;
    st = check_buffers({{Q ? q : nullptr, Q ? span(M, (int64_t)Hq * D, q_ld, 2) : 0, kIn},
                        {K ? k : nullptr, K ? span(M, (int64_t)Hk * D, k_ld, 2) : 0, kIn},
                        {Q ? q_weight : nullptr, hd, kIn}, {K ? k_weight : nullptr, hd, kIn},
                        {cos, table, kIn}, {sin, table, kIn}, {positions, 4 * (size_t)M, kIn},
                        {Q ? q_out : nullptr, 2 * nq, kOut}, {Q ? q_codes : nullptr, nq, kOut},
                        {Q ? q_scale : nullptr, 4 * nq / g, kOut}, {Q ? q_rstd : nullptr, 4 * (size_t)M * (size_t)Hq, kOut},
                        {K ? k_out : nullptr, 2 * nk, kOut}, {K ? k_codes : nullptr, nk, kOut},
                        {K ? k_scale : nullptr, 4 * nk / g, kOut}, {K ? k_rstd : nullptr, 4 * (size_t)M * (size_t)Hk, kOut}});
    if (st != COAT_OK) return st;
    coat::QkArgs a{};
    a.q = coat::HeadSide{q, q_out, q_ld, Hq, q_weight, q_codes, q_scale, q_rstd, nullptr};
    a.k = coat::HeadSide{k, k_out, k_ld, Hk, k_weight, k_codes, k_scale, k_rstd, nullptr};
    a.cos = cos; a.sin = sin; a.positions = positions;
    a.M = M; a.max_pos = max_pos; a.D = D; a.rot = rot; a.G = G;
    a.interleaved = interleaved; a.eps = eps;
    return from_cuda(coat::launch_qk_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_qk_norm_rope_ckpt_backward_workspace_bytes(int64_t M, int32_t D) {
    if (M < 1 || M >= (1LL << 31) || D < 16 || D > 256 || D % 16 != 0) return 0;
    const int sms = coat::device_sms();
    return sms > 0 ? 4 * (size_t)coat::qk_bwd_partials(sms) * (size_t)D : 0;
}

coat_status coat_qk_norm_rope_ckpt_backward(const uint16_t* dq_out, const uint16_t* dk_out, const uint8_t* q_codes,
                                            const float* q_scale, const float* q_rstd, const uint8_t* k_codes,
                                            const float* k_scale, const float* k_rstd, int32_t Hq, int32_t Hk, int32_t D,
                                            const float* q_weight, const float* k_weight, const float* cos,
                                            const float* sin, int64_t max_pos, int32_t rot, const int32_t* positions,
                                            int32_t interleaved, int64_t M, int32_t G, uint16_t* dq, int64_t dq_ld,
                                            uint16_t* dk, int64_t dk_ld, uint16_t* dq_weight, uint16_t* dk_weight,
                                            void* workspace, size_t workspace_bytes, void* stream) {
    if (!cos || !sin || !positions || !workspace) return COAT_ERR_INVALID_ARG;
    if (Hq > 0 && (!dq_out || !q_codes || !q_scale || !q_rstd || !q_weight || !dq || !dq_weight)) return COAT_ERR_INVALID_ARG;
    if (Hk > 0 && (!dk_out || !k_codes || !k_scale || !k_rstd || !k_weight || !dk || !dk_weight)) return COAT_ERR_INVALID_ARG;
    coat_status st = check_qk_shape(M, Hq, dq_ld, Hk, dk_ld, D, rot, max_pos, G);
    if (st != COAT_OK) return st;
    const bool Q = Hq > 0, K = Hk > 0;
    if ((Q && !aligned16(dq)) || (K && !aligned16(dk))) return COAT_ERR_MISALIGNED;
    const size_t sq = Q ? span(M, (int64_t)Hq * D, dq_ld, 2) : 0, sk = K ? span(M, (int64_t)Hk * D, dk_ld, 2) : 0;
    if (Q && K && overlaps(dq, sq, dk, sk) &&
        !(dq_ld == dk_ld && rows_apart(dq, (int64_t)Hq * D, dk, (int64_t)Hk * D, M, dq_ld)))
        return COAT_ERR_INVALID_ARG;
    const size_t nq = (size_t)M * (size_t)Hq * (size_t)D, nk = (size_t)M * (size_t)Hk * (size_t)D;
    const size_t table = 2 * (size_t)max_pos * (size_t)rot, hd = 4 * (size_t)D, g = (size_t)G;
    st = check_buffers({{Q ? dq_out : nullptr, 2 * nq, kIn}, {K ? dk_out : nullptr, 2 * nk, kIn},
                        {Q ? q_codes : nullptr, nq, kIn}, {K ? k_codes : nullptr, nk, kIn},
                        {Q ? q_scale : nullptr, 4 * nq / g, kIn}, {K ? k_scale : nullptr, 4 * nk / g, kIn},
                        {Q ? q_rstd : nullptr, 4 * (size_t)M * (size_t)Hq, kIn},
                        {K ? k_rstd : nullptr, 4 * (size_t)M * (size_t)Hk, kIn},
                        {Q ? q_weight : nullptr, hd, kIn}, {K ? k_weight : nullptr, hd, kIn},
                        {cos, table, kIn}, {sin, table, kIn}, {positions, 4 * (size_t)M, kIn},
                        {Q ? dq : nullptr, sq, kOutRows}, {K ? dk : nullptr, sk, kOutRows},
                        {Q ? dq_weight : nullptr, 2 * (size_t)D, kOut}, {K ? dk_weight : nullptr, 2 * (size_t)D, kOut},
                        {workspace, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    const size_t need = coat_qk_norm_rope_ckpt_backward_workspace_bytes(M, D);
    if (need == 0) return COAT_ERR_CUDA;
    if (workspace_bytes < need) return COAT_ERR_INVALID_ARG;
    coat::QkArgs a{};
    // the kernels only read the checkpoint in this direction
    a.q = coat::HeadSide{dq_out, dq, dq_ld, Hq, q_weight, const_cast<uint8_t*>(q_codes), const_cast<float*>(q_scale),
                         const_cast<float*>(q_rstd), dq_weight};
    a.k = coat::HeadSide{dk_out, dk, dk_ld, Hk, k_weight, const_cast<uint8_t*>(k_codes), const_cast<float*>(k_scale),
                         const_cast<float*>(k_rstd), dk_weight};
    a.cos = cos; a.sin = sin; a.positions = positions;
    a.M = M; a.max_pos = max_pos; a.D = D; a.rot = rot; a.G = G;
    a.interleaved = interleaved; a.partial = static_cast<float*>(workspace);
    return from_cuda(coat::launch_qk_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t coat_ckpt_weight_grad_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!shape_ok(M, N) || !shape_ok(M, K)) return 0;
    const int sms = coat::device_sms();
    return sms > 0 ? coat::wgrad_workspace(M, N, K, sms) : 0;
}

coat_status coat_ckpt_weight_grad(const uint16_t* dy, int64_t dy_ld, const uint8_t* q, const float* scale,
                                  const float* row_scale, const float* col_scale, int64_t M, int64_t N, int64_t K,
                                  int32_t G, uint16_t* dw, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dy || !q || !scale || !dw || (workspace_bytes > 0 && !workspace)) return COAT_ERR_INVALID_ARG;
    if (!group_ok(G)) return COAT_ERR_UNSUPPORTED_G;
    if (!shape_ok(M, N) || !shape_ok(M, K) || N % 8 != 0 || !width_ok(K, G) || !stride_ok(dy_ld, N)) return COAT_ERR_INVALID_ARG;
    const size_t nx = (size_t)M * (size_t)K;
    const coat_status st = check_buffers({{dy, span(M, N, dy_ld, 2), kIn}, {q, nx, kIn}, {scale, 4 * nx / (size_t)G, kIn},
                                          {row_scale, 4 * (size_t)M, kIn}, {col_scale, 4 * (size_t)K, kIn},
                                          {dw, 2 * (size_t)N * (size_t)K, kOut},
                                          {workspace_bytes > 0 ? workspace : nullptr, workspace_bytes, kOut}});
    if (st != COAT_OK) return st;
    if (workspace_bytes < coat_ckpt_weight_grad_workspace_bytes(M, N, K)) return COAT_ERR_INVALID_ARG;
    const coat::WgradArgs a{dy, dy_ld, q, scale, row_scale, col_scale, M, N, K, G, dw, static_cast<float*>(workspace)};
    return from_cuda(coat::launch_wgrad(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
