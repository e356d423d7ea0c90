// qz_api_moe.cu -- extern "C" entry points of a block of experts in FP8 (routing,
// the experts' products, the residual norm): host-side validation and dispatch.
// Nothing here allocates; a rejected call launches nothing.
#include "qz_internal.cuh"
#include "qz_gemm.cuh"
#include "qz_moe.cuh"

#include <cmath>

using namespace qz;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 31;

qz_status moe_gemm_checks(const MoeGemmArgs& a) {
    if (a.tokens < 0 || a.rows < 0 || a.experts < 1 || a.N < 1 || a.K < 1) return QZ_ERR_INVALID_ARG;
    if (a.experts > kMoeMaxExperts || a.N % 128 || a.K % 128 || a.rows >= kMaxRows || a.tokens >= kMaxRows ||
        (int64_t)a.experts * a.N >= kMaxRows)
        return QZ_ERR_SHAPE;
    if (a.rows == 0) return QZ_OK;
    if (!a.offsets || !a.qW || !a.sW || (a.tokens && (!a.qA || !a.sA))) return QZ_ERR_INVALID_ARG;
    if (!a.Y && (!a.codes || !a.scales)) return QZ_ERR_INVALID_ARG;
    if (!is_aligned(a.qA, 16) || !is_aligned(a.qW, 16) || !is_aligned(a.Y, 16) || !is_aligned(a.codes, 16) ||
        !is_aligned(a.sA, 4) || !is_aligned(a.sW, 4) || !is_aligned(a.scales, 4) || !is_aligned(a.row_token, 4) ||
        !is_aligned(a.offsets, 4))
        return QZ_ERR_ALIGNMENT;
    return QZ_OK;
}

} // namespace

extern "C" {

qz_status qz_moe_route(const void* logits, qz_dtype lt, int64_t tokens, int64_t ldl, const float* bias,
                       const int32_t* n_tokens, const qz_moe_routing* routing, int32_t* ids, float* weights,
                       int32_t* offsets, int32_t* row_token, int32_t* token_row, void* ws, size_t ws_bytes, void* stream) {
    if (!routing || !offsets || (lt != QZ_F32 && lt != QZ_BF16) || tokens < 0) return QZ_ERR_INVALID_ARG;
    const qz_moe_routing& r = *routing;
    if (r.experts < 1 || r.top_k < 1 || r.groups < 1 || (r.score != QZ_SCORE_SOFTMAX && r.score != QZ_SCORE_SIGMOID) ||
        (r.renormalize != 0 && r.renormalize != 1) || !std::isfinite(r.scale) || r.top_groups < 1 ||
        r.top_groups > r.groups || r.group_best < 1 || r.group_best > 2)
        return QZ_ERR_INVALID_ARG;
    if (r.experts > kMoeMaxExperts || r.top_k > kMoeMaxTopK || r.groups > kMoeMaxGroups || r.experts % r.groups ||
        r.group_best > r.experts / r.groups || r.top_k > r.top_groups * (r.experts / r.groups))
        return QZ_ERR_SHAPE;
    if (tokens >= kMaxRows || tokens * r.top_k >= kMaxRows) return QZ_ERR_SHAPE;
    if (tokens && (!logits || !ids || !weights || !row_token || !token_row || ldl < r.experts)) return QZ_ERR_INVALID_ARG;
    if (!is_aligned(logits, lt == QZ_F32 ? 4 : 2)) return QZ_ERR_ALIGNMENT;
    const void* p[7] = {bias, n_tokens, ids, weights, offsets, row_token, token_row};
    for (const void* x : p)
        if (!is_aligned(x, 4)) return QZ_ERR_ALIGNMENT;
    const size_t need = ws_moe_route(tokens, r.experts, r.top_k);
    if (need && (!ws || ws_bytes < need || !is_aligned(ws, 16))) return QZ_ERR_WORKSPACE;
    QZ_TRY(device_check());
    const RouteArgs a = {logits, tokens, ldl, bias, n_tokens, r, ids, weights, offsets, row_token, token_row};
    return moe_route_launch(a, lt, ws, (cudaStream_t)stream);
}

qz_status qz_moe_gemm_fp8(const uint8_t* qA, const float* sA, int64_t tokens, const int32_t* row_token, int64_t rows,
                          const int32_t* offsets, int experts, const uint8_t* qW, const float* sW, uint16_t* Y, int N,
                          int K, void* stream) {
    const MoeGemmArgs a = {qA, sA, tokens, row_token, rows, offsets, experts, qW, sW, Y, nullptr, nullptr, N, K};
    QZ_TRY(moe_gemm_checks(a));
    if (rows == 0) return QZ_OK;
    QZ_TRY(device_check());
    return moe_gemm_fp8_launch(a, (cudaStream_t)stream);
}

qz_status qz_moe_gemm_fp8_swiglu(const uint8_t* qA, const float* sA, int64_t tokens, const int32_t* row_token,
                                 int64_t rows, const int32_t* offsets, int experts, const uint8_t* qW, const float* sW,
                                 uint8_t* y_codes, float* y_scales, int I, int K, void* stream) {
    if (I < 1) return QZ_ERR_INVALID_ARG;
    if (I % 128 || I >= 1 << 30) return QZ_ERR_SHAPE;
    const MoeGemmArgs a = {qA, sA, tokens, row_token, rows, offsets, experts, qW, sW, nullptr, y_codes, y_scales, 2 * I, K};
    QZ_TRY(moe_gemm_checks(a));
    if (rows == 0) return QZ_OK;
    QZ_TRY(device_check());
    return moe_gemm_fp8_launch(a, (cudaStream_t)stream);
}

qz_status qz_residual_rmsnorm(const void* x, qz_dtype xt, int64_t tokens, int hidden, int64_t ldx,
                              const qz_block_output* block, void* x_out, int64_t ldo, const void* gamma, float eps,
                              uint16_t* normed, uint8_t* codes, float* scales, void* stream) {
    if ((xt != QZ_F32 && xt != QZ_BF16) || tokens < 0 || hidden < 1) return QZ_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps <= 0.0f) return QZ_ERR_INVALID_ARG;
    if (hidden % 8 || hidden > 16384 || (codes && hidden % 128) || tokens >= kMaxRows) return QZ_ERR_SHAPE;
    if (block && (block->k < 1 || block->rows < 0 || !std::isfinite(block->alpha))) return QZ_ERR_INVALID_ARG;
    if (block && (block->k > kMoeMaxTopK || block->rows >= kMaxRows)) return QZ_ERR_SHAPE;
    if (tokens == 0) return QZ_OK;                // tensors of no elements have null pointers
    if ((codes == nullptr) != (scales == nullptr) || (!gamma && (normed || codes))) return QZ_ERR_INVALID_ARG;
    if (!x_out && !normed && !codes) return QZ_ERR_INVALID_ARG;
    if (!x || ldx < hidden || (x_out && ldo < hidden)) return QZ_ERR_INVALID_ARG;
    if (block && ((block->rows && !block->y) || block->ldy < hidden)) return QZ_ERR_INVALID_ARG;
    if (block && !block->token_row && block->rows < tokens * block->k) return QZ_ERR_INVALID_ARG;
    const int64_t es = xt == QZ_F32 ? 4 : 2;
    if (!is_aligned(x, 16) || !is_aligned(x_out, 16) || !is_aligned(gamma, 16) || !is_aligned(normed, 16) ||
        !is_aligned(codes, 16) || !is_aligned(scales, 4) || (ldx * es) % 16 || (x_out && (ldo * es) % 16))
        return QZ_ERR_ALIGNMENT;
    if (block && (!is_aligned(block->y, 16) || (block->ldy * 2) % 16 || !is_aligned(block->token_row, 4) ||
                  !is_aligned(block->weights, 4) || !is_aligned(block->gamma, 16)))
        return QZ_ERR_ALIGNMENT;
    QZ_TRY(device_check());
    const NormArgs a = {x, tokens, ldx, hidden, block != nullptr, block ? *block : qz_block_output{}, x_out, ldo, gamma, eps,
                        normed, codes, scales};
    return residual_rmsnorm_launch(a, xt, (cudaStream_t)stream);
}

} // extern "C"
