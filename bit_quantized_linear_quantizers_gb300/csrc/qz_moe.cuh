// qz_moe.cuh -- launchers of a block of experts in FP8: routing, the experts'
// products, the residual norm.
#pragma once

#include "qz_paged.cuh"

namespace qz {

constexpr int kMoeMaxExperts = 512, kMoeMaxTopK = 16, kMoeMaxGroups = 32;

struct RouteArgs {
    const void* logits;
    int64_t tokens, ldl;
    const float* bias;
    const int32_t* n_tokens;
    qz_moe_routing r;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* row_token;
    int32_t* token_row;
};
size_t ws_moe_route(int64_t tokens, int64_t experts, int64_t top_k);
qz_status moe_route_launch(const RouteArgs& a, qz_dtype lt, void* ws, cudaStream_t st);

struct MoeGemmArgs {
    const uint8_t* qA;
    const float* sA;
    int64_t tokens;
    const int32_t* row_token;
    int64_t rows;
    const int32_t* offsets;
    int experts;
    const uint8_t* qW;
    const float* sW;
    uint16_t* Y;              // plain output, or
    uint8_t* codes;           // SwiGLU's codes and scales (N = 2 I)
    float* scales;
    int N, K;
};
qz_status moe_gemm_fp8_launch(const MoeGemmArgs& a, cudaStream_t st);
qz_status moe_gemm_error_read_and_clear();

struct NormArgs {
    const void* x;
    int64_t tokens, ldx;
    int hidden;
    bool has_block;
    qz_block_output b;
    void* x_out;
    int64_t ldo;
    const void* gamma;
    float eps;
    uint16_t* normed;
    uint8_t* codes;
    float* scales;
};
qz_status residual_rmsnorm_launch(const NormArgs& a, qz_dtype xt, cudaStream_t st);

} // namespace qz
