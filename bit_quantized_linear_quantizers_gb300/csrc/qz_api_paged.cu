// qz_api_paged.cu -- extern "C" entry points of the paged FP8 KV cache (block
// tables, the write of new tokens, attention): host-side validation, workspace
// checks and dispatch. Nothing here allocates; a rejected call launches nothing.
#include "qz_internal.cuh"
#include "qz_gemm.cuh"
#include "qz_paged.cuh"

#include <cmath>

using namespace qz;

static bool page_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128; }

static qz_status cache_checks(const qz_paged_kv* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return QZ_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->heads < 1) return QZ_ERR_INVALID_ARG;
    if (!page_ok(c->page_size) || (c->head_dim != 64 && c->head_dim != 128) || c->heads > 32767) return QZ_ERR_SHAPE;
    if ((int64_t)c->num_pages * c->page_size >= (int64_t)1 << 31) return QZ_ERR_SHAPE;
    if (c->page_stride < (int64_t)c->heads * c->page_size * c->head_dim) return QZ_ERR_INVALID_ARG;
    if (!is_aligned(c->k_codes, 16) || !is_aligned(c->v_codes, 16) || c->page_stride % 16 ||
        !is_aligned(c->k_scale, 4) || !is_aligned(c->v_scale, 4))
        return QZ_ERR_ALIGNMENT;
    return QZ_OK;
}

extern "C" {

qz_status qz_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                          int32_t* block_table, int max_blocks, int64_t ld_table,
                          const int32_t* free_pages, int n_free, const int32_t* free_head,
                          int32_t* kv_lens, int32_t* cu_new, int32_t* slot_map, int32_t* positions, int n_slots,
                          int32_t* free_head_out, void* stream) {
    if (B < 0 || max_blocks < 0 || n_free < 0 || n_slots < 0 || ld_table < max_blocks) return QZ_ERR_INVALID_ARG;
    if (!free_head || !cu_new || !free_head_out || (n_free && !free_pages) || (n_slots && !slot_map))
        return QZ_ERR_INVALID_ARG;
    if (B && (!ctx_lens || !new_lens || !kv_lens || (max_blocks && !block_table))) return QZ_ERR_INVALID_ARG;
    if (!page_ok(page_size)) return QZ_ERR_SHAPE;
    if ((int64_t)max_blocks * page_size >= (int64_t)1 << 31) return QZ_ERR_SHAPE;
    const void* p[9] = {ctx_lens, new_lens, block_table, free_pages, free_head, kv_lens, cu_new, slot_map, positions};
    for (const void* x : p)
        if (x && !is_aligned(x, 4)) return QZ_ERR_ALIGNMENT;
    if (!is_aligned(free_head_out, 4)) return QZ_ERR_ALIGNMENT;
    QZ_TRY(device_check());
    return block_tables_launch(ctx_lens, new_lens, B, page_size, block_table, max_blocks, ld_table, free_pages, n_free,
                               free_head, kv_lens, cu_new, slot_map, positions, n_slots, free_head_out,
                               (cudaStream_t)stream);
}

qz_status qz_kv_append_fp8_paged(const void* k, const void* v, qz_dtype xt, int64_t tokens, int64_t ldk, int64_t ldv,
                                 const int32_t* slot_map, const qz_paged_kv* cache, void* stream) {
    QZ_TRY(cache_checks(cache));
    if ((xt != QZ_F32 && xt != QZ_BF16) || tokens < 0) return QZ_ERR_INVALID_ARG;
    if (tokens == 0) return QZ_OK;
    if (!k || !v || !slot_map) return QZ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)cache->heads * cache->head_dim, es = xt == QZ_F32 ? 4 : 2;
    if (ldk < row || ldv < row) return QZ_ERR_INVALID_ARG;
    if (tokens >= (int64_t)1 << 31) return QZ_ERR_SHAPE;
    if (!is_aligned(k, 16) || !is_aligned(v, 16) || (ldk * es) % 16 || (ldv * es) % 16 || !is_aligned(slot_map, 4))
        return QZ_ERR_ALIGNMENT;
    QZ_TRY(device_check());
    return kv_append_paged_launch(k, v, xt, tokens, ldk, ldv, slot_map, *cache, (cudaStream_t)stream);
}

qz_status qz_attn_fp8_paged(const uint16_t* q, int64_t ldq, int64_t tokens, int heads_q, const int32_t* cu_q, int B,
                            int max_q, const qz_paged_kv* cache, const int32_t* block_table, int max_blocks,
                            int64_t ld_table, const int32_t* kv_lens, float sm_scale, int causal, uint16_t* out,
                            int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream) {
    QZ_TRY(cache_checks(cache));
    if (tokens < 0 || B < 0 || max_q < 0 || heads_q < 1 || max_blocks < 0 || ld_table < max_blocks ||
        !std::isfinite(sm_scale) || (causal != 0 && causal != 1))
        return QZ_ERR_INVALID_ARG;
    if (heads_q % cache->heads || heads_q / cache->heads > 256) return QZ_ERR_SHAPE;
    if (tokens == 0 || B == 0 || max_q == 0) return QZ_OK;
    if (!q || !cu_q || !kv_lens || !out || (max_blocks && !block_table)) return QZ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)heads_q * cache->head_dim;
    if (ldq < row || ldo < row) return QZ_ERR_INVALID_ARG;
    if (tokens >= (int64_t)1 << 31 || (int64_t)max_blocks * cache->page_size >= (int64_t)1 << 31) return QZ_ERR_SHAPE;
    if (!is_aligned(q, 16) || !is_aligned(out, 16) || ldq % 8 || ldo % 8 || !is_aligned(cu_q, 4) ||
        !is_aligned(kv_lens, 4) || (block_table && !is_aligned(block_table, 4)) || (lse && !is_aligned(lse, 4)))
        return QZ_ERR_ALIGNMENT;
    const size_t need = ws_attn_paged((int64_t)max_q * (heads_q / cache->heads), cache->head_dim);
    if (need && (!ws || ws_bytes < need || !is_aligned(ws, 16))) return QZ_ERR_WORKSPACE;
    QZ_TRY(device_check());
    const AttnArgs a = {q, ldq, tokens, heads_q, cu_q, B, max_q, *cache, block_table, max_blocks, ld_table, kv_lens,
                        sm_scale, causal, out, ldo, lse};
    return attn_paged_launch(a, ws, (cudaStream_t)stream);
}

} // extern "C"
