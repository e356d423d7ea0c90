// qz_paged.cuh -- launchers of the paged FP8 KV cache: block tables, the write
// of new tokens, attention; and the device helpers they share.
#pragma once

#include "qz_gemm.cuh"

namespace qz {

qz_status block_tables_launch(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                              int32_t* block_table, int max_blocks, int64_t ld_table, const int32_t* free_pages,
                              int n_free, const int32_t* free_head, int32_t* kv_lens, int32_t* cu_new,
                              int32_t* slot_map, int32_t* positions, int n_slots, int32_t* free_head_out,
                              cudaStream_t st);
qz_status kv_append_paged_launch(const void* k, const void* v, qz_dtype xt, int64_t tokens, int64_t ldk, int64_t ldv,
                                 const int32_t* slot_map, const qz_paged_kv& cache, cudaStream_t st);

struct AttnArgs {
    const uint16_t* q;
    int64_t ldq, tokens;
    int heads_q;
    const int32_t* cu_q;
    int B, max_q;
    qz_paged_kv kv;
    const int32_t* block_table;
    int max_blocks;
    int64_t ld_table;
    const int32_t* kv_lens;
    float sm_scale;
    int causal;
    uint16_t* out;
    int64_t ldo;
    float* lse;
};
size_t ws_attn_paged(int64_t rows, int64_t head_dim);
qz_status attn_paged_launch(const AttnArgs& a, void* ws, cudaStream_t st);
// the requests of at most max_rows query rows per KV head (attn_fp8_decode.cu)
size_t ws_attn_decode();
qz_status attn_decode_launch(const AttnArgs& a, int max_rows, bool beside, void* ws, cudaStream_t st);
qz_status attn_decode_error_read_and_clear();
// the requests of at least min_rows query rows per KV head (attn_fp8_prefill.cu)
size_t ws_attn_prefill();
qz_status attn_prefill_launch(const AttnArgs& a, int min_rows, void* ws, bool* joined, cudaStream_t st);
qz_status attn_prefill_error_read_and_clear();

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch under programmatic dependent launch; the kernel itself waits for the
// stream's earlier work before it touches memory.
template <typename... KArgs, typename... Args>
qz_status launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? launch_status() : QZ_ERR_CUDA;
}

} // namespace qz
