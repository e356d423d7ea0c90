// attn_fp8.cu -- attention over the paged FP8 KV cache, simple form: one CTA per
// (query token, KV head), one warp per query head of the group, one key at a time.
//   x_j = sm_scale * sum_d q_d K_jd;  O = sum_j softmax(x)_j V_j;  lse = ln sum_j e^x_j
// with a running maximum and sum. Each warp re-reads K and V for its query head.
#include "qz_internal.cuh"
#include "qz_paged.cuh"

#include <algorithm>

namespace qz {

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

template <int D>
__global__ void __launch_bounds__(kWarps * 32)
attn_simple_kernel(const AttnArgs a, int shift, int min_rows) {
    constexpr int C = D / 32;                     // channels per lane
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int lo = 0, hi = a.B - 1;                     // the last request that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu_q + mid) <= t) lo = mid; else hi = mid - 1;
    }
    const int n = min(__ldg(a.cu_q + lo + 1) - __ldg(a.cu_q + lo), a.max_q), i = (int)(t - __ldg(a.cu_q + lo));
    if (i < 0 || i >= n || n * (a.heads_q / a.kv.heads) < min_rows) return;
    const int L = (int)min((int64_t)max(__ldg(a.kv_lens + lo), 0), (int64_t)a.max_blocks << shift);
    const int seen = a.causal ? min(L, max(L - n + i + 1, 0)) : L;
    const int G = a.heads_q / a.kv.heads, mask = (1 << shift) - 1;
    const float c = a.sm_scale * kLog2e;
    const int32_t* row = a.block_table + (int64_t)lo * a.ld_table;
    for (int g = warp; g < G; g += kWarps) {
        const int hq = h * G + g;
        float q[C], o[C], m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int j = 0; j < C; j++) {
            q[j] = bf16_bits_to_f32(a.q[t * a.ldq + (int64_t)hq * D + lane * C + j]);
            o[j] = 0.0f;
        }
        for (int k = 0; k < seen; k++) {
            const int p = __ldg(row + (k >> shift));
            if (p < 0 || p >= a.kv.num_pages) continue;
            const int64_t at = (int64_t)p * a.kv.page_stride + (((int64_t)h << shift) + (k & mask)) * D + lane * C;
            const int64_t sc = (int64_t)p * a.kv.heads + h;
            float x = 0.0f;
#pragma unroll
            for (int j = 0; j < C; j++) x = fmaf(q[j], e4m3_value(a.kv.k_codes[at + j]), x);
            for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
            x *= a.kv.k_scale[sc] * c;
            const float m2 = fmaxf(m, x), f = exp2f(m - m2), e = exp2f(x - m2), w = e * a.kv.v_scale[sc];
            m = m2;
            l = fmaf(l, f, e);
#pragma unroll
            for (int j = 0; j < C; j++) o[j] = fmaf(w, e4m3_value(a.kv.v_codes[at + j]), o[j] * f);
        }
        const float r = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
        for (int j = 0; j < C; j++)
            a.out[t * a.ldo + (int64_t)hq * D + lane * C + j] = __bfloat16_as_ushort(__float2bfloat16_rn(o[j] * r));
        if (a.lse && lane == 0) a.lse[t * a.heads_q + hq] = l > 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
    }
}

} // namespace

constexpr int kDecodeRows = 64;                   // rows per KV head up to which a request takes the decode kernel

size_t ws_attn_paged(int64_t, int64_t) { return ws_attn_decode(); }

qz_status attn_paged_launch(const AttnArgs& a, void* ws, cudaStream_t st) {
    QZ_TRY(attn_decode_launch(a, kDecodeRows, ws, st));
    if ((int64_t)a.max_q * (a.heads_q / a.kv.heads) <= kDecodeRows) return QZ_OK;
    const int P = a.kv.page_size, shift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
    auto* fn = a.kv.head_dim == 64 ? attn_simple_kernel<64> : attn_simple_kernel<128>;
    return launch_pdl(fn, dim3((unsigned)a.tokens, a.kv.heads), dim3(kWarps * 32), 0, st, a, shift, kDecodeRows + 1);
}

} // namespace qz
