// moe_gemm_fp8.cu -- the experts' products over ragged rows, block-scaled FP8:
//   P[r, n] = sum_kb sA[a, kb] sW[e, n/128, kb] sum_{k in kb} qA[a, k] qW[e, n, k]
// with a = row_token[r] and e the expert whose rows contain r; output in bf16, or SwiGLU of
// the gate and up columns encoded as E4M3 with a scale per 128 columns.
//
// Simple form: a CTA takes 16 rows of one expert and 128 columns (of gate and of up with SwiGLU),
// a thread one column; the rows' codes lie in shared memory, widened, a block of 128 of K at a time.
#include "qz_moe.cuh"

namespace qz {

namespace {

constexpr int kRows = 16;

template <bool SWIGLU>
__global__ void __launch_bounds__(SWIGLU ? 256 : 128)
moe_gemm_kernel(const MoeGemmArgs a) {
    __shared__ float sx[kRows][128];
    __shared__ float ss[kRows];
    __shared__ int64_t sat[kRows];
    pdl_wait();
    // the expert and the rows of tile blockIdx.y
    int e = 0, lo = 0, hi = 0;
    int64_t left = blockIdx.y;
    for (; e < a.experts; e++) {
        lo = (int)min(max((int64_t)a.offsets[e], (int64_t)0), a.rows);
        hi = (int)min(max((int64_t)a.offsets[e + 1], (int64_t)lo), a.rows);
        const int64_t tiles = (hi - lo + kRows - 1) / kRows;
        if (left < tiles) break;
        left -= tiles;
    }
    if (e == a.experts) return;
    const int r0 = lo + (int)left * kRows, nr = min(kRows, hi - r0), nkb = a.K / 128;
    const int half = threadIdx.x >> 7, c = threadIdx.x & 127;
    const int n0 = blockIdx.x * 128 + (half ? a.N / 2 : 0);
    if (threadIdx.x < kRows) {
        int64_t at = -1;
        if ((int)threadIdx.x < nr) at = a.row_token ? a.row_token[r0 + threadIdx.x] : r0 + threadIdx.x;
        sat[threadIdx.x] = at < a.tokens ? at : -1;
    }
    __syncthreads();
    const uint8_t* w = a.qW + ((int64_t)e * a.N + n0 + c) * a.K;
    const float* ws = a.sW + ((int64_t)e * (a.N / 128) + n0 / 128) * nkb;
    float acc[kRows] = {};
    for (int kb = 0; kb < nkb; kb++) {
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * 128; i += blockDim.x) {
            const int64_t at = sat[i >> 7];
            sx[i >> 7][i & 127] = at >= 0 ? e4m3_value(a.qA[at * a.K + kb * 128 + (i & 127)]) : 0.0f;
        }
        if (threadIdx.x < kRows) ss[threadIdx.x] = sat[threadIdx.x] >= 0 ? a.sA[sat[threadIdx.x] * nkb + kb] : 0.0f;
        __syncthreads();
        float p[kRows] = {};
        for (int k = 0; k < 128; k += 4) {
            const uint32_t q = *reinterpret_cast<const uint32_t*>(w + kb * 128 + k);
            for (int j = 0; j < 4; j++) {
                const float v = e4m3_value(q >> (8 * j));
#pragma unroll
                for (int r = 0; r < kRows; r++) p[r] = fmaf(sx[r][k + j], v, p[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; r++) acc[r] = fmaf(p[r], ss[r] * ws[kb], acc[r]);
    }
    if constexpr (!SWIGLU) {
        for (int r = 0; r < nr; r++) {
            const __nv_bfloat16 y = __float2bfloat16_rn(acc[r]);
            a.Y[(int64_t)(r0 + r) * a.N + n0 + c] = *reinterpret_cast<const uint16_t*>(&y);
        }
    } else {
        __syncthreads();
        if (half)
#pragma unroll
            for (int r = 0; r < kRows; r++) sx[r][c] = acc[r];
        __syncthreads();
        float h[kRows];
        if (!half)
#pragma unroll
            for (int r = 0; r < kRows; r++) h[r] = acc[r] / (1.0f + expf(-acc[r])) * sx[r][c];
        __syncthreads();
        if (!half)
#pragma unroll
            for (int r = 0; r < kRows; r++) sx[r][c] = h[r];
        __syncthreads();
        if (half) return;
        const int I = a.N / 2;
        for (int r = 0; r < nr; r++) {
            float am = 0.0f;
            for (int i = 0; i < 128; i++) am = fmaxf(am, fabsf(sx[r][i]));
            const float sc = div1(fmaxf(am, kAmaxMin), Recip(kFp8Max));
            const float v = sx[r][c];
            a.codes[(int64_t)(r0 + r) * I + n0 + c] = (uint8_t)e4m3_code(sign_of(div1(v, Recip(sc)), v));
            if (c == 0) a.scales[(int64_t)(r0 + r) * (I / 128) + n0 / 128] = sc;
        }
    }
}

} // namespace

qz_status moe_gemm_fp8_launch(const MoeGemmArgs& a, cudaStream_t st) {
    const int64_t tiles = a.rows / kRows + (a.rows < a.experts ? a.rows : a.experts);
    if (a.Y) return launch_pdl(moe_gemm_kernel<false>, dim3(a.N / 128, (unsigned)tiles), dim3(128), 0, st, a);
    return launch_pdl(moe_gemm_kernel<true>, dim3(a.N / 256, (unsigned)tiles), dim3(256), 0, st, a);
}

} // namespace qz
