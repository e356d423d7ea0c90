// residual_norm.cu -- the norm around a block, in one pass over the residual stream:
//   z = sum_j w[j] y[row_j]  (the experts' rows by their gates, or the block's one row)
//   z = z gamma_y / sqrt(mean z^2 + eps)     (where the block has a norm behind it)
//   r = x + alpha z;   n = r gamma / sqrt(mean r^2 + eps)
// and of r and n what the next block reads: r in x's type, n in bf16, n as E4M3 codes
// with a scale per 128 columns. Bound by memory: everything is read and written once.
//
// A CTA per row. A thread holds NC chunks of 8 columns in registers from the first load
// to the last store, so that the row is never read again after its sum of squares is
// known; its loads (x, and a chunk of each of the k rows of y) do not wait for one
// another. 16 neighbouring threads hold 128 neighbouring columns: a scale's amax is
// four shuffles.
#include "qz_moe.cuh"

namespace qz {

namespace {

constexpr int kMaxThreads = 512;

template <typename T> __device__ __forceinline__ void load8(const T* p, float v[8]);
template <> __device__ __forceinline__ void load8<float>(const float* p, float v[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void widen8(const uint4& a, float v[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <> __device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float v[8]) {
    widen8(*reinterpret_cast<const uint4*>(p), v);
}
__device__ __forceinline__ uint4 bf16x8(const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float v[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float v[8]) { *reinterpret_cast<uint4*>(p) = bf16x8(v); }

// Sum over the CTA, in the same order for everybody; `red` holds a value per warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < warps; i++) s += red[i];
    return s;
}

// T: x's type (float, or bf16 as its bits); NC: chunks of 8 columns a thread.
template <typename T, int NC>
__global__ void __launch_bounds__(kMaxThreads)
residual_rmsnorm_kernel(const NormArgs a) {
    __shared__ float red[2][kMaxThreads / 32];
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int chunks = a.hidden >> 3;
    const T* x = static_cast<const T*>(a.x) + t * a.ldx;
    float r[NC][8];
#pragma unroll
    for (int i = 0; i < NC; i++) {
        const int c = i * blockDim.x + threadIdx.x;
#pragma unroll
        for (int e = 0; e < 8; e++) r[i][e] = 0.0f;
        if (c < chunks) load8<T>(x + 8 * c, r[i]);
    }
    if (a.has_block) {
        float z[NC][8];
#pragma unroll
        for (int i = 0; i < NC; i++)
#pragma unroll
            for (int e = 0; e < 8; e++) z[i][e] = 0.0f;
        for (int j = 0; j < a.b.k; j++) {
            const int64_t at = t * a.b.k + j;
            const int64_t row = a.b.token_row ? (int64_t)a.b.token_row[at] : at;
            if (row < 0 || row >= a.b.rows) continue;
            const float w = a.b.weights ? a.b.weights[at] : 1.0f;
#pragma unroll
            for (int i = 0; i < NC; i++) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < chunks) {
                    float v[8];
                    load8<uint16_t>(a.b.y + row * a.b.ldy + 8 * c, v);
#pragma unroll
                    for (int e = 0; e < 8; e++) z[i][e] = fmaf(w, v[e], z[i][e]);
                }
            }
        }
        if (a.b.gamma) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) s = fmaf(z[i][e], z[i][e], s);
            const float inv = 1.0f / sqrtf(block_sum(s, red[0]) / (float)a.hidden + a.eps);
#pragma unroll
            for (int i = 0; i < NC; i++) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < chunks) {
                    float g[8];
                    load8<T>(static_cast<const T*>(a.b.gamma) + 8 * c, g);
#pragma unroll
                    for (int e = 0; e < 8; e++) z[i][e] = z[i][e] * inv * g[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NC; i++)
#pragma unroll
            for (int e = 0; e < 8; e++) r[i][e] = fmaf(a.b.alpha, z[i][e], r[i][e]);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; i++) {
        const int c = i * blockDim.x + threadIdx.x;
        if (a.x_out && c < chunks) store8(static_cast<T*>(a.x_out) + t * a.ldo + 8 * c, r[i]);
#pragma unroll
        for (int e = 0; e < 8; e++) s = fmaf(r[i][e], r[i][e], s);
    }
    if (a.gamma) {
        const float inv = 1.0f / sqrtf(block_sum(s, red[1]) / (float)a.hidden + a.eps);
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int c = i * blockDim.x + threadIdx.x;
            float n[8];
#pragma unroll
            for (int e = 0; e < 8; e++) n[e] = 0.0f;
            if (c < chunks) {
                float g[8];
                load8<T>(static_cast<const T*>(a.gamma) + 8 * c, g);
#pragma unroll
                for (int e = 0; e < 8; e++) n[e] = r[i][e] * inv * g[e];
                if (a.normed) store8(a.normed + t * a.hidden + 8 * c, n);
            }
            if (a.codes) {
                float am = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) am = fmaxf(am, fabsf(n[e]));
                am = warp_max(am, 16);
                if (c < chunks) {
                    const float sc = div1(fmaxf(am, kAmaxMin), Recip(kFp8Max));
                    const Recip d(sc);
                    uint32_t p[4];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        p[e] = e4m3x2(sign_of(div1(n[2 * e], d), n[2 * e]), sign_of(div1(n[2 * e + 1], d), n[2 * e + 1]));
                    *reinterpret_cast<uint2*>(a.codes + t * a.hidden + 8 * c) =
                        make_uint2(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410));
                    if ((c & 15) == 0) a.scales[t * (a.hidden / 128) + c / 16] = sc;
                }
            }
        }
    }
    pdl_trigger();
}

template <typename T>
qz_status launch(const NormArgs& a, cudaStream_t st) {
    const int chunks = a.hidden / 8;
    const int nc = chunks <= kMaxThreads ? 1 : chunks <= 2 * kMaxThreads ? 2 : 4;
    const int threads = ((chunks + nc - 1) / nc + 31) / 32 * 32;
    const dim3 grid((unsigned)a.tokens);
    switch (nc) {
    case 1: return launch_pdl(residual_rmsnorm_kernel<T, 1>, grid, dim3(threads), 0, st, a);
    case 2: return launch_pdl(residual_rmsnorm_kernel<T, 2>, grid, dim3(threads), 0, st, a);
    default: return launch_pdl(residual_rmsnorm_kernel<T, 4>, grid, dim3(threads), 0, st, a);
    }
}

} // namespace

qz_status residual_rmsnorm_launch(const NormArgs& a, qz_dtype xt, cudaStream_t st) {
    return xt == QZ_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

} // namespace qz
