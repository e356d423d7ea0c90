// residual_norm.cu -- the norm around a block, in one pass over the residual stream:
//   z = sum_j w[j] y[row_j]  (the experts' rows by their gates, or the block's one row)
//   z = z gamma_y / sqrt(mean z^2 + eps)     (where the block has a norm behind it)
//   r = x + alpha z;   n = r gamma / sqrt(mean r^2 + eps)
// and of r and n what the next block reads: r in x's type, n in bf16, n as E4M3 codes
// with a scale per 128 columns. Bound by memory: everything is read and written once.
//
// A thread holds NC chunks of 8 columns in registers from the first load to the last store,
// so that the row is never read again after its sum of squares is known. 16 neighbouring threads hold 128
// neighbouring columns: a scale's amax is four shuffles. Two forms:
//  STREAM   one row of the block, or none, and no norm behind it: a persistent grid, and the next row's loads are under
//           way while this row is summed, normed and stored (8192 rows of 4096 bf16: 62 -> 53 us)
//  GATHER   a CTA per row and 64 warps an SM (32 registers): here the loads are many or the sums two, and other rows hide
//           them better than a deeper row does (8192 x 8 rows of 2048: 73 us, with the next row's loads under way 95, with
//           two of the eight rows in flight and 40 registers 115; 5000 rows of 4096 fp32 normed twice: 54, 59 and 79)
#include "qz_moe.cuh"

#include <algorithm>

namespace qz {

namespace {

constexpr int kMaxThreads = 1024, kSmThreads = 1024;          // of a CTA; of an SM's that are resident with 64 registers
constexpr int kGroupThreads = 256;                            // rows of fewer threads share a CTA of as many

// Eight values as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    static __device__ __forceinline__ void read(const uint16_t* p, float v[8]) {
        Raw8 r;
        r.load(p);
        r.values(v);
    }
    __device__ __forceinline__ void values(float v[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    static __device__ __forceinline__ void read(const float* p, float v[8]) {
        Raw8 r;
        r.load(p);
        r.values(v);
    }
    __device__ __forceinline__ void values(float v[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

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

// g v / root. The quotient is rounded once, as a division is: 1 / root is held in two parts, the first of them rounded down, so
// that both are positive and a zero keeps its sign. (v times the rounded reciprocal gave 0.99999994 for a row of 49s, 10 % more
// of the bf16 values off and scales of the codes off by a last place, in the same time.) A sum of squares past fp32's range
// has an infinite root: all finite values become 0.
struct Root {
    float inv, rest;
    __device__ __forceinline__ Root(float sum, int n, float eps) {
        const float root = sqrtf(sum / (float)n + eps);
        inv = __frcp_rd(root);
        rest = inv == 0.0f ? 0.0f : fmaf(-root, inv, 1.0f) * inv;
    }
    // g = g v / root for eight values, two an instruction where that spills nothing (one chunk a thread: 8192 rows of 4096
    // bf16 53.8 us, by one 54.5; two chunks: 2000 rows of 16384 fp32 101 and 94)
    template <bool PAIRS> __device__ __forceinline__ void scale(const float v[8], float g[8]) const {
        if constexpr (!PAIRS) {
#pragma unroll
            for (int e = 0; e < 8; e++) g[e] *= fmaf(v[e], inv, v[e] * rest);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2)
                asm("{ .reg .b64 v, g, i, r;\n\t"
                    "mov.b64 v, {%2, %3}; mov.b64 g, {%0, %1}; mov.b64 i, {%4, %4}; mov.b64 r, {%5, %5};\n\t"
                    "mul.rn.f32x2 r, v, r;\n\t"
                    "fma.rn.f32x2 v, v, i, r;\n\t"
                    "mul.rn.f32x2 g, v, g;\n\t"
                    "mov.b64 {%0, %1}, g; }"
                    : "+f"(g[e]), "+f"(g[e + 1]) : "f"(v[e]), "f"(v[e + 1]), "f"(inv), "f"(rest));
        }
    }
};

// Codes of chunk c of row t, with a scale per 16 chunks; all lanes of a warp come here.
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t t, int c, bool there, const float n[8]) {
    float am = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e++) am = fmaxf(am, fabsf(n[e]));
    am = warp_max(am, 16);
    if (!there) return;
    const float sc = div1(fmaxf(am, kAmaxMin), Recip(kFp8Max));
    const Recip d(sc);
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; e++) p[e] = e4m3x2(sign_of(div1(n[2 * e], d), n[2 * e]), sign_of(div1(n[2 * e + 1], d), n[2 * e + 1]));
    *reinterpret_cast<uint2*>(a.codes + t * a.hidden + 8 * c) = make_uint2(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410));
    if ((c & 15) == 0) a.scales[t * (a.hidden / 128) + c / 16] = sc;
}

// T: x's type (float, or bf16 as its bits); NC: chunks of 8 columns a thread. per_row: threads of a row, a multiple of 32.
template <typename T, int NC>
__global__ void __launch_bounds__(kMaxThreads)
rmsnorm_stream_kernel(const __grid_constant__ NormArgs a, const int per_row) {
    __shared__ float s_red[2][kMaxThreads / 32];
    pdl_wait();
    const int group = threadIdx.x / per_row, groups = blockDim.x / per_row, tid = threadIdx.x % per_row, lane = threadIdx.x & 31;
    const int chunks = a.hidden >> 3, warps = per_row >> 5;
    int slot = 0;
    // Sum over the row's threads, in the same order for everybody.
    auto row_sum = [&](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (warps == 1) return v;
        float* red = s_red[slot] + group * warps;
        slot ^= 1;                                            // the next sum's warps may be ahead of this one's readers
        if (lane == 0) red[tid >> 5] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(per_row) : "memory");
        float s = 0.0f;
        for (int i = 0; i < warps; i++) s += red[i];
        return s;
    };
    Raw8<T> gamma[NC], x[NC];
    Raw8<uint16_t> y[NC];
    float gate = 1.0f;
    auto read = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int c = i * per_row + tid;
            x[i].zero();
            y[i].zero();
            if (t < a.tokens && c < chunks) {
                x[i].load(static_cast<const T*>(a.x) + t * a.ldx + 8 * c);
                if (a.has_block) y[i].load(a.b.y + t * a.b.ldy + 8 * c);
            }
        }
        if (a.has_block && a.b.weights && t < a.tokens) gate = a.b.weights[t];
    };
#pragma unroll
    for (int i = 0; i < NC; i++) {
        const int c = i * per_row + tid;
        gamma[i].zero();
        if (a.gamma && c < chunks) gamma[i].load(static_cast<const T*>(a.gamma) + 8 * c);
    }
    int64_t t = (int64_t)blockIdx.x * groups + group;
    read(t);
    for (; t < a.tokens;) {
        const int64_t next = t + (int64_t)gridDim.x * groups;
        float r[NC][8], z[NC][8];
#pragma unroll
        for (int i = 0; i < NC; i++) {
            x[i].values(r[i]);
            y[i].values(z[i]);
        }
        if (a.has_block) {
            if (a.b.weights) {
#pragma unroll
                for (int i = 0; i < NC; i++)
#pragma unroll
                    for (int e = 0; e < 8; e++) z[i][e] *= gate;
            }
#pragma unroll
            for (int i = 0; i < NC; i++)
#pragma unroll
                for (int e = 0; e < 8; e++) r[i][e] = fmaf(a.b.alpha, z[i][e], r[i][e]);
        }
        read(next);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int c = i * per_row + tid;
            if (a.x_out && c < chunks) store8(static_cast<T*>(a.x_out) + t * a.ldo + 8 * c, r[i]);
#pragma unroll
            for (int e = 0; e < 8; e++) s = fmaf(r[i][e], r[i][e], s);
        }
        if (a.gamma) {
            const Root root(row_sum(s), a.hidden, a.eps);
#pragma unroll
            for (int i = 0; i < NC; i++) {
                const int c = i * per_row + tid;
                float n[8];
                gamma[i].values(n);
                root.scale<NC == 1>(r[i], n);
                if (a.normed && c < chunks) store8(a.normed + t * a.hidden + 8 * c, n);
                if (a.codes) store_codes(a, t, c, c < chunks, n);
            }
        }
        t = next;
    }
    pdl_trigger();
}

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

// GATHER, or a norm behind the block: a CTA per row.
template <typename T, int NC>
__global__ void __launch_bounds__(kMaxThreads, NC == 1 ? 2 : 1)
residual_rmsnorm_kernel(const __grid_constant__ NormArgs a) {
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
        if (c < chunks) Raw8<T>::read(x + 8 * c, r[i]);
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
                    Raw8<uint16_t>::read(a.b.y + row * a.b.ldy + 8 * c, v);
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
            const Root root(block_sum(s, red[0]), a.hidden, a.eps);
#pragma unroll
            for (int i = 0; i < NC; i++) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < chunks) {
                    float g[8];
                    Raw8<T>::read(static_cast<const T*>(a.b.gamma) + 8 * c, g);
                    root.scale<NC == 1>(z[i], g);
#pragma unroll
                    for (int e = 0; e < 8; e++) z[i][e] = g[e];
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
        const Root root(block_sum(s, red[1]), a.hidden, a.eps);
#pragma unroll
        for (int i = 0; i < NC; i++) {
            const int c = i * blockDim.x + threadIdx.x;
            float n[8];
#pragma unroll
            for (int e = 0; e < 8; e++) n[e] = 0.0f;
            if (c < chunks) {
                Raw8<T>::read(static_cast<const T*>(a.gamma) + 8 * c, n);
                root.scale<NC == 1>(r[i], n);
                if (a.normed) store8(a.normed + t * a.hidden + 8 * c, n);
            }
            if (a.codes) store_codes(a, t, c, c < chunks, n);
        }
    }
    pdl_trigger();
}

template <typename T, int NC>
qz_status stream_launch(const NormArgs& a, cudaStream_t st) {
    const int per_row = ((a.hidden / 8 + NC - 1) / NC + 31) / 32 * 32, groups = std::max(1, kGroupThreads / per_row);
    const int threads = per_row * groups;
    const int64_t ctas = (a.tokens + groups - 1) / groups, most = (int64_t)num_sms() * std::max(1, kSmThreads / threads);
    return launch_pdl(rmsnorm_stream_kernel<T, NC>, dim3((unsigned)std::min(ctas, most)), dim3(threads), 0, st, a, per_row);
}

template <typename T>
qz_status launch(const NormArgs& a, cudaStream_t st) {
    const int chunks = a.hidden / 8;
    if (!a.has_block || (a.b.k == 1 && !a.b.token_row && !a.b.gamma))
        return chunks <= kMaxThreads ? stream_launch<T, 1>(a, st) : stream_launch<T, 2>(a, st);
    const int nc = chunks <= kMaxThreads ? 1 : 2;
    const dim3 grid((unsigned)a.tokens), block(((chunks + nc - 1) / nc + 31) / 32 * 32);
    if (nc == 1) return launch_pdl(residual_rmsnorm_kernel<T, 1>, grid, block, 0, st, a);
    return launch_pdl(residual_rmsnorm_kernel<T, 2>, grid, block, 0, st, a);
}

} // namespace

qz_status residual_rmsnorm_launch(const NormArgs& a, qz_dtype xt, cudaStream_t st) {
    return xt == QZ_F32 ? launch<float>(a, st) : launch<uint16_t>(a, st);
}

} // namespace qz
