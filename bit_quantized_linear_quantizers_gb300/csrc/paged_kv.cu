// paged_kv.cu -- the bookkeeping and the writes of the paged FP8 KV cache:
//  * block tables and slot maps of a step from the requests' lengths;
//  * new tokens quantized into their pages, one scale per (page, head)
//    ("量化部署实战", KV Cache 量化, 伪量化实现: scale = max(amax, 1e-12) / 448,
//    code = E4M3(clamp(x / scale))).
#include "qz_internal.cuh"
#include "qz_paged.cuh"

#include <algorithm>

namespace qz {

namespace {

// --------------------------------------------------- block tables, slot maps

constexpr int kTableThreads = 1024;

// Inclusive sums over the block of two counts packed in one word (pages in the
// high half, tokens in the low half; each total is below 2^31, so no carry).
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* warp_sums, uint64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    uint64_t w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return v + (warp > 0 ? before : 0);
}

// Every CTA sums all the lengths itself (4 bytes per request and array; no
// second launch, no traffic between CTAs) and maps its share of the tokens; CTA
// 0 also writes the per-request outputs. The token at offset 0 of a page is the
// one that records the page in the table, so each entry has one writer. Bound by latency: 3.1 us for 64
// requests of one token, 3.7 for 500 of up to 384 (a floor of 0.1 for their bytes).
__global__ void __launch_bounds__(kTableThreads)
block_tables_kernel(const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int B, int shift,
                    int32_t* block_table, int max_blocks, int64_t ld_table, const int32_t* __restrict__ free_pages,
                    int n_free, const int32_t* __restrict__ free_head, int32_t* __restrict__ kv_lens,
                    int32_t* __restrict__ cu_new, int32_t* __restrict__ slot_map, int32_t* __restrict__ positions,
                    int n_slots, int32_t* __restrict__ free_head_out) {
    __shared__ uint64_t warp_sums[32];
    __shared__ int32_t s_cu[kTableThreads], s_ctx[kTableThreads], s_have[kTableThreads];
    __shared__ int64_t s_at[kTableThreads];
    __shared__ int s_head;
    pdl_wait();
    const int tid = threadIdx.x;
    const int page = 1 << shift, mask = page - 1;
    const int64_t head = __ldg(free_head);
    int64_t pages = 0, tokens = 0;                // of the requests before this chunk
    if (tid == 0) s_head = (int)head;
    for (int b0 = 0; b0 < B; b0 += kTableThreads) {
        const int b = b0 + tid;
        int ctx = 0, add = 0;
        if (b < B) {
            ctx = max(__ldg(ctx_lens + b), 0);
            add = max(__ldg(new_lens + b), 0);
        }
        const int have = (int)(((int64_t)ctx + mask) >> shift);
        const int64_t want = ((int64_t)ctx + add + mask) >> shift;
        const bool fits = want <= max_blocks;
        const int need = fits ? (int)want - have : 0;
        uint64_t total;
        const uint64_t upto = block_scan((uint64_t)(uint32_t)need << 32 | (uint32_t)add, warp_sums, total);
        const int64_t last = head + pages + (int64_t)(upto >> 32);       // one past the request's last free page
        const int64_t cu = tokens + (int64_t)(uint32_t)upto - add;
        const bool ok = fits && (need == 0 || (last <= n_free && last - need >= 0));
        s_cu[tid] = (int)cu;
        s_ctx[tid] = ctx;
        s_have[tid] = ok ? have : -1;
        s_at[tid] = last - need;
        if (ok && need > 0) atomicMax(&s_head, (int)last);               // a maximum: the order does not matter
        if (blockIdx.x == 0 && b < B) {
            kv_lens[b] = ok ? ctx + add : ctx;
            cu_new[b] = (int)cu;
        }
        __syncthreads();
        const int64_t t_end = tokens + (int64_t)(uint32_t)total;
        const int n = min(kTableThreads, B - b0);
        for (int64_t t = (int64_t)blockIdx.x * kTableThreads + tid; t < t_end; t += (int64_t)gridDim.x * kTableThreads) {
            if (t < tokens) continue;
            int lo = 0, hi = n - 1;               // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_cu[mid] <= t) lo = mid; else hi = mid - 1;
            }
            const int pos = s_ctx[lo] + (int)(t - s_cu[lo]), j = pos >> shift, had = s_have[lo];
            int slot = -1;
            if (had >= 0) {                       // admitted: j < want <= max_blocks
                int32_t* row = block_table + (int64_t)(b0 + lo) * ld_table;
                const int p = j < had ? row[j] : __ldg(free_pages + s_at[lo] + (j - had));
                if ((pos & mask) == 0) row[j] = p;
                slot = p >= 0 && p <= 0x7fffffff >> shift ? (p << shift) + (pos & mask) : -1;
            }
            if (t < n_slots) {
                slot_map[t] = slot;
                if (positions) positions[t] = pos;
            }
        }
        pages += (int64_t)(total >> 32);
        tokens = t_end;
        __syncthreads();
    }
    for (int64_t t = tokens + (int64_t)blockIdx.x * kTableThreads + tid; t < n_slots;
         t += (int64_t)gridDim.x * kTableThreads) {
        slot_map[t] = -1;
        if (positions) positions[t] = 0;
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) {
        cu_new[B] = (int)tokens;
        free_head_out[0] = s_head;
    }
    pdl_trigger();
}

// ------------------------------------------------------------- cache write

constexpr int kAppendThreads = 256;
constexpr int kStrip = 16;                        // tokens that one warp holds in registers
template <typename T> constexpr int kAppendCtas = sizeof(T) == 2 ? 4 : 3;        // CTAs that an SM holds

__device__ __forceinline__ void e4m3_codes8(const float v[8], const Recip& d, uint32_t& lo, uint32_t& hi) {
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        div1x2(v[j], v[j + 1], d, y[j], y[j + 1]);
        y[j] = sign_of(y[j], v[j]);
        y[j + 1] = sign_of(y[j + 1], v[j + 1]);
    }
    lo = e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16;
    hi = e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16;
}

// Eight input values as they lie in memory (bf16: 16 bytes, fp32: 32), held so until
// they are encoded: widened on arrival, 16 tokens of bf16 took 64 registers a lane instead
// of 32, and half as many CTAs fitted an SM.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void load(const uint16_t* p) { w = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float amax() const {
        uint32_t m = 0;                           // both halves at once: the order of the bits below the sign is the values'
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) m = __vmaxu2(m, x[i] & 0x7FFF7FFFu);
        if ((m & 0xFFFFu) > 0x7F80u || (m >> 16) > 0x7F80u) {          // a NaN: left out of the maximum, as fmaxf does
            float v[8], f = 0.0f;
            widen(v);
#pragma unroll
            for (int i = 0; i < 8; i++) f = fmaxf(f, fabsf(v[i]));
            return f;
        }
        return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
    __device__ __forceinline__ float amax() const {
        return fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(a.z), fabsf(a.w))),
                     fmaxf(fmaxf(fabsf(b.x), fabsf(b.y)), fmaxf(fabsf(b.z), fabsf(b.w))));
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
};

// A group of W = page_size / 16 warps takes the pages whose first new token
// lies in its window of `window` tokens, for one head of K or V (blockIdx.y).
// Warp w of the group holds tokens 16w .. 16w+15 of the page's run in
// registers, D / 8 lanes of 8 values per token, so x is read once; the amax
// goes through shared memory. A group takes page after page in series: slots, rows,
// maximum, codes. Prompts are bound by that chain rather than by a unit (16 thousand bf16 tokens, 8 heads of
// 128, pages of 16: 27 us, 62 % of the measured copy rate, SMs 55 % busy; 5, 6 or 8 CTAs on an SM 36, 40, 46: they
// spill), single tokens by latency (64 of them: 5.4 us).
template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas<T>)
kv_append_kernel(const T* __restrict__ k, const T* __restrict__ v, int64_t tokens, int64_t ldk, int64_t ldv,
                 const int32_t* __restrict__ slot_map, qz_paged_kv c, int shift, int window) {
    constexpr int kWarps = kAppendThreads / 32;
    constexpr int kRowLanes = D / 8, kRows = 32 / kRowLanes, kSteps = kStrip / kRows;
    __shared__ float red[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = 1 << shift, W = P / kStrip;
    const int group = warp / W, wig = warp % W;
    const int h = blockIdx.y >> 1;
    const bool isv = blockIdx.y & 1;
    const T* x = (isv ? v : k) + (int64_t)h * D;
    const int64_t ld = isv ? ldv : ldk;
    uint8_t* codes = (isv ? c.v_codes : c.k_codes) + (int64_t)h * P * D;
    float* scales = (isv ? c.v_scale : c.k_scale) + h;
    auto page_of = [&](int64_t t) {
        if (t < 0 || t >= tokens) return -1;
        const int s = __ldg(slot_map + t), p = s >> shift;
        return s >= 0 && p < c.num_pages ? p : -1;
    };
    const int64_t w0 = ((int64_t)blockIdx.x * (kWarps / W) + group) * window;
    const int64_t w1 = min(w0 + window, tokens);
    for (int64_t c0 = w0; c0 < w1; c0 += 32) {    // uniform over the group
        const int64_t t = c0 + lane;
        const int p = t < w1 ? page_of(t) : -1;
        uint32_t leaders = __ballot_sync(0xffffffffu, p >= 0 && page_of(t - 1) != p);
        while (leaders) {
            const int l = __ffs(leaders) - 1;
            leaders &= leaders - 1;
            const int64_t t0 = c0 + l;
            const int pg = __shfl_sync(0xffffffffu, p, l);
            int n = 0;                            // tokens of the page's run, at most P
            for (int i = 0; i < P; i += 32) {
                const uint32_t same = __ballot_sync(0xffffffffu, i + lane < P && page_of(t0 + i + lane) == pg);
                n += same == 0xffffffffu ? 32 : __ffs(~same) - 1;
                if (same != 0xffffffffu) break;
            }
            const int off0 = __ldg(slot_map + t0) & (P - 1);
            const int r0 = wig * kStrip + lane / kRowLanes, d0 = (lane % kRowLanes) * 8;
            Raw8<T> val[kSteps];
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < kSteps; i++) {
                const int r = r0 + i * kRows;
                if (r < n) val[i].load(x + (t0 + r) * ld + d0);
                else val[i].zero();
            }
#pragma unroll
            for (int i = 0; i < kSteps; i++) m = fmaxf(m, val[i].amax());
            m = warp_max(m, 32);
            if (W > 1) {                          // the group's warps alone
                if (lane == 0) red[warp] = m;
                asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");
                for (int i = 0; i < W; i++) m = fmaxf(m, red[group * W + i]);
            }
            const int64_t si = (int64_t)pg * c.heads;
            const float fresh = div_rn(fmaxf(m, kAmaxMin), kFp8Max);
            const float was = off0 ? scales[si] : 0.0f;
            const float s = fmaxf(was, fresh);
            uint8_t* base = codes + (int64_t)pg * c.page_stride;
            const Recip d(s);
#pragma unroll
            for (int i = 0; i < kSteps; i++) {
                const int r = r0 + i * kRows;
                if (r < n) {
                    const int off = __ldg(slot_map + t0 + r) & (P - 1);
                    uint2 o;
                    float y[8];
                    val[i].widen(y);
                    e4m3_codes8(y, d, o.x, o.y);
                    *reinterpret_cast<uint2*>(base + off * D + d0) = o;
                }
            }
            if (off0 && s > was)                  // older tokens: the values they stood for, under the new scale
                for (int i = wig * 32 + lane; i < off0 * (D / 8); i += W * 32) {
                    uint2 o = reinterpret_cast<uint2*>(base)[i];
                    float y[8];
#pragma unroll
                    for (int j = 0; j < 8; j++) y[j] = __fmul_rn(e4m3_value((j < 4 ? o.x : o.y) >> (8 * (j & 3))), was);
                    e4m3_codes8(y, d, o.x, o.y);
                    reinterpret_cast<uint2*>(base)[i] = o;
                }
            if (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(W * 32) : "memory");   // `was` and `red` read by all
            else __syncwarp();
            if (wig == 0 && lane == 0) scales[si] = s;
        }
    }
    pdl_trigger();
}

int log2_page(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

template <typename T>
qz_status append_launch(const T* k, const T* v, int64_t tokens, int64_t ldk, int64_t ldv, const int32_t* slots,
                        const qz_paged_kv& c, cudaStream_t st) {
    const int P = c.page_size, groups = kAppendThreads / 32 / (P / kStrip);
    // Window of a group: one token while that gives every group work at once
    // (single tokens, each its own page), up to a page when there are many. (1200 fp32 tokens of 4 heads
    // of 64: 4.2 us so, 6.0 with windows of one token, which are mostly empty; 64 single tokens of 8 heads of 128: 5.4 us,
    // 7.8 with windows that leave half the groups without one.)
    const int64_t units = tokens * c.heads * 2, room = (int64_t)num_sms() * kAppendCtas<T> * groups;
    const int window = (int)std::min<int64_t>(P, std::max<int64_t>(1, units / room));
    const int64_t gx = (tokens + (int64_t)window * groups - 1) / ((int64_t)window * groups);
    if (gx > 0x7fffffff || c.heads > 32767) return QZ_ERR_SHAPE;
    const dim3 grid((unsigned)gx, (unsigned)c.heads * 2), block(kAppendThreads);
    auto* fn = c.head_dim == 64 ? kv_append_kernel<T, 64> : kv_append_kernel<T, 128>;
    return launch_pdl(fn, grid, block, 0, st, k, v, tokens, ldk, ldv, slots, c, log2_page(P), window);
}

} // namespace

qz_status block_tables_launch(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                              int32_t* block_table, int max_blocks, int64_t ld_table, const int32_t* free_pages,
                              int n_free, const int32_t* free_head, int32_t* kv_lens, int32_t* cu_new,
                              int32_t* slot_map, int32_t* positions, int n_slots, int32_t* free_head_out,
                              cudaStream_t st) {
    const int ctas = std::max(1, std::min((n_slots + kTableThreads - 1) / kTableThreads, num_sms()));
    return launch_pdl(block_tables_kernel, dim3(ctas), dim3(kTableThreads), 0, st, ctx_lens, new_lens, B,
                      log2_page(page_size), block_table, max_blocks, ld_table, free_pages, n_free, free_head, kv_lens,
                      cu_new, slot_map, positions, n_slots, free_head_out);
}

qz_status kv_append_paged_launch(const void* k, const void* v, qz_dtype xt, int64_t tokens, int64_t ldk, int64_t ldv,
                                 const int32_t* slot_map, const qz_paged_kv& cache, cudaStream_t st) {
    if (xt == QZ_F32)
        return append_launch((const float*)k, (const float*)v, tokens, ldk, ldv, slot_map, cache, st);
    return append_launch((const uint16_t*)k, (const uint16_t*)v, tokens, ldk, ldv, slot_map, cache, st);
}

} // namespace qz
