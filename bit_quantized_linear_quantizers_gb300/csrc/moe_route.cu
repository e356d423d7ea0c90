// moe_route.cu -- routing of tokens to experts and the order of their rows.
//
// Selection: a warp per token, expert e in lane e % 32. The top_k are taken one by one:
// every lane's best key, a warp maximum over the keys as ordered integers, the lowest
// index among those that have it. Without bias and groups the keys are the logits, which
// order the experts exactly as their scores do.
//
// With them keys are rounded sums, and two that 32 bits cannot tell apart could change
// places. Every comparison that decides something is therefore checked against a bound
// on its rounding errors, and a token that has one too close is chosen again in 64 bits
// (pick_wide). That is rare: the bound is a few units in the last place of the scores.
//
// The plan: the rows of an expert in the order of the tokens, whatever order CTAs run in.
// A CTA of kBlockTokens tokens counts its pairs per expert and gives each pair its rank
// among them; the second kernel adds, per expert, the counts of the CTAs before it and the rows of the
// experts before it. Up to kBlockTokens tokens are one CTA and one launch.
#include "qz_moe.cuh"

#include <cfloat>
#include <climits>

namespace qz {

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kBlockTokens = 128, kWarpTokens = kBlockTokens / kWarps;
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// NaN counts as -inf, +inf as the largest finite value.
__device__ __forceinline__ float finite_logit(float l) { return fminf(l != l ? -INFINITY : l, FLT_MAX); }
__device__ __forceinline__ float finite_bias(float b) { return fminf(b != b ? -INFINITY : b, FLT_MAX); }

// Integers in the order of the floats; 0 is below all of them (closed experts).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);              // -0 and +0 are one value
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}
__device__ __forceinline__ double sigmoid(double l) {
    const double e = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ double warp_max_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// (best, second) of two pairs of largest values.
template <typename V>
__device__ __forceinline__ void merge2(V& b, V& s, V ob, V os) {
    const V lo = b < ob ? b : ob;
    b = b < ob ? ob : b;
    s = s < os ? os : s;
    s = s < lo ? lo : s;
}

// A group's score of its best two keys; nothing open: -inf.
template <typename V>
__device__ __forceinline__ V group_score(V b, V s, int best) {
    return best == 2 && s > (V)-INFINITY ? b + s : b;
}

// How far a key v of a score s may be off by rounding, in units of 2^-24 of s: the argument of a softmax term's
// exponential up to 104 (one unit for each e-fold below the largest), expf 4, the sum over 16 + 5 terms, product and
// reciprocal 3; a sigmoid has no such argument and no such sum. The sum with the bias adds a unit of v.
__device__ __forceinline__ float margin(float s, float v, bool softmax) {
    return s * ((softmax ? 132.0f : 12.0f) * 0x1p-24f) + fabsf(v) * 0x1p-23f;
}

// What one lane knows of its experts.
template <int EPL>
struct Lane {
    float l[EPL];                     // logits (-inf: none)
    float b[EPL];                     // bias, 0 without one
};

// The choice of one token in 64 bits. Returns the lane's choice (lane j the j-th expert, -1: none).
template <int EPL>
__device__ __noinline__ int pick_wide(const Lane<EPL>& x, const qz_moe_routing& r, bool biased, int lane) {
    double key[EPL];
    double m = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; i++) m = fmax(m, (double)x.l[i]);
    m = fmax(warp_max_d(m), (double)-FLT_MAX);
    double sum = 0.0;
    if (r.score == QZ_SCORE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < EPL; i++) sum += exp((double)x.l[i] - m);
        sum = warp_sum(sum);
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const double s = r.score == QZ_SCORE_SOFTMAX ? exp((double)x.l[i] - m) / sum : sigmoid((double)x.l[i]);
        key[i] = x.l[i] == -INFINITY ? -INFINITY : s + (double)x.b[i];
    }
    if (r.groups > 1) {
        const int size = r.experts / r.groups;
        double mine = -INFINITY;                               // lane g: the score of group g
        for (int g = 0; g < r.groups; g++) {
            double b = -INFINITY, s = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                if ((lane + 32 * i) / size == g) merge2<double>(b, s, key[i], -INFINITY);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                merge2<double>(b, s, __shfl_xor_sync(kFull, b, o), __shfl_xor_sync(kFull, s, o));
            if (lane == g) mine = group_score(b, s, r.group_best);
        }
        uint32_t kept = 0;
        for (int n = 0; n < r.top_groups; n++) {
            const double top = warp_max_d(mine);
            const uint32_t who = __ballot_sync(kFull, mine == top && top > -INFINITY);
            if (!who) break;
            const int g = __ffs(who) - 1;
            kept |= 1u << g;
            if (lane == g) mine = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!(kept >> min((lane + 32 * i) / size, 31) & 1)) key[i] = -INFINITY;
    }
    if (!biased) {                                             // inside the groups logits decide
#pragma unroll
        for (int i = 0; i < EPL; i++) key[i] = key[i] > -INFINITY ? (double)x.l[i] : -INFINITY;
    }
    int chosen = -1;
    for (int j = 0; j < r.top_k; j++) {
        double best = -INFINITY;
        int at = INT_MAX;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (key[i] > best) {
                best = key[i];
                at = lane + 32 * i;
            }
        const double top = warp_max_d(best);
        if (top == -INFINITY) break;
        at = __reduce_min_sync(kFull, best == top ? at : INT_MAX);
        if (lane == j) chosen = at;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 32 * i == at) key[i] = -INFINITY;
    }
    return chosen;
}

template <int EPL>
__device__ __forceinline__ int pick(const Lane<EPL>& x, const qz_moe_routing& r, bool biased, int lane) {
    const bool grouped = r.groups > 1, soft = r.score == QZ_SCORE_SOFTMAX;
    uint32_t key[EPL];
    float s[EPL];
    if (!biased && !grouped) {
#pragma unroll
        for (int i = 0; i < EPL; i++) key[i] = x.l[i] == -INFINITY ? 0u : ordered(x.l[i]);
    } else {
        float m = -INFINITY, inv = 1.0f;
        if (r.score == QZ_SCORE_SOFTMAX) {
#pragma unroll
            for (int i = 0; i < EPL; i++) m = fmaxf(m, x.l[i]);
            m = fmaxf(warp_max(m, 32), -FLT_MAX);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++) sum += s[i] = expf(x.l[i] - m);
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            s[i] = r.score == QZ_SCORE_SOFTMAX ? s[i] * inv : sigmoid(x.l[i]);
            key[i] = x.l[i] == -INFINITY || x.b[i] == -INFINITY ? 0u : ordered(fminf(s[i] + x.b[i], FLT_MAX));
        }
    }
    bool close = false;
    if (grouped) {
        const int size = r.experts / r.groups;
        float mine = -INFINITY, slack = 0.0f;                  // lane g: the score of group g and its margin
        for (int g = 0; g < r.groups; g++) {
            float b = -INFINITY, c = -INFINITY, top = 0.0f, far = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                if ((lane + 32 * i) / size == g && key[i]) {
                    merge2<float>(b, c, unordered(key[i]), -INFINITY);
                    top = fmaxf(top, s[i]);
                    far = fmaxf(far, fabsf(unordered(key[i])));
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                merge2<float>(b, c, __shfl_xor_sync(kFull, b, o), __shfl_xor_sync(kFull, c, o));
                top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
                far = fmaxf(far, __shfl_xor_sync(kFull, far, o));
            }
            if (lane == g) {
                mine = group_score(b, c, r.group_best);
                slack = 2.0f * margin(top, far, soft) + fabsf(mine) * 0x1p-23f;
            }
        }
        uint32_t kept = 0;
        float last = 0.0f, last_slack = 0.0f;
        for (int n = 0; n <= r.top_groups; n++) {
            const uint32_t u = mine == -INFINITY ? 0u : ordered(mine);
            const uint32_t top = __reduce_max_sync(kFull, u);
            if (!top) break;
            const int g = __ffs(__ballot_sync(kFull, u == top)) - 1;
            const float v = unordered(top), w = __shfl_sync(kFull, slack, g);
            if (n == r.top_groups) {
                close = !(last - v > last_slack + w);
            } else {
                kept |= 1u << g;
                last = v;
                last_slack = w;
                if (lane == g) mine = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (!(kept >> min((lane + 32 * i) / size, 31) & 1)) key[i] = 0u;
        if (!biased) {                                         // inside the groups logits decide
#pragma unroll
            for (int i = 0; i < EPL; i++) key[i] = key[i] ? ordered(x.l[i]) : 0u;
        }
    }
    int chosen = -1;
    float last = 0.0f, last_s = 0.0f, last_l = 0.0f, last_b = 0.0f;
    const int rounds = biased ? r.top_k + 1 : r.top_k;         // with a bias the runner-up has to be well behind too
    for (int j = 0; j < rounds; j++) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (!top) break;
        const int e = __reduce_min_sync(kFull, best == top ? lane + 32 * at : INT_MAX);
        if (biased) {
            float s0 = 0.0f, l0 = 0.0f, b0 = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++)
                if (i == e / 32) {
                    s0 = s[i];
                    l0 = x.l[i];
                    b0 = x.b[i];
                }
            s0 = __shfl_sync(kFull, s0, e & 31);
            l0 = __shfl_sync(kFull, l0, e & 31);
            b0 = __shfl_sync(kFull, b0, e & 31);
            const float v = unordered(top);
            // two experts of one logit and one bias are a true tie
            if (j > 0 && !(last - v > margin(last_s, last, soft) + margin(s0, v, soft)) && !(l0 == last_l && b0 == last_b)) close = true;
            last = v;
            last_s = s0;
            last_l = l0;
            last_b = b0;
        }
        if (lane == j && j < r.top_k) chosen = e;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 32 * i == e) key[i] = 0u;
    }
    return close ? pick_wide<EPL>(x, r, biased, lane) : chosen;
}

// The weight of the lane's choice (chosen < 0: none), with logits at hand.
template <int EPL>
__device__ __forceinline__ float weight_of(const Lane<EPL>& x, float l, bool there, const qz_moe_routing& r) {
    float w = 0.0f;
    if (r.renormalize) {
        // relative to the largest chosen logit, so that scores which underflow keep their ratios
        float m = warp_max(there ? l : -INFINITY, 32);
        if (r.score == QZ_SCORE_SOFTMAX) {
            w = there ? expf(l - m) : 0.0f;
        } else {
            m = fminf(m, 0.0f);
            if (there) w = l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / (1.0f + expf(l));
        }
        const float sum = warp_sum(w);
        return there ? w / sum * r.scale : 0.0f;
    }
    if (r.score == QZ_SCORE_SOFTMAX) {
        float m = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) m = fmaxf(m, x.l[i]);
        m = fmaxf(warp_max(m, 32), -FLT_MAX);
#pragma unroll
        for (int i = 0; i < EPL; i++) sum += expf(x.l[i] - m);
        sum = warp_sum(sum);
        return there ? expf(l - m) / sum * r.scale : 0.0f;
    }
    return there ? sigmoid(l) * r.scale : 0.0f;
}

template <typename T, int EPL>
__global__ void __launch_bounds__(kThreads)
moe_select_kernel(const RouteArgs a, int* __restrict__ block_counts) {
    __shared__ int s_count[kWarps][kMoeMaxExperts];            // per warp and expert: pairs, then those before the warp
    __shared__ int s_scan[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.r.experts, k = a.r.top_k;
    const bool alone = gridDim.x == 1;
    const int64_t t0 = (int64_t)blockIdx.x * kBlockTokens;
    for (int e = lane; e < E; e += 32) s_count[warp][e] = 0;
    __syncwarp();
    int64_t live = a.tokens;
    if (a.n_tokens) live = min(live, (int64_t)max(*a.n_tokens, 0));
    Lane<EPL> x;
#pragma unroll
    for (int i = 0; i < EPL; i++) x.b[i] = a.bias && lane + 32 * i < E ? finite_bias(a.bias[lane + 32 * i]) : 0.0f;
    int id[kWarpTokens], rank[kWarpTokens];                    // lane j: the token's j-th choice
#pragma unroll
    for (int n = 0; n < kWarpTokens; n++) {
        const int64_t t = t0 + warp * kWarpTokens + n;
        id[n] = -1;
        rank[n] = 0;
        if (t >= a.tokens) continue;
        if (t < live) {
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
#pragma unroll
            for (int i = 0; i < EPL; i++) x.l[i] = lane + 32 * i < E ? finite_logit(load_logit(row + lane + 32 * i)) : -INFINITY;
            id[n] = pick<EPL>(x, a.r, a.bias != nullptr, lane);
            const bool there = id[n] >= 0;
            const float l = there ? finite_logit(load_logit(row + id[n])) : 0.0f;
            const float w = weight_of<EPL>(x, l, there, a.r);
            if (lane < k) a.weights[t * k + lane] = w;
            // a token's choices are different experts: no two lanes meet at a counter
            if (there) {
                rank[n] = s_count[warp][id[n]];
                s_count[warp][id[n]] = rank[n] + 1;
            }
            __syncwarp();
        } else if (lane < k) {
            a.weights[t * k + lane] = 0.0f;
        }
        if (lane < k) a.ids[t * k + lane] = id[n];
    }
    __syncthreads();
    // pairs of the warps before; the CTA's own count per expert
    int mine = 0;
    const int e = threadIdx.x;
    if (e < E)
        for (int w = 0; w < kWarps; w++) {
            const int c = s_count[w][e];
            s_count[w][e] = mine;
            mine += c;
        }
    static_assert(kThreads >= kMoeMaxExperts, "a thread per expert");
    int total = 0;
    if (alone) {
        // offsets: exclusive sums over the experts
        int v = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kFull, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) s_scan[warp] = v;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < kWarps; w++) {
            before += w < warp ? s_scan[w] : 0;
            total += s_scan[w];
        }
        const int off = before + v - mine;
        if (e < E) {
            a.offsets[e] = off;
            for (int w = 0; w < kWarps; w++) s_count[w][e] += off;
        }
        if (e == 0) a.offsets[E] = total;
    } else if (e < E) {
        block_counts[(int64_t)blockIdx.x * E + e] = mine;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kWarpTokens; n++) {
        const int64_t t = t0 + warp * kWarpTokens + n;
        if (t >= a.tokens || lane >= k) continue;
        const int row = id[n] >= 0 ? s_count[warp][id[n]] + rank[n] : -1;
        a.token_row[t * k + lane] = row;                       // several CTAs: the rank within this one
        if (alone && row >= 0) a.row_token[row] = (int32_t)t;
    }
    if (alone)
        for (int64_t i = total + threadIdx.x; i < a.tokens * k; i += kThreads) a.row_token[i] = -1;
    pdl_trigger();
}

// Rows of the pairs of one CTA of the selection, from the counts of all of them.
__global__ void __launch_bounds__(kThreads)
moe_place_kernel(const RouteArgs a, const int* __restrict__ block_counts) {
    __shared__ int s_base[kMoeMaxExperts];
    __shared__ int s_scan[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.r.experts, k = a.r.top_k, e = threadIdx.x;
    int all = 0, before = 0;
    if (e < E)
        for (int b = 0; b < (int)gridDim.x; b++) {
            const int c = block_counts[(int64_t)b * E + e];
            before += b < (int)blockIdx.x ? c : 0;
            all += c;
        }
    int v = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    int total = 0, warps_before = 0;
    for (int w = 0; w < kWarps; w++) {
        warps_before += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
    }
    const int off = warps_before + v - all;
    if (e < E) s_base[e] = off + before;
    if (blockIdx.x == 0) {
        if (e < E) a.offsets[e] = off;
        if (e == 0) a.offsets[E] = total;
    }
    __syncthreads();
    const int64_t n = a.tokens * k, i0 = (int64_t)blockIdx.x * kBlockTokens * k;
    for (int i = threadIdx.x; i < kBlockTokens * k && i0 + i < n; i += kThreads) {
        const int id = a.ids[i0 + i];
        if (id < 0) continue;
        const int row = s_base[id] + a.token_row[i0 + i];
        a.token_row[i0 + i] = row;
        a.row_token[row] = (int32_t)((i0 + i) / k);
    }
    for (int64_t i = total + (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) a.row_token[i] = -1;
    pdl_trigger();
}

int64_t select_blocks(int64_t tokens) { return tokens <= kBlockTokens ? 1 : (tokens + kBlockTokens - 1) / kBlockTokens; }

template <typename T>
qz_status select_launch(const RouteArgs& a, int* counts, cudaStream_t st) {
    const dim3 grid((unsigned)select_blocks(a.tokens)), block(kThreads);
    const int per_lane = (a.r.experts + 31) / 32;
    if (per_lane <= 1) return launch_pdl(moe_select_kernel<T, 1>, grid, block, 0, st, a, counts);
    if (per_lane <= 2) return launch_pdl(moe_select_kernel<T, 2>, grid, block, 0, st, a, counts);
    if (per_lane <= 4) return launch_pdl(moe_select_kernel<T, 4>, grid, block, 0, st, a, counts);
    if (per_lane <= 8) return launch_pdl(moe_select_kernel<T, 8>, grid, block, 0, st, a, counts);
    return launch_pdl(moe_select_kernel<T, 16>, grid, block, 0, st, a, counts);
}

} // namespace

size_t ws_moe_route(int64_t tokens, int64_t experts, int64_t) {
    if (tokens <= kBlockTokens || experts < 1) return 0;
    return (size_t)select_blocks(tokens) * (size_t)experts * sizeof(int);
}

qz_status moe_route_launch(const RouteArgs& a, qz_dtype lt, void* ws, cudaStream_t st) {
    int* counts = static_cast<int*>(ws);
    QZ_TRY(lt == QZ_F32 ? select_launch<float>(a, counts, st) : select_launch<uint16_t>(a, counts, st));
    if (select_blocks(a.tokens) == 1) return QZ_OK;
    return launch_pdl(moe_place_kernel, dim3((unsigned)select_blocks(a.tokens)), dim3(kThreads), 0, st, a, (const int*)counts);
}

} // namespace qz
