// moe_route.cu -- routing of tokens to experts and the order of their rows.
//
// Selection: a warp per token, expert e in lane e % 32. The top_k are taken one by one: every
// lane's best key, a warp maximum over the keys as ordered integers, the lowest index among
// those that have it. Without bias the keys are the logits, which order the experts exactly
// as their scores do, and no score but those of the chosen is formed. A group's score is found by the
// 32 / groups lanes that share the group, over the keys in shared memory.
//
// With a bias, and for groups, keys are rounded sums, and two that 32 bits cannot tell apart could change places. Every
// comparison that decides something is checked against a bound on its rounding errors. Experts too close to
// one another are compared again in 64 bits, a lane each (sort_wide; sigmoid only: a softmax needs all terms of its
// sum again); a token whose groups are too close, or that has more such experts than lanes, is chosen in
// 64 bits altogether (pick_wide). At 8000 tokens of 256 experts about one token in 200 is.
//
// The plan: the rows of an expert in the order of the tokens, whatever order CTAs run in. A
// CTA counts its pairs per warp and expert and gives each pair its rank; the second kernel adds, per expert, the counts of
// the CTAs before it and the rows of the experts before it. Up to kAlone tokens are one CTA and one launch.
//
// What bounds it: the chain of about 100 cycles per chosen expert (with 32 warps an SM the issue of about 400
// instructions a token), two launches, and the latency of the counts between them; the bytes are little.
#include "qz_moe.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>

namespace qz {

namespace {

constexpr int kWarps = 32, kThreads = kWarps * 32;
constexpr int kAlone = 128;                                    // tokens that one CTA takes by itself
constexpr int kMinTokens = 64, kMaxBlocks = 256;               // else: tokens a CTA at least, CTAs at most
constexpr int kPlaceThreads = 512;
constexpr uint32_t kFull = 0xffffffffu;
static_assert(kThreads >= kMoeMaxExperts && kPlaceThreads >= kMoeMaxExperts, "a thread per expert");

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_bits_to_f32(*p); }

// NaN counts as -inf, +inf as the largest finite value.
__device__ __forceinline__ float finite(float v) { return fminf(v != v ? -INFINITY : v, FLT_MAX); }

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
    return __fdiv_rn(l >= 0.0f ? 1.0f : e, 1.0f + e);
}
__device__ __forceinline__ double sigmoid(double l) {
    const double e = exp(-fabs(l));
    return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

template <typename V> __device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <typename V> __device__ __forceinline__ V warp_most(V v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const V u = __shfl_xor_sync(kFull, v, o);
        v = u > v ? u : v;
    }
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

// How far two keys may seem from each other by rounding, over the difference that they have: in units of 2^-24 of the
// largest score, twice: the argument of a softmax term's exponential up to 104 (one unit for each e-fold below
// the largest), expf 4, the sum over 16 + 5 terms, product and reciprocal 3; a sigmoid has expf, sum and quotient.
// The sum with the bias adds a unit of each key.
__device__ __forceinline__ float margin(float most, float key, bool softmax) {
    return most * ((softmax ? 2 * 132.0f : 2 * 8.0f) * 0x1p-24f) + fabsf(key) * 0x1p-22f;
}

// The choice of one token in 64 bits, every term of it. Lane j gets the j-th expert, -1: none.
template <typename T>
__device__ __noinline__ int pick_wide(const T* row, const float* bias, const qz_moe_routing* rt, int lane, double* keys) {
    const qz_moe_routing r = *rt;
    double most = -FLT_MAX, sum = 0.0;
    if (r.score == QZ_SCORE_SOFTMAX) {
        for (int e = lane; e < r.experts; e += 32) most = fmax(most, (double)finite(load_logit(row + e)));
        most = warp_most(most);
        for (int e = lane; e < r.experts; e += 32) sum += exp((double)finite(load_logit(row + e)) - most);
        sum = warp_sum(sum);
    }
    auto key_of = [&](int e) {
        const float l = finite(load_logit(row + e)), b = bias ? finite(bias[e]) : 0.0f;
        if (l == -INFINITY || b == -INFINITY) return (double)-INFINITY;
        return (r.score == QZ_SCORE_SOFTMAX ? exp((double)l - most) / sum : sigmoid((double)l)) + (double)b;
    };
    uint32_t kept = 0xffffffffu;
    const int size = r.experts / r.groups;
    if (r.groups > 1) {
        double mine = -INFINITY;                               // lane g: the score of group g
        for (int g = 0; g < r.groups; g++) {
            double b = -INFINITY, s = -INFINITY;
            for (int e = g * size + lane; e < (g + 1) * size; e += 32) merge2<double>(b, s, key_of(e), -INFINITY);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                merge2<double>(b, s, __shfl_xor_sync(kFull, b, o), __shfl_xor_sync(kFull, s, o));
            if (lane == g) mine = r.group_best == 2 && s > -INFINITY ? b + s : b;
        }
        kept = 0;
        for (int n = 0; n < r.top_groups; n++) {
            const double top = warp_most(mine);
            const uint32_t who = __ballot_sync(kFull, mine == top && top > -INFINITY);
            if (!who) break;
            kept |= who & -who;
            if (lane == __ffs(who) - 1) mine = -INFINITY;
        }
    }
    int chosen = -1;
    double last = INFINITY;                                    // key and index of the choice before: the next is behind it
    int last_e = -1;
    for (int j = 0; j < r.top_k; j++) {
        double best = -INFINITY;
        int at = INT_MAX;
        for (int e = lane; e < r.experts; e += 32) {
            if (!(kept >> (r.groups > 1 ? e / size : 0) & 1)) continue;
            double k = key_of(e);
            if (!bias && k > -INFINITY) k = (double)finite(load_logit(row + e));       // inside the groups logits decide
            const bool behind = k < last || (k == last && e > last_e);
            if (behind && k > best) {
                best = k;
                at = e;
            }
        }
        const double top = warp_most(best);
        if (top == -INFINITY) break;
        at = __reduce_min_sync(kFull, best == top ? at : INT_MAX);
        if (lane == j) chosen = at;
        last = top;
        last_e = at;
    }
    return chosen;
}

// n candidates, one a lane, in the order of their keys in 64 bits: lane j gets the j-th.
template <typename T>
__device__ __noinline__ int sort_wide(const T* row, const float* bias, int id, int n, int lane) {
    double key = -INFINITY;
    if (lane < n) key = sigmoid((double)finite(load_logit(row + id))) + (double)finite(bias[id]);
    int rank = 0;
    for (int i = 0; i < n; i++) {
        const double k = __shfl_sync(kFull, key, i);
        const int e = __shfl_sync(kFull, id, i);
        rank += k > key || (k == key && e < id);
    }
    int got = -1;
    for (int i = 0; i < n; i++)
        if (__shfl_sync(kFull, rank, i) == lane) got = __shfl_sync(kFull, id, i);
        else (void)__shfl_sync(kFull, id, i);
    return got;
}

// The choice of one token. l: the lane's logits, finite or -inf.
template <typename T, int EPL>
__device__ __forceinline__ int pick(const float (&l)[EPL], const float (&b)[EPL], const T* row, const float* bias,
                                    const qz_moe_routing& r, int lane, uint32_t* keys) {
    const bool grouped = r.groups > 1, soft = r.score == QZ_SCORE_SOFTMAX;
    uint32_t key[EPL];
    float most = 1.0f;                                         // no score is larger
    if (!bias && !grouped) {
#pragma unroll
        for (int i = 0; i < EPL; i++) key[i] = l[i] == -INFINITY ? 0u : ordered(l[i]);
    } else {
        float s[EPL], inv = 1.0f;
        if (soft) {
            float m = -FLT_MAX, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; i++) m = fmaxf(m, l[i]);
            m = warp_max(m, 32);
#pragma unroll
            for (int i = 0; i < EPL; i++) sum += s[i] = expf(l[i] - m);
            sum = warp_sum(sum);
            inv = sum > 0.0f ? 1.0f / sum : 0.0f;
            most = inv;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const float v = soft ? s[i] * inv : sigmoid(l[i]);
            key[i] = l[i] == -INFINITY || b[i] == -INFINITY ? 0u : ordered(fminf(v + b[i], FLT_MAX));
        }
    }
    if (grouped) {
        // the 32 / groups (rounded down to a power of two) lanes of a group look at its experts by turns
        const int size = r.experts / r.groups, share = 32 - __clz(32 / r.groups) - 1, lanes = 1 << share;
        const int g = lane >> share;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = lane + 32 * i;
            if (e < r.experts) keys[e + (e >> 5)] = key[i];
        }
        __syncwarp();
        uint32_t best = 0, second = 0;
        if (g < r.groups)
            for (int e = g * size + (lane & (lanes - 1)); e < (g + 1) * size; e += lanes) merge2<uint32_t>(best, second, keys[e + (e >> 5)], 0u);
        for (int o = lanes >> 1; o > 0; o >>= 1)
            merge2<uint32_t>(best, second, __shfl_xor_sync(kFull, best, o), __shfl_xor_sync(kFull, second, o));
        // a group's score as an ordered integer, in its first lane
        uint32_t mine = 0;
        if (g < r.groups && (lane & (lanes - 1)) == 0 && best)
            mine = ordered(r.group_best == 2 && second ? unordered(best) + unordered(second) : unordered(best));
        uint32_t kept = 0;
        float last = 0.0f;
        bool close = false;
        for (int n = 0; n <= r.top_groups; n++) {
            const uint32_t top = __reduce_max_sync(kFull, mine);
            if (!top) break;
            const float v = unordered(top);
            if (n == r.top_groups) {
                close = !(last - v > 2.0f * margin(most, fmaxf(fabsf(last), fabsf(v)), soft));
            } else {
                const int first = __ffs(__ballot_sync(kFull, mine == top)) - 1;
                kept |= 1u << (first >> share);
                last = v;
                if (lane == first) mine = 0;
            }
        }
        // without a bias and by one logit a group the comparison of the keys was that of scores, which may be equal in 32
        // bits where the logits are not
        if (close) return pick_wide<T>(row, bias, &r, lane, nullptr);
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = lane + 32 * i;
            if (!(kept >> min(e / size, 31) & 1)) key[i] = 0u;
            else if (!bias && key[i]) key[i] = ordered(l[i]);  // inside the groups logits decide
        }
    }
    int chosen = -1, n = 0, more = INT_MAX;                    // more: choices wanted beyond the last one that was clear
    bool close = false;
    float last = 0.0f, kth = 0.0f;
    for (int j = 0; j < 32; j++) {
        if (j == r.top_k && !bias) break;
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
        if (bias) {
            const float v = unordered(top);
            const bool near = j > 0 && !(last - v > margin(most, fmaxf(fabsf(last), fabsf(v)), soft));
            if (j < r.top_k) close |= near;
            // behind the last choice: those that might belong before it
            else if (!(kth - v > margin(most, fmaxf(fabsf(kth), fabsf(v)), soft))) close = true;
            else break;
            last = v;
            if (j == r.top_k - 1) kth = v;
            if (j == 31) more = 0;
        }
        const int e = __reduce_min_sync(kFull, best == top ? lane + 32 * at : INT_MAX);
        if (lane == j) chosen = e;
        n++;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 32 * i == e) key[i] = 0u;
    }
    if (close) {
        if (soft || more == 0) return pick_wide<T>(row, bias, &r, lane, nullptr);
        chosen = sort_wide<T>(row, bias, chosen, n, lane);
    }
    return lane < r.top_k ? chosen : -1;
}

// The weight of the lane's choice (there: it has one) of logit l0.
template <int EPL>
__device__ __forceinline__ float weight_of(const float (&l)[EPL], float l0, bool there, const qz_moe_routing& r) {
    float w = 0.0f;
    if (r.renormalize) {
        // relative to the largest chosen logit, so that scores which underflow keep their ratios
        float m = warp_max(there ? l0 : -INFINITY, 32);
        if (r.score == QZ_SCORE_SOFTMAX) {
            w = there ? expf(l0 - m) : 0.0f;
        } else {
            m = fminf(m, 0.0f);
            if (there) w = l0 >= 0.0f ? 1.0f / (1.0f + expf(-l0)) : expf(l0 - m) / (1.0f + expf(l0));
        }
        const float sum = warp_sum(w);
        return there ? w / sum * r.scale : 0.0f;
    }
    if (r.score == QZ_SCORE_SOFTMAX) {
        float m = -FLT_MAX, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) m = fmaxf(m, l[i]);
        m = warp_max(m, 32);
#pragma unroll
        for (int i = 0; i < EPL; i++) sum += expf(l[i] - m);
        sum = warp_sum(sum);
        return there ? expf(l0 - m) / sum * r.scale : 0.0f;
    }
    return there ? sigmoid(l0) * r.scale : 0.0f;
}

// Dynamic shared memory: counts [warps][experts], then with groups the keys of each warp [warps][experts + experts / 32].
__host__ __device__ __forceinline__ int key_words(int experts) { return experts + (experts >> 5) + 1; }

template <typename T, int EPL>
__global__ void __launch_bounds__(kThreads)
moe_select_kernel(const __grid_constant__ RouteArgs a, const int per_warp, int* __restrict__ block_counts) {
    extern __shared__ int s_dyn[];
    __shared__ int s_scan[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.r.experts, k = a.r.top_k;
    int* count = s_dyn + warp * E;                             // pairs per expert, then those of the warps before
    uint32_t* keys = reinterpret_cast<uint32_t*>(s_dyn + kWarps * E) + warp * key_words(E);
    const bool alone = gridDim.x == 1;
    for (int e = lane; e < E; e += 32) count[e] = 0;
    __syncwarp();
    int64_t live = a.tokens;
    if (a.n_tokens) live = min(live, (int64_t)max(*a.n_tokens, 0));
    float b[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) b[i] = a.bias && lane + 32 * i < E ? finite(a.bias[lane + 32 * i]) : 0.0f;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * per_warp, t1 = min(t0 + per_warp, a.tokens);
    for (int64_t t = t0; t < t1; t++) {
        int id = -1, rank = -1;
        float w = 0.0f;
        if (t < live) {
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
            float l[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++) l[i] = lane + 32 * i < E ? finite(load_logit(row + lane + 32 * i)) : -INFINITY;
            id = pick<T, EPL>(l, b, row, a.bias, a.r, lane, keys);
            const bool there = id >= 0;
            w = weight_of<EPL>(l, there ? finite(load_logit(row + id)) : 0.0f, there, a.r);
            // a token's choices are different experts: no two lanes meet at a counter
            if (there) {
                rank = count[id];
                count[id] = rank + 1;
            }
            __syncwarp();
        }
        if (lane < k) {
            a.ids[t * k + lane] = id;
            a.weights[t * k + lane] = w;
            a.token_row[t * k + lane] = rank;                  // among the warp's pairs of the expert
        }
    }
    __syncthreads();
    int mine = 0;                                              // thread e: the CTA's pairs of expert e
    const int e = threadIdx.x;
    if (e < E) {
#pragma unroll 8
        for (int w = 0; w < kWarps; w++) {
            const int c = s_dyn[w * E + e];
            s_dyn[w * E + e] = mine;
            mine += c;
        }
    }
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
#pragma unroll 8
            for (int w = 0; w < kWarps; w++) s_dyn[w * E + e] += off;
        }
        if (e == 0) a.offsets[E] = total;
    } else if (e < E) {
        block_counts[(int64_t)blockIdx.x * E + e] = mine;
    }
    __syncthreads();
    // from ranks in the warp to ranks in the CTA, or rows
    for (int64_t i = t0 * k + lane; i < t1 * k; i += 32) {
        const int id = a.ids[i];
        if (id < 0) continue;
        const int row = count[id] + a.token_row[i];
        a.token_row[i] = row;
        if (alone) a.row_token[row] = (int32_t)(i / k);
    }
    if (alone)
        for (int64_t i = total + threadIdx.x; i < a.tokens * k; i += kThreads) a.row_token[i] = -1;
    pdl_trigger();
}

// Rows of the pairs of one CTA of the selection, from the counts of all of them.
__global__ void __launch_bounds__(kPlaceThreads)
moe_place_kernel(const __grid_constant__ RouteArgs a, const int block_tokens, const int* __restrict__ block_counts) {
    __shared__ int s_all[kPlaceThreads], s_before[kPlaceThreads];
    __shared__ int s_base[kMoeMaxExperts];
    __shared__ int s_scan[kPlaceThreads / 32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.r.experts, k = a.r.top_k;
    // `parts` threads share an expert's column of counts
    const int parts = kPlaceThreads / E, part = threadIdx.x / E, e = threadIdx.x % E;
    int all = 0, before = 0;
    if (part < parts) {
#pragma unroll 8
        for (int b = part; b < (int)gridDim.x; b += parts) {
            const int c = block_counts[(int64_t)b * E + e];
            before += b < (int)blockIdx.x ? c : 0;
            all += c;
        }
    }
    s_all[threadIdx.x] = all;
    s_before[threadIdx.x] = before;
    __syncthreads();
    all = before = 0;
    if (threadIdx.x < E)
        for (int p = 0; p < parts; p++) {
            all += s_all[p * E + threadIdx.x];
            before += s_before[p * E + threadIdx.x];
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
#pragma unroll
    for (int w = 0; w < kPlaceThreads / 32; w++) {
        warps_before += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
    }
    const int off = warps_before + v - all;
    if (threadIdx.x < E) s_base[threadIdx.x] = off + before;
    if (blockIdx.x == 0) {
        if (threadIdx.x < E) a.offsets[threadIdx.x] = off;
        if (threadIdx.x == 0) a.offsets[E] = total;
    }
    __syncthreads();
    const int64_t n = a.tokens * k, i0 = (int64_t)blockIdx.x * block_tokens * k, i1 = min(i0 + (int64_t)block_tokens * k, n);
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kPlaceThreads) {
        const int id = a.ids[i];
        if (id < 0) continue;
        const int row = s_base[id] + a.token_row[i];
        a.token_row[i] = row;
        a.row_token[row] = (int32_t)(i / k);
    }
    for (int64_t i = total + (int64_t)blockIdx.x * kPlaceThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kPlaceThreads) a.row_token[i] = -1;
    pdl_trigger();
}

// Tokens a warp and CTAs. One CTA up to kAlone tokens; more CTAs than kMaxBlocks would read too many counts.
struct Split {
    int per_warp, blocks;
};
Split split_of(int64_t tokens) {
    if (tokens <= kAlone) return {(int)std::max<int64_t>(1, (tokens + kWarps - 1) / kWarps), 1};
    const int64_t block = std::max<int64_t>(kMinTokens, (tokens + kMaxBlocks - 1) / kMaxBlocks);
    const int per_warp = (int)((block + kWarps - 1) / kWarps);
    return {per_warp, (int)((tokens + (int64_t)per_warp * kWarps - 1) / ((int64_t)per_warp * kWarps))};
}

template <typename T, int EPL>
qz_status select_kernel(const RouteArgs& a, const Split& s, int* counts, cudaStream_t st) {
    const int words = kWarps * (a.r.experts + (a.r.groups > 1 ? key_words(a.r.experts) : 0));
    if (words * 4 > 48 * 1024) QZ_TRY(opt_in_smem((const void*)moe_select_kernel<T, EPL>, words * 4));
    return launch_pdl(moe_select_kernel<T, EPL>, dim3(s.blocks), dim3(kThreads), words * 4, st, a, s.per_warp, counts);
}

template <typename T>
qz_status select_launch(const RouteArgs& a, const Split& s, int* counts, cudaStream_t st) {
    const int per_lane = (a.r.experts + 31) / 32;
    if (per_lane <= 2) return select_kernel<T, 2>(a, s, counts, st);
    if (per_lane <= 4) return select_kernel<T, 4>(a, s, counts, st);
    if (per_lane <= 8) return select_kernel<T, 8>(a, s, counts, st);
    return select_kernel<T, 16>(a, s, counts, st);
}

} // namespace

size_t ws_moe_route(int64_t tokens, int64_t experts, int64_t) {
    const Split s = split_of(tokens);
    return s.blocks == 1 || experts < 1 ? 0 : (size_t)s.blocks * (size_t)experts * sizeof(int);
}

qz_status moe_route_launch(const RouteArgs& a, qz_dtype lt, void* ws, cudaStream_t st) {
    int* counts = static_cast<int*>(ws);
    const Split s = split_of(a.tokens);
    QZ_TRY(lt == QZ_F32 ? select_launch<float>(a, s, counts, st) : select_launch<uint16_t>(a, s, counts, st));
    if (s.blocks == 1) return QZ_OK;
    return launch_pdl(moe_place_kernel, dim3(s.blocks), dim3(kPlaceThreads), 0, st, a, s.per_warp * kWarps, (const int*)counts);
}

} // namespace qz
