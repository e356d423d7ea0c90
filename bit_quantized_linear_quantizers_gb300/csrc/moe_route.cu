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
// one another are compared again in 64 bits, a lane each (sort_wide), and so are the best of groups that are
// (groups_wide). A softmax with a bias needs all terms of its sum again, and more such experts than lanes need all
// keys: such a token is chosen in 64 bits altogether (pick_wide; 15 to 25 us, where the others take 3).
//
// The plan: the rows of an expert in the order of the tokens, whatever order CTAs run in. A
// CTA counts its pairs per warp and expert and gives each pair its rank; the second kernel adds, per expert, the counts of
// the CTAs before it and the rows of the experts before it. Up to kAlone tokens are one CTA and one launch.
//
// What bounds it: for few tokens the chain of about 100 cycles per chosen expert, two launches, and the latency of the
// counts between them; for many the issue of about 500 instructions a token (16384 of 128 experts: 18 us), 2100 with a bias
// and groups (8000 of 256 experts: 33 us). The bytes are little.
#include "qz_moe.cuh"

#include <algorithm>
#include <cfloat>
#include <climits>

namespace qz {

namespace {

constexpr int kWarps = 16;                                     // of a selecting CTA, at most; two CTAs an SM
constexpr int kAlone = 16;                                     // tokens that one CTA takes by itself
constexpr int kMaxBlocks = 304;                                // two CTAs of kWarps an SM
constexpr int kPlaceThreads = 512, kParts = 16;                // threads that share an expert's counts, at most
constexpr uint32_t kFull = 0xffffffffu;
static_assert(kWarps * 32 >= kMoeMaxExperts && kPlaceThreads >= kMoeMaxExperts, "a thread per expert");

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
    return __fdividef(l >= 0.0f ? 1.0f : e, 1.0f + e);
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
// the largest), expf 4, the sum over 16 + 5 terms, product and reciprocal 3; a sigmoid has 1.5 + 1 + 4.
// The sum with the bias adds a unit of each key.
__device__ __forceinline__ float margin(float most, float key, bool softmax) {
    return most * ((softmax ? 2 * 132.0f : 2 * 7.0f) * 0x1p-24f) + fabsf(key) * 0x1p-22f;
}

// The choice of one token with a bias in 64 bits, every term of it, EPL experts a lane. Lane j gets the j-th expert, -1: none.
template <typename T, int EPL>
__device__ __noinline__ int pick_wide(const T* row, const float* bias, const qz_moe_routing* rt, int lane) {
    const qz_moe_routing r = *rt;
    double key[EPL], most = -FLT_MAX, sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 32 * i;
        key[i] = e < r.experts ? (double)finite(load_logit(row + e)) : (double)-INFINITY;
        most = fmax(most, key[i]);
    }
    const bool soft = r.score == QZ_SCORE_SOFTMAX;
    if (soft) most = warp_most(most);
#pragma unroll 1
    for (int i = 0; i < EPL; i++) sum += soft ? exp(key[i] - most) : 0.0;
    if (soft) sum = warp_sum(sum);
#pragma unroll 1
    for (int i = 0; i < EPL; i++) {
        const int e = lane + 32 * i;
        const float b = e < r.experts ? finite(bias[e]) : 0.0f;
        const bool open = key[i] > -INFINITY && b > -INFINITY;
        const double s = soft ? exp(key[i] - most) / sum : sigmoid(key[i]);
        key[i] = open ? s + (double)b : -INFINITY;
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
            if (lane == g) mine = r.group_best == 2 && s > -INFINITY ? b + s : b;
        }
        uint32_t kept = 0;
        for (int n = 0; n < r.top_groups; n++) {
            const double top = warp_most(mine);
            const uint32_t who = __ballot_sync(kFull, mine == top && top > -INFINITY);
            if (!who) break;
            kept |= who & -who;
            if (lane == __ffs(who) - 1) mine = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = lane + 32 * i;
            if (!(kept >> min(e / size, 31) & 1)) key[i] = -INFINITY;
        }
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
        const double top = warp_most(best);
        if (top == -INFINITY) break;
        at = __reduce_min_sync(kFull, best == top ? at : INT_MAX);
        if (lane == j) chosen = at;
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (lane + 32 * i == at) key[i] = -INFINITY;
    }
    return chosen;
}

// The groups that are kept where some are too close to the border for 32 bits: those surely above it, and the best of
// the near ones by their scores in 64 bits, of the keys that can be among their best. Lane g says of group g whether
// it is sure or near; largest: no score is larger. Not for a softmax with a bias, whose terms need their sum.
template <typename T>
__device__ __noinline__ uint32_t groups_wide(const T* row, const float* bias, const qz_moe_routing* rt, int lane, const uint32_t* keys,
                                             bool sure, bool near, float largest) {
    const qz_moe_routing r = *rt;
    const int size = r.experts / r.groups;
    const bool soft = r.score == QZ_SCORE_SOFTMAX;
    const uint32_t surely = __ballot_sync(kFull, sure), nearly = __ballot_sync(kFull, near);
    double most = -FLT_MAX;
    if (soft) {
        for (int e = lane; e < r.experts; e += 32) most = fmax(most, (double)finite(load_logit(row + e)));
        most = warp_most(most);
    }
    double exact = -INFINITY;
    for (uint32_t left = nearly; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        uint32_t b = 0, s = 0;
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) merge2<uint32_t>(b, s, keys[e + (e >> 5)], 0u);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) merge2<uint32_t>(b, s, __shfl_xor_sync(kFull, b, o), __shfl_xor_sync(kFull, s, o));
        const float from = unordered(r.group_best == 2 && s ? s : b);
        double eb = -INFINITY, es = -INFINITY;
        for (int e = g * size + lane; e < (g + 1) * size; e += 32) {
            const uint32_t k = keys[e + (e >> 5)];
            if (!k) continue;
            const float v = unordered(k);
            if (from - v > margin(largest, fmaxf(fabsf(from), fabsf(v)), soft)) continue;
            const double l = (double)finite(load_logit(row + e));
            merge2<double>(eb, es, (soft ? exp(l - most) : sigmoid(l)) + (bias ? (double)finite(bias[e]) : 0.0), -INFINITY);
        }
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) merge2<double>(eb, es, __shfl_xor_sync(kFull, eb, o), __shfl_xor_sync(kFull, es, o));
        if (lane == g) exact = r.group_best == 2 && es > -INFINITY ? eb + es : eb;
    }
    int rank = __popc(surely);
    for (uint32_t left = nearly; left; left &= left - 1) {
        const int g = __ffs(left) - 1;
        const double v = __shfl_sync(kFull, exact, g);
        rank += v > exact || (v == exact && g < lane);
    }
    return surely | __ballot_sync(kFull, near && rank < r.top_groups);
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
    for (int i = 0; i < n; i++) {
        const int place = __shfl_sync(kFull, rank, i), e = __shfl_sync(kFull, id, i);
        if (place == lane) got = e;
    }
    return got;
}

// A score for comparisons alone. The fast exponential is off by 2 + 1.16 |l| units in the last place, of which s (1 - s), at
// most a quarter, reaches s: 1.5 units of 2^-24 of the largest score.
__device__ __forceinline__ float key_sigmoid(float l) {
    const float e = __expf(-fabsf(l));
    return __fdividef(l >= 0.0f ? 1.0f : e, 1.0f + e);
}

// A lane's two best experts (register numbers a1, a2) of those behind (key ck, register ci): smaller keys, and equal ones
// of larger index. A key of 0: there is none.
template <int EPL>
__device__ __forceinline__ void best_two(const uint32_t (&key)[EPL], uint32_t ck, int ci, uint32_t& b1, int& a1, uint32_t& b2, int& a2) {
    b1 = b2 = 0;
    a1 = a2 = 0;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint32_t v = key[i] < ck || (key[i] == ck && i > ci) ? key[i] : 0u;
        if (v > b1) {
            b2 = b1;
            a2 = a1;
            b1 = v;
            a1 = i;
        } else if (v > b2) {
            b2 = v;
            a2 = i;
        }
    }
}

// The choice of one token. l: the lane's logits, finite or -inf.
template <typename T, int EPL, bool SIMPLE>
__device__ __forceinline__ int pick(const float (&l)[EPL], const float (&b)[EPL], const T* row, const float* bias,
                                    const qz_moe_routing& r, int lane, uint32_t* keys) {
    const bool grouped = !SIMPLE && r.groups > 1, soft = r.score == QZ_SCORE_SOFTMAX;
    uint32_t key[EPL];
    float most = 1.0f;                                         // no score is larger
    if (SIMPLE || (!bias && !grouped)) {
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
            const float v = soft ? s[i] * inv : key_sigmoid(l[i]);
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
        // a group's score in its first lane, finite, so that differences are numbers: two that the limit makes equal are
        // compared in 64 bits. It is off by the roundings of its keys, which may be far larger than their sum.
        const bool open = g < r.groups && (lane & (lanes - 1)) == 0 && best;
        float score = 0.0f, off = 0.0f;
        uint32_t mine = 0;
        if (open) {
            const float k1 = unordered(best), k2 = r.group_best == 2 && second ? unordered(second) : 0.0f;
            score = fmaxf(fminf(k1 + k2, FLT_MAX), -FLT_MAX);
            off = margin(most, fminf(fabsf(k1) + fabsf(k2), FLT_MAX), soft);
            mine = ordered(score);
        }
        uint32_t kept = 0;
        for (int n = 0; n < r.top_groups; n++) {
            const uint32_t top = __reduce_max_sync(kFull, mine);
            if (!top) break;
            const int first = __ffs(__ballot_sync(kFull, mine == top)) - 1;
            kept |= 1u << (first >> share);
            if (lane == first) mine = 0;
        }
        // the least that a kept group may have, and the most that another one may
        const bool in = open && (kept >> g & 1);
        const float least = unordered(__reduce_min_sync(kFull, in ? ordered(score - off) : kFull));
        const uint32_t other = __reduce_max_sync(kFull, open && !in ? ordered(score + off) : 0u);
        if (other && !(least > unordered(other))) {
            if (soft && bias) return pick_wide<T, EPL>(row, bias, &r, lane);
            const bool sure = in && score - off > unordered(other), near = open && !sure && (in || score + off >= least);
            const uint32_t which = (sure ? 1u : 0u) | (near ? 2u : 0u), of = __shfl_sync(kFull, which, min(lane, r.groups - 1) << share);
            kept = groups_wide<T>(row, bias, &r, lane, keys, lane < r.groups && (of & 1), lane < r.groups && (of & 2), most);
        }
        const float per = 1.0f / (float)size;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            // its group: e / size, exact for such small numbers half a step away from the next quotient
            const int of = __float2int_rd(((float)(lane + 32 * i) + 0.5f) * per);
            if (!(kept >> min(of, 31) & 1)) key[i] = 0u;
            else if (!bias && key[i]) key[i] = ordered(l[i]);  // inside the groups logits decide
        }
    }
    int chosen = -1, n = 0, more = INT_MAX;                    // more: choices wanted beyond the last one that was clear
    bool close = false;
    float last = 0.0f, kth = 0.0f;
    // every lane's two best at hand: rarely more of the chosen lie in one lane, and it looks again
    uint32_t b1, b2, ck = 0xffffffffu;
    int a1, a2, ci = EPL, left = 2;
    best_two<EPL>(key, ck, ci, b1, a1, b2, a2);
    for (int j = 0; j < 32; j++) {
        if (j == r.top_k && (SIMPLE || !bias)) break;
        const uint32_t top = __reduce_max_sync(kFull, b1);
        if (!top) break;
        if (!SIMPLE && bias) {
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
        const int e = __reduce_min_sync(kFull, b1 == top ? lane + 32 * a1 : INT_MAX);
        if (lane == j) chosen = e;
        n++;
        if ((e & 31) == lane) {
            ck = b1;
            ci = a1;
            b1 = b2;
            a1 = a2;
            left--;
        }
        if (__any_sync(kFull, left == 0) && left == 0) {
            best_two<EPL>(key, ck, ci, b1, a1, b2, a2);
            left = 2;
        }
    }
    if (!SIMPLE && close) {
        if (soft || more == 0) return pick_wide<T, EPL>(row, bias, &r, lane);
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

// Dynamic shared memory: counts [warps][experts], then with groups the keys of each warp.
__host__ __device__ __forceinline__ int key_words(int experts) { return experts + (experts >> 5) + 1; }
// A CTA's counts in the workspace: experts, rounded up to reads of four.
__host__ __device__ __forceinline__ int count_words(int experts) { return (experts + 3) & ~3; }

// Exclusive sums over the CTA's threads, and the sum of all.
__device__ __forceinline__ int scan(int mine, int* s_scan, int& total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int v = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    const int w = lane < (int)(blockDim.x >> 5) ? s_scan[lane] : 0;
    total = __reduce_add_sync(kFull, w);
    return __reduce_add_sync(kFull, lane < warp ? w : 0) + v - mine;
}

// SIMPLE: neither a bias nor groups. Two CTAs an SM leave 64 registers a thread; with a bias or groups the forms of 2, 4, 8 and
// 16 experts a lane spill 44, 104, 252 and 612 bytes.
template <typename T, int EPL, bool SIMPLE>
__global__ void __launch_bounds__(kWarps * 32, 2)
moe_select_kernel(const __grid_constant__ RouteArgs a, const int per_warp, int* __restrict__ block_counts) {
    extern __shared__ int s_dyn[];
    __shared__ int s_scan[kWarps];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, E = a.r.experts, k = a.r.top_k;
    const int tokens = (int)a.tokens;
    int* count = s_dyn + warp * E;                             // pairs per expert, then those of the warps before
    uint32_t* keys = reinterpret_cast<uint32_t*>(s_dyn + warps * E) + warp * key_words(E);
    const bool alone = gridDim.x == 1;
    const float* bias = SIMPLE ? nullptr : a.bias;
    for (int e = lane; e < E; e += 32) count[e] = 0;
    __syncwarp();
    const int live = a.n_tokens ? min(tokens, max(*a.n_tokens, 0)) : tokens;
    float b[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) b[i] = bias && lane + 32 * i < E ? finite(bias[lane + 32 * i]) : 0.0f;
    const int t0 = (int)min(((int64_t)blockIdx.x * warps + warp) * per_warp, a.tokens), t1 = (int)min((int64_t)t0 + per_warp, a.tokens);
    auto logits_of = [&](int t, float (&l)[EPL]) {
        const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
#pragma unroll
        for (int i = 0; i < EPL; i++) l[i] = lane + 32 * i < E ? finite(load_logit(row + lane + 32 * i)) : -INFINITY;
    };
    float next[EPL];
    if (t0 < min(t1, live)) logits_of(t0, next);
    for (int t = t0; t < t1; t++) {
        int id = -1, rank = -1;
        float w = 0.0f;
        if (t < live) {
            const T* row = static_cast<const T*>(a.logits) + t * a.ldl;
            float l[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++) l[i] = next[i];
            if (t + 1 < min(t1, live)) logits_of(t + 1, next);
            id = pick<T, EPL, SIMPLE>(l, b, row, bias, a.r, lane, keys);
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
            const uint32_t at = (uint32_t)t * k + lane;
            a.ids[at] = id;
            a.weights[at] = w;
            a.token_row[at] = rank;                            // among the warp's pairs of the expert
        }
    }
    __syncthreads();
    int mine = 0;                                              // thread e: the CTA's pairs of expert e (there is one for each)
    const int e = threadIdx.x;
    if (e < E) {
#pragma unroll 8
        for (int w = 0; w < warps; w++) {
            const int v = s_dyn[w * E + e];
            s_dyn[w * E + e] = mine;
            mine += v;
        }
        if (!alone) block_counts[(int64_t)blockIdx.x * count_words(E) + e] = mine;
    } else if (!alone && e < count_words(E)) {
        block_counts[(int64_t)blockIdx.x * count_words(E) + e] = 0;
    }
    int total = 0;
    if (alone) {
        const int off = scan(mine, s_scan, total);
        if (e < E) {
            a.offsets[e] = off;
#pragma unroll 8
            for (int w = 0; w < warps; w++) s_dyn[w * E + e] += off;
        }
        if (e == 0) a.offsets[E] = total;
    }
    __syncthreads();
    // from ranks in the warp to ranks in the CTA, or rows
    for (uint32_t i = (uint32_t)t0 * k + lane; i < (uint32_t)t1 * k; i += 32) {
        const int id = a.ids[i];
        if (id < 0) continue;
        const int row = count[id] + a.token_row[i];
        a.token_row[i] = row;
        if (alone) a.row_token[row] = (int32_t)(i / (uint32_t)k);
    }
    if (alone)
        for (uint32_t i = total + threadIdx.x; i < (uint32_t)tokens * k; i += blockDim.x) a.row_token[i] = -1;
    pdl_trigger();
}

// Rows of the pairs of one CTA of the selection, from the counts of all of them.
__global__ void __launch_bounds__(kPlaceThreads)
moe_place_kernel(const __grid_constant__ RouteArgs a, const int block_tokens, const int* __restrict__ block_counts) {
    __shared__ int4 s_all[kPlaceThreads], s_before[kPlaceThreads];       // one each for the threads that share the counts
    __shared__ int s_base[kMoeMaxExperts];
    __shared__ int s_scan[kPlaceThreads / 32];
    pdl_wait();
    const int E = a.r.experts, words = count_words(E), quads = words >> 2;
    const uint32_t k = a.r.top_k;
    // `parts` threads share four experts' columns of counts
    const int parts = min(kParts, kPlaceThreads / quads), part = threadIdx.x / quads, quad = threadIdx.x % quads;
    // the first pair of each thread, in flight beside the counts
    const uint32_t n = (uint32_t)a.tokens * k, i0 = (uint32_t)blockIdx.x * block_tokens * k, i1 = min(i0 + (uint32_t)block_tokens * k, n);
    int id = -1, rank = 0;
    if (i0 + threadIdx.x < i1) {
        id = a.ids[i0 + threadIdx.x];
        rank = a.token_row[i0 + threadIdx.x];
    }
    if (part < parts) {
        int4 all = make_int4(0, 0, 0, 0), before = all;
        const int4* at = reinterpret_cast<const int4*>(block_counts) + part * quads + quad;
#pragma unroll 8
        for (int b = part; b < (int)gridDim.x; b += parts, at += parts * quads) {
            const int4 c = *at;
            const int m = b < (int)blockIdx.x ? -1 : 0;
            before = make_int4(before.x + (c.x & m), before.y + (c.y & m), before.z + (c.z & m), before.w + (c.w & m));
            all = make_int4(all.x + c.x, all.y + c.y, all.z + c.z, all.w + c.w);
        }
        s_all[part * quads + quad] = all;
        s_before[part * quads + quad] = before;
    }
    __syncthreads();
    int all = 0, before = 0;
    const int e = threadIdx.x;
    if (e < E)
        for (int p = 0; p < parts; p++) {
            all += reinterpret_cast<const int*>(s_all)[p * words + e];
            before += reinterpret_cast<const int*>(s_before)[p * words + e];
        }
    int total;
    const int off = scan(all, s_scan, total);
    if (e < E) s_base[e] = off + before;
    if (blockIdx.x == 0) {
        if (e < E) a.offsets[e] = off;
        if (e == 0) a.offsets[E] = total;
    }
    __syncthreads();
    for (uint32_t i = i0 + threadIdx.x; i < i1;) {
        if (id >= 0) {
            const int row = s_base[id] + rank;
            a.token_row[i] = row;
            a.row_token[row] = (int32_t)(i / k);
        }
        i += kPlaceThreads;
        if (i < i1) {
            id = a.ids[i];
            rank = a.token_row[i];
        }
    }
    for (uint32_t i = total + blockIdx.x * kPlaceThreads + threadIdx.x; i < n; i += gridDim.x * kPlaceThreads) a.row_token[i] = -1;
    pdl_trigger();
}

// Warps a CTA, tokens a warp and CTAs. One CTA up to kAlone tokens; more CTAs than kMaxBlocks would read too many counts.
struct Split {
    int warps, per_warp, blocks;
};
Split split_of(int64_t tokens, int64_t experts) {
    if (tokens <= kAlone) {
        const int warps = (int)std::max<int64_t>((experts + 31) / 32, tokens);
        return {warps, (int)std::max<int64_t>(1, (tokens + warps - 1) / warps), 1};
    }
    const int per_warp = (int)((tokens + (int64_t)kWarps * kMaxBlocks - 1) / ((int64_t)kWarps * kMaxBlocks));
    return {kWarps, per_warp, (int)((tokens + (int64_t)per_warp * kWarps - 1) / ((int64_t)per_warp * kWarps))};
}

template <typename T, int EPL>
qz_status select_kernel(const RouteArgs& a, const Split& s, int* counts, cudaStream_t st) {
    const bool simple = !a.bias && a.r.groups == 1;
    const auto fn = simple ? moe_select_kernel<T, EPL, true> : moe_select_kernel<T, EPL, false>;
    const int bytes = 4 * s.warps * (a.r.experts + (a.r.groups > 1 ? key_words(a.r.experts) : 0));
    if (bytes > 40 * 1024) QZ_TRY(opt_in_smem((const void*)fn, bytes));         // the 48 KB of a launch hold the static arrays too
    return launch_pdl(fn, dim3(s.blocks), dim3(s.warps * 32), bytes, st, a, s.per_warp, counts);
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
    const Split s = split_of(tokens, experts);
    return s.blocks == 1 ? 0 : (size_t)s.blocks * count_words((int)experts) * sizeof(int);
}

qz_status moe_route_launch(const RouteArgs& a, qz_dtype lt, void* ws, cudaStream_t st) {
    int* counts = static_cast<int*>(ws);
    const Split s = split_of(a.tokens, a.r.experts);
    QZ_TRY(lt == QZ_F32 ? select_launch<float>(a, s, counts, st) : select_launch<uint16_t>(a, s, counts, st));
    if (s.blocks == 1) return QZ_OK;
    return launch_pdl(moe_place_kernel, dim3(s.blocks), dim3(kPlaceThreads), 0, st, a, s.per_warp * s.warps, (const int*)counts);
}

} // namespace qz
