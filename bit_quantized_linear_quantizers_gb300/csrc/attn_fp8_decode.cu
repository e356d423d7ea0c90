// attn_fp8_decode.cu -- attention over the paged FP8 KV cache for few query rows
// per KV head (single tokens, a few tokens each): the keys and values are read
// once, so HBM is the bound.
//
// Products: mma.sync in f16, transposed, so that the query rows are the narrow side:
//   S^T [16 keys x 8 rows] = K q^T,  O^T [16 channels x 8 rows] += V^T P^T
// E4M3 codes widen to f16 exactly (two per instruction). FP8 operands of mma.sync
// are no way around that: on sm_103a they are widened inside, both of them, for every
// instruction (measured 7.1 cycles per SM for m16n8k32 with fresh operands, against
// 2 x 2.0 for the f16 form; 900 instructions for 32 keys instead of ~300). A bf16
// query is exact in f16 after its row is scaled by a power of two that brings its amax
// into [2^14, 2^15), down to 2^-29 of the amax. The scores of 8 keys x 8 rows turn
// into the second product's operand by movmatrix.
//
// The value scale of a page goes into the exponent instead of into V:
//   t_j = x_j log2(e) + log2 sv_j,  p_j = 2^(t_j - m + 8)
//   O = sum_j p_j c_j,  l = sum_j p_j / sv_j,  result O / l,
// since p_j = 2^(x_j log2 e) sv_j up to a factor common to O and l. m is raised only
// where a t passes m + 6 (p stays below 2^14 and keeps f16's 11 bits down to 2^-14), so
// few units rescale O. m, l and O are fp32.
//
// Work split: the units (32 keys) of every item (request, KV head, row tile), each
// item with a charge of kItemCost units for its q, its joining and its output in front,
// laid end to end over all requests and cut into equal shares, one CTA of 8 warps per
// SM (without the charge, a CTA with 70 items of a unit each ran six times as long as the
// others). Each
// warp takes every eighth unit of the CTA's share from a ring of its own (3 stages of
// 8 KB: 192 KB in flight per SM, against ~45 KB that the latency asks for), so no warp
// waits for another inside a share. The pages and scales of its next 32 units are looked
// up together, a lane for each, and passed on by shuffles: looked up unit by unit they were
// a third of the instructions; by a ninth warp for all rings, that warp's copies were
// the bound (112 us for 64 x <= 8192 keys with no arithmetic at all). V's fragments come
// transposed from shared memory by ldmatrix on bytes. At the end of a
// (request, head) the eight states join in shared memory; what spans several
// CTAs is joined by a second, small launch in a fixed order.
#include "qz_internal.cuh"
#include "attn_fp8.cuh"

#include <algorithm>

namespace qz {

namespace {

__device__ unsigned int g_attn_decode_err;

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kKeys = 32;                         // keys of a unit
constexpr int kStages = 3;
constexpr int kWholeKeys = 1024;                  // keys up to which few items take a CTA each
constexpr int kItemCost = 18;                     // units that an item's q, joining and output take (6: 98 us for 64 x <= 8192 keys,
                                                  // 12: 91.4, 24: 89.9)
constexpr float kPShift = 8.0f, kGrow = 6.0f;      // p = 2^(t - m + 8); growth of the maximum that m lets pass

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four E4M3 codes -> f16: bytes 0, 1 and 2, 3.
__device__ __forceinline__ void widen4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{ .reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi) : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16(float x0, float x1) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    return h;
}
// 8 x 8 transpose of 16-bit values over the warp (thread (g, t) holds row g, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t transpose_f16(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two 16 x 16 byte matrices transposed: lane l gives the address of row l (16 bytes). Rows
// are keys, columns channels: r[0] and r[2] hold rows 4t .. 4t+3 and 16 + 4t .. of channel g,
// r[1] and r[3] of channel 8 + g.
__device__ __forceinline__ void ldmatrix_t8(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
struct DecodeParams {
    CUtensorMap tm_k, tm_v;                       // codes as (head_dim, heads * page_size, num_pages)
    AttnArgs a;
    int shift;                                    // log2 page_size
    int max_rows;                                 // requests with more rows per KV head are not taken
    int whole;                                    // one item per CTA (row tiles per request and head), no joining launch; 0: shares
    int beside;                                   // the launch before is the prefill kernel on other requests: wait at the end
    int* head;                                    // [CTAs][8]: what the CTA left for the joining launch: 0: the part of an
                                                  // item begun before (0 or -1), 1: it goes on, 2: an item that goes on
                                                  // begins here (0 or -1), 3 .. 6: its first token, tokens, first row, KV head
    float* part;                                  // [CTAs][2] partial states
};

// A request's part of the work: rows (queries x heads of the group), keys, units.
struct Req {
    int q0, n, L, tiles, subs;                    // first token, tokens, keys, row tiles, units per (head, tile)
};

template <int R>
__device__ __forceinline__ Req load_req(const DecodeParams& P, int b, int G) {
    Req r;
    r.q0 = P.a.cu_q[b];
    r.n = min(P.a.cu_q[b + 1] - r.q0, P.a.max_q);
    r.n = (int)min((int64_t)r.n, P.a.tokens - r.q0);
    if (r.n < 0 || r.q0 < 0) r.n = 0;
    r.L = (int)min((int64_t)max(P.a.kv_lens[b], 0), (int64_t)P.a.max_blocks << P.shift);
    const int64_t rows = (int64_t)r.n * G;
    r.tiles = rows > P.max_rows ? 0 : (int)((rows + R - 1) / R);
    r.subs = (r.L + kKeys - 1) / kKeys;
    return r;
}

// The walk over the items that a CTA's share touches. An item lies at a .. a + kItemCost
// + subs of the line, counted from the share's begin; its units follow its charge.
template <int R>
struct Walk {
    int b, h, tile, a, share;
    Req r;
    __device__ bool valid() const { return a < share && b < 0x7fffffff; }
    __device__ int lo() const { return min(max(-a - kItemCost, 0), r.subs); }
    __device__ int hi() const { return min(max(share - a - kItemCost, 0), r.subs); }
    // some of its units are in the share; an item without keys belongs to the share that it begins in
    __device__ bool mine() const { return r.subs ? lo() < hi() : a >= 0; }
    __device__ void next(const DecodeParams& P, int G) {
        a += kItemCost + r.subs;
        if (++tile < r.tiles) return;
        tile = 0;
        if (++h < P.a.kv.heads) return;
        h = 0;
        do {
            if (++b >= P.a.B) { b = 0x7fffffff; return; }
            r = load_req<R>(P, b, G);
        } while (r.tiles == 0);
    }
    __device__ void next_mine(const DecodeParams& P, int G) {
        do next(P, G); while (valid() && !mine());
    }
};

template <int D, int R>
struct DecodeLayout {
    static constexpr int HALF = kKeys * D;                          // bytes of K (or V) of a unit
    static constexpr int STAGE = 2 * HALF;
    static constexpr int RING = kWarps * kStages * STAGE;
    static constexpr int JOIN_W = R == 8 ? kWarps : kWarps / 2;     // states that join at once
    static constexpr int JOIN_F = JOIN_W * R * D;                   // floats
    static constexpr int META = RING + JOIN_F * 4;
    static constexpr int SMEM = META + 1408 + 1024;                 // barriers, states; alignment
    static constexpr int PART = R * D + 2 * R;                      // floats of a partial state
};

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
attn_decode_kernel(const __grid_constant__ DecodeParams P) {
    using Lay = DecodeLayout<D, R>;
    constexpr int KS = D / 16;                    // 16-deep steps of K q^T
    constexpr int MT = D / 16;                    // 16-channel tiles of O^T
    constexpr int NR = R / 8;                     // 8-row tiles
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* join = reinterpret_cast<float*>(smem + Lay::RING);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Lay::META);                   // [warp][stage]
    float* s_m = reinterpret_cast<float*>(smem + Lay::META + 256);                    // [warp][R]
    float* s_l = s_m + kWarps * 16;
    int64_t* s_sum = reinterpret_cast<int64_t*>(s_l + kWarps * 16);                   // [warp]
    int* s_start = reinterpret_cast<int*>(s_sum + kWarps);                            // request, unit inside it

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = P.a.heads_q / P.a.kv.heads;
    const uint32_t bar0 = smem_u32(bars + warp * kStages), ring = smem_u32(smem) + warp * kStages * Lay::STAGE;
    if (lane == 0) {
        for (int s = 0; s < kStages; s++) mbar_init(bar0 + s * 8, 1);
        fence_barrier_init();
        if (warp == 0) {
            prefetch_tmap(&P.tm_k);
            prefetch_tmap(&P.tm_v);
        }
    }
    // The prefill kernel lets this one start when its CTAs have waited for the stream's earlier work
    // themselves and begin to leave; the two share no memory that either writes. The wait for its end
    // comes last, so that whatever waits for this kernel waits for both.
    // At the start a fence stands in for it: L1 may hold lines from before that earlier work, and the loads below
    // are plain ones, not those of the read-only path, so that they stay behind it.
    if (P.beside) __threadfence();
    else pdl_wait();
    pdl_trigger();                                // the joining launch may come up; it waits for this one's end

    int* header = P.head + blockIdx.x * 8;
    Walk<R> cur;
    if (P.whole) {
        const int id = blockIdx.x / P.whole;
        cur.tile = blockIdx.x % P.whole;
        cur.h = id % P.a.kv.heads;
        cur.b = id / P.a.kv.heads;
        cur.r = load_req<R>(P, cur.b, G);
        cur.a = 0;
        cur.share = cur.tile < cur.r.tiles ? kItemCost + cur.r.subs : 0;
    } else {
        // ---- the CTA's share: all units counted, then the request that holds its first one
        auto units_of = [&](int b) -> int64_t {
            if (b >= P.a.B) return 0;
            const Req r = load_req<R>(P, b, G);
            return (int64_t)P.a.kv.heads * r.tiles * (r.subs + kItemCost);
        };
        const int64_t mine0 = units_of(threadIdx.x);
        int64_t sum = mine0;
        for (int b = threadIdx.x + kThreads; b < P.a.B; b += kThreads) sum += units_of(b);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        int64_t total = 0;
        for (int w = 0; w < kWarps; w++) total += s_sum[w];
        const int64_t per = max((int64_t)(kWarps + kItemCost), (total + gridDim.x - 1) / gridDim.x);
        const int64_t u0 = per * blockIdx.x, u1 = min(u0 + per, total);
        if (threadIdx.x == 0) header[0] = header[2] = -1;
        if (u0 >= u1) {
            if (P.beside) pdl_wait();
            return;
        }
        int64_t before = 0;
        for (int b0 = 0; b0 < P.a.B; b0 += kThreads) {
            int64_t v = b0 == 0 ? mine0 : units_of(b0 + threadIdx.x);
            const int64_t own = v;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = v;
            __syncthreads();
            int64_t all = 0, base = before;
            for (int w = 0; w < kWarps; w++) {
                if (w < warp) base += s_sum[w];
                all += s_sum[w];
            }
            const int64_t first = base + v - own;
            if (u0 >= first && u0 < first + own) {
                s_start[0] = b0 + threadIdx.x;
                *reinterpret_cast<int64_t*>(s_start + 2) = u0 - first;
            }
            before += all;
            if (before > u0) break;                   // uniform
        }
        __syncthreads();

        cur.b = s_start[0];
        cur.r = load_req<R>(P, cur.b, G);
        cur.share = (int)(u1 - u0);                   // (a share of 2^31 units would be 2^36 keys)
        {
            const int64_t inside = *reinterpret_cast<int64_t*>(s_start + 2), len = cur.r.subs + kItemCost;
            const int item0 = (int)(inside / len);
            cur.h = item0 / cur.r.tiles;
            cur.tile = item0 % cur.r.tiles;
            cur.a = -(int)(inside % len);
        }
    }
    if (!P.whole && !cur.mine()) cur.next_mine(P, G);

    // q of an item: row g of each 8, channels t*16 .. of each 64-channel half, as it lies in memory
    uint4 raw[NR][D / 32];
    auto load_q = [&](const Walk<R>& it) {
#pragma unroll
        for (int rr = 0; rr < NR; rr++) {
            const int row = it.tile * R + rr * 8 + g, i = row / G, a = row - i * G;
            const bool there = it.valid() && i < it.r.n;
            const uint16_t* src = P.a.q + (int64_t)(it.r.q0 + i) * P.a.ldq + (int64_t)(it.h * G + a) * D + t * 16;
#pragma unroll
            for (int j = 0; j < D / 32; j++)
                raw[rr][j] = there ? *reinterpret_cast<const uint4*>(src + (j >> 1) * 64 + (j & 1) * 8) : make_uint4(0, 0, 0, 0);
        }
    };
    load_q(cur);

    // ---- the warp's next 32 units, one per lane: pages, rows in them, scales
    struct Batch { int p0, p1, y; float k0, v0, k1, v1; };            // y < 0: no unit; p < 0: no page
    Walk<R> ahead = cur;                          // at the item of the batch's first unit
    int ahead_base = 0, looked = warp;            // units of the share before that item; the batch's first unit
    auto look_up = [&]() {                        // leaves the walk at the next batch
        Walk<R> w = ahead;
        int base = ahead_base;
        const int u = looked + lane * kWarps;
        while (w.valid() && u >= base + w.hi() - w.lo()) {
            base += w.hi() - w.lo();
            w.next(P, G);
        }
        Batch k = {-1, -1, -1, 0.0f, 1.0f, 0.0f, 1.0f};
        if (w.valid()) {
            const int key = (w.lo() + u - base) * kKeys;
            k.y = (w.h << P.shift) + (key & ((1 << P.shift) - 1));
            const int32_t* row = P.a.block_table + (int64_t)w.b * P.a.ld_table + (key >> P.shift);
            k.p0 = *row;
            if (P.shift == 4 && key + 16 < w.r.L) k.p1 = row[1];
        }
        ahead_base = __shfl_sync(0xffffffffu, base, 31);              // (the last lane's item, or the end)
        ahead.b = __shfl_sync(0xffffffffu, w.b, 31);
        ahead.h = __shfl_sync(0xffffffffu, w.h, 31);
        ahead.tile = __shfl_sync(0xffffffffu, w.tile, 31);
        ahead.a = __shfl_sync(0xffffffffu, w.a, 31);
        ahead.r.q0 = __shfl_sync(0xffffffffu, w.r.q0, 31);
        ahead.r.n = __shfl_sync(0xffffffffu, w.r.n, 31);
        ahead.r.L = __shfl_sync(0xffffffffu, w.r.L, 31);
        ahead.r.tiles = __shfl_sync(0xffffffffu, w.r.tiles, 31);
        ahead.r.subs = __shfl_sync(0xffffffffu, w.r.subs, 31);
        looked += 32 * kWarps;
        return k;
    };
    auto load_scales = [&](Batch& k) {
        if (k.p0 >= P.a.kv.num_pages) k.p0 = -1;
        if (k.p1 >= P.a.kv.num_pages) k.p1 = -1;
        const int h = k.y >> P.shift;
        if (k.p0 >= 0) {
            const int64_t i = (int64_t)k.p0 * P.a.kv.heads + h;
            k.k0 = P.a.kv.k_scale[i];
            k.v0 = value_scale(P.a.kv.v_scale[i]);
        }
        if (P.shift == 4 && k.p1 >= 0) {
            const int64_t i = (int64_t)k.p1 * P.a.kv.heads + h;
            k.k1 = P.a.kv.k_scale[i];
            k.v1 = value_scale(P.a.kv.v_scale[i]);
        }
    };
    bool dead = false;                            // a wait gave up: no more copies, and no waits but the last ones
    int dead_at = -1;
    int issued = 0, fill = 0;                     // units whose copies are issued; their stage
    auto issue = [&](const Batch& b) {            // copies of the warp's next unit, in lane `issued` of its batch
        const int from = issued & 31;
        const int p0 = __shfl_sync(0xffffffffu, b.p0, from), p1 = __shfl_sync(0xffffffffu, b.p1, from);
        const int y = __shfl_sync(0xffffffffu, b.y, from);
        if (y < 0) return;
        if (lane == 0 && !dead) {
            const uint32_t dst = ring + fill * Lay::STAGE, bar = bar0 + fill * 8;
            if (P.shift == 4) {                   // two pages of 16 keys
                mbar_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * Lay::HALF);
                if (p0 >= 0) {
                    tma_load_3d(dst, &P.tm_k, 0, y, p0, bar);
                    tma_load_3d(dst + Lay::HALF, &P.tm_v, 0, y, p0, bar);
                }
                if (p1 >= 0) {
                    tma_load_3d(dst + Lay::HALF / 2, &P.tm_k, 0, y, p1, bar);
                    tma_load_3d(dst + Lay::HALF + Lay::HALF / 2, &P.tm_v, 0, y, p1, bar);
                }
            } else {
                mbar_arrive_expect_tx(bar, (p0 >= 0) * Lay::STAGE);
                if (p0 >= 0) {
                    tma_load_3d(dst, &P.tm_k, 0, y, p0, bar);
                    tma_load_3d(dst + Lay::HALF, &P.tm_v, 0, y, p0, bar);
                }
            }
        }
        issued++;
        if (++fill == kStages) fill = 0;
        __syncwarp();
    };
    // Batches: copies are issued from `front`, units computed from `back`, which is the same one but for the
    // stages in flight across a batch's end; `next` is on its way meanwhile.
    Batch front = look_up();
    if (front.p0 >= P.a.kv.num_pages) front.p0 = -1;
    if (front.p1 >= P.a.kv.num_pages) front.p1 = -1;
#pragma unroll 1
    for (int s = 0; s < kStages; s++) issue(front);
    load_scales(front);
    Batch back = front, next = {-1, -1, -1, 0.0f, 1.0f, 0.0f, 1.0f};
    int done = 0;                                 // units that this warp has computed
    int st = 0;                                   // stage of the warp's next unit, and its phase
    uint32_t phase = 0;
    const float c0 = fabsf(P.a.sm_scale) * kLog2e;
    int unit = 0;                                 // units of the share before the item
    // Row of the V matrices that this lane addresses: rows 4t + {0, 1, 2, 3} are keys 2t, 2t + 1, 8 + 2t,
    // 9 + 2t, the depth that P's fragment gives to lane t of a quad.
    const int slot = lane & 15, vrow = (lane & 16) + (slot & 2 ? 8 : 0) + (slot >> 2) * 2 + (slot & 1);
    const uint32_t voff = Lay::HALF + vrow * D + (D == 128 ? (vrow & 7) << 4 : ((vrow >> 1) & 3) << 4);

    while (cur.valid()) {
        if (cur.r.subs == 0) {                    // no keys: zeros
            for (int c = threadIdx.x; c < R * D / 8; c += kThreads) {
                const int row = cur.tile * R + c / (D / 8), i = row / G, a = row - i * G;
                if (i >= cur.r.n) break;
                const int64_t token = cur.r.q0 + i;
                *reinterpret_cast<uint4*>(P.a.out + token * P.a.ldo + (int64_t)(cur.h * G + a) * D + c % (D / 8) * 8) =
                    make_uint4(0, 0, 0, 0);
                if (P.a.lse && c % (D / 8) == 0) P.a.lse[token * P.a.heads_q + cur.h * G + a] = -INFINITY;
            }
            cur.next_mine(P, G);
            load_q(cur);
            continue;
        }
        const int sub = cur.lo(), here = cur.hi() - sub;               // units of this item in this share
        // ---- q of this item: row g of each 8 in f16, in the order the keys are read; per thread the factor
        // and the seen keys of rows 2t, 2t + 1 of each 8, which its scores belong to
        uint32_t qf[NR][KS][2];
        float crow[NR][2];
        int seen[NR][2];
#pragma unroll
        for (int n = 0; n < NR; n++) {
            float v[D / 4];
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 32; j++) {    // 16 bytes: channels t*16 + (j & 1)*8 of the 64-channel half j >> 1
                const uint32_t x[4] = {raw[n][j].x, raw[n][j].y, raw[n][j].z, raw[n][j].w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    v[j * 8 + 2 * e] = __uint_as_float(x[e] << 16);
                    v[j * 8 + 2 * e + 1] = __uint_as_float(x[e] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int e = 0; e < D / 4; e++) m = fmaxf(m, fabsf(v[e]));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            float up, down;
            row_scale(m, up, down);               // to [2^7, 2^8), and on to [2^14, 2^15)
            const float sgn = (P.a.sm_scale < 0.0f ? -up : up) * 128.0f, c = c0 * down * (1.0f / 128.0f);
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int e = 0; e < 2; e++)
                    qf[n][k][e] = pack_f16(v[4 * k + 2 * e] * sgn, v[4 * k + 2 * e + 1] * sgn);
#pragma unroll
            for (int e = 0; e < 2; e++) {
                crow[n][e] = __shfl_sync(0xffffffffu, c, (2 * t + e) * 4);
                const int i = (cur.tile * R + n * 8 + 2 * t + e) / G;
                seen[n][e] = i >= cur.r.n ? 0 : P.a.causal ? min(max(cur.r.L - cur.r.n + i + 1, 0), cur.r.L) : cur.r.L;
            }
        }
        float o[MT][NR][4];                       // channel 16 mt + g (+ 8: [2], [3]), rows 2t, 2t + 1
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int n = 0; n < NR; n++) {
#pragma unroll
            for (int j = 0; j < MT; j++)
#pragma unroll
                for (int e = 0; e < 4; e++) o[j][n][e] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }

        // ---- this warp's units of the item: share indices = warp mod 8
        int first = unit + ((warp - unit) & (kWarps - 1));
#pragma unroll 1
        for (int u = first; u < unit + here; u += kWarps) {
            const int key0 = (sub + (u - unit)) * kKeys;
            const int from = done & 31;
            if (from == 0) back = front;          // (the copies' batch turned over at most kStages units ago)
            const float k0 = __shfl_sync(0xffffffffu, back.k0, from), v0 = __shfl_sync(0xffffffffu, back.v0, from);
            float k1 = k0, v1 = v0;
            bool p0 = __shfl_sync(0xffffffffu, back.p0, from) >= 0, p1 = p0;
            if (P.shift == 4) {
                k1 = __shfl_sync(0xffffffffu, back.k1, from);
                v1 = __shfl_sync(0xffffffffu, back.v1, from);
                p1 = __shfl_sync(0xffffffffu, back.p1, from) >= 0;
            }
            if (!dead && !mbar_wait<false>(bar0 + st * 8, phase, &g_attn_decode_err)) dead = true;
            if (__any_sync(0xffffffffu, dead) && dead_at < 0) dead = true, dead_at = done;
            uint8_t* kt = smem + (warp * kStages + st) * Lay::STAGE;

            // S^T = K q^T: two tiles of 16 keys
            float s[2][NR][4];                    // key 16 mt + g (+ 8: [2], [3]), rows 2t, 2t + 1
#pragma unroll
            for (int mt = 0; mt < 2; mt++) {
#pragma unroll
                for (int n = 0; n < NR; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) s[mt][n][e] = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 64; c++) {                    // 16 channels of this thread, 4 steps
                    uint4 x[2];
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int r = mt * 16 + e * 8 + g, ch = D == 128 ? ((t + 4 * c) ^ g) : (t ^ ((r >> 1) & 3));
                        x[e] = *reinterpret_cast<const uint4*>(kt + r * D + ch * 16);
                    }
                    const uint32_t x0[4] = {x[0].x, x[0].y, x[0].z, x[0].w}, x1[4] = {x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        uint32_t a0, a1, a2, a3;
                        widen4(x0[k], a0, a2);
                        widen4(x1[k], a1, a3);
#pragma unroll
                        for (int n = 0; n < NR; n++)
                            mma_f16(s[mt][n], a0, a1, a2, a3, qf[n][4 * c + k][0], qf[n][4 * c + k][1]);
                    }
                }
            }
            // (a term of 0 that is NaN under an infinite key scale)
            const float lv[2] = {fmaf(k0, 0.0f, __log2f(v0)), fmaf(k1, 0.0f, __log2f(v1))}, iv[2] = {__frcp_rn(v0), __frcp_rn(v1)};
            const int live = cur.r.L - key0;      // keys of the unit that exist
            const bool nil0 = !p0 || v0 <= kLeastScale, nil1 = !p1 || v1 <= kLeastScale;     // no values
            const bool edge = live < kKeys || nil0 || nil1 || (P.a.causal && key0 + kKeys > cur.r.L - cur.r.n + 1);
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NR; n++)
#pragma unroll
                for (int mt = 0; mt < 2; mt++) {
                    const float a0 = crow[n][0] * (mt ? k1 : k0), a1 = crow[n][1] * (mt ? k1 : k0);
                    s[mt][n][0] = fmaf(s[mt][n][0], a0, lv[mt]);
                    s[mt][n][1] = fmaf(s[mt][n][1], a1, lv[mt]);
                    s[mt][n][2] = fmaf(s[mt][n][2], a0, lv[mt]);
                    s[mt][n][3] = fmaf(s[mt][n][3], a1, lv[mt]);
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (16 * mt + 8 * (e >> 1) + g >= seen[n][e & 1] - key0 || !(mt ? p1 : p0)) s[mt][n][e] = -INFINITY;
                    }
                }
            if (edge) {
                // rows of V that were never written may hold NaN codes, and 0 * NaN is no 0
                if (lane >= live || (lane < 16 ? nil0 : nil1))
#pragma unroll
                    for (int c = 0; c < D / 16; c++)
                        *reinterpret_cast<uint4*>(kt + Lay::HALF + lane * D + c * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();         // before the stage's next copy
                __syncwarp();
            }
            float mx[NR][2];                      // of this thread's keys
#pragma unroll
            for (int n = 0; n < NR; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    mx[n][e] = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
                    raise |= mx[n][e] > m[n][e] + kGrow;              // (an m of -inf: anything seen)
                }
            if (__any_sync(0xffffffffu, raise)) {
                float f[NR][2];
#pragma unroll
                for (int n = 0; n < NR; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        float x = mx[n][e];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        x = fmaxf(x, m[n][e]);
                        f[n][e] = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - x);
                        m[n][e] = x;
                        l[n][e] *= f[n][e];
                    }
#pragma unroll
                for (int j = 0; j < MT; j++)
#pragma unroll
                    for (int n = 0; n < NR; n++)
#pragma unroll
                        for (int e = 0; e < 4; e++) o[j][n][e] *= f[n][e & 1];
            }
            uint32_t pf[NR][4];                   // P^T: depth steps of keys 0-15 and 16-31
#pragma unroll
            for (int n = 0; n < NR; n++) {
                const float f0 = m[n][0] == -INFINITY ? 0.0f : kPShift - m[n][0];   // nothing seen yet: every p is 0
                const float f1 = m[n][1] == -INFINITY ? 0.0f : kPShift - m[n][1];
#pragma unroll
                for (int mt = 0; mt < 2; mt++) {
                    const float a = ex2(s[mt][n][0] + f0), b = ex2(s[mt][n][1] + f1);
                    const float c = ex2(s[mt][n][2] + f0), d = ex2(s[mt][n][3] + f1);
                    l[n][0] = fmaf(a + c, iv[mt], l[n][0]);
                    l[n][1] = fmaf(b + d, iv[mt], l[n][1]);
                    pf[n][2 * mt] = transpose_f16(pack_f16(a, b));
                    pf[n][2 * mt + 1] = transpose_f16(pack_f16(c, d));
                }
            }
            // O^T += V^T P^T, 16 channels at a time
            const uint32_t va = smem_u32(kt) + voff;
#pragma unroll
            for (int j = 0; j < MT; j++) {
                uint32_t b[4], a0, a1, a2, a3;
                ldmatrix_t8(b, va ^ (uint32_t)(j * 16));              // the swizzled 16-byte chunk j of the rows
                widen4(b[0], a0, a2);
                widen4(b[1], a1, a3);
#pragma unroll
                for (int n = 0; n < NR; n++) mma_f16(o[j][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
                widen4(b[2], a0, a2);
                widen4(b[3], a1, a3);
#pragma unroll
                for (int n = 0; n < NR; n++) mma_f16(o[j][n], a0, a1, a2, a3, pf[n][2], pf[n][3]);
            }
            __syncwarp();                         // the stage has been read
            if (++st == kStages) { st = 0; phase ^= 1; }
            done++;
            // the next batch: looked up half a batch early, its scales a quarter
            if (from == 15) next = look_up();
            if (from == 23) load_scales(next);
            if ((issued & 31) == 0) front = next; // (issued runs kStages ahead of done)
            issue(front);
        }

        // ---- the item's end in this share: join the warps, the next item's q on its way
        Walk<R> nxt = cur;
        nxt.next_mine(P, G);
        load_q(nxt);
#pragma unroll
        for (int n = 0; n < NR; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
                l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
                if (g == 0) {
                    s_m[warp * 16 + n * 8 + 2 * t + e] = m[n][e];
                    s_l[warp * 16 + n * 8 + 2 * t + e] = l[n][e];
                }
            }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NR; n++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const int row = n * 8 + 2 * t + e;
                float x = -INFINITY;
                for (int w = 0; w < kWarps; w++) x = fmaxf(x, s_m[w * 16 + row]);
                const float f = m[n][e] == -INFINITY ? 0.0f : ex2(m[n][e] - x);
#pragma unroll
                for (int j = 0; j < MT; j++) {
                    o[j][n][e] *= f;
                    o[j][n][2 + e] *= f;
                }
            }
        // A state as [row][channel], bits 3 and 4 of the channel turned by the row's (every lane of a store
        // in a bank of its own). The upper warps' states first where not all fit at once.
        auto at = [&](int row, int ch) { return row * D + (ch ^ ((row >> 1 & 3) * 8)); };
        auto put = [&](float* to) {
#pragma unroll
            for (int n = 0; n < NR; n++)
#pragma unroll
                for (int e = 0; e < 2; e++)
#pragma unroll
                    for (int j = 0; j < MT; j++) {
                        to[at(n * 8 + 2 * t + e, j * 16 + g)] = o[j][n][e];
                        to[at(n * 8 + 2 * t + e, j * 16 + 8 + g)] = o[j][n][2 + e];
                    }
        };
        constexpr int JW = Lay::JOIN_W;
        if (JW < kWarps) {
            if (warp >= JW) put(join + (warp - JW) * R * D);
            __syncthreads();
            if (warp < JW) {
                float* own = join + warp * R * D;
#pragma unroll
                for (int n = 0; n < NR; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++)
#pragma unroll
                        for (int j = 0; j < MT; j++) {
                            o[j][n][e] += own[at(n * 8 + 2 * t + e, j * 16 + g)];
                            o[j][n][2 + e] += own[at(n * 8 + 2 * t + e, j * 16 + 8 + g)];
                        }
                put(own);                         // the places that this thread has read
            }
        } else {
            put(join + warp * R * D);
        }
        __syncthreads();
        const bool begins = sub == 0, ends = sub + here == cur.r.subs;
        float* dst = P.part + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * Lay::PART;
#pragma unroll
        for (int c = threadIdx.x; c < R * D / 4; c += kThreads) {     // four channels of a row per thread
            const int row = c / (D / 4), d0 = c % (D / 4) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float mr = -INFINITY, lr = 0.0f;
#pragma unroll
            for (int w = 0; w < JW; w++) {
                const float4 y = *reinterpret_cast<const float4*>(join + w * R * D + at(row, d0));
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
#pragma unroll
            for (int w = 0; w < kWarps; w++) mr = fmaxf(mr, s_m[w * 16 + row]);
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float mw = s_m[w * 16 + row], lw = s_l[w * 16 + row];
                lr += mw == -INFINITY && lw == 0.0f ? 0.0f : lw * ex2(mw - mr);
            }
            if (!(begins && ends)) {
                *reinterpret_cast<float4*>(dst + row * D + d0) = x;
                if (d0 == 0) {
                    dst[R * D + row] = mr;
                    dst[R * D + R + row] = lr;
                }
                continue;
            }
            const int i = (cur.tile * R + row) / G, a = cur.tile * R + row - i * G;
            if (i < cur.r.n) {
                const float inv = lr > 0.0f ? 1.0f / lr : (lr == lr ? 0.0f : lr);
                const int64_t token = cur.r.q0 + i;
                const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.x * inv, x.y * inv), y1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
                *reinterpret_cast<uint2*>(P.a.out + token * P.a.ldo + (int64_t)(cur.h * G + a) * D + d0) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
                if (P.a.lse && d0 == 0)
                    P.a.lse[token * P.a.heads_q + cur.h * G + a] =
                        lr > 0.0f ? (mr - kPShift + __log2f(lr)) * kLn2 : (lr == lr ? -INFINITY : lr);
            }
        }
        if (!(begins && ends) && threadIdx.x == 0) {
            if (begins) {                         // the joining launch starts here
                header[2] = 0;
                header[3] = cur.r.q0;
                header[4] = cur.r.n;
                header[5] = cur.tile * R;
                header[6] = cur.h;
            } else {
                header[0] = 0;
                header[1] = !ends;                // goes on in the next CTA
            }
        }
        __syncthreads();                          // the states, s_m and s_l have been read
        unit += here;
        cur = nxt;
    }
    // copies still in flight (a wait that gave up): their stages must not outlive the CTA. The units counted as issued
    // after it had no copies: a wait for each of them would run its whole limit.
    if (dead)
        for (int k = dead_at; k < min(issued, dead_at + kStages); k++)
            mbar_wait(bar0 + k % kStages * 8, (k / kStages) & 1, &g_attn_decode_err);
    if (P.beside) pdl_wait();
}

// Joins the states of an item that several CTAs share, in the order of its keys:
// CTA c's launch-mate takes the item whose first part CTA c left.
template <int D, int R>
__global__ void __launch_bounds__(256)
attn_join_kernel(const __grid_constant__ DecodeParams P, int parts) {
    using Lay = DecodeLayout<D, R>;
    constexpr int V = R * D / 256;                // channels of a thread: 4 (R = 8, D = 128) ...
    pdl_trigger();
    pdl_wait();
    const int* own = P.head + blockIdx.x * 8;
    if (own[2] >= 0) {
        const int G = P.a.heads_q / P.a.kv.heads;
        const int q0 = own[3], n = own[4], row0 = own[5], h = own[6];
        const int row = threadIdx.x * V / D, d0 = threadIdx.x * V % D;
        const float* src = P.part + ((int64_t)blockIdx.x * 2 + 1) * Lay::PART;
        float m = src[R * D + row], l = src[R * D + R + row], o[V];
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = src[row * D + d0 + i];
        bool more = true;
        for (int c = blockIdx.x + 1; more && c < parts; c++) {
            src = P.part + (int64_t)c * 2 * Lay::PART;
            more = P.head[c * 8 + 1] != 0;
            const float m2 = src[R * D + row], l2 = src[R * D + R + row], mm = fmaxf(m, m2);
            const float f = m == -INFINITY ? (l == l ? 0.0f : l) : ex2(m - mm);
            const float f2 = m2 == -INFINITY ? (l2 == l2 ? 0.0f : l2) : ex2(m2 - mm);
            l = l * f + l2 * f2;
#pragma unroll
            for (int i = 0; i < V; i++) o[i] = o[i] * f + src[row * D + d0 + i] * f2;
            m = mm;
        }
        const int rw = row0 + row, i = rw / G, a = rw - i * G;
        if (i < n) {
            const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
            uint16_t* out = P.a.out + (int64_t)(q0 + i) * P.a.ldo + (int64_t)(h * G + a) * D + d0;
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const __nv_bfloat162 w = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
                *reinterpret_cast<__nv_bfloat162*>(out + e) = w;
            }
            if (P.a.lse && d0 == 0)
                P.a.lse[(int64_t)(q0 + i) * P.a.heads_q + h * G + a] =
                    l > 0.0f ? (m - kPShift + __log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
        }
    }
}

template <int D, int R>
qz_status launch_decode(DecodeParams& P, int64_t most_rows, void* ws, cudaStream_t st) {
    using Lay = DecodeLayout<D, R>;
    // Few and short items (by the table's width): a CTA each, which spares the shares' reckoning and the joining
    // launch (one request on 8 KV heads, whole against split: 517 keys 7.9 against 10.7 us, 2048 keys 14.6
    // against 12.4).
    const int64_t tiles = (most_rows + R - 1) / R, items = (int64_t)P.a.B * P.a.kv.heads * tiles;
    P.whole = items <= num_sms() && (int64_t)P.a.max_blocks * P.a.kv.page_size <= kWholeKeys ? (int)tiles : 0;
    const int ctas = P.whole ? (int)items : num_sms();
    P.head = reinterpret_cast<int*>(ws);
    P.part = reinterpret_cast<float*>(static_cast<char*>(ws) + ((size_t)ctas * 32 + 255) / 256 * 256);
    QZ_TRY(opt_in_smem((const void*)attn_decode_kernel<D, R>, Lay::SMEM));
    QZ_TRY(launch_pdl(attn_decode_kernel<D, R>, dim3(ctas), dim3(kThreads), Lay::SMEM, st, P));
    if (P.whole) return QZ_OK;
    return launch_pdl(attn_join_kernel<D, R>, dim3(ctas), dim3(256), 0, st, P, ctas);
}

} // namespace

size_t ws_attn_decode() {
    const size_t ctas = (size_t)num_sms();
    return (ctas * 32 + 255) / 256 * 256 + ctas * 2 * DecodeLayout<128, 16>::PART * 4;
}

// Requests of at most max_rows rows per KV head; the others are left alone. beside: launched directly
// after the prefill kernel of the same call, with a workspace of its own.
qz_status attn_decode_launch(const AttnArgs& a, int max_rows, bool beside, void* ws, cudaStream_t st) {
    DecodeParams P;
    P.beside = beside;
    P.a = a;
    P.shift = a.kv.page_size == 16 ? 4 : a.kv.page_size == 32 ? 5 : a.kv.page_size == 64 ? 6 : 7;
    P.max_rows = max_rows;
    const uint64_t D = (uint64_t)a.kv.head_dim, rows = (uint64_t)a.kv.heads * a.kv.page_size;
    const uint32_t box = (uint32_t)std::min(a.kv.page_size, kKeys);
    if (!encode_tmap_3d_u8(&P.tm_k, a.kv.k_codes, D, rows, (uint64_t)a.kv.num_pages, D, (uint64_t)a.kv.page_stride,
                           (uint32_t)D, box, (int)D) ||
        !encode_tmap_3d_u8(&P.tm_v, a.kv.v_codes, D, rows, (uint64_t)a.kv.num_pages, D, (uint64_t)a.kv.page_stride,
                           (uint32_t)D, box, (int)D))
        return QZ_ERR_CUDA;
    const int64_t most = std::min<int64_t>((int64_t)a.max_q * (a.heads_q / a.kv.heads), max_rows);
    if (most <= 8)
        return D == 64 ? launch_decode<64, 8>(P, most, ws, st) : launch_decode<128, 8>(P, most, ws, st);
    return D == 64 ? launch_decode<64, 16>(P, most, ws, st) : launch_decode<128, 16>(P, most, ws, st);
}

qz_status attn_decode_error_read_and_clear() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_decode_err, sizeof(v)) != cudaSuccess) return QZ_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_attn_decode_err, &z, sizeof(z)) != cudaSuccess) return QZ_ERR_CUDA;
    return v ? QZ_ERR_TIMEOUT : QZ_OK;
}

} // namespace qz
