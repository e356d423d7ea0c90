// attn_fp8_prefill.cu -- attention over the paged FP8 KV cache for many query rows
// per KV head (prompts, chunks of prompts, cross attention of prompts): bound by
// the tensor cores, so both products run on tcgen05 with accumulators in TMEM.
//
// Rows: the query heads of a KV head and the tokens of a request are packed into
// one row index (token * group + head), so a key tile is read once for the group.
// A CTA takes 256 rows (two 128-row tiles, one warpgroup of softmax each) and
// walks the keys in tiles of 128:
//   S = q K^T    kind::f8f6f4. K enters as stored; bf16 q is the sum of two E4M3
//                parts (hi = E4M3(q), lo = E4M3(q - hi): 4 + 4 significant bits, after a
//                power of two brings the row's amax into [128, 256); exact above 2^-10 of the amax,
//                off by at most 2^-17 of it below), two MMAs at twice the bf16 rate each: the
//                time of a bf16 product, and no widening of K.
//   O += P V     kind::f16, P from TMEM in f16 (11 bits), V widened from E4M3 to f16 (exact)
//                by a warpgroup of its own. Splitting P into two E4M3 parts as well would
//                spare the widening but costs 14 issue cycles per pair of scores and
//                scheduler against 2 (measured conversion rates: e4m3x2.f16x2 4.0 cycles
//                per warp, f16x2.e4m3x2 2.25, f16x2.f32 2.0): more than the MMAs take.
// The page's value scale goes into the exponent, as in the decode kernel:
//   t = x log2(e) + log2 sv, p = 2^(t - m + 8), O = sum p c, l = sum p / sv.
// m is raised only when p outgrows f16 (sums of 16 above 2^15), which spares the
// maximum of most tiles and most rescalings of O.
//
// One warp issues the MMAs of both row tiles in turn: while one's softmax runs, the
// other's P V and next S do. S's TMEM columns hold P afterwards. A pair of row tiles
// takes 32 MMAs of 64 cycles for 128 keys; the S products read both operands from shared
// memory at its full 128 bytes a cycle. Measured, graph replays: 8192 tokens, 32 heads on
// 8 KV heads of 128, causal: 435 us (1.26 PFLOP/s, 66 % of the 1.91 that a bf16 product
// reaches); 4864 rows a head by 8192 keys without a mask: 471 us (72 %). What is missing is
// the chain S -> softmax -> P V of a row tile, which its partner's MMAs do not cover to the
// end: the same hand-offs without any arithmetic take 2290 to 2760 cycles a pair
// of tiles against 2048 of MMAs.
//
// One CTA per SM stays for the launch: a scheduler warp takes the items (row tile,
// KV head, part of the keys) of CTAs not yet launched (cluster launch control), the
// longest first, one item ahead of the roles, so copies, q and the first S of the next item
// run under the output of the last one. A launch of few row tiles splits their keys into
// parts, whose states a second launch joins in order.
#include "qz_internal.cuh"
#include "attn_fp8.cuh"

#include <algorithm>

namespace qz {

namespace {

__device__ unsigned int g_attn_prefill_err;

constexpr int kThreads = 512;                     // warps 0-7 softmax, 8-11 widen V, 12 TMA, 13 items, 14 MMA
constexpr int kM = 128, kRows = 2 * kM, kN = 128; // rows of a tile, of a CTA; keys of a tile
constexpr int kKStages = 3, kVStages = 2, kScStages = 4;
constexpr int kSplitKeys = 512;
constexpr float kPShift = 8.0f;
constexpr float kMost = 32768.0f;                  // a sum of 16 p up to which each fits f16 (largest 65504)
constexpr float kTiny = 1e-30f;                   // added to the factor of a raw score: an infinite one stays so under it

struct PrefillParams {
    CUtensorMap tm_k, tm_v;                       // codes as (head_dim, heads * page_size, num_pages), one page's rows a box
    AttnArgs a;
    int shift;
    int min_rows;                                 // requests with fewer rows per KV head are not taken
    int tiles;                                    // upper bound of row tiles over all requests
    int splits;                                   // parts of an item's keys; with more than one:
    int* head;                                    //   [tiles * heads][2] request (-1: none) and first row
    float* part;                                  //   [tiles * heads][splits] states: O [256][D], m [256], l [256]
};

// What a role reads about an item.
struct Item {
    int b, row0, h, q0, n, L, t0, nk[2], part;    // t0: first key tile; nk: key tiles of each row tile; part: -1 or its state
};

template <int D>
struct PrefillLayout {
    static constexpr int Q = kM * D;                                // one part of one row tile
    static constexpr int KT = kN * D;                               // a key tile (codes)
    static constexpr int VH = kN * D * 2;                           // a value tile in f16
    static constexpr int Q_OFF = 0;                                 // [tile][part]
    static constexpr int K_OFF = Q_OFF + 4 * Q;
    static constexpr int V_OFF = K_OFF + kKStages * KT;
    static constexpr int VH_OFF = V_OFF + kVStages * KT;
    static constexpr int SC_OFF = VH_OFF + 2 * VH;                  // [stage][8] float4: scales of 16 keys
    static constexpr int BAR_OFF = SC_OFF + kScStages * 8 * 16;
    static constexpr int SMEM = BAR_OFF + 640 + 1024;
    static constexpr int PART = kRows * D + 2 * kRows;              // floats of a part's state
    static constexpr uint32_t S_COL = 0, O_COL = 256;               // TMEM columns: S0 S1 O0 O1
    static constexpr uint32_t IDESC_S = idesc_dense(0u, 0u, kM, kN);                     // E4M3 x E4M3
    static constexpr uint32_t IDESC_O = idesc_dense(0u, 0u, kM, D) | 1u << 16;           // f16 x f16, B MN-major
};

// Shared-memory descriptors as two words, so that the issuing thread adds an offset
// to the low one only: the low word holds the address (in 16-byte units) and the
// leading offset, the high word is a constant of the layout. One thread issues 32
// MMAs of 64 cycles per pair of row tiles: with descriptors built per MMA the issue
// took 156 cycles each, more than twice the MMAs themselves.
// K-major operand of D-byte rows under the D-byte swizzle (8-row atoms stacked).
template <int D>
__device__ __forceinline__ uint32_t sdesc_k_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | 1u << 16; }
template <int D>
__device__ constexpr uint32_t sdesc_k_hi() { return (uint32_t)(8 * D) >> 4 | 1u << 14 | (D == 128 ? 2u : 4u) << 29; }
// MN-major f16 operand: 64-channel blocks (128 bytes per key, 128-byte swizzle over 8
// keys), the blocks kN * 128 bytes apart (leading offset), 8-key groups 1024 apart.
__device__ __forceinline__ uint32_t sdesc_v_lo(uint32_t saddr) {
    return (saddr & 0x3FFFFu) >> 4 | (uint32_t)((kN * 128) >> 4) << 16;
}
constexpr uint32_t kDescVHi = 1024u >> 4 | 1u << 14 | 2u << 29;

// The MMA warp issues them converged, through an elected lane: operands of a branch of one
// lane are moved to the uniform registers anew for every MMA (4864 rows a head by 8192 keys: 543 us
// so, 503 elected).
__device__ __forceinline__ void mma_s(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool acc) {
    asm volatile("{ .reg .pred p, q; .reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0; elect.sync _|q, 0xffffffff;\n\t"
                 "mov.b64 a, {%1, %3}; mov.b64 b, {%2, %3};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p; }"
                 ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_o(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool acc) {
    asm volatile("{ .reg .pred p, q; .reg .b64 b;\n\tsetp.ne.b32 p, %5, 0; elect.sync _|q, 0xffffffff;\n\t"
                 "mov.b64 b, {%2, %3};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p; }"
                 ::"r"(d), "r"(a), "r"(b_lo), "r"(kDescVHi), "r"(idesc), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t bar) {
    asm volatile("{ .reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar) : "memory");
}

// (a, b) * s + c and (a, b) += (x, y) on the paired fp32 instructions.
__device__ __forceinline__ void fma2(float a, float b, float s, float c, float& x, float& y) {
    asm("{ .reg .b64 v, m, k, r;\n\tmov.b64 v, {%2, %3}; mov.b64 m, {%4, %4}; mov.b64 k, {%5, %5};\n\t"
        "fma.rn.f32x2 r, v, m, k;\n\tmov.b64 {%0, %1}, r; }"
        : "=f"(x), "=f"(y) : "f"(a), "f"(b), "f"(s), "f"(c));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
    asm("{ .reg .b64 v, r;\n\tmov.b64 v, {%0, %1}; mov.b64 r, {%2, %3};\n\t"
        "add.rn.f32x2 v, v, r;\n\tmov.b64 {%0, %1}, v; }"
        : "+f"(a), "+f"(b) : "f"(x), "f"(y));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
                 "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

template <int REGS> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

// The bounded wait of this kernel: few polls with a long suspend hint.
constexpr uint32_t kHintNs = 1000, kPolls = 1u<<21;
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kPolls; i++) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity), "r"(kHintNs) : "memory");
        if (ok) return true;
    }
    atomicExch(&g_attn_prefill_err, (unsigned int)QZ_ERR_TIMEOUT);
    return false;
}

// Cluster launch control: asks for the item of a CTA that has not been launched.
__device__ __forceinline__ void try_cancel(uint32_t result, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(result), "r"(bar) : "memory");
}
// Its blockIdx.x, or -1 where there is none left.
__device__ __forceinline__ int canceled_cta(uint32_t result) {
    uint32_t ok, x = 0;
    asm volatile("{ .reg .pred p; .reg .b128 r;\n\t"
                 "ld.shared.b128 r, [%2];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r; }"
                 : "=r"(ok), "=r"(x) : "r"(result) : "memory");
    return ok ? (int)x : -1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_kernel(const __grid_constant__ PrefillParams P) {
    using L = PrefillLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    // barriers: K full/empty, raw V full/empty, widened V full/empty, scales full, S full, P full, O done, q, drain,
    // item full/empty, scheduler
    constexpr int KF = 0, KE = KF + kKStages, VF = KE + kKStages, VE = VF + kVStages, HF = VE + kVStages, HE = HF + 2,
                  SC = HE + 2, SF = SC + kScStages, PF = SF + 2, OD = PF + 2, QF = OD + 2, DR = QF + 2, IF = DR + 1, IE = IF + 2, CB = IE + 2, NBAR = CB + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBAR);
    uint8_t* canceled = smem + L::BAR_OFF + 384;                    // 16 bytes
    Item* items = reinterpret_cast<Item*>(smem + L::BAR_OFF + 400); // two: a role's current one stays here, not in registers
    int* classes = reinterpret_cast<int*>(smem + L::BAR_OFF + 512);  // [32] row tiles of the requests of a class
    float4* sc = reinterpret_cast<float4*>(smem + L::SC_OFF);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = P.a.heads_q / P.a.kv.heads;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kKStages; s++) { mbar_init(bar(KF + s), 1); mbar_init(bar(KE + s), 1); }
        for (int s = 0; s < kVStages; s++) { mbar_init(bar(VF + s), 1); mbar_init(bar(VE + s), 4); }
        for (int s = 0; s < 2; s++) {
            mbar_init(bar(HF + s), 4);
            mbar_init(bar(HE + s), 1);
            mbar_init(bar(SF + s), 1);
            mbar_init(bar(PF + s), 4);
            mbar_init(bar(OD + s), 1);
            mbar_init(bar(QF + s), 4);
        }
        for (int s = 0; s < kScStages; s++) mbar_init(bar(SC + s), 1);
        for (int s = 0; s < 2; s++) {
            mbar_init(bar(IF + s), 1);
            mbar_init(bar(IE + s), 14);           // 8 softmax, 4 widening, the TMA and the MMA warp
        }
        mbar_init(bar(CB), 1);
        mbar_init(bar(DR), 1);
        fence_barrier_init();
        prefetch_tmap(&P.tm_k);
        prefetch_tmap(&P.tm_v);
    }
    if (warp == 13) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();
    const int pages_tile = kN >> P.shift;         // boxes of a key tile

    // The k-th item of this CTA: is there one (its b >= 0), and the role's leave of it.
    auto has_item = [&](int k) { return warp_wait(bar(IF + (k & 1)), (k >> 1) & 1) && items[k & 1].b >= 0; };
    auto done_item = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(IE + (k & 1)));
    };

    if (warp < 8) {
        // ------------------------------------------------------- softmax
        reg_inc<184>();                           // 8 x 184 + 8 x 72 = 16 x 128 registers a lane; fewer spill
        const int w = warp >> 2, q = warp & 3;
        const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
        const uint32_t s_addr = lane_base + L::S_COL + w * kN, o_addr = lane_base + L::O_COL + w * D;
        const int r = q * 32 + lane;              // row of the tile
        // The thread's row of an item's q as two E4M3 parts in shared memory, in the swizzled order of the
        // K-major operand; returns the factor of its scores. The row tile's last S before has completed.
        auto put_q = [&](const Item& x) {
            if (x.nk[w] == 0) return 0.0f;
            const int row = x.row0 + w * kM + r, i = row / G;
            const uint16_t* src = P.a.q + (int64_t)(x.q0 + i) * P.a.ldq + (int64_t)(x.h * G + row - i * G) * D;
            uint4 raw[D / 8];
            float m = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 8; c++)
                raw[c] = i < x.n ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
                const uint32_t y[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                for (int e = 0; e < 4; e++)
                    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(y[e] << 16)), fabsf(__uint_as_float(y[e] & 0xFFFF0000u))));
            }
            float up, down;
            row_scale(m, up, down);
            const float factor = fabsf(P.a.sm_scale) * kLog2e * down;
            if (P.a.sm_scale < 0.0f) up = -up;
            uint8_t* hi = smem + L::Q_OFF + (w * 2) * L::Q + r * D;
#pragma unroll
            for (int c = 0; c < D / 16; c++) {    // 16 channels
                uint32_t hw[4], lw[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint4 y = raw[2 * c + (e >> 1)];
                    const uint32_t y0 = e & 1 ? y.z : y.x, y1 = e & 1 ? y.w : y.y;
                    split4(__uint_as_float(y0 << 16) * up, __uint_as_float(y0 & 0xFFFF0000u) * up,
                           __uint_as_float(y1 << 16) * up, __uint_as_float(y1 & 0xFFFF0000u) * up, hw[e], lw[e]);
                }
                const int ch = D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
                *reinterpret_cast<uint4*>(hi + ch * 16) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                *reinterpret_cast<uint4*>(hi + L::Q + ch * 16) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(QF + w));
            return factor;
        };
        bool more = has_item(0);
        float next_crow = more ? put_q(items[0]) : 0.0f;
        uint32_t od = 0;                          // phase of the row tile's O
        int tw = 0;                               // key tiles that this row tile has taken, over all items
        int tc = 0;                               // key tiles of the CTA before this item
        bool ok = true;
        for (int k = 0; more; k++) {
            const Item& it = items[k & 1];
            const int nk = it.nk[w];
            const int i = (it.row0 + w * kM + r) / G;
            const bool there = i < it.n;
            const float crow = next_crow;
            // keys that the row sees, counted from the item's first key tile
            const int seen = (!there ? 0 : P.a.causal ? min(max(it.L - it.n + i + 1, 0), it.L) : it.L) - it.t0 * kN;
            // the fewest that a row of this warp sees (rows past the end see none, and are not stored)
            int least = there ? seen : 0x7fffffff;
            for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
            float m = -INFINITY, l = 0.0f;
            for (int t = 0; t < nk; t++, tw++) {
                const int ts = tc + t;
                // A row tile without keys in an item skips the phases of that item's scales, so the wait of its next tile could
                // come two uses of a slot early, where the parity is the same. An item's first tile waits for its S
                // before: K was copied after the scales of the slot's last use were stored. From then on the S of the tile
                // before says so, and the scales come first. (Two waits on chosen barriers: a third one in line here
                // cost the 8192-token prompt 2 %.)
                const uint32_t b_sc = bar(SC + ts % kScStages), p_sc = (ts / kScStages) & 1, b_s = bar(SF + w), p_s = tw & 1;
                if (!warp_wait(t ? b_sc : b_s, t ? p_sc : p_s) || !warp_wait(t ? b_s : b_sc, t ? p_s : p_sc)) { ok = false; break; }
                tc_fence_after();
                const float4* con = sc + (ts % kScStages) * 8;        // (k scale, log2 v scale, 1 / v scale, +-kTiny) per 16 keys
                const int lim = seen - t * kN;
                const bool edge = least < (t + 1) * kN;                   // some row of the warp does not see the whole tile
                if (edge) {                       // infinite, against the scale's sign, where a row does not see a key: p 0
#pragma unroll 1
                    for (int c = 0; c < kN; c += 16) {
                        uint32_t x[16];
                        tmem_ld16(s_addr + c, x);
                        const uint32_t out = 0xFF800000u ^ (__float_as_uint(con[c >> 4].w) & 0x80000000u);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e++)
                            if (e >= lim - c) x[e] = out;
                        tmem_st16(s_addr + c, x);
                    }
                    tmem_wait_st();
                }
                // One pass without a maximum, 64 keys at a time: p under the m so far. Only where a sum shows that p
                // may have grown past f16's range (or no m is known yet) is the maximum of what is left of S taken,
                // m raised, what stands under the old m scaled and the pass made again. P of 64 keys stays in
                // registers until their S is read and found in range, since it takes the columns of S's keys before.
                // Rolled, and pieces of 16 columns off the common path: the code has to stay in the instruction cache beside
                // the other roles' (all 128 keys in one pass: 8192-token prompt 422 us instead of 433, but 16 prompts
                // of up to 448 tokens by 1500 keys 45.8 instead of 42.6 and a step of chunks and single tokens 135
                // instead of 130). Sixteen softmax warps, two threads a row, need registers that are not
                // there: 640 us.
#pragma unroll 1
                for (int half = 0; half < 2; half++) {
                    uint32_t pk[32];
                    float sum;
                    bool raise = half == 0 && m == -INFINITY && lim > 0;
                    int raised = 0;
                    while (true) {
                        if (__any_sync(0xffffffffu, raise)) {
                            raised++;
                            tmem_wait_st();       // P of keys 0-63 and a scaled O may still be on their way, and are read below
                            float mx = -INFINITY;
#pragma unroll 1
                            for (int c = 4 * half; c < 8; c++) {
                                uint32_t x[16];
                                tmem_ld16(s_addr + c * 16, x);
                                const float4 cn = con[c];
                                tmem_wait_ld();
                                const float ca = fmaf(crow, cn.x, cn.w);
#pragma unroll
                                for (int e = 0; e < 16; e++) mx = fmaxf(mx, fmaf(__uint_as_float(x[e]), ca, cn.y));
                            }
                            // by a whole number of doublings: the P that is stored scales exactly
                            const float up = !raise || !(mx > m) ? 0.0f : m == -INFINITY ? INFINITY : ceilf(mx - m);
                            const float f = m == -INFINITY ? 0.0f : ex2(-up);
                            if (up > 0.0f) m = m == -INFINITY ? mx : m + up;
                            l *= f;
                            if (half) {           // P of keys 0-63
                                const __half2 f2 = __float2half2_rn(f);
#pragma unroll 1
                                for (int c = 0; c < 32; c += 16) {
                                    uint32_t x[16];
                                    tmem_ld16(s_addr + c, x);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; e++) {
                                        const __half2 y = __hmul2(*reinterpret_cast<__half2*>(&x[e]), f2);
                                        x[e] = *reinterpret_cast<const uint32_t*>(&y);
                                    }
                                    tmem_st16(s_addr + c, x);
                                }
                            }
                            if (t > 0) {          // O so far
#pragma unroll 1
                                for (int c = 0; c < D; c += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(o_addr + c, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st16(o_addr + c, o);
                                }
                            }
                        }
                        const float off = m == -INFINITY ? 0.0f : kPShift - m;
                        float top = 0.0f;
                        uint32_t s[2][32];
                        sum = 0.0f;
                        tmem_ld32(s_addr + half * 64, s[0]);
#pragma unroll
                        for (int cc = 0; cc < 2; cc++) {
                            tmem_wait_ld();
                            if (cc == 0) tmem_ld32(s_addr + half * 64 + 32, s[1]);      // in flight during this chunk
#pragma unroll
                            for (int gr = 0; gr < 2; gr++) {
                                const float4 cn = con[half * 4 + cc * 2 + gr];
                                const uint32_t* y = s[cc] + gr * 16;
                                const float ca = fmaf(crow, cn.x, cn.w), cb = cn.y + off;
                                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    float p0, p1;
                                    fma2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]), ca, cb, p0, p1);
                                    p0 = ex2(p0);
                                    p1 = ex2(p1);
                                    add2(s0, s1, p0, p1);
                                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[cc * 16 + gr * 8 + e / 2]) : "f"(p1), "f"(p0));
                                }
                                const float both = s0 + s1;
                                top = fmaxf(top, both);
                                sum = fmaf(both, cn.z, sum);
                            }
                        }
                        // Under a maximum taken here a p is at most 2^8. (Scores so large that their rounding alone
                        // exceeds that would come back for ever: m is raised twice for a half at most, once for rows without
                        // an m, which rows of NaN are in every tile, and once for what has outgrown it.)
                        raise = top > kMost && there;
                        if (raised == 2 || !__any_sync(0xffffffffu, raise)) break;
                    }
                    l += sum;
                    tmem_st32(s_addr + half * 32, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PF + w));
            }
            if (!ok) break;
            // ---- the next item's q first: its S runs while this item's output leaves
            tc += max(it.nk[0], it.nk[1]);
            more = has_item(k + 1);
            if (more) next_crow = put_q(items[(k + 1) & 1]);
            if (nk > 0 && !warp_wait(bar(OD + w), od)) break;
            od ^= nk > 0;
            const int a = it.row0 + w * kM + r - i * G;
            tc_fence_after();
            if (it.part >= 0) {                  // a part of the keys: the state as it is
                float* dst = P.part + (int64_t)it.part * L::PART;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    if (nk > 0) {
                        tmem_ld16(o_addr + c, o);
                        tmem_wait_ld();
                    }
                    float4* d4 = reinterpret_cast<float4*>(dst + (w * kM + r) * D + c);
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        d4[e] = nk > 0 ? make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]))
                                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                dst[kRows * D + w * kM + r] = m;
                dst[kRows * D + kRows + w * kM + r] = l;
            } else {
                const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
                uint16_t* out = P.a.out + (int64_t)(it.q0 + i) * P.a.ldo + (int64_t)(it.h * G + a) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    uint32_t o[16];
                    if (nk > 0) {
                        tmem_ld16(o_addr + c, o);
                        tmem_wait_ld();
                    }
                    const bool empty = nk == 0 || l == 0.0f;          // a row that saw nothing
                    if (there) {
#pragma unroll
                        for (int e = 0; e < 16; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[e + 2 * j]) * inv,
                                                                               __uint_as_float(o[e + 2 * j + 1]) * inv);
                                y[j] = empty ? 0u : *reinterpret_cast<const uint32_t*>(&v);
                            }
                            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if (there && P.a.lse)
                    P.a.lse[(int64_t)(it.q0 + i) * P.a.heads_q + it.h * G + a] =
                        l > 0.0f ? (m - kPShift + __log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
            }
            tc_fence_before();
            done_item(k);
        }
    } else if (warp < 12) {
        // ------------------------------------------------- V codes to f16
        reg_dec<72>();
        const int tid = threadIdx.x - 256;
        constexpr int CH = D / 16, STEP = 128 / CH;                   // 16-code chunks of a row; rows per step
        // rows STEP apart keep the swizzle (a multiple of 8), so a step only adds to the addresses
        const int r0 = tid / CH, c = tid % CH, sw = r0 & 7, odd = c >> 2, c0 = (c & 3) * 2;
        const uint8_t* src0 = smem + L::V_OFF + r0 * D + c * 16;
        uint8_t* dst0 = smem + L::VH_OFF + odd * (kN * 128) + r0 * 128;
        const int o1 = ((c0 + odd) ^ sw) << 4, o2 = ((c0 + 1 - odd) ^ sw) << 4;     // the second block's halves swapped: other banks
        bool ok = true;
        int kt = 0;                               // key tiles of the CTA so far
        for (int k = 0; ok && has_item(k); k++) {
            const Item& it = items[k & 1];
            const int nkv = max(it.nk[0], it.nk[1]);
            for (int t = 0; t < nkv; t++, kt++) {
                const int st = kt & 1;
                if (!warp_wait(bar(VF + st), (kt >> 1) & 1)) { ok = false; break; }
                if (!warp_wait(bar(HE + st), ((kt >> 1) & 1) ^ 1)) { ok = false; break; }
                const uint8_t* src = src0 + st * L::KT;
                uint8_t* dst = dst0 + st * L::VH;
                const int live = it.L - (it.t0 + t) * kN;             // rows behind the last key were never written: zeros
                // rolled: in bursts, this traffic holds up the S products, which alone read 128 bytes of
                // shared memory a cycle (at an earlier step, 4864 rows a head by 4096 keys: unrolled 8 times
                // 365 us, twice 309, rolled 292; 251 now)
#pragma unroll 1
                for (int j = 0; j < CH; j++) {
                    uint4 x = *reinterpret_cast<const uint4*>(src + j * STEP * D);
                    if (r0 + j * STEP >= live) x = make_uint4(0, 0, 0, 0);
                    const uint32_t in[4] = {x.x, x.y, x.z, x.w};
                    uint32_t y[8];
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        asm("{ .reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi; }"
                            : "=r"(y[2 * e]), "=r"(y[2 * e + 1]) : "r"(in[e]));
                    const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
                    *reinterpret_cast<uint4*>(dst + j * STEP * 128 + o1) = odd ? hi : lo;
                    *reinterpret_cast<uint4*>(dst + j * STEP * 128 + o2) = odd ? lo : hi;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(HF + st));
                    mbar_arrive(bar(VE + st));
                }
            }
            done_item(k);
        }
    } else {
        reg_dec<72>();
        if (warp == 12) {
            // ------------------------------------------------- TMA, scales
            bool ok = true;
            int kt = 0, ks = 0;
            uint32_t kph = 1;          // K stage and the parity its release is waited for with
            for (int k = 0; ok && has_item(k); k++) {
                const Item& it = items[k & 1];
                const int nkv = max(it.nk[0], it.nk[1]), h = it.h;
                const int32_t* tab = P.a.block_table + (int64_t)it.b * P.a.ld_table;
                const int page_end = (it.L + (1 << P.shift) - 1) >> P.shift;
                auto page_at = [&](int t) {       // lane's page of tile t, num_pages (out of bounds: reads as zeros) if none
                    const int j = (it.t0 + t) * pages_tile + lane;
                    int p = -1;
                    if (lane < pages_tile && j < page_end) p = __ldg(tab + j);
                    return p >= 0 && p < P.a.kv.num_pages ? p : P.a.kv.num_pages;
                };
                auto scales_of = [&](int p) {
                    float4 cn = make_float4(0.0f, -INFINITY, 0.0f, kTiny);
                    if (lane < pages_tile && p < P.a.kv.num_pages) {
                        const int64_t i = (int64_t)p * P.a.kv.heads + h;
                        cn.x = __ldg(P.a.kv.k_scale + i);
                        cn.z = __ldg(P.a.kv.v_scale + i);
                    }
                    return cn;
                };
                // pages two tiles ahead of their copies, scales one
                int p = nkv > 0 ? page_at(0) : 0, p1 = nkv > 1 ? page_at(1) : 0;
                float4 cn = scales_of(nkv > 0 ? p : P.a.kv.num_pages);
                for (int t = 0; t < nkv; t++, kt++) {
                    const int vs = kt & 1;
                    const int p2 = t + 2 < nkv ? page_at(t + 2) : 0;
                    const float4 cn1 = scales_of(t + 1 < nkv ? p1 : P.a.kv.num_pages);
                    ok = warp_wait(bar(KE + ks), kph);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(KF + ks), L::KT);
                    __syncwarp();
                    if (lane < pages_tile)
                        tma_load_3d(sbase + L::K_OFF + ks * L::KT + (lane << P.shift) * D, &P.tm_k, 0, h << P.shift, p, bar(KF + ks));
                    // scales per 16 keys (a page covers page_size / 16 of them)
                    const int reps = 1 << (P.shift - 4);
                    const int pv = cn.z <= kLeastScale ? P.a.kv.num_pages : p;       // no values: zeros
                    if (p < P.a.kv.num_pages) {
                        const float v = value_scale(cn.z);
                        cn.y = fmaf(cn.x, 0.0f, __log2f(v));        // (NaN under an infinite key scale)
                        cn.z = __frcp_rn(v);
                        cn.w = copysignf(kTiny, cn.x);
                    }
                    if (lane < pages_tile)
                        for (int j = 0; j < reps; j++) sc[(kt % kScStages) * 8 + lane * reps + j] = cn;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(SC + kt % kScStages));
                    if (++ks == kKStages) { ks = 0; kph ^= 1; }
                    ok = warp_wait(bar(VE + vs), ((kt >> 1) & 1) ^ 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar(VF + vs), L::KT);
                    __syncwarp();
                    if (lane < pages_tile)
                        tma_load_3d(sbase + L::V_OFF + vs * L::KT + (lane << P.shift) * D, &P.tm_v, 0, h << P.shift, pv, bar(VF + vs));
                    p = p1;
                    p1 = p2;
                    cn = cn1;
                }
                done_item(k);
            }
            // no copy outlives the CTA (at once unless a wait gave up: the roles have read every tile)
            if (!ok) {
                for (int j = max(0, kt - kKStages); j <= kt; j++) warp_wait(bar(KF + j % kKStages), (j / kKStages) & 1);
                for (int j = max(0, kt - kVStages); j < kt; j++) warp_wait(bar(VF + (j & 1)), (j >> 1) & 1);
            }
        } else if (warp == 13) {
            // ------------------------------------------------------ items
            // Requests in classes of similar length (two for each power of two of key tiles), the longest first,
            // and a request's last row tiles first: what begins last is short.
            auto request = [&](int b, int& start, int& n, int& cls) {               // its row tiles
                if (b >= P.a.B) return 0;
                start = __ldg(P.a.cu_q + b);
                n = min(__ldg(P.a.cu_q + b + 1) - start, P.a.max_q);
                const int64_t rows = (int64_t)max(n, 0) * G;
                const int kt = max((__ldg(P.a.kv_lens + b) + kN - 1) / kN, 1), lg = 31 - __clz(kt);
                cls = 31 - min(2 * lg + (lg > 0 ? kt >> (lg - 1) & 1 : 0), 31);
                return rows < P.min_rows ? 0 : (int)((rows + kRows - 1) / kRows);
            };
            classes[lane] = 0;
            __syncwarp();
            for (int b = lane; b < P.a.B; b += 32) {
                int start, n, cls;
                const int own = request(b, start, n, cls);
                if (own) atomicAdd(classes + cls, own);               // whole numbers: any order
            }
            __syncwarp();
            int upto = classes[lane];             // row tiles of the classes up to this lane's
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += u;
            }
            int id = blockIdx.x, asked = 0;
            for (int k = 0; ; ) {
                Item it;
                it.b = -1;
                if (id >= 0) {
                    it.h = id % P.a.kv.heads;
                    const int rest = id / P.a.kv.heads, split = rest % P.splits, want = rest / P.splits;
                    const uint32_t past = __ballot_sync(0xffffffffu, upto > want);
                    if (past) {
                        const int cls = __ffs(past) - 1;
                        int before = cls ? __shfl_sync(0xffffffffu, upto, cls - 1) : 0;
                        for (int b0 = 0; b0 < P.a.B; b0 += 32) {
                            int start = 0, n = 0, c = -1;
                            int own = request(b0 + lane, start, n, c);
                            if (c != cls) own = 0;
                            int v = own;
                            for (int o = 1; o < 32; o <<= 1) {
                                const int u = __shfl_up_sync(0xffffffffu, v, o);
                                if (lane >= o) v += u;
                            }
                            const int first = before + v - own;
                            const uint32_t hit = __ballot_sync(0xffffffffu, want >= first && want < first + own);
                            if (hit) {
                                const int l0 = __ffs(hit) - 1;
                                it.b = b0 + l0;
                                it.row0 = (__shfl_sync(0xffffffffu, own, l0) - 1 - (want - __shfl_sync(0xffffffffu, first, l0))) * kRows;
                                it.q0 = __shfl_sync(0xffffffffu, start, l0);
                                it.n = __shfl_sync(0xffffffffu, n, l0);
                                break;
                            }
                            before += __shfl_sync(0xffffffffu, v, 31);
                        }
                    }
                    if (P.splits > 1 && split == 0 && lane == 0) {
                        P.head[(want * P.a.kv.heads + it.h) * 2] = it.b;
                        P.head[(want * P.a.kv.heads + it.h) * 2 + 1] = it.row0;
                    }
                    if (it.b >= 0) {
                        it.n = it.q0 < 0 ? 0 : (int)min((int64_t)it.n, P.a.tokens - it.q0);
                        it.L = (int)min((int64_t)max(__ldg(P.a.kv_lens + it.b), 0), (int64_t)P.a.max_blocks << P.shift);
                        // key tiles of each row tile: up to what its last row sees, cut to this part
                        int full[2];
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            const int first = it.row0 + w * kM, last = min(first + kM, it.n * G) - 1;
                            const int sees = last < first ? 0 : P.a.causal ? min(max(it.L - it.n + last / G + 1, 0), it.L) : it.L;
                            full[w] = (sees + kN - 1) / kN;
                        }
                        const int all = max(full[0], full[1]);
                        it.t0 = (int)((int64_t)all * split / P.splits);
                        const int t1 = (int)((int64_t)all * (split + 1) / P.splits);
#pragma unroll
                        for (int w = 0; w < 2; w++) it.nk[w] = max(min(full[w], t1) - it.t0, 0);
                        it.part = P.splits > 1 ? (want * P.a.kv.heads + it.h) * P.splits + split : -1;
                    }
                }
                if (it.b >= 0 || id < 0) {
                    if (lane == 0) {
                        items[k & 1] = it;
                        mbar_arrive(bar(IF + (k & 1)));
                    }
                    if (id < 0) break;
                    k++;                          // its place is free once every role has left the item before last
                    if (!warp_wait(bar(IE + (k & 1)), ((k >> 1) & 1) ^ 1)) break;
                }
                if (lane == 0) {
                    fence_proxy_async_smem();     // the last answer has been read
                    mbar_arrive_expect_tx(bar(CB), 16);
                    try_cancel(smem_u32(canceled), bar(CB));
                }
                __syncwarp();
                if (!warp_wait(bar(CB), asked & 1)) break;
                asked++;
                id = canceled_cta(smem_u32(canceled));
            }
        } else if (warp == 14) {
            // -------------------------------------------------------- MMA
            const uint32_t s0 = tmem + L::S_COL, o0 = tmem + L::O_COL;
            const uint32_t q_lo = sdesc_k_lo<D>(sbase + L::Q_OFF), k_lo = sdesc_k_lo<D>(sbase + L::K_OFF),
                           v_lo = sdesc_v_lo(sbase + L::VH_OFF);
            bool ok = true;
            int kt = 0, ks = 0;                   // key tiles; K stage
            uint32_t kph = 0, qph0 = 0, qph1 = 0, pph0 = 0, pph1 = 0;
            for (int k = 0; ok && has_item(k); k++) {
                const int nk0 = items[k & 1].nk[0], nk1 = items[k & 1].nk[1], nkv = max(nk0, nk1);
                if (nkv > 0) {                    // the whole warp; one lane's MMAs and commits
                    // A wait that gives up leaves the warp together and the MMAs to run on what is there, until
                    // the tile's vote: the election needs every lane.
                    auto wait = [&](int i, uint32_t parity) { ok = ok && warp_wait(bar(i), parity); };
                    auto score = [&](const int w, uint32_t ka) {      // S of row tile w, both parts of q
                        const uint32_t sd = s0 + w * kN, qa = q_lo + w * (2 * L::Q >> 4);
#pragma unroll
                        for (int j = 0; j < D / 32; j++) mma_s(sd, qa + j * 2, ka + j * 2, sdesc_k_hi<D>(), L::IDESC_S, j > 0);
#pragma unroll
                        for (int j = 0; j < D / 32; j++) mma_s(sd, qa + (L::Q >> 4) + j * 2, ka + j * 2, sdesc_k_hi<D>(), L::IDESC_S, true);
                        commit_elect(bar(SF + w));
                    };
                    auto value = [&](const int w, uint32_t va, bool acc) {          // O += P V
                        const uint32_t sd = s0 + w * kN, od = o0 + w * D;
                        mma_o(od, sd, va, L::IDESC_O, acc);
#pragma unroll
                        for (int j = 1; j < kN / 16; j++) mma_o(od, sd + j * 8, va + j * (2048 >> 4), L::IDESC_O, true);
                    };
                    wait(KF + ks, kph);
                    if (nk0 > 0) {
                        wait(QF, qph0);
                        qph0 ^= 1;
                        tc_fence_after();
                        score(0, k_lo + ks * (L::KT >> 4));
                    }
                    if (nk1 > 0) {
                        wait(QF + 1, qph1);
                        qph1 ^= 1;
                        tc_fence_after();
                        score(1, k_lo + ks * (L::KT >> 4));
                    }
                    commit_elect(bar(KE + ks));
                    ok = __all_sync(0xffffffffu, ok);
                    for (int t = 0; t < nkv && ok; t++, kt++) {
                        if (++ks == kKStages) { ks = 0; kph ^= 1; }
                        wait(HF + (kt & 1), (kt >> 1) & 1);
                        if (t + 1 < nkv) wait(KF + ks, kph);
                        const uint32_t ka = k_lo + ks * (L::KT >> 4), va = v_lo + (kt & 1) * (L::VH >> 4);
                        if (t < nk0) {
                            wait(PF, pph0);
                            pph0 ^= 1;
                            tc_fence_after();
                            value(0, va, t > 0);
                            if (t + 1 < nk0) score(0, ka);
                            else commit_elect(bar(OD));
                        }
                        if (t < nk1) {
                            wait(PF + 1, pph1);
                            pph1 ^= 1;
                            tc_fence_after();
                            value(1, va, t > 0);
                            if (t + 1 < nk1) score(1, ka);
                            else commit_elect(bar(OD + 1));
                        }
                        commit_elect(bar(HE + (kt & 1)));
                        if (t + 1 < nkv) commit_elect(bar(KE + ks));
                        ok = __all_sync(0xffffffffu, ok);
                    }
                }
                done_item(k);
            }
            commit_elect(bar(DR));                // no MMA outlives the CTA's tensor memory
            warp_wait(bar(DR), 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the states of an item's key parts in order: 8 rows of one item per CTA.
template <int D>
__global__ void __launch_bounds__(2 * D)
attn_prefill_join_kernel(const __grid_constant__ PrefillParams P) {
    using L = PrefillLayout<D>;
    pdl_trigger();
    pdl_wait();
    const int idx = blockIdx.y, b = P.head[idx * 2];
    if (b < 0) return;
    const int G = P.a.heads_q / P.a.kv.heads, h = idx % P.a.kv.heads;
    const int r = blockIdx.x * 8 + threadIdx.x / (D / 4), d0 = threadIdx.x % (D / 4) * 4;
    const int q0 = __ldg(P.a.cu_q + b);
    int n = min(__ldg(P.a.cu_q + b + 1) - q0, P.a.max_q);
    n = q0 < 0 ? 0 : (int)min((int64_t)n, P.a.tokens - q0);
    const int row = P.head[idx * 2 + 1] + r, i = row / G, a = row - i * G;
    if (i >= n) return;
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < P.splits; s++) {
        const float* src = P.part + ((int64_t)idx * P.splits + s) * L::PART;
        const float m2 = src[kRows * D + r], l2 = src[kRows * D + kRows + r], mm = fmaxf(m, m2);
        const float4 x = *reinterpret_cast<const float4*>(src + r * D + d0);
        const float f = m == -INFINITY ? (l == l ? 0.0f : l) : ex2(m - mm);
        const float f2 = m2 == -INFINITY ? (l2 == l2 ? 0.0f : l2) : ex2(m2 - mm);
        l = l * f + l2 * f2;
        o.x = o.x * f + x.x * f2;
        o.y = o.y * f + x.y * f2;
        o.z = o.z * f + x.z * f2;
        o.w = o.w * f + x.w * f2;
        m = mm;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(o.x * inv, o.y * inv), y1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(P.a.out + (int64_t)(q0 + i) * P.a.ldo + (int64_t)(h * G + a) * D + d0) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    if (P.a.lse && d0 == 0)
        P.a.lse[(int64_t)(q0 + i) * P.a.heads_q + h * G + a] =
            l > 0.0f ? (m - kPShift + __log2f(l)) * kLn2 : (l == l ? -INFINITY : l);
}

template <int D>
qz_status launch_prefill(PrefillParams& P, int64_t ctas, void* ws, cudaStream_t st) {
    using L = PrefillLayout<D>;
    const int items = P.tiles * P.a.kv.heads;
    P.head = reinterpret_cast<int*>(ws);
    P.part = reinterpret_cast<float*>(static_cast<char*>(ws) + ((size_t)items * 8 + 255) / 256 * 256);
    QZ_TRY(opt_in_smem((const void*)attn_prefill_kernel<D>, L::SMEM));
    QZ_TRY(launch_pdl(attn_prefill_kernel<D>, dim3((unsigned)ctas), dim3(kThreads), L::SMEM, st, P));
    if (P.splits == 1) return QZ_OK;
    return launch_pdl(attn_prefill_join_kernel<D>, dim3(kRows / 8, items), dim3(2 * D), 0, st, P);
}

} // namespace

// States of a launch that splits its items: at most one part per SM.
size_t ws_attn_prefill() {
    return (size_t)num_sms() * (PrefillLayout<128>::PART * 4 + 8) + 256;
}

// Requests of at least min_rows rows per KV head; the others are left alone.
qz_status attn_prefill_launch(const AttnArgs& a, int min_rows, void* ws, bool* joined, cudaStream_t st) {
    PrefillParams P;
    P.a = a;
    P.shift = a.kv.page_size == 16 ? 4 : a.kv.page_size == 32 ? 5 : a.kv.page_size == 64 ? 6 : 7;
    P.min_rows = min_rows;
    const uint64_t D = (uint64_t)a.kv.head_dim, rows = (uint64_t)a.kv.heads * a.kv.page_size;
    const uint32_t box = (uint32_t)a.kv.page_size;
    if (!encode_tmap_3d_u8(&P.tm_k, a.kv.k_codes, D, rows, (uint64_t)a.kv.num_pages, D, (uint64_t)a.kv.page_stride,
                           (uint32_t)D, box, (int)D) ||
        !encode_tmap_3d_u8(&P.tm_v, a.kv.v_codes, D, rows, (uint64_t)a.kv.num_pages, D, (uint64_t)a.kv.page_stride,
                           (uint32_t)D, box, 0))
        return QZ_ERR_CUDA;
    // row tiles of the requests: at most one partly filled each, and a request taken has min_rows rows
    const int64_t all = a.tokens * (a.heads_q / a.kv.heads);
    const int64_t tiles = all / kRows + std::min<int64_t>(a.B, all / min_rows + 1);
    // Parts of the keys: as many as fill the SMs where the row tiles fill less than half of them, each of
    // kSplitKeys keys or more (by the table's width; the lengths are on the device).
    const int64_t keys = (int64_t)a.max_blocks * a.kv.page_size;
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(num_sms() / (tiles * a.kv.heads), keys / kSplitKeys));
    if (tiles * a.kv.heads * splits > 0x7fffffff) return QZ_ERR_SHAPE;
    P.tiles = (int)tiles;
    P.splits = (int)splits;
    *joined = splits > 1;                         // a second launch follows
    const int64_t ctas = tiles * a.kv.heads * splits;
    return a.kv.head_dim == 64 ? launch_prefill<64>(P, ctas, ws, st) : launch_prefill<128>(P, ctas, ws, st);
}

qz_status attn_prefill_error_read_and_clear() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_prefill_err, sizeof(v)) != cudaSuccess) return QZ_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_attn_prefill_err, &z, sizeof(z)) != cudaSuccess) return QZ_ERR_CUDA;
    return v ? QZ_ERR_TIMEOUT : QZ_OK;
}

} // namespace qz
