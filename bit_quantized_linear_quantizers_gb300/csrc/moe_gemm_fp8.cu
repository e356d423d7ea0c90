// moe_gemm_fp8.cu -- the experts' products over ragged rows, block-scaled FP8 on tcgen05:
//   P[r, n] = sum_kb sA[a, kb] sW[e, n/128, kb] sum_{k in kb} qA[a, k] qW[e, n, k]
// with a = row_token[r] and e the expert whose rows contain r; output in bf16, or SwiGLU of
// the gate and up columns encoded as E4M3 with a scale per 128 columns.
//
// A work item is 128 rows of one expert by 256 columns (two boxes of 128 weight rows; with
// SwiGLU one of the gate and the same one of the up projection, so that h is made where P
// is). The number of items is known on the GPU alone: a warp reads the offsets and hands the
// items out through a ring in shared memory, an expert's row tiles before its next columns,
// so that the CTAs of one moment share weights and rows in L2.
//
// CTA of 16 warps, one per SM:
//  warp 0      weights: TMA boxes of 128 x 128 bytes into a 4-stage ring
//  warp 1      MMA: per block of 128 of K four tcgen05.mma (M 128, N 256, K 32) into one of two
//              accumulators of 256 columns in tensor memory
//  warp 2      items (warp 3 completes the warpgroup)
//  warps 4-7   rows: gathered by their tokens in copies of 16 bytes (cp.async), as TMA boxes of 32 rows where
//              they lie in order. The copies arrive on the stage's barrier by themselves, and the
//              MMA's warp orders them before its own reads. (Gathered by TMA, four rows a copy, a block of
//              128 rows took 2400 cycles; by one warp's copies 1900.)
//  warps 8-15  promotion: block scales are fp32, so every block's partial sums leave tensor
//              memory to be added as acc += P_kb * (sA sW). A thread holds one row of 64 columns of
//              each of the two boxes.
// With many rows neither the tensor pipe, L2 nor shared memory is at its limit. The cycle of an accumulator (MMA 512 cycles,
// hand-off, promotion, hand-off, about 1200), two blocks of K by turns, gives 660 cycles a block, which this loop takes with
// operands that lie there already; with rows, scales and items on their way it takes 860 (960 with SwiGLU), and where those
// 200 to 300 go is not known. What lies between is kept short: scales are read by the promoting threads
// themselves, groups of four blocks ahead (staged in shared memory they came 300 cycles late), and waits are few.
// With few rows the bound is the weights' way from memory, and the promotion and the gather of rows that
// are not there are left out. Where items are fewer than SMs (rows <= 32), a cluster shares an item's K.
#include "qz_moe.cuh"
#include "qz_tc.cuh"

#include <algorithm>
#include <cstring>

namespace qz {

namespace {

__device__ unsigned int g_moe_err;

constexpr int BM = 128, BN = 256, BK = 128, STAGES = 4;
constexpr int A_BYTES = BM * BK, HALF_BYTES = 128 * BK;
constexpr int STAGE_BYTES = A_BYTES + 2 * HALF_BYTES;
constexpr int FEED_WARPS = 8, EPI_WARPS = 8, THREADS = (FEED_WARPS + EPI_WARPS) * 32;
constexpr int REGS_FEED = 72, REGS_EPI = 184;     // 256 * 72 + 256 * 184 = 512 * 128, what the CTA is launched with
constexpr int INFO = 4;                           // items in flight
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr int STG_WARP = 32 * 128;                // a warp's output: 32 rows of 64 bf16
constexpr int STG_OFF = STAGES * STAGE_BYTES;
constexpr int INFO_OFF = STG_OFF + EPI_WARPS * STG_WARP;
constexpr int BAR_OFF = INFO_OFF + INFO * 16;
constexpr int BARS = 2 * STAGES + 2 + 2 * INFO + 4;
constexpr int SMEM_BYTES = BAR_OFF + BARS * 8 + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory of a CTA");
constexpr int SPLIT_ROWS = 32, MAX_SPLITS = 4;    // rows of a shared item: one warp's lanes
constexpr int PART_BYTES = SPLIT_ROWS * BN * 4;
static_assert((MAX_SPLITS - 1) * PART_BYTES <= STAGES * STAGE_BYTES, "the others' sums fit in the ring");

template <int REGS> __device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS)); }
template <int REGS> __device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS)); }

// A thread's sums: 64 columns of the first box, 64 of the second. add: += v * s for 32 of them from AT on; volatile, so
// that it stays behind the wait for the reads of v. Paired instructions take half the issue slots: lane by lane it was 396
// instead of 374 us for 4001 tokens by 2 of 8 experts [4096, 14336], 318 instead of 308 for 65536 rows with SwiGLU. (The
// pairs stay in place for a whole item: formed anew from floats for every block, they cost more than they save.)
struct Sums {
    uint64_t a[64];
    struct Values {
        float v[128];
        __device__ __forceinline__ float& operator[](int i) { return v[i]; }
    };
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 64; i++) a[i] = 0;
    }
    template <int AT> __device__ __forceinline__ void add(const uint32_t (&v)[32], float s) {
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
#pragma unroll
        for (int i = 0; i < 16; i++)
            asm volatile("{ .reg .b64 x; mov.b64 x, {%1, %2}; fma.rn.f32x2 %0, x, %3, %0; }"
                         : "+l"(a[AT / 2 + i]) : "r"(v[2 * i]), "r"(v[2 * i + 1]), "l"(s2));
    }
    __device__ __forceinline__ Values values() const {
        Values o;
#pragma unroll
        for (int i = 0; i < 64; i++) asm("mov.b64 {%0, %1}, %2;" : "=f"(o.v[2 * i]), "=f"(o.v[2 * i + 1]) : "l"(a[i]));
        return o;
    }
};

// g / (1 + exp(-g)) by 2^x and 1/x of the special-function unit in their forms without subnormals. The exponent t is rounded, up
// to 44 half units of the result at g = -87: what it lost, c, is added to first order (its square is below 2^-37), so that
// the error is the same for gates of any size, 10 half units (without it up to 64; the scales of the codes are fp32).
// 65536 rows: 316 us, 308 without it, 356 with expf. The limits keep c finite where 2^t is 0 or past the reciprocal's
// range: exp(-g) is 0 from g = 88 on, where 1 + exp(-g) is 1 long since, and the reciprocal is 0 above 2^126, where g's
// share is nothing.
__device__ __forceinline__ float silu(float g) {
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Rest = -1.9046543e-9f;
    const float x = fminf(fmaxf(-g, -128.0f), 88.0f), t = x * kLog2e;
    const float c = fmaf(t, -kLn2Rest, fmaf(t, -kLn2, x));     // x - t ln 2
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + fmaf(e, c, e)));
    return g * r;
}

// One block of K: D = A B^T of 128 x 128-byte and 256 x 128-byte tiles behind one another at `stage`, K = 32 bytes an
// MMA, then arrivals on two barriers. The warp issues it converged, through an elected lane: operands of a branch of
// one lane are moved to the uniform registers anew for every instruction (490 cycles a block so).
__device__ __forceinline__ void mma_block(uint32_t d, uint32_t stage, uint32_t idesc, uint32_t bar0, uint32_t bar1) {
    const uint64_t ad = sdesc_k_sw128(stage), bd = sdesc_k_sw128(stage + A_BYTES);
    asm volatile("{ .reg .pred q, f, t; .reg .b64 a, b;\n\t"
                 "elect.sync _|q, 0xffffffff; setp.eq.u32 t, 0, 0; setp.eq.u32 f, 0, 1;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, f;\n\t"
                 "add.s64 a, %1, 2; add.s64 b, %2, 2;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
                 "add.s64 a, %1, 4; add.s64 b, %2, 4;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
                 "add.s64 a, %1, 6; add.s64 b, %2, 6;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5]; }"
                 ::"r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(bar0), "r"(bar1) : "memory");
}

// The bounded wait of this kernel. 15 warps wait at a time, and each poll takes the shared-memory pipe that the scales'
// reads and the arrivals need: few polls, with a long suspend hint.
constexpr uint32_t kHintNs = 1000, kPolls = 1u << 21;
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    for (uint32_t i = 0; i < kPolls; i++) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(bar), "r"(parity), "r"(kHintNs) : "memory");
        if (ok) return true;
    }
    atomicExch(&g_moe_err, (unsigned int)QZ_ERR_TIMEOUT);
    return false;
}

// The same for the two waits that every block of K stands behind, with the system's own limit: 434 -> 418 us for 4001
// tokens by 2 of 8 experts [4096, 14336].
__device__ __forceinline__ bool block_wait(uint32_t bar, uint32_t parity) { return mbar_wait<false>(bar, parity, &g_moe_err); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
}
// An arrival on `bar` (one of those it counts) once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ int one(int v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ bool all(bool v) { return __all_sync(0xffffffffu, v); }

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// An expert's rows, cut to those that exist.
__device__ __forceinline__ int2 expert_rows(const MoeGemmArgs& a, int e) {
    const int R = (int)a.rows, b = min(max(a.offsets[e], 0), R);
    return make_int2(b, min(max(a.offsets[e + 1], b), R));
}
__device__ __forceinline__ int row_tiles(int2 r) { return (r.y - r.x) / BM + ((r.y - r.x) % BM != 0); }

// nt: column tiles of an expert. splits: CTAs (a cluster) that share an item's blocks of K.
template <bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1)
moe_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmY, const __grid_constant__ MoeGemmArgs a,
                const int nt, const int splits) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bars = sbase + BAR_OFF;
    volatile int4* info = reinterpret_cast<volatile int4*>(smem + INFO_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + BAR_OFF + BARS * 8);
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (STAGES + s); };
    auto tfull = [&](int b) { return bars + 8 * (2 * STAGES + b); };
    auto ifull = [&](int i) { return bars + 8 * (2 * STAGES + 2 + i); };
    auto iempty = [&](int i) { return bars + 8 * (2 * STAGES + 2 + INFO + i); };
    auto peaks = [&](int q) { return bars + 8 * (2 * STAGES + 2 + 2 * INFO + q); };

    // What a warp's lanes have in common goes through one(): loops and addresses that depend on it are then known to be
    // the warp's, and the operands of its tensor instructions stay in uniform registers.
    const int warp = one(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int nkb = a.K / BK;
    const int rank = (int)(blockIdx.x % splits);                    // in the cluster
    const int kb0 = nkb * rank / splits, kb1 = nkb * (rank + 1) / splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(full(s), EPI_WARPS + (a.row_token ? 129 : 2));    // the accumulator; the weights' thread; the rows': one, or 128 that copy
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; b++) mbar_init(tfull(b), 1);
        for (int i = 0; i < INFO; i++) {
            mbar_init(ifull(i), 1);
            mbar_init(iempty(i), 2 + 4 + EPI_WARPS);
        }
        for (int q = 0; q < 4; q++) mbar_init(peaks(q), EPI_WARPS / 4);
        fence_barrier_init();
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = one(*tmem_slot);
    pdl_wait();

    // The next item (x < 0: no more); every warp but warp 3 takes each of them once.
    uint32_t taken = 0;
    auto next_item = [&](int4& it) {
        const int i = taken % INFO;
        if (!all(warp_wait(ifull(i), (taken / INFO) & 1))) return false;
        it.x = one(info[i].x);
        it.y = one(info[i].y);
        it.z = one(info[i].z);
        it.w = one(info[i].w);
        if (lane == 0) mbar_arrive(iempty(i));
        taken++;
        return it.x >= 0;
    };

    if (warp < FEED_WARPS) {
        reg_dec<REGS_FEED>();
        int4 item;                                 // expert, first row, rows, column tile
        if (warp == 0) {
            // --------------------------------------------------------- weights
            uint32_t it = 0;
            bool ok = true;
            while (ok && next_item(item)) {
                const int n0 = item.x * a.N + item.w * (SWIGLU ? 128 : BN);
                const bool two = SWIGLU || item.w * BN + 128 < a.N;
                for (int kb = kb0; kb < kb1; kb++, it++) {
                    const int s = it % STAGES;
                    ok = all(warp_wait(empty(s), ((it / STAGES) & 1) ^ 1));
                    if (!ok) break;
                    if (lane == 0) {
                        const uint32_t dst = sbase + s * STAGE_BYTES + A_BYTES;
                        mbar_arrive_expect_tx(full(s), two ? 2 * HALF_BYTES : HALF_BYTES);
                        tma_load_2d(dst, &tmB, kb * BK, n0, full(s));
                        if (two) tma_load_2d(dst + HALF_BYTES, &tmB, kb * BK, n0 + (SWIGLU ? a.N / 2 : 128), full(s));
                    }
                    __syncwarp();
                }
            }
            // all copies into this CTA's shared memory have landed before it may exit
            for (uint32_t j = it > STAGES ? it - STAGES : 0; j < it; j++)
                warp_wait(empty(j % STAGES), (j / STAGES) & 1);
        } else if (warp >= 4) {
            // ------------------------------------------------------------ rows
            // Gathered: warp p has rows 32 p .. 32 p + 31, lane l copies chunk l % 8 of every fourth of them from
            // l / 8 on. A row whose token is not there is any row here, the promotion writes zeros for it.
            const int part = warp - 4, c = lane & 7, sub = lane >> 3;
            const uint8_t* src = (a.tokens ? a.qA : a.qW) + 16 * c;
            const uint32_t even = (c ^ sub) << 4, odd = (c ^ (4 + sub)) << 4;   // swizzle of rows sub, 4 + sub, 8 + sub, ...
            uint32_t it = 0;
            bool ok = true;
            while (ok && next_item(item)) {
                const int here = item.z - 32 * part;                            // rows from this warp's first on
                int at[8];                                                      // this lane's rows, in qA
                if (a.row_token) {
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        const int tok = sub + 4 * j < here ? a.row_token[item.y + 32 * part + sub + 4 * j] : 0;
                        at[j] = tok >= 0 && tok < a.tokens ? tok : 0;
                    }
                }
                for (int kb = kb0; kb < kb1; kb++, it++) {
                    const int s = it % STAGES;
                    if (!a.row_token && part) continue;
                    ok = all(warp_wait(empty(s), ((it / STAGES) & 1) ^ 1));
                    if (!ok) break;
                    const uint32_t dst = sbase + s * STAGE_BYTES;
                    if (a.row_token) {
                        const uint8_t* from = src + kb * BK;
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            if (4 * j < here) cp_async16(dst + (32 * part + sub + 4 * j) * BK + (j & 1 ? odd : even), from + (int64_t)at[j] * a.K);
                        cp_async_arrive(full(s));
                    } else {
                        const int boxes = (item.z + 31) / 32;
                        if (lane == 0) mbar_arrive_expect_tx(full(s), boxes * 32 * BK);
                        __syncwarp();
                        if (lane < boxes) tma_load_2d(dst + lane * 32 * BK, &tmA, kb * BK, item.y + 32 * lane, full(s));
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------- MMA
            // One wait a block: its stage counts the promotion of the block two before it, which had the same
            // accumulator, beside its operands. (With a barrier each the tensor core stood still 200 cycles a block: it takes
            // instructions only a few ahead, and a wait behind them costs as much when it is over already.)
            uint32_t it = 0;
            bool ok = true;
            while (ok && next_item(item)) {
                const bool two = SWIGLU || item.w * BN + 128 < a.N;
                const uint32_t idesc = two ? idesc_dense(0u, 0u, BM, BN) : idesc_dense(0u, 0u, BM, 128);
                for (int kb = kb0; kb < kb1; kb++, it++) {
                    const int b = it & 1, s = it % STAGES;
                    ok = all(block_wait(full(s), (it / STAGES) & 1));
                    if (!ok) break;
                    if (a.row_token) fence_proxy_async_smem();               // the gathered rows came by the generic proxy
                    tc_fence_after();
                    mma_block(tmem_base + b * BN, sbase + s * STAGE_BYTES, idesc, empty(s), tfull(b));
                }
            }
            // the last accumulators are complete before tensor memory is released
            if (it > 0) warp_wait(tfull((it - 1) & 1), ((it - 1) >> 1) & 1);
        } else if (warp == 2) {
            // ----------------------------------------------------------- items
            // lane l: the row tiles before expert l * per; an item of the list is row tile p of an
            // expert's column tile n, p running first
            const int per = (a.experts + 31) / 32, e0 = lane * per;
            int mine = 0;
            for (int j = 0; j < per && e0 + j < a.experts; j++) mine += row_tiles(expert_rows(a, e0 + j));
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const int64_t total = (int64_t)__shfl_sync(0xffffffffu, upto, 31) * nt;
            const int first = upto - mine;
            bool ok = true;
            for (uint32_t n = 0; ok; n++) {
                const int64_t i = blockIdx.x / splits + (int64_t)n * (gridDim.x / splits);
                int4 v = make_int4(-1, 0, 0, 0);
                // a cluster has one item: more than the host's bound come from offsets that do not ascend
                if (i < total && (splits == 1 || n == 0)) {
                    // the lane whose experts hold the item, then the expert among them
                    const uint32_t who = __ballot_sync(0xffffffffu, (int64_t)first * nt <= i && mine > 0);
                    const int l = 31 - __clz(who);
                    const int64_t base = (int64_t)__shfl_sync(0xffffffffu, first, l) * nt;
                    const int e = l * per + lane;
                    const int2 r = lane < per && e < a.experts ? expert_rows(a, e) : make_int2(0, 0);
                    const int tiles = row_tiles(r);
                    int before = tiles;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int u = __shfl_up_sync(0xffffffffu, before, o);
                        if (lane >= o) before += u;
                    }
                    const int64_t at = i - base - (int64_t)(before - tiles) * nt;       // within this lane's expert
                    const int w = __ffs(__ballot_sync(0xffffffffu, at >= 0 && at < (int64_t)tiles * nt)) - 1;
                    if (lane == w) {
                        const int p = (int)(at % tiles);
                        v = make_int4(e, r.x + p * BM, min(BM, r.y - r.x - p * BM), (int)(at / tiles));
                    }
                    v.x = __shfl_sync(0xffffffffu, v.x, w);
                    v.y = __shfl_sync(0xffffffffu, v.y, w);
                    v.z = __shfl_sync(0xffffffffu, v.z, w);
                    v.w = __shfl_sync(0xffffffffu, v.w, w);
                }
                const int slot = n % INFO;
                ok = warp_wait(iempty(slot), ((n / INFO) & 1) ^ 1);
                if (ok && lane == 0) {
                    info[slot].x = v.x;
                    info[slot].y = v.y;
                    info[slot].z = v.z;
                    info[slot].w = v.w;
                    mbar_arrive(ifull(slot));
                }
                __syncwarp();
                if (v.x < 0) break;
            }
        }
        if (splits > 1) {
            cluster_sync();
            cluster_sync();
        }
    } else {
        // ------------------------------------------------- promotion and output
        reg_inc<REGS_EPI>();
        const int q = warp & 3, h = (warp - FEED_WARPS) >> 2;          // lane quarter of tensor memory, half of each box
        const int r = q * 32 + lane;                          // row of the tile
        uint8_t* stg = smem + STG_OFF + (warp - FEED_WARPS) * STG_WARP;
        // Scales are read four blocks of K at a time and a group ahead, an item's first ones before the output of the item
        // before it; its row's token a whole item ahead.
        const bool vec = ((nkb | kb0) & 3) == 0 && ((reinterpret_cast<uintptr_t>(a.sA) | reinterpret_cast<uintptr_t>(a.sW)) & 15) == 0;
        const float *sa = a.sA, *sw = a.sW;
        int up = 0, token = 0;                                // from the first box's weight scales to the second's; the row in qA
        float4 na, nw0, nw1;                                  // a group in flight
        auto read_group = [&](int kb) {
            if (vec && kb + 4 <= kb1) {
                na = __ldg(reinterpret_cast<const float4*>(sa + kb));
                nw0 = __ldg(reinterpret_cast<const float4*>(sw + kb));
                nw1 = __ldg(reinterpret_cast<const float4*>(sw + up + kb));
            } else {
                auto one = [&](const float* p, int i) { return kb + i < kb1 ? __ldg(p + kb + i) : 0.0f; };
                na = make_float4(one(sa, 0), one(sa, 1), one(sa, 2), one(sa, 3));
                nw0 = make_float4(one(sw, 0), one(sw, 1), one(sw, 2), one(sw, 3));
                nw1 = make_float4(one(sw + up, 0), one(sw + up, 1), one(sw + up, 2), one(sw + up, 3));
            }
        };
        auto row_of = [&](const int4& i) {                    // a row behind the tile's last repeats that one
            const int row = i.y + min(r, i.z - 1);
            return a.row_token ? a.row_token[row] : row;
        };
        auto begin = [&](const int4& i, int tok) {            // the item's first group; a token that is not there counts as any
            const bool two = SWIGLU || i.w * BN + 128 < a.N;
            sa = a.sA + (int64_t)(tok >= 0 && tok < a.tokens ? tok : 0) * nkb;
            sw = a.sW + ((size_t)i.x * (a.N / 128) + (SWIGLU ? i.w : 2 * i.w)) * nkb;
            up = two ? (SWIGLU ? a.N / 256 : 1) * nkb : 0;
            if (a.tokens) read_group(kb0);
        };
        na = nw0 = nw1 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane == 0) {                                      // the first two blocks find their accumulators empty
            mbar_arrive(full(0));
            mbar_arrive(full(1));
        }
        uint32_t it = 0;
        int done = 0;
        bool ok = true, synced = false;
        int4 item, next;
        bool more = next_item(next);
        if (more) {
            token = row_of(next);
            begin(next, token);
        }
        while (ok && more) {
            item = next;
            const bool there = token >= 0 && token < a.tokens;
            more = next_item(next);
            if (more) token = row_of(next);
            const bool active = q * 32 < item.z;              // some row of the warp exists
            const bool two = SWIGLU || item.w * BN + 128 < a.N;
            Sums sums;
            sums.zero();
            float4 s0, s1;                                    // the group's scales of the two boxes
            for (int kb = kb0; kb < kb1; kb++, it++) {
                const int b = it & 1;
                if (((kb - kb0) & 3) == 0) {
                    s0 = make_float4(na.x * nw0.x, na.y * nw0.y, na.z * nw0.z, na.w * nw0.w);
                    s1 = make_float4(na.x * nw1.x, na.y * nw1.y, na.z * nw1.z, na.w * nw1.w);
                    if (kb + 4 < kb1 && a.tokens) read_group(kb + 4);
                }
                ok = all(block_wait(tfull(b), (it >> 1) & 1));
                if (!ok) break;
                tc_fence_after();
                if (active) {
                    const uint32_t t = tmem_base + ((uint32_t)(q * 32) << 16) + b * BN + h * 64;
                    uint32_t x[32];
                    tmem_ld32(t, x);
                    tmem_wait_ld();
                    sums.add<0>(x, s0.x);
                    tmem_ld32(t + 32, x);
                    tmem_wait_ld();
                    sums.add<32>(x, s0.x);
                    tmem_ld32(t + 128, x);
                    tmem_wait_ld();
                    sums.add<64>(x, s1.x);
                    tmem_ld32(t + 160, x);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full((it + 2) % STAGES));                // all of it is in registers
                    sums.add<96>(x, s1.x);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full((it + 2) % STAGES));
                }
                s0 = make_float4(s0.y, s0.z, s0.w, 0.0f);
                s1 = make_float4(s1.y, s1.z, s1.w, 0.0f);
            }
            if (!ok) break;
            Sums::Values acc = sums.values();
            if (more) begin(next, token);
            if (splits > 1) {
                // the sums of an item's parts meet in rank 0, in the order of the ranks
                cluster_sync();                               // its ring is free
                const uint32_t mine = sbase + ((h * 32) * 32 + lane) * 16;
                if (rank > 0 && q == 0) {
                    uint32_t dst;
                    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(mine + (rank - 1) * PART_BYTES));
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * 512), "f"(acc[4 * i]),
                                     "f"(acc[4 * i + 1]), "f"(acc[4 * i + 2]), "f"(acc[4 * i + 3]) : "memory");
                }
                cluster_sync();
                synced = true;
                if (rank > 0) break;
                if (q == 0)
                    for (int p = 0; p < splits - 1; p++)
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const float4 v = *reinterpret_cast<const float4*>(smem + ((h * 32) * 32 + lane) * 16 + p * PART_BYTES + i * 512);
                            acc[4 * i] += v.x;
                            acc[4 * i + 1] += v.y;
                            acc[4 * i + 2] += v.z;
                            acc[4 * i + 3] += v.w;
                        }
            }
            if (!there) {                                     // a row of zeros
#pragma unroll
                for (int i = 0; i < 128; i++) acc[i] = 0.0f;
            }
            const size_t out = (size_t)(item.y + r);
            if constexpr (SWIGLU) {
                // column i of h: gate acc[i], up acc[64 + i]; a scale's 128 columns lie in two threads
                float* peak = reinterpret_cast<float*>(smem + STG_OFF) + (done & 1) * 256;
                float am = 0.0f;
                if (active) {
#pragma unroll
                    for (int i = 0; i < 64; i++) {
                        acc[i] = silu(acc[i]) * acc[64 + i];
                        am = fmaxf(am, fabsf(acc[i]));
                    }
                }
                peak[h * 128 + r] = am;
                // the two warps of these rows meet, with a limit: the other may have given up
                __syncwarp();
                if (lane == 0) mbar_arrive(peaks(q));
                ok = all(warp_wait(peaks(q), done & 1));
                if (!ok) break;
                if (r < item.z) {
                    const float sc = div1(fmaxf(fmaxf(am, peak[(h ^ 1) * 128 + r]), kAmaxMin), Recip(kFp8Max));
                    const Recip d(sc);
                    const int I = a.N / 2;
                    uint4* codes = reinterpret_cast<uint4*>(a.codes + out * I + item.w * 128 + h * 64);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        uint32_t p[8];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const float v = acc[16 * j + 2 * e], w = acc[16 * j + 2 * e + 1];
                            p[e] = e4m3x2(sign_of(div1(v, d), v), sign_of(div1(w, d), w));
                        }
                        codes[j] = make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                                              __byte_perm(p[4], p[5], 0x5410), __byte_perm(p[6], p[7], 0x5410));
                    }
                    if (h == 0) a.scales[out * (I / 128) + item.w] = sc;
                }
                done++;
            } else if (active) {
#pragma unroll
                for (int s = 0; s < 2; s++) {
                    if (s == 1 && !two) break;
                    const int c0 = item.w * BN + s * 128 + h * 64;
                    if (lane == 0) bulk_wait_read0();                     // the previous store has read the block
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; j++) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const __nv_bfloat162 p = __floats2bfloat162_rn(acc[s * 64 + j * 8 + 2 * e], acc[s * 64 + j * 8 + 2 * e + 1]);
                            w[e] = *reinterpret_cast<const uint32_t*>(&p);
                        }
                        *reinterpret_cast<uint4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (q * 32 + 32 <= item.z) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&tmY, smem_u32(stg), c0, item.y + q * 32);
                    } else {
                        // the tile's last rows: what lies behind them is another expert's
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const int rr = 4 * j + (lane >> 3), ch = lane & 7;
                            if (q * 32 + rr < item.z)
                                *reinterpret_cast<uint4*>(a.Y + (size_t)(item.y + q * 32 + rr) * a.N + c0 + ch * 8) =
                                    *reinterpret_cast<const uint4*>(stg + rr * 128 + ((ch ^ (rr & 7)) << 4));
                        }
                        __syncwarp();
                    }
                }
            }
        }
        if (!SWIGLU && lane == 0) bulk_wait_all0();           // stores complete before the CTA exits
        __syncwarp();
        if (splits > 1 && !synced) {
            cluster_sync();
            cluster_sync();
        }
    }
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

} // namespace

qz_status moe_gemm_error_read_and_clear() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_moe_err, sizeof(v)) != cudaSuccess) return QZ_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_moe_err, &z, sizeof(z)) != cudaSuccess) return QZ_ERR_CUDA;
    return v ? QZ_ERR_TIMEOUT : QZ_OK;
}

qz_status moe_gemm_fp8_launch(const MoeGemmArgs& a, cudaStream_t st) {
    CUtensorMap ta, tb, ty;
    // without tokens every row is one of zeros: what the map of the rows reaches is not used
    const void* rows = a.tokens ? a.qA : a.qW;
    const uint64_t tokens = a.tokens ? (uint64_t)a.tokens : 1, K = (uint64_t)a.K;
    if (!encode_tmap_2d_u8(&ta, rows, K, tokens, K, BK, 32) ||
        !encode_tmap_2d_u8(&tb, a.qW, K, (uint64_t)a.experts * a.N, K, BK, 128))
        return QZ_ERR_CUDA;
    memset(&ty, 0, sizeof(ty));                   // SwiGLU's codes are stored without TMA
    if (a.Y && !encode_tmap_2d_swz(&ty, a.Y, 2, (uint64_t)a.N, (uint64_t)a.rows, (uint64_t)a.N * 2, 64, 32, 128))
        return QZ_ERR_CUDA;
    const int nt = a.Y ? (a.N + BN - 1) / BN : a.N / 256;
    const int64_t items = (a.rows / BM + std::min<int64_t>(a.experts, a.rows)) * nt;       // at most
    const int sms = num_sms(), nkb = a.K / BK;
    int splits = 1;
    while (a.rows <= SPLIT_ROWS && splits < MAX_SPLITS && 2 * splits * items <= sms && nkb >= 4 * splits) splits *= 2;
    const int grid = splits > 1 ? (int)items * splits : (int)std::min<int64_t>(items, sms);
    const void* fn = a.Y ? (const void*)moe_gemm_kernel<false> : (const void*)moe_gemm_kernel<true>;
    QZ_TRY(opt_in_smem(fn, SMEM_BYTES));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    const cudaError_t r = a.Y ? cudaLaunchKernelEx(&cfg, moe_gemm_kernel<false>, ta, tb, ty, a, nt, splits)
                              : cudaLaunchKernelEx(&cfg, moe_gemm_kernel<true>, ta, tb, ty, a, nt, splits);
    return r == cudaSuccess ? launch_status() : QZ_ERR_CUDA;
}

} // namespace qz
