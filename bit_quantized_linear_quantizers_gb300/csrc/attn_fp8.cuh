// attn_fp8.cuh -- what the attention kernels over the paged FP8 cache share.
#pragma once

#include "qz_paged.cuh"
#include "qz_tc.cuh"

namespace qz {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values as E4M3 parts: hi = E4M3(x), lo = E4M3(x - hi); 16 bits each. The
// f16 step in between keeps 11 bits (the values lie in [-256, 256]).
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    uint32_t h, back;
    uint16_t e, f;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(e) : "r"(h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(e));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(back));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(f) : "r"(h));
    hi = e;
    lo = f;
}

// Four values -> one register of each part (value i in byte i).
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t& hi, uint32_t& lo) {
    uint32_t ha, la, hb, lb;
    split2(x0, x1, ha, la);
    split2(x2, x3, hb, lb);
    hi = ha | hb << 16;
    lo = la | lb << 16;
}

// The power of two that brings a row's amax into [128, 256), and its inverse
// (both normal numbers: amax below 2^-106 is scaled by 2^113 only); 1 for a row of zeros. A row
// with an infinity is made NaN: every score of it is infinite or NaN, so its softmax is NaN.
__device__ __forceinline__ void row_scale(float amax, float& up, float& down) {
    const int ex = (int)(__float_as_uint(amax) >> 23) & 255;
    const int se = min(max(134 + 127 - ex, 6), 240);
    up = amax > 0.0f ? __uint_as_float((uint32_t)se << 23) : 1.0f;
    if (ex == 255) up = __int_as_float(0x7FFFFFFF);
    down = amax > 0.0f ? __uint_as_float((uint32_t)(254 - se) << 23) : 1.0f;
}

// Least value scale that enters the exponent and l = sum p / sv: p <= 2^15 and 2^31 keys leave l below 2^126. Pages
// of this scale or less (0 among them) keep their share of l; their codes are taken as 0.
constexpr float kLeastScale = 0x1p-80f;
// NaN stays, and the logarithm of a negative scale is NaN.
__device__ __forceinline__ float value_scale(float v) { return fabsf(v) < kLeastScale ? kLeastScale : v; }

// 3-D TMA load of a box (channels, rows, page).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

} // namespace qz
