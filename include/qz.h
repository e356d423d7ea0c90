/*
 * qz.h -- C ABI of libqz: low-bit quantizers and quantized linear layers for
 * one GB300 (sm_103a) GPU.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Ownership: every data pointer is a DEVICE pointer owned by the caller. The
 *   library never allocates or frees device memory. Scratch that a call needs
 *   comes from a caller buffer `ws` of at least qz_workspace_size(...) bytes.
 * Streams: `stream` is a cudaStream_t passed as void* (NULL = the legacy
 *   default stream). Every call only enqueues work on that stream and returns
 *   without synchronising; outputs are valid in stream order. A workspace must
 *   not be shared by calls that may run concurrently.
 * Early start: most calls launch under programmatic dependent launch, so their
 *   kernels may begin while the previous kernel on the stream is still running.
 *   Each waits for that kernel before it reads or writes anything, with one
 *   exception. The INT4 W4A16 GEMMs (qz_gemm_w4a16, _grouped, _zp) read qweight,
 *   scale_bf16 and zero BEFORE that wait, so the weight stream overlaps the
 *   previous kernel's tail. The library tracks the outputs of its own INT4
 *   quantizers per device and stream. A W4A16 call whose weights such a call may
 *   still be writing is launched only after the stream's earlier work. Weights
 *   written by other code must not come from the kernel enqueued directly
 *   before the W4A16 call on its stream. Any synchronisation, copy or other
 *   kernel between the two is enough.
 * Layout: row-major, leading dimension in elements. Packed 4-bit codes put
 *   the even-index element in the low nibble of each byte. bf16 data is passed
 *   as uint16_t bit patterns. Scales use the row-major layouts given per call.
 * Errors: every call returns a qz_status. Arguments are validated on the host
 *   before anything is enqueued, so a rejected call launches nothing and
 *   leaves every output untouched. No call aborts, throws or prints.
 *   QZ_ERR_CUDA reports a launch or runtime error seen right after enqueueing.
 * Numerics: the codes and scales of every quantizer are defined by the fake-
 *   quant functions of "量化部署实战" (anrans.github.io), section 伪量化实现,
 *   computed in IEEE fp32 (bf16 inputs are widened exactly to fp32 first):
 *   E4M3 rounds to nearest even and saturates at +-448; E2M1 rounds to the
 *   nearest of +-{0, .5, 1, 1.5, 2, 3, 4, 6} with exact ties going to the
 *   smaller magnitude; the clamp floor 1e-12 is the fp32 value nearest 1e-12.
 *   NaN or infinite inputs are outside the contract (no fault, undefined codes).
 */
#ifndef QZ_H
#define QZ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum qz_status {
    QZ_OK = 0,
    QZ_ERR_INVALID_ARG = 1,   /* null pointer, unknown enum value, negative size */
    QZ_ERR_SHAPE = 2,         /* size not divisible as required, or out of the supported range */
    QZ_ERR_ALIGNMENT = 3,     /* pointer or leading dimension not aligned as required */
    QZ_ERR_UNSUPPORTED = 4,   /* no usable sm_103 device, or the path is not available */
    QZ_ERR_CUDA = 5,          /* a CUDA runtime call or kernel launch failed */
    QZ_ERR_TIMEOUT = 6,       /* a bounded device-side wait gave up (see qz_device_error) */
    QZ_ERR_WORKSPACE = 7      /* ws is NULL or smaller than qz_workspace_size() */
} qz_status;

typedef enum qz_dtype { QZ_F32 = 0, QZ_BF16 = 1 } qz_dtype;

typedef enum qz_fp8_gran {
    QZ_FP8_PER_TENSOR = 0,    /* one scale for the tensor                      scales[1]             */
    QZ_FP8_PER_ROW = 1,       /* one scale per row (output channel / token)    scales[rows]          */
    QZ_FP8_BLOCK_128x128 = 2, /* one scale per (br x 128) block, br=min(128,rows) scales[rows/br][cols/128] */
    QZ_FP8_GROUP_1x128 = 3    /* one scale per row per 128 columns             scales[rows][cols/128] */
} qz_fp8_gran;

typedef enum qz_scale_mode {
    QZ_SCALE_COMPUTE = 0,     /* scale = max(amax, 1e-12) / 448 from the data written   */
    QZ_SCALE_GIVEN = 1        /* use the caller's (calibrated) scale, read from device  */
} qz_scale_mode;

typedef enum qz_op {
    QZ_OP_QUANTIZE_FP8 = 0,   /* d0 = rows, d1 = cols, d2 = granularity   */
    QZ_OP_QUANTIZE_NVFP4 = 1, /* d0 = rows, d1 = cols                      */
    QZ_OP_KV_WRITE_FP8 = 2,   /* d0 = elements per tensor (B*H*T*D)        */
    QZ_OP_GEMM_W4A16 = 3,     /* d0 = M, d1 = N, d2 = K                    */
    QZ_OP_GEMM_FP8_BLOCK = 4, /* d0 = M, d1 = N, d2 = K                    */
    QZ_OP_GEMM_NVFP4 = 5,     /* d0 = M, d1 = N, d2 = K                    */
    QZ_OP_GEMM_MXFP4 = 6,     /* d0 = M, d1 = N, d2 = K                    */
    QZ_OP_GEMM_NVFP4_GROUPED = 7, /* d0 = problem count, d1 = largest K    */
    QZ_OP_PREPARE_FP4_SCALES = 8, /* d0 = rows, d1 = K, d2 = 1 NVFP4 / 0 MXFP4:
                                     bytes of the prepared output (not scratch) */
    QZ_OP_QUANTIZE_NVFP4_GROUPED = 9, /* d0 = tensor count                   */
    QZ_OP_KV_WRITE_FP8_PER_HEAD = 10, /* d0 = B*H, d1 = T*D                   */
    QZ_OP_KV_WRITE_FP8_CHANNEL_ZP = 11, /* d0 = B*H, d1 = T, d2 = D           */
    QZ_OP_COL_AMAX = 12,                /* d0 = rows, d1 = cols               */
    QZ_OP_ATTN_FP8_PAGED = 13,          /* d0 = query rows of the largest request per KV
                                           head (max_q * heads_q / heads), d1 = head_dim */
    QZ_OP_MOE_ROUTE = 14                /* d0 = tokens, d1 = experts, d2 = top_k */
} qz_op;

typedef enum qz_smooth_op {
    QZ_SMOOTH_NONE = 0,       /* x' = x                                          */
    QZ_SMOOTH_DIVIDE = 1,     /* x' = x / f[col]  (activations, SmoothQuant)     */
    QZ_SMOOTH_MULTIPLY = 2    /* x' = x * f[col]  (weights as B^T, SmoothQuant)  */
} qz_smooth_op;

/* Bytes of workspace the call `op` needs for the given sizes (0 if none).
 * Returns 0 for an unknown op. Sizes that the call itself would reject still
 * return a (harmless) value. Workspace contents need no initialisation. */
size_t qz_workspace_size(qz_op op, int64_t d0, int64_t d1, int64_t d2);

/* Human-readable name of a status (static string, never NULL). */
const char* qz_status_string(qz_status s);

/* Reads and clears the library's device-side error word on the current
 * device (set when a bounded wait inside a GEMM kernel gives up). Returns
 * QZ_ERR_TIMEOUT if it was set, QZ_OK if not, QZ_ERR_CUDA if the read failed.
 * Synchronises with the legacy default stream. */
qz_status qz_device_error(void);

/* Self-test of the failure detection (the pages have no counterpart; this is
 * a property of this library's kernels). Launches one CTA on `stream` that
 * waits on an mbarrier nothing ever completes, using the same bounded wait as
 * every GEMM kernel but giving up after `polls` polls (1 <= polls <= 2^20,
 * each poll suspends for at most tens of nanoseconds). The wait runs out,
 * records QZ_ERR_TIMEOUT in the device error word and the kernel returns, so
 * the next qz_device_error() reports QZ_ERR_TIMEOUT and the CUDA context stays
 * usable. Returns QZ_ERR_INVALID_ARG for polls out of range. */
qz_status qz_selftest_bounded_wait(uint32_t polls, void* stream);

/* ------------------------------------------------------------ quantizers */

/* FP8 E4M3 quantization of x[rows, cols] (leading dim ldx >= cols) at one of
 * four scale granularities ("量化部署实战", 伪量化实现: fp8_per_tensor,
 * fp8_per_row, fp8_blockwise with (128,128) for weights and (1,128) for
 * activations; 格式速查: FP8 E4M3 row):
 *   scale = max(amax_unit, 1e-12) / 448;  code = E4M3(clamp(x / scale, +-448))
 *   dequant = E4M3value(code) * scale    (fp32, one rounding)
 * codes:   [rows, cols] bytes, dense.
 * scales:  fp32, shape per qz_fp8_gran.
 * dequant: nullable; fp32 [rows, cols], dense.
 * ws:      PER_TENSOR needs qz_workspace_size(QZ_OP_QUANTIZE_FP8, rows, cols, 0)
 *          bytes; the other granularities need none (ws may be NULL).
 * Shapes:  BLOCK_128x128 needs cols % 128 == 0 and rows % min(128, rows) == 0;
 *          GROUP_1x128 needs cols % 128 == 0. rows == 0 or cols == 0 is a no-op
 *          returning QZ_OK, except PER_TENSOR (amax undefined) -> QZ_ERR_SHAPE.
 * Alignment: x 16-byte aligned with ldx*elemsize % 16 == 0 and cols % 8 == 0
 *          give the vector path; PER_TENSOR and PER_ROW also accept any other
 *          x/ldx/cols (scalar path). BLOCK/GROUP require the vector conditions
 *          (QZ_ERR_ALIGNMENT), and codes/dequant must then be 8/16-byte aligned. */
qz_status qz_quantize_fp8(const void* x, qz_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                          qz_fp8_gran gran, uint8_t* codes, float* scales, float* dequant,
                          void* ws, size_t ws_bytes, void* stream);

/* MXFP4 quantization, one power-of-two (E8M0) scale per 32 consecutive
 * elements of a row ("量化部署实战", 伪量化实现: mxfp4; "量化：让每一步搬更少的
 * 字节", 新一代低位格式: MXFP4):
 *   E = floor(log2(max(amax32, 1e-12))) (exact, from the exponent field)
 *   scale = 2^(E-2); scale_e8m0 = E - 2 + 127
 *   code = E2M1(clamp(x / scale, +-6));  dequant = E2M1value(code) * scale
 * codes: [rows, cols/2] bytes (even element in the low nibble).
 * scale_e8m0: [rows, cols/32] bytes. dequant: nullable fp32 [rows, cols].
 * Shapes: cols % 32 == 0. Alignment: x 16 B, ldx*elemsize % 16 == 0, codes 4 B,
 * dequant 16 B. rows == 0 is a no-op. No workspace. */
qz_status qz_quantize_mxfp4(const void* x, qz_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                            uint8_t* codes, uint8_t* scale_e8m0, float* dequant, void* stream);

/* NVFP4 quantization, one E4M3 scale per 16 consecutive elements of a row
 * plus one fp32 scale per tensor ("量化部署实战", 伪量化实现: nvfp4;
 * 格式速查: NVFP4 row), in the page's order:
 *   g = max(amax_tensor, 1e-12) / (448 * 6)         -> *global_scale
 *   b = E4M3(amax16 / 6 / g)                         -> scale_e4m3
 *   s = max(E4M3value(b), 1e-12) * g
 *   code = E2M1(clamp(x / s, +-6));  dequant = E2M1value(code) * s
 * global_amax_in: nullable device pointer; when given, its value replaces the
 *   computed tensor amax (calibrated or shared across slices) and no
 *   workspace is needed.
 * codes: [rows, cols/2]; scale_e4m3: [rows, cols/16]; global_scale: 1 fp32.
 * ws: qz_workspace_size(QZ_OP_QUANTIZE_NVFP4, rows, cols, 0) bytes when
 *   global_amax_in is NULL. Shapes: cols % 16 == 0; rows == 0 -> QZ_ERR_SHAPE
 *   unless global_amax_in is given (then a no-op). Alignment as MXFP4. */
qz_status qz_quantize_nvfp4(const void* x, qz_dtype xt, int64_t rows, int64_t cols, int64_t ldx,
                            uint8_t* codes, uint8_t* scale_e4m3, float* global_scale,
                            const float* global_amax_in, float* dequant,
                            void* ws, size_t ws_bytes, void* stream);

/* One tensor of qz_quantize_nvfp4_grouped: contiguous x [rows, cols] (cols %
 * 16 == 0) and its outputs, laid out as qz_quantize_nvfp4 writes them. */
typedef struct qz_nvfp4_tensor {
    const void* x;
    int64_t rows, cols;
    uint8_t* codes;
    uint8_t* scale_e4m3;
    float* global_scale;
} qz_nvfp4_tensor;

/* NVFP4 quantization of `count` independent tensors (the activations of a
 * decoder step's linears, "量化部署实战", 精度比较: each linear quantizes its
 * input) in two launches: the same computation as one qz_quantize_nvfp4 call
 * with a computed tensor amax per tensor, bit for bit. All tensors share the
 * dtype xt. count <= 256. Alignment: x 16 B, codes 4 B. ws:
 * qz_workspace_size(QZ_OP_QUANTIZE_NVFP4_GROUPED, count, 0, 0) bytes. */
qz_status qz_quantize_nvfp4_grouped(const qz_nvfp4_tensor* tensors, int count, qz_dtype xt,
                                    void* ws, size_t ws_bytes, void* stream);

/* Symmetric INT4 weight quantization with one bf16 scale per group of 128
 * along K, for a row-major weight w[K, N] (leading dim ldw >= N)
 * ("量化部署实战", 格式速查: W4A16 row, integers -8..7 with a scale per 128;
 * "量化：让每一步搬更少的字节", 量化在做什么: q = round(x / s), x^ = q * s;
 * "LLM 推理优化 · 量化学习笔记" 5.1: q = clamp(round(x / s), qmin, qmax)):
 *   s = bf16_rne(max(amax_group, 1e-12) / 7);  q = clamp(rint(w / s), -8, 7)
 * qweight: int32 [K/8, N]; element k of column n sits in bits 4*(k%8)..+3 of
 *   qweight[k/8][n], two's complement.
 * scale_bf16: [K/128, N] bf16 bits. dequant: nullable fp32 [K, N] = q * s.
 * Shapes: K % 128 == 0, N % 64 == 0. Alignment: w 16 B, ldw*elemsize % 16 == 0,
 * qweight and dequant 16 B, scale_bf16 16 B. K == 0 or N == 0 is a no-op. */
qz_status qz_quantize_int4_g128(const void* w, qz_dtype wt, int64_t K, int64_t N, int64_t ldw,
                                int32_t* qweight, uint16_t* scale_bf16, float* dequant,
                                void* stream);

/* FP8 KV-cache write: per-tensor E4M3 quantization of K and of V, each with
 * its own scale ("量化部署实战", 伪量化实现: FP8KVCache.update applies
 * fp8_per_tensor to k and to v; KV Cache 量化: calibrated offline scales).
 * k, v: bf16 [B, H, T, D] contiguous (n = B*H*T*D elements each).
 * k_codes, v_codes: n bytes each. k_scale, v_scale: one fp32 each (device).
 * mode COMPUTE: scales = max(amax, 1e-12) / 448 written to k_scale/v_scale;
 *   needs qz_workspace_size(QZ_OP_KV_WRITE_FP8, n, 0, 0) bytes.
 * mode GIVEN: k_scale/v_scale are read (must be finite and > 0); no workspace.
 * Alignment: k, v 16 B; codes 8 B. n == 0 -> QZ_ERR_SHAPE (COMPUTE), no-op (GIVEN). */
qz_status qz_kv_write_fp8(const uint16_t* k, const uint16_t* v, int B, int H, int T, int D,
                          uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale,
                          qz_scale_mode mode, void* ws, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------- GEMMs */

/* W4A16 GEMM ("量化：让每一步搬更少的字节", 路线一: one kernel that fuses the
 * INT4 unpack, the dequantization and the matrix product):
 *   Y[m, n] = bf16_rne( sum_g s[g, n] * sum_{k in g} A[m, k] * q[k, n] )
 * accumulated in fp32. A: bf16 [M, K] row-major. qweight, scale_bf16: the
 * layouts written by qz_quantize_int4_g128. Y: bf16 [M, N].
 * Shapes: 1 <= M <= 64, K % 128 == 0, N % 64 == 0.
 * Alignment: all pointers 16 B. ws: qz_workspace_size(QZ_OP_GEMM_W4A16, M, N, K). */
qz_status qz_gemm_w4a16(const uint16_t* A, const int32_t* qweight, const uint16_t* scale_bf16,
                        uint16_t* Y, int M, int N, int K, void* ws, size_t ws_bytes, void* stream);

/* One W4A16 problem of a grouped launch (all pointers device, layouts as in
 * qz_gemm_w4a16). */
typedef struct qz_w4a16_problem {
    const uint16_t* A;
    const int32_t* qweight;
    const uint16_t* scale_bf16;
    uint16_t* Y;
    int M, N, K;
} qz_w4a16_problem;

/* Runs `count` independent W4A16 problems (a decoder step's linears, whose
 * inputs are all ready) in as few launches as the kernel parameter space
 * allows (per launch: up to 120 problems of at most 8 tokens and K <= 8192,
 * 256 for deeper K, 56 at 9-16 tokens, 80 at 17-64), split into equal
 * shares. The kernel is chosen by the largest M of the group. Each problem
 * obeys the rules of qz_gemm_w4a16; outputs must not overlap. count <= 256.
 * ws: qz_workspace_size(QZ_OP_GEMM_W4A16, Mmax, sum of N, Kmax) bytes
 * suffices. */
qz_status qz_gemm_w4a16_grouped(const qz_w4a16_problem* problems, int count,
                                void* ws, size_t ws_bytes, void* stream);

/* FP8 block-scaled GEMM ("量化部署实战", 练习 2: inside each 128-wide K block
 * the tensor cores multiply-accumulate FP8, then the partial sum is multiplied
 * by that block's activation and weight scales and added into the fp32 result):
 *   Y[i, j] = bf16_rne( sum_kb sA[i, kb] * sB[j/128, kb] * sum_{k in kb} qA[i,k] * qB[j,k] )
 * qA: E4M3 [M, K] (1x128 groups, as written by qz_quantize_fp8 GROUP_1x128);
 * sA: fp32 [M, K/128]. qB: E4M3 [N, K] = B^T, K-major (128x128 blocks, as
 * written by qz_quantize_fp8 BLOCK_128x128 on B^T); sB: fp32 [N/128, K/128].
 * Y: bf16 [M, N]. Shapes: M % 128 == 0, N % 256 == 0, K % 128 == 0, K >= 128.
 * Alignment: all pointers 16 B. */
qz_status qz_gemm_fp8_block(const uint8_t* qA, const float* sA, const uint8_t* qB, const float* sB,
                            uint16_t* Y, int M, int N, int K, void* ws, size_t ws_bytes, void* stream);

/* NVFP4 GEMM (Blackwell FP4 tensor cores; "量化部署实战", 格式速查: NVFP4):
 *   Y[i, j] = bf16_rne( gA * gB * sum_b sA[i,b] * sB[j,b] * sum_{k in b} qA[i,k] * qB[j,k] )
 * qA: [M, K/2] packed E2M1, sA: E4M3 [M, K/16], gA: fp32 device scalar;
 * qB, sB, gB likewise for B^T [N, K]; layouts as written by qz_quantize_nvfp4.
 * Y: bf16 [M, N]. Shapes: M % 128 == 0, N % 256 == 0, K % 256 == 0.
 * Alignment: all pointers 16 B. */
qz_status qz_gemm_nvfp4(const uint8_t* qA, const uint8_t* sA, const float* gA,
                        const uint8_t* qB, const uint8_t* sB, const float* gB,
                        uint16_t* Y, int M, int N, int K, void* ws, size_t ws_bytes, void* stream);

/* MXFP4 GEMM: Y[i, j] = bf16_rne( sum_b 2^(eA[i,b]-127) * 2^(eB[j,b]-127) *
 * sum_{k in b} qA[i,k] * qB[j,k] ), blocks of 32 along K. Layouts as written by
 * qz_quantize_mxfp4 on A [M, K] and B^T [N, K]. Shapes and alignment as NVFP4. */
qz_status qz_gemm_mxfp4(const uint8_t* qA, const uint8_t* eA, const uint8_t* qB, const uint8_t* eB,
                        uint16_t* Y, int M, int N, int K, void* ws, size_t ws_bytes, void* stream);

/* Re-lays a row-major block-scale matrix, as the FP4 quantizers write it
 * (NVFP4: E4M3 [rows, K/16], nv = 1; MXFP4: E8M0 [rows, K/32], nv = 0), into the
 * order the FP4 tensor cores read scale factors in: per 128 rows and 4
 * consecutive scales, a 512-byte block where byte (m%32)*16 + (m/32)*4 + k holds
 * the scale k of row m (rows beyond `rows` up to a multiple of 128 are 0).
 * Weights are static, so their scales are re-laid once and handed to
 * qz_gemm_nvfp4_grouped; the single-problem GEMMs do this per call in their
 * workspace. This is a layout step of this library; the pages define no
 * layout for the scales beyond the row-major block order.
 * out: qz_workspace_size(QZ_OP_PREPARE_FP4_SCALES, rows, K, nv) bytes, 16 B
 * aligned, caller-owned. Shapes: rows >= 1, K % 256 == 0. */
qz_status qz_prepare_fp4_scales(const uint8_t* scales, int rows, int K, int nv, uint8_t* out, void* stream);

/* One problem of qz_gemm_nvfp4_grouped: Y = A B with A NVFP4 codes [M, K/2],
 * row-major E4M3 scales [M, K/16] and tensor scale gA (as qz_quantize_nvfp4
 * writes them), B^T NVFP4 codes [N, K/2] with its scales already re-laid by
 * qz_prepare_fp4_scales(nv = 1) and tensor scale gB, Y bf16 [M, N]. */
typedef struct qz_nvfp4_problem {
    const uint8_t* qA;
    const uint8_t* sA;
    const float* gA;
    const uint8_t* qB;
    const uint8_t* sB_prepared;
    const float* gB;
    uint16_t* Y;
    int M, N, K;
} qz_nvfp4_problem;

/* Runs `count` independent NVFP4 GEMMs of decode shape (the linears of a
 * decoder step, "量化部署实战", 精度比较: every linear of the block quantized)
 * with one scale re-layout launch for all A operands and one GEMM launch per
 * 72 problems, the problems' 128 x 256 output tiles shared out over the SMs.
 * Same arithmetic as qz_gemm_nvfp4. Shapes per problem: 1 <= M <= 128,
 * N % 256 == 0, K % 256 == 0. count <= 256. Alignment: codes, prepared scales
 * and Y 16 B, sA 4 B. ws: qz_workspace_size(QZ_OP_GEMM_NVFP4_GROUPED, count,
 * largest K, 0) bytes. */
qz_status qz_gemm_nvfp4_grouped(const qz_nvfp4_problem* problems, int count, void* ws, size_t ws_bytes,
                                void* stream);

/* -------------------------------------------- variants (zero points, KV, INT8) */

/* FP8 KV-cache write with one scale per (batch, head) for K and for V
 * ("量化部署实战", KV Cache 量化: per_head, the amax over the head's T x D
 * values; calibrated scales per 实际部署时):
 *   scale[b, h] = max(amax over k[b, h, :, :], 1e-12) / 448; code = E4M3(x / scale)
 * k, v: bf16 [B, H, T, D] contiguous; codes: n bytes each; k_scale, v_scale:
 * fp32 [B, H] (device). mode COMPUTE writes the scales and needs
 * qz_workspace_size(QZ_OP_KV_WRITE_FP8_PER_HEAD, B*H, T*D, 0) bytes of ws; mode
 * GIVEN reads them (finite, > 0) and needs no workspace.
 * Shapes: B, H, T >= 1, D % 8 == 0. Alignment: k, v 16 B; codes 8 B. */
qz_status qz_kv_write_fp8_per_head(const uint16_t* k, const uint16_t* v, int B, int H, int T, int D,
                                   uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* v_scale,
                                   qz_scale_mode mode, void* ws, size_t ws_bytes, void* stream);

/* FP8 KV-cache write with K per channel and a zero point, V per token
 * ("量化部署实战", KV Cache 量化: K carries a constant bias per channel plus a
 * small variation; quantizing K per channel with a zero point absorbs the bias,
 * and the KIVI split quantizes K per channel and V per token; "LLM 推理优化 ·
 * 量化学习笔记" 5.1: asymmetric quantization adds a zero point). The codes stay
 * E4M3, so the zero point lives in value space. For each channel (b, h, d), over
 * its T tokens:
 *   z = fl(0.5 * fl(max + min));  s = max(max_t |fl(x - z)|, 1e-12) / 448
 *   k_code = E4M3(clamp(fl(x - z) / s, +-448)); dequant = fl(fl(value * s) + z)
 * and for each token (b, h, t): v_scale = max(amax over its D values, 1e-12) / 448,
 * v_code = E4M3(v / v_scale).
 * k_scale, k_zero: fp32 [B, H, D]; v_scale: fp32 [B, H, T]; codes [B, H, T, D].
 * ws: qz_workspace_size(QZ_OP_KV_WRITE_FP8_CHANNEL_ZP, B*H, T, D) bytes.
 * Shapes: B, H, T >= 1, D one of 8, 16, 32, 64, 128, 256. Alignment: k, v 16 B,
 * codes 8 B. */
qz_status qz_kv_write_fp8_channel_zp(const uint16_t* k, const uint16_t* v, int B, int H, int T, int D,
                                     uint8_t* k_codes, uint8_t* v_codes, float* k_scale, float* k_zero,
                                     float* v_scale, void* ws, size_t ws_bytes, void* stream);

/* INT4 weight quantization with a zero point: unsigned codes 0..15, one bf16
 * scale and one integer zero point per group of 128 along K ("量化部署实战",
 * 格式速查: W4A16, a scale per 128 "+ 零点"; "LLM 推理优化 · 量化学习笔记" 5.1:
 * q = clamp(round(x / s) + z, ...)). Per group and column the range is widened
 * to include 0 (lo = min(min, 0), hi = max(max, 0)):
 *   s = bf16_rne(max(hi - lo, 1e-12) / 15);  z = clamp(rint(-lo / s), 0, 15)
 *   q = clamp(rint(w / s) + z, 0, 15);         dequant = (q - z) * s
 * qweight: int32 [K/8, N], element k in bits 4*(k%8)..+3 (unsigned);
 * scale_bf16: [K/128, N]; zero: uint8 [K/128, N]; dequant nullable fp32 [K, N].
 * Shapes: K % 128 == 0, N % 64 == 0. Alignment as qz_quantize_int4_g128. */
qz_status qz_quantize_int4_g128_zp(const void* w, qz_dtype wt, int64_t K, int64_t N, int64_t ldw,
                                   int32_t* qweight, uint16_t* scale_bf16, uint8_t* zero, float* dequant,
                                   void* stream);

/* W4A16 GEMM with zero points (the fused unpack + dequant + matmul of
 * "量化：让每一步搬更少的字节", 路线一, on the codes of qz_quantize_int4_g128_zp):
 *   Y[m, n] = bf16_rne( sum_g s[g, n] * sum_{k in g} A[m, k] * (q[k, n] - z[g, n]) )
 * fp32 accumulation. Shapes: 1 <= M <= 16, K % 128 == 0, N % 64 == 0.
 * Alignment: A, qweight, scale, Y 16 B; zero 4 B. */
qz_status qz_gemm_w4a16_zp(const uint16_t* A, const int32_t* qweight, const uint16_t* scale_bf16,
                           const uint8_t* zero, uint16_t* Y, int M, int N, int K, void* stream);

/* Weight-only FP4 GEMMs ("量化部署实战", 精度比较: W4A16 NVFP4 and W4A16
 * MXFP4): bf16 activations times FP4 weights given as B^T [N, K] exactly as the
 * FP4 quantizers write them, fp32 accumulation, bf16 output:
 *   NVFP4: Y[m, n] = bf16_rne( gB * sum_k A[m, k] * e2m1(q[n, k]) * e4m3(s[n, k/16]) )
 *   MXFP4: Y[m, n] = bf16_rne( sum_k A[m, k] * e2m1(q[n, k]) * 2^(e[n, k/32] - 127) )
 * qB: [N, K/2]; sB: E4M3 [N, K/16]; gB: fp32 device scalar; eB: E8M0 [N, K/32].
 * MXFP4 scale codes must lie in 66..192 (scales 2^-61 .. 2^65).
 * Shapes: 1 <= M <= 16, K % 128 == 0, N % 32 == 0. Alignment: A, qB, Y 16 B;
 * sB 2 B. */
qz_status qz_gemm_w4a16_nvfp4(const uint16_t* A, const uint8_t* qB, const uint8_t* sB, const float* gB,
                              uint16_t* Y, int M, int N, int K, void* stream);
qz_status qz_gemm_w4a16_mxfp4(const uint16_t* A, const uint8_t* qB, const uint8_t* eB,
                              uint16_t* Y, int M, int N, int K, void* stream);

/* Per-column amax of x[rows, cols] (the per-channel statistic of SmoothQuant,
 * "量化：让每一步搬更少的字节", 路线二: max|X_j| over the tokens, max|W_j| over
 * the output channels of a weight stored as B^T): out[c] = max_r |x[r, c]|.
 * ws: qz_workspace_size(QZ_OP_COL_AMAX, rows, cols, 0) bytes.
 * Shapes: rows >= 1, cols % 8 == 0. Alignment: x, out 16 B. */
qz_status qz_col_amax(const void* x, qz_dtype xt, int64_t rows, int64_t cols, float* out, void* ws,
                      size_t ws_bytes, void* stream);

/* SmoothQuant migration factors ("量化：让每一步搬更少的字节", 路线二:
 * s_j = max|X_j|^a / max|W_j|^(1-a), a = 0.5 for most models):
 *   s[j] = fl(sqrt(max(x_amax[j], 1e-12))) / fl(sqrt(max(w_amax[j], 1e-12)))
 * alpha must be 0.5 (QZ_ERR_UNSUPPORTED otherwise). n >= 1. */
qz_status qz_smooth_factors(const float* x_amax, const float* w_amax, int64_t n, float alpha, float* s,
                            void* stream);

/* INT8 quantization per row ("量化部署实战", 格式速查: W8A8 INT8, integers
 * -128..127, per token for activations and per output channel for weights;
 * "量化：让每一步搬更少的字节", 量化在做什么: s = amax / 127), after the optional
 * SmoothQuant factor of each column (op DIVIDE for activations, MULTIPLY for
 * a weight stored as B^T [N, K]; factors nullable for op NONE):
 *   x' = fl(x / f[c]) or fl(x * f[c]);  s = max(amax_row(x'), 1e-12) / 127
 *   q = clamp(rint(x' / s), -128, 127);  dequant = q * s
 * codes int8 [rows, cols]; scales fp32 [rows]; dequant nullable fp32.
 * Shapes: cols % 8 == 0. Alignment: x, factors, dequant 16 B; codes 8 B. */
qz_status qz_quantize_int8_rows(const void* x, qz_dtype xt, int64_t rows, int64_t cols, const float* factors,
                                qz_smooth_op op, int8_t* codes, float* scales, float* dequant, void* stream);

/* INT8 W8A8 GEMM ("量化：让每一步搬更少的字节", 路线二):
 *   Y[i, j] = bf16_rne( sA[i] * sB[j] * sum_k qA[i, k] * qB[j, k] )
 * qA int8 [M, K], qB int8 [N, K] (B^T), sA fp32 [M], sB fp32 [N]; the integer
 * products are summed exactly while |sum| < 2^24 (fp16 tensor cores on the
 * widened codes, fp32 accumulation). Shapes: M % 128 == 0, N % 256 == 0,
 * K % 64 == 0. Alignment: all pointers 16 B. */
qz_status qz_gemm_int8(const int8_t* qA, const float* sA, const int8_t* qB, const float* sB, uint16_t* Y,
                       int M, int N, int K, void* stream);

/* FP8 block-scaled GEMM whose epilogue also quantizes its output for the next
 * layer ("量化部署实战", 练习 2: the activation's (1, 128) scales are computed at
 * the end of the previous kernel, avoiding another read and write): the same
 * arithmetic as qz_gemm_fp8_block, then each row's 128-column groups of the
 * bf16 output y are quantized exactly as qz_quantize_fp8(GROUP_1x128) would:
 *   y_scale = max(amax(y_group), 1e-12) / 448;  y_code = E4M3(y / y_scale)
 * y_codes: [M, N] bytes; y_scales: fp32 [M, N/128]; Y (bf16 [M, N]) nullable:
 * stored too when given. Shapes, layouts and alignment as qz_gemm_fp8_block. */
qz_status qz_gemm_fp8_block_quant(const uint8_t* qA, const float* sA, const uint8_t* qB, const float* sB,
                                  uint16_t* Y, uint8_t* y_codes, float* y_scales, int M, int N, int K,
                                  void* stream);

/* NVFP4 GEMM whose epilogue quantizes its output to NVFP4 for the next layer
 * ("量化部署实战", 练习 2: activation scales computed at the end of the previous
 * kernel; 格式速查: NVFP4, E2M1 + E4M3 per 16 + fp32 per tensor). The same
 * arithmetic as qz_gemm_nvfp4 up to the bf16 output y, which is then encoded
 * exactly as qz_quantize_nvfp4(y, global_amax_in = y_amax) would:
 *   g = max(*y_amax, 1e-12) / 2688 (written to y_global);
 *   per 16 columns: s_code = E4M3(amax16 / 6 / g), s = max(e4m3(s_code), 1e-12) * g,
 *   codes = E2M1(y / s).
 * The tensor amax is the caller's (a calibrated or previous-step value): the
 * kernel cannot know the output's own amax before every tile is done. Blocks
 * whose amax exceeds it saturate as in the quantizer.
 * y_codes: [M, N/2] bytes (16 B aligned); y_scales: E4M3 [M, N/16] (8 B aligned);
 * y_amax, y_global: one fp32 each (device). No bf16 output is written. Other
 * shapes, layouts, workspace and alignment as qz_gemm_nvfp4. */
qz_status qz_gemm_nvfp4_quant(const uint8_t* qA, const uint8_t* sA, const float* gA,
                              const uint8_t* qB, const uint8_t* sB, const float* gB,
                              const float* y_amax, uint8_t* y_codes, uint8_t* y_scales, float* y_global,
                              int M, int N, int K, void* ws, size_t ws_bytes, void* stream);

/* MXFP4 GEMM whose epilogue quantizes its output to MXFP4 for the next layer
 * (as qz_gemm_nvfp4_quant; 格式速查: MXFP4, E2M1 + an E8M0 scale per 32). The
 * same arithmetic as qz_gemm_mxfp4 up to the bf16 output y, then encoded
 * exactly as qz_quantize_mxfp4(y) would: per 32 columns,
 * scale = 2^(floor(log2 max(amax32, 1e-12)) - 2), codes = E2M1(y / scale).
 * No tensor amax is needed. y_codes: [M, N/2] bytes (16 B aligned); y_e8m0:
 * [M, N/32] (4 B aligned). No bf16 output is written. Other shapes, layouts,
 * workspace and alignment as qz_gemm_mxfp4. */
qz_status qz_gemm_mxfp4_quant(const uint8_t* qA, const uint8_t* eA, const uint8_t* qB, const uint8_t* eB,
                              uint8_t* y_codes, uint8_t* y_e8m0, int M, int N, int K,
                              void* ws, size_t ws_bytes, void* stream);

/* NVFP4 GEMM that allocates nothing and takes no workspace. (The quantization
 * pages have no counterpart: this is an interface convenience of this library.)
 * Some callers cannot call cudaMalloc or hand this library a workspace: runtimes
 * whose device memory is planned once at start-up and parcelled out by their own
 * arena (plug-ins get no allocator), and latency-critical loops that must not
 * risk cudaMalloc/cudaFree synchronising the device or failing mid-step. This
 * call computes exactly what qz_gemm_nvfp4 computes, with the same arguments
 * minus ws/ws_bytes; its scratch (the scale factors re-laid for the tensor
 * cores) lives in a fixed device array of QZ_NVFP4_NOALLOC_SCRATCH_BYTES that
 * the library defines, which every GPU that loads the library holds until the
 * process exits.
 * Limit: round_up(M*K/16, 1024) + round_up(N*K/16, 1024) must not exceed
 *   QZ_NVFP4_NOALLOC_SCRATCH_BYTES (4 MiB: e.g. M + N <= 16384 at K = 4096);
 *   larger sizes return QZ_ERR_SHAPE and launch nothing.
 * Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture on the device. The address belongs to the
 *   device's primary context (the CUDA runtime's); it is not looked up again,
 *   so it is stale after cudaDeviceReset or under another context.
 * Sharing: every call uses the same array and leaves its last contents there;
 *   nothing in it needs to start at zero (each call writes every byte it later
 *   reads). Calls whose executions overlap on the GPU (different streams, no
 *   ordering between them) race on the array and must be serialised by the
 *   caller. Other rules, layouts and errors: as qz_gemm_nvfp4. */
#define QZ_NVFP4_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)
qz_status qz_gemm_nvfp4_noalloc(const uint8_t* qA, const uint8_t* sA, const float* gA,
                                const uint8_t* qB, const uint8_t* sB, const float* gB,
                                uint16_t* Y, int M, int N, int K, void* stream);

/* ------------------------------------------------- paged FP8 KV cache
 * A cache of pages of page_size tokens: E4M3 codes [num_pages, heads, page_size,
 * head_dim] for K and for V and one fp32 scale per (page, head) of each
 * ("量化部署实战", KV Cache 量化: FP8 codes with a scale per head; here per head
 * and block of tokens). The value of a code is E4M3value(code) * scale. */
typedef struct qz_paged_kv {
    uint8_t* k_codes;         /* 16 B aligned */
    uint8_t* v_codes;
    float* k_scale;           /* [num_pages, heads], dense */
    float* v_scale;
    int64_t page_stride;      /* bytes from one page to the next in k_codes and in v_codes:
                                 >= heads * page_size * head_dim, a multiple of 16 */
    int num_pages;            /* num_pages * page_size < 2^31 */
    int page_size;            /* 16, 32, 64 or 128 */
    int heads;                /* KV heads, 1..32767 */
    int head_dim;             /* 64 or 128 */
} qz_paged_kv;

/* Block tables and slot maps of one step, from the requests' lengths. Request b
 * holds ctx_lens[b] tokens and gets new_lens[b] more (negative lengths count as
 * 0). With have = ceil(ctx / page_size), want = ceil((ctx + new) / page_size) and
 * need = want - have (0 where want > max_blocks: refused), pages are taken from
 * free_pages in request order, from entry *free_head on: request b is admitted if
 * want <= max_blocks and (need == 0 or *free_head + need[0] + ... + need[b] <= n_free).
 *   block_table[b, have .. want-1] <- the pages taken (admitted requests; the rest
 *     of the table is left as it is; row stride ld_table >= max_blocks)
 *   cu_new[B + 1]   exclusive sums of new_lens (tokens of a step are packed)
 *   kv_lens[b]      ctx + new, or ctx where refused
 *   slot_map[t]     page * page_size + offset of token t, -1 where its request was
 *                   refused, where its page is negative or its slots would pass 2^31,
 *                   and for t past the last token (padding of a fixed-size step)
 *   positions[t]    position of token t in its request (nullable; 0 in the padding)
 *   free_head_out   the first entry of free_pages still free
 * n_slots: entries of slot_map and positions; tokens past it are not mapped, but
 * their pages are taken. Sums of lengths and of pages must stay below 2^31. Apart
 * from block_table, outputs must not overlap inputs. B = 0 writes cu_new[0],
 * free_head_out and the padding. Shapes: page_size 16, 32, 64 or 128. */
qz_status qz_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int B, int page_size,
                          int32_t* block_table, int max_blocks, int64_t ld_table,
                          const int32_t* free_pages, int n_free, const int32_t* free_head,
                          int32_t* kv_lens, int32_t* cu_new, int32_t* slot_map, int32_t* positions, int n_slots,
                          int32_t* free_head_out, void* stream);

/* Write of new tokens into the cache. k, v: [tokens, heads, head_dim] of type xt,
 * rows ldk and ldv elements apart (>= heads * head_dim; the heads of a token dense).
 * slot_map[t]: token t's slot, as qz_block_tables gives it; slots outside the cache
 * are skipped. The tokens of a page follow one another in slot_map, and no page is
 * named by two such runs. Per page and head, for K and for V:
 *   f = max(amax over the new tokens, 1e-12) / 448
 *   first new offset 0: s = f; otherwise s = max(scale, f), and where that is larger
 *   than scale the older codes c (offsets below it) become E4M3(clamp(x / s)) of
 *   x = fl(E4M3value(c) * scale), the value they stood for
 *   code = E4M3(clamp(x / s, +-448)); scale = s
 * so a page's values never saturate whatever order they came in. Alignment: k, v 16 B,
 * ldk and ldv multiples of 16 bytes. No workspace. tokens == 0 is a no-op. */
qz_status qz_kv_append_fp8_paged(const void* k, const void* v, qz_dtype xt, int64_t tokens, int64_t ldk, int64_t ldv,
                                 const int32_t* slot_map, const qz_paged_kv* cache, void* stream);

/* Attention over the cache. Tokens cu_q[b] .. cu_q[b+1]-1 of q are request b's, its
 * keys and values the first kv_lens[b] tokens of the pages block_table[b, :]. Query
 * head a reads KV head a / (heads_q / heads). With n = cu_q[b+1] - cu_q[b], L = kv_lens[b]:
 *   x[i, j] = sm_scale * sum_d q[i, d] * K[j, d]
 *   seen: j < L, and for causal j <= L - n + i (the last query sees every key)
 *   O[i] = sum_j softmax_j(x[i, j]) V[j];  lse[i] = ln sum_j exp(x[i, j])
 * A row that sees nothing gives O = 0 and lse = -inf. Not causal: a cross
 * attention to states of another length.
 * Numerics: q enters as two E4M3 parts, exact for elements above 2^-10 of their row's amax
 * and off by at most 2^-17 of it below; requests of few rows a KV head (n * heads_q / heads,
 * up to 32) as f16 instead, exact down to 2^-29 of the amax. Sums are fp32. The
 * probabilities are rounded to f16 before they meet V (11 bits; one whose product with its
 * value scale is below 2^-31 of the row's largest may be lost). O is rounded once to bf16.
 * q: bf16 [tokens, heads_q, head_dim], rows ldq elements apart; out: bf16, rows ldo
 * apart; lse: nullable fp32 [tokens, heads_q]. Rows of no request are not written.
 * max_q: the largest n; longer requests are cut off there. Entries of block_table past a
 * request's pages are not read; entries outside the cache count as keys that are not seen.
 * What lies in a page behind the last token may hold any codes.
 * A value scale of magnitude 2^-80 or less counts as 0, whatever the codes under it; other
 * negative ones and infinite ones as NaN. Key scales may have either sign; an infinite one counts as NaN. A NaN
 * scale or code makes every row NaN that sees its key and may do so to other rows of its
 * request and KV head, but to none of another request. Inf or NaN in a row of q makes
 * that row NaN where it sees a key, and no other row.
 * Shapes: heads_q % heads == 0, heads_q / heads <= 256, max_blocks * page_size < 2^31.
 * Alignment: q, out 16 B, ldq, ldo multiples of 8.
 * ws: qz_workspace_size(QZ_OP_ATTN_FP8_PAGED, max_q * heads_q / heads, head_dim, 0). */
qz_status qz_attn_fp8_paged(const uint16_t* q, int64_t ldq, int64_t tokens, int heads_q, const int32_t* cu_q, int B,
                            int max_q, const qz_paged_kv* cache, const int32_t* block_table, int max_blocks,
                            int64_t ld_table, const int32_t* kv_lens, float sm_scale, int causal, uint16_t* out,
                            int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------- a block of experts in FP8
 * What a decoder block of experts needs around the products that quantized weights are
 * for: the choice of experts and the order of their rows (qz_moe_route), the products
 * over those rows (qz_moe_gemm_fp8_swiglu, qz_moe_gemm_fp8), and the residual norm that
 * joins the experts' rows by their gates and encodes the next product's input
 * (qz_residual_rmsnorm). None of them needs a count on the host, so a step can be
 * captured into a CUDA graph and replayed with other routings. */

typedef enum qz_score {
    QZ_SCORE_SOFTMAX = 0,     /* s = softmax over the token's experts */
    QZ_SCORE_SIGMOID = 1      /* s = 1 / (1 + exp(-l))                */
} qz_score;

typedef struct qz_moe_routing {
    int experts;              /* 1..512 */
    int top_k;                /* 1..16, <= top_groups * experts / groups */
    qz_score score;
    int renormalize;          /* 1: the chosen scores are divided by their sum */
    float scale;              /* finite factor of the weights */
    int groups;               /* divides experts, 1..32; experts of a group are consecutive */
    int top_groups;           /* 1..groups */
    int group_best;           /* 1 or 2 (<= experts / groups): how many of its best keys make a group's score */
} qz_moe_routing;

/* Routing of tokens to experts. logits: [tokens, experts] of type lt, rows ldl elements
 * apart. A NaN logit counts as -inf, +inf as the largest fp32 value. For token t:
 *   s[e] the score of expert e;  key[e] = s[e] + bias[e] (bias: nullable fp32 [experts])
 *   experts with logit -inf, or with bias NaN or -inf, are closed (a bias of +inf counts as the
 *   largest fp32 value)
 *   groups > 1: a group's score is the sum of the group_best largest keys of its open experts (of
 *   as many as there are); experts outside the best top_groups groups are closed
 *   ids[t, :] = the top_k open experts by key, in descending order (without bias by logit,
 *   which orders them alike); ties, of groups too, go to the lowest index
 *   weights[t, j] = scale * s[ids[t, j]], divided by the sum over j where renormalize is set
 * Keys are compared as in 64 bits, where 32 would decide otherwise too; weights are fp32 throughout, good to
 * some units of 2^-24. Where fewer than top_k experts are open, the rest of the token's ids is -1 with weight 0.
 * n_tokens: nullable device int32; tokens from *n_tokens on are padding of a fixed-size step:
 * all their ids are -1.
 * The plan of the products: the pairs (t, j) with ids[t, j] = e have the rows offsets[e] ..
 * offsets[e + 1] - 1, in the order of t. offsets: [experts + 1]; row_token[r] = t (-1 from row
 * offsets[experts] on); token_row[t, j] = r (-1 where ids is).
 * ids, weights, token_row: [tokens, top_k]; row_token: [tokens * top_k].
 * Shapes: tokens * top_k < 2^31. Alignment: logits its element size, the others 4 B.
 * ws: qz_workspace_size(QZ_OP_MOE_ROUTE, tokens, experts, top_k). tokens == 0 writes offsets. */
qz_status qz_moe_route(const void* logits, qz_dtype lt, int64_t tokens, int64_t ldl, const float* bias,
                       const int32_t* n_tokens, const qz_moe_routing* routing, int32_t* ids, float* weights,
                       int32_t* offsets, int32_t* row_token, int32_t* token_row, void* ws, size_t ws_bytes, void* stream);

/* The experts' products, block-scaled FP8 as qz_gemm_fp8_block ("量化部署实战", 练习 2). Row r
 * with offsets[e] <= r < offsets[e + 1] is multiplied by the weight of expert e:
 *   P[r, n] = sum_kb sA[a, kb] * sW[e, n/128, kb] * sum_{k in kb} qA[a, k] * qW[e, n, k],
 *   a = row_token[r], or r where row_token is NULL;  fp32 accumulation
 * qz_moe_gemm_fp8:        Y[r, :] = bf16_rne(P[r, :]), Y bf16 [rows, N]
 * qz_moe_gemm_fp8_swiglu: N = 2 I, rows 0 .. I-1 of a weight are the gate's, the others the up
 *   projection's: h = g * u / (1 + exp(-g)) with g = P[r, i], u = P[r, I + i] in fp32, encoded as
 *   qz_quantize_fp8(GROUP_1x128) encodes h: y_codes [rows, I], y_scales fp32 [rows, I/128]. h is good to 10 * 2^-24
 *   of itself for any g (exp and the quotient are the GPU's approximations, corrected), 0 where exp(-g) passes 2^126
 * qA: E4M3 [tokens, K], sA: fp32 [tokens, K/128] (qz_quantize_fp8 GROUP_1x128, or
 * qz_residual_rmsnorm). qW: E4M3 [experts, N, K], sW: fp32 [experts, N/128, K/128]
 * (qz_quantize_fp8 BLOCK_128x128 on the weights as one tensor of experts * N rows).
 * offsets: device int32 [experts + 1], ascending, as qz_moe_route writes them; what lies outside
 * 0 .. rows is cut off. Rows of no expert are not written. A row whose row_token lies outside
 * 0 .. tokens-1 is a row of zeros. A NaN in a row of qA or sA reaches that row alone.
 * The same call gives the same bits. With more than 32 rows a row's bits depend on its own inputs alone; with up to 32
 * several CTAs may share its K, and its sums then have another order than in a call of other sizes.
 * Shapes: experts 1..512, rows and tokens < 2^31, experts * N < 2^31, K % 128 == 0, N % 128 == 0 (I % 128 == 0).
 * Alignment: qA, qW, outputs 16 B, the others 4 B. rows == 0 is a no-op. No workspace. */
qz_status qz_moe_gemm_fp8(const uint8_t* qA, const float* sA, int64_t tokens, const int32_t* row_token, int64_t rows,
                          const int32_t* offsets, int experts, const uint8_t* qW, const float* sW, uint16_t* Y, int N,
                          int K, void* stream);
qz_status qz_moe_gemm_fp8_swiglu(const uint8_t* qA, const float* sA, int64_t tokens, const int32_t* row_token,
                                 int64_t rows, const int32_t* offsets, int experts, const uint8_t* qW, const float* sW,
                                 uint8_t* y_codes, float* y_scales, int I, int K, void* stream);

/* What a block adds to the residual stream (qz_residual_rmsnorm). */
typedef struct qz_block_output {
    const uint16_t* y;        /* bf16 [rows, hidden], rows ldy elements apart */
    int64_t rows, ldy;
    int k;                    /* rows of y per token, 1..16 */
    const int32_t* token_row; /* [tokens, k]: their places in y, those outside 0 .. rows-1 add nothing; NULL:
                                 token t has the rows t*k .. t*k + k-1 */
    const float* weights;     /* nullable fp32 [tokens, k]: the gates */
    float alpha;              /* finite scale of the block's output */
    const void* gamma;        /* nullable [hidden], of x's type: norm of the block's output */
} qz_block_output;

/* Residual, norm and quantization around a block, in one pass:
 *   z[t] = sum_j weights[t, j] * y[token_row[t, j]];  with block->gamma: z *= block->gamma / sqrt(mean(z^2) + eps)
 *   r = x + alpha * z (r = x where block is NULL);  n = r * gamma / sqrt(mean(r^2) + eps)
 * x: [tokens, hidden] of type xt, rows ldx elements apart. x_out: nullable, r in xt, rows ldo
 * apart; it may be x itself (but nothing else that the call reads). gamma: nullable [hidden] of type xt; without
 * it there are no n and no codes. normed: nullable, n in bf16, dense. codes, scales: nullable together, n as
 * qz_quantize_fp8(GROUP_1x128) encodes it: [tokens, hidden] and fp32 [tokens, hidden/128].
 * All sums are fp32 and n, its codes and x_out come from the unrounded fp32 r, each rounded once. A row of r whose sum of
 * squares passes fp32's range gives n = 0, one with infinities the same but NaN in their places, one with a NaN
 * gives NaN; none of them reaches another row.
 * Shapes: hidden % 8 == 0, 8..16384; hidden % 128 == 0 with codes. eps finite, > 0. tokens < 2^31; tokens == 0 is a no-op.
 * Alignment: x, x_out, y, gammas, normed, codes 16 B, ldx, ldo, ldy multiples of 16 bytes, the others 4 B. */
qz_status qz_residual_rmsnorm(const void* x, qz_dtype xt, int64_t tokens, int hidden, int64_t ldx,
                              const qz_block_output* block, void* x_out, int64_t ldo, const void* gamma, float eps,
                              uint16_t* normed, uint8_t* codes, float* scales, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QZ_H */
