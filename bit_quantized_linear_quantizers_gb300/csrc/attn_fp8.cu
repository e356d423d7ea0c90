// attn_fp8.cu -- attention over the paged FP8 KV cache: which kernel takes which
// request. The lengths are on the device, so the choice is made there, by the
// query rows per KV head (tokens x heads of the group): both kernels look at every
// request and skip the other's.
#include "qz_internal.cuh"
#include "qz_paged.cuh"

namespace qz {

namespace {
// Rows per KV head up to which a request takes the decode kernel, which reads the
// keys once per 16 rows; the prefill kernel reads them once per 256 but computes
// 128 rows at least. Measured, decode against prefill kernel, 8 KV heads of 128, 4096 keys
// and more: 32 requests of 32 rows 119 against 131 us, of 64 rows 226 against 131, of
// 128 rows 432 against 134; one request of 32 rows 20.1 against 23.1, of 64 rows 20.9
// against 23.1, of 128 rows 27.5 against 23.6.
constexpr int kDecodeRows = 32;

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
} // namespace

// The two kernels of a call may overlap: a workspace each.
size_t ws_attn_paged(int64_t rows, int64_t) {
    return rows <= kDecodeRows ? ws_attn_decode() : round256(ws_attn_decode()) + ws_attn_prefill();
}

qz_status attn_paged_launch(const AttnArgs& a, void* ws, cudaStream_t st) {
    const int64_t rows = (int64_t)a.max_q * (a.heads_q / a.kv.heads);
    if (rows <= kDecodeRows) return attn_decode_launch(a, kDecodeRows, false, ws, st);
    void* ws2 = static_cast<char*>(ws) + round256(ws_attn_decode());
    bool joined = false;
    if (a.B == 1) return attn_prefill_launch(a, 1, ws2, &joined, st);     // one request: no second launch for what it is not
    QZ_TRY(attn_prefill_launch(a, kDecodeRows + 1, ws2, &joined, st));
    return attn_decode_launch(a, kDecodeRows, !joined, ws, st);
}

} // namespace qz
