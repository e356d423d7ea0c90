"""The attention call's workspace: a short, missing or misaligned one is refused before any launch (CPU)."""
import ctypes

import pytest

import bit_quantized_linear_quantizers_gb300 as qz

WORKSPACE = 7                         # QZ_ERR_WORKSPACE
FAKE = 0x10000                        # aligned, never dereferenced


@pytest.mark.parametrize("max_q", [1, 16, 17, 400])
def test_attention_workspace_is_checked(max_q):
    cache = qz._PagedKV(k_codes=FAKE, v_codes=FAKE, k_scale=FAKE, v_scale=FAKE, page_stride=8 * 16 * 128, num_pages=4,
                        page_size=16, heads=8, head_dim=128)
    heads, row = 16, 16 * 128
    need = qz.lib.qz_workspace_size(qz.OP_ATTN_FP8_PAGED, max_q * heads // 8, 128, 0)
    assert need > 0
    for ws, size in ((FAKE, need - 1), (FAKE, 0), (None, need), (FAKE + 8, need)):
        assert qz.lib.qz_attn_fp8_paged(FAKE, row, max_q, heads, FAKE, 2, max_q, ctypes.byref(cache), FAKE, 4, 4, FAKE, 0.1, 1,
                                        FAKE, row, None, ws, size, None) == WORKSPACE
