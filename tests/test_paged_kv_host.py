"""The paged FP8 KV cache's refusals, on the CPU: host validation behind the C ABI (every call carries an
invalid argument or nothing to do, so none can launch) and the binding's own checks."""
import ctypes

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qzm

FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
NULL = None


@pytest.fixture(scope="module")
def qz():
    return qzm


def _cache(qz, **kw):
    c = dict(k_codes=0x10000, v_codes=0x10000, k_scale=0x10000, v_scale=0x10000, page_stride=8 * 16 * 128, num_pages=4,
             page_size=16, heads=8, head_dim=128)
    c.update(kw)
    return ctypes.byref(qz._PagedKV(**c))


BAD_CACHES = [(dict(k_codes=0), 1), (dict(v_scale=0), 1), (dict(num_pages=0), 1), (dict(heads=0), 1),
              (dict(page_stride=8 * 16 * 128 - 16), 1), (dict(page_size=24), 2), (dict(head_dim=96), 2),
              (dict(num_pages=1 << 27), 2), (dict(heads=40000, page_stride=1 << 40), 2), (dict(k_codes=0x10008), 3),
              (dict(page_stride=8 * 16 * 128 + 8), 3), (dict(k_scale=0x10002), 3)]


def test_block_tables_validation(qz):
    f = qz.lib.qz_block_tables
    # ctx, new, B, page, table, max_blocks, ld, free, n_free, head, kv, cu, slots, pos, n_slots, head_out, stream
    ok = [FAKE, FAKE, 2, 16, FAKE, 4, 4, FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE, 2, FAKE, NULL]

    def call(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i, v, want in [(0, NULL, 1), (1, NULL, 1), (2, -1, 1), (3, 8, 2), (3, 48, 2), (4, NULL, 1), (5, -1, 1), (6, 3, 1),
                       (7, NULL, 1), (8, -1, 1), (9, NULL, 1), (10, NULL, 1), (11, NULL, 1), (12, NULL, 1), (14, -1, 1),
                       (15, NULL, 1), (0, ODD, 3), (12, ODD, 3), (15, ODD, 3)]:
        assert call(i, v) == want, (i, v)
    big = list(ok)
    big[5], big[6] = 1 << 27, 1 << 27
    assert f(*big) == 2


def test_paged_append_validation(qz):
    f = qz.lib.qz_kv_append_fp8_paged
    row = 8 * 128
    # k, v, dtype, tokens, ldk, ldv, slots, cache, stream
    for bad, want in BAD_CACHES:
        assert f(FAKE, FAKE, 1, 4, row, row, FAKE, _cache(qz, **bad), NULL) == want, bad
    c = _cache(qz)
    assert f(FAKE, FAKE, 1, 4, row, row, FAKE, None, NULL) == 1
    assert f(FAKE, FAKE, 2, 4, row, row, FAKE, c, NULL) == 1
    assert f(FAKE, FAKE, 1, -1, row, row, FAKE, c, NULL) == 1
    assert f(FAKE, FAKE, 1, 0, row, row, FAKE, c, NULL) == 0
    assert f(NULL, FAKE, 1, 4, row, row, FAKE, c, NULL) == 1
    assert f(FAKE, FAKE, 1, 4, row, row, NULL, c, NULL) == 1
    assert f(FAKE, FAKE, 1, 4, row - 8, row, FAKE, c, NULL) == 1
    assert f(FAKE, FAKE, 1, 1 << 31, row, row, FAKE, c, NULL) == 2
    assert f(ODD, FAKE, 1, 4, row, row, FAKE, c, NULL) == 3
    assert f(FAKE, FAKE, 1, 4, row, row + 4, FAKE, c, NULL) == 3


def test_paged_attention_validation(qz):
    f = qz.lib.qz_attn_fp8_paged
    row = 32 * 128
    # q, ldq, tokens, heads_q, cu, B, max_q, cache, table, max_blocks, ld, kv, scale, causal, out, ldo, lse, ws, bytes, st
    ok = [FAKE, row, 4, 32, FAKE, 2, 2, _cache(qz), FAKE, 4, 4, FAKE, 0.1, 1, FAKE, row, NULL, FAKE, 1 << 40, NULL]

    def call(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for bad, want in BAD_CACHES:
        assert call(7, _cache(qz, **bad)) == want, bad
    for i, v, want in [(0, NULL, 1), (1, row - 8, 1), (2, -1, 1), (3, 0, 1), (3, 36, 2), (3, 8 * 257, 2), (4, NULL, 1),
                       (5, -1, 1), (6, -1, 1), (7, None, 1), (8, NULL, 1), (9, -1, 1), (10, 3, 1), (11, NULL, 1),
                       (12, float("nan"), 1), (12, float("inf"), 1), (13, 2, 1), (14, NULL, 1), (15, row - 8, 1),
                       (2, 1 << 31, 2), (0, ODD, 3), (14, ODD, 3), (1, row + 4, 3), (15, row + 4, 3), (16, ODD, 3),
                       (4, ODD, 3), (11, ODD, 3)]:
        assert call(i, v) == want, (i, v)
    for i in (2, 5, 6):                                                                # nothing to do
        assert call(i, 0) == 0


def _cpu_cache(pages=4, heads=2, page=16, dim=64):
    codes = torch.zeros((2, pages, heads, page, dim), dtype=torch.uint8)
    scales = torch.zeros((2, pages, heads))
    return codes, scales


def test_paged_cache_checks_its_tensors():
    codes, scales = _cpu_cache()
    c = qzm.PagedKV(codes[0], codes[1], scales[0], scales[1])
    assert (c.num_pages, c.heads, c.page_size, c.head_dim, c._c.page_stride) == (4, 2, 16, 64, 2 * 16 * 64)
    both = torch.zeros((4, 2, 2, 16, 64), dtype=torch.uint8)
    assert qzm.PagedKV(both[:, 0], both[:, 1], scales[0], scales[1])._c.page_stride == 4 * 16 * 64
    for bad, match in [((codes[0][0], codes[1][0], scales[0], scales[1]), "pages"),
                       ((codes[0], codes[1][:3], scales[0], scales[1]), "one shape"),
                       ((codes[0].transpose(1, 2), codes[1].transpose(1, 2), scales[0], scales[1]), "dense"),
                       ((codes[0].int(), codes[1], scales[0], scales[1]), "1-byte"),
                       ((both[:, 0], codes[1], scales[0], scales[1]), "stride"),
                       ((codes[0], codes[1], scales[0][:3], scales[1]), "k_scale"),
                       ((codes[0], codes[1], scales[0], scales[1].double()), "v_scale")]:
        with pytest.raises(ValueError, match=match):
            qzm.PagedKV(*bad)


def test_paged_calls_refuse_what_the_c_call_cannot_see(monkeypatch):
    monkeypatch.setattr(qzm, "_device", lambda: -1)
    codes, scales = _cpu_cache()
    c = qzm.PagedKV(codes[0], codes[1], scales[0], scales[1])
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="slot_map"):
        qzm.qz_kv_append_fp8_paged(k, k, i32(2), c)
    with pytest.raises(ValueError, match="same number"):
        qzm.qz_kv_append_fp8_paged(k, k[:2], i32(3), c)
    with pytest.raises(ValueError, match="k: expected"):
        qzm.qz_kv_append_fp8_paged(k[:, :1], k, i32(3), c)
    with pytest.raises(ValueError, match="dense"):
        qzm.qz_kv_append_fp8_paged(k, torch.zeros((3, 4, 64), dtype=torch.bfloat16)[:, ::2], i32(3), c)
    with pytest.raises(TypeError):
        qzm.qz_kv_append_fp8_paged(k.half(), k.half(), i32(3), c)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    for args, match in [((q[..., :32], c, i32(2, 3), i32(2), i32(3), 2, 0.1), "q: expected"),
                        ((q, c, i32(6), i32(2), i32(3), 2, 0.1), "block_table"),
                        ((q, c, i32(2, 3).long(), i32(2), i32(3), 2, 0.1), "block_table"),
                        ((q, c, i32(2, 3), i32(3), i32(3), 2, 0.1), "kv_lens"),
                        ((q, c, i32(2, 3), i32(2), i32(2), 2, 0.1), "cu_q")]:
        with pytest.raises(ValueError, match=match):
            qzm.qz_attn_fp8_paged(*args)
    with pytest.raises(TypeError):
        qzm.qz_attn_fp8_paged(q.float(), c, i32(2, 3), i32(2), i32(3), 2, 0.1)
    with pytest.raises(ValueError, match="out"):
        qzm.qz_attn_fp8_paged(q, c, i32(2, 3), i32(2), i32(3), 2, 0.1, out=q[:2])
    with pytest.raises(ValueError, match="lse"):
        qzm.qz_attn_fp8_paged(q, c, i32(2, 3), i32(2), i32(3), 2, 0.1, lse=torch.zeros(5))
    with pytest.raises(ValueError, match="ctx_lens"):
        qzm.qz_block_tables(i32(3), i32(2), i32(2, 4), i32(9), i32(1), 16, 5)
    with pytest.raises(ValueError, match="slot_map"):
        qzm.qz_block_tables(i32(2), i32(2), i32(2, 4), i32(9), i32(1), 16, 5, slot_map=i32(4))
    monkeypatch.setattr(qzm, "_device", lambda: 0)
    with pytest.raises(ValueError, match="cache: .*on cpu"):
        qzm.qz_kv_append_fp8_paged(k, k, i32(3), c)
