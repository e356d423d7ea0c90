"""The paged FP8 KV cache on the GPU: block tables against a loop over requests, the cache write
bit for bit against the oracle's quantizer, attention against its formula in 64 bits.

Tolerance of attention, derived from the arithmetic that include/qz.h states (x in natural units,
p the softmax, vs the scale of a value's page, c its code's value, sums over the keys j of a row):
* the two E4M3 parts of q leave at most 2^-17 of the row's amax, and the fp32 sums of D <= 128 products add at
  most as much: |dx| <= 2^-16 * |sm_scale| * amax(q) * sum_d |K_jd| + 2^-21 * |x|;
* a probability keeps 8 significant bits down to 2^-9 of the largest p * vs, with steps of at most
  2^-17 of that below it, so O is off by at most
  (2.5 * dx + 2^-8) * sum_j p_j |V_j| + 2^-17 * max_j(p_j vs_j) * sum_j |c_j| + half a bf16 ulp;
* lse: dx + 2^-18 * (1 + |lse|).
"""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import oracle
import synthetic as syn
from gpu_util import assert_same_bytes, dev_bf16, dev_f32, host

pytestmark = pytest.mark.gpu

VALUE = np.array([oracle.e4m3_decode(c) for c in range(256)], np.float64)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ block tables

def ref_tables(ctx, new, table, free, head, P, n_slots):
    table, cu, kv, slots, pos = table.copy(), [0], [], [], []
    blocks, upto, out = table.shape[1], head, head
    for b, (c, n) in enumerate(zip(ctx, new)):
        c, n = max(c, 0), max(n, 0)
        have, want = -(-c // P), -(-(c + n) // P)
        need = want - have if want <= blocks else 0
        upto += need
        ok = want <= blocks and (need == 0 or upto <= len(free))
        if ok and need:
            table[b, have:want] = free[upto - need:upto]
            out = upto
        kv.append(c + n if ok else c)
        cu.append(cu[-1] + n)
        for i in range(c, c + n):
            pos.append(i)
            slots.append(table[b, i // P] * P + i % P if ok and table[b, i // P] >= 0 else -1)
    slots = (slots + [-1] * n_slots)[:n_slots]
    pos = (pos + [0] * n_slots)[:n_slots]
    return table, np.array(slots), np.array(pos), np.array(cu), np.array(kv), out


TABLE_CASES = {
    "one token": ([0], [1], 16, 4, 4, 0, 1),
    "page edges": ([0, 15, 16, 17, 31, 32], [16, 1, 1, 15, 2, 33], 16, 8, 64, 2, 68),
    "nothing new": ([5, 0, 64], [0, 0, 0], 32, 2, 3, 1, 4),
    "negative lengths": ([-3, 4, 10], [5, -2, 3], 16, 3, 9, 0, 8),
    "padding": ([3, 100], [2, 7], 64, 4, 9, 3, 40),
    "fewer slots than tokens": ([3, 100], [20, 70], 16, 12, 30, 0, 50),
    "list runs out": ([0, 10, 5, 128, 3], [40, 200, 1, 1, 300], 32, 40, 9, 1, 542),
    "table too narrow": ([10, 60, 7], [90, 10, 3], 16, 5, 30, 0, 103),
    "list used up": ([16, 3, 15], [1, 1, 1], 16, 4, 2, 2, 3),
    "no requests": ([], [], 16, 4, 5, 3, 6),
}


@pytest.mark.parametrize("name", TABLE_CASES)
def test_block_tables(name):
    check_tables(*TABLE_CASES[name])


@pytest.mark.parametrize("B, P", [(1, 128), (333, 16), (1024, 64), (1025, 32), (2500, 16)])
def test_block_tables_many_requests(B, P):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 300, B), rng.integers(0, 70, B) * rng.integers(0, 2, B)
    need = int(np.sum(-(-(ctx + new) // P) + ctx // -P))
    check_tables(ctx.tolist(), new.tolist(), P, 400 // P + 1, max(1, need * 9 // 10), 0, int(new.sum()) + 5)


def check_tables(ctx, new, P, blocks, n_free, head, n_slots):
    B = len(ctx)
    rng = np.random.default_rng(P)
    pages = rng.permutation(2 * n_free + B * blocks + 1).astype(np.int32)
    free, rest = pages[:n_free], pages[n_free:]
    wide = np.full((B, blocks + 3), -7, np.int32)            # rows further apart than they are long
    for b in range(B):
        have = min(-(-max(ctx[b], 0) // P), blocks)
        wide[b, :have] = rest[b * blocks:b * blocks + have]
    want = ref_tables(ctx, new, wide[:, :blocks], free, head, P, n_slots)
    dwide = torch.from_numpy(wide).cuda()
    got = qz.qz_block_tables(i32(ctx), i32(new), dwide[:, :blocks], torch.from_numpy(free).cuda(), i32([head]), P, n_slots)
    slots, pos, cu, kv, out = (host(t) for t in got)
    assert np.array_equal(host(dwide)[:, :blocks], want[0]) and np.all(host(dwide)[:, blocks:] == -7)
    assert np.array_equal(slots, want[1]) and np.array_equal(pos, want[2])
    assert np.array_equal(cu, want[3]) and np.array_equal(kv, want[4]) and out[0] == want[5]


# ------------------------------------------------------------ the cache write

def new_cache(pages, H, P, D, seed=0, interleaved=False):
    """A cache whose pages hold arbitrary finite codes; also the host copy of its parts."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (pages, 2, H, P, D)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x13
    scales = (np.abs(rng.standard_normal((2, pages, H))) * 0.05 + 1e-3).astype(np.float32)
    if interleaved:                                           # K and V of a page side by side
        both = torch.from_numpy(codes).cuda()
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.from_numpy(np.ascontiguousarray(codes[:, i])).cuda() for i in (0, 1))
    cache = qz.PagedKV(k, v, torch.from_numpy(scales[0]).cuda(), torch.from_numpy(scales[1]).cuda())
    return cache, [codes[:, 0].copy(), codes[:, 1].copy()], [scales[0].copy(), scales[1].copy()]


def ref_append(x, slots, codes, scales):
    """x fp32 [T, H, D] (exact values), codes [pages, H, P, D], scales [pages, H]: in place."""
    P = codes.shape[2]
    t = 0
    while t < len(slots):
        page = slots[t] // P
        u = t + 1
        while u < len(slots) and slots[u] // P == page and u - t < P:
            u += 1
        if slots[t] >= 0 and page < codes.shape[0]:
            off = slots[t] % P
            for h in range(codes.shape[1]):
                f = np.float32(max(np.float32(np.abs(x[t:u, h]).max()), np.float32(1e-12))) / np.float32(448)
                s = f if off == 0 else max(scales[page, h], f)
                if off and s > scales[page, h]:
                    old = VALUE[codes[page, h, :off]].astype(np.float32) * scales[page, h]
                    codes[page, h, :off] = oracle.quant_fp8_given(old, s, want_deq=False)[0]
                for r in range(t, u):
                    codes[page, h, slots[r] % P] = oracle.quant_fp8_given(x[r, h][None], s, want_deq=False)[0][0]
                scales[page, h] = s
        t = u


@pytest.mark.parametrize("H, P, D, bf16, lens", [
    (2, 16, 128, True, [(0, 1)]),
    (8, 16, 128, True, [(5, 1), (16, 1), (31, 1), (0, 1)]),
    (3, 32, 64, False, [(0, 100), (7, 25), (31, 1), (64, 33), (3, 0)]),
    (1, 64, 64, True, [(63, 2), (1, 200)]),
    (2, 128, 128, False, [(127, 1), (0, 257), (100, 40)]),
    (2, 128, 64, True, [(1, 126), (128, 128)]),
    (4, 64, 128, True, [(b * 5, 1) for b in range(70)]),
    (2, 16, 64, True, [(0, 3000)]),
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_matches_the_quantizer(H, P, D, bf16, lens, interleaved):
    rng = np.random.default_rng(P + D)
    pages = sum(-(-(c + n) // P) for c, n in lens) + 3
    cache, codes, scales = new_cache(pages, H, P, D, seed=P, interleaved=interleaved)
    order, at, slots = rng.permutation(pages), 0, []
    for c, n in lens:
        mine = order[at:at + -(-(c + n) // P)]
        at += len(mine)
        slots += [int(mine[i // P]) * P + i % P for i in range(c, c + n)]
    T = len(slots)
    qkv = rng.standard_normal((T, 3 * H, D)).astype(np.float32) * np.where(np.arange(T) % 3 == 0, 30, 0.5)[:, None, None]
    qkv[T // 2] = 0.0                                         # a token of zeros (scale floor where it is alone)
    if bf16:
        bits = syn.to_bf16_bits(qkv.astype(np.float32))
        dev, qkv = dev_bf16(bits), syn.bf16_bits_to_f32(bits)
    else:
        qkv = qkv.astype(np.float32)
        dev = dev_f32(qkv)
    for _ in range(2):                                        # writing the same tokens again changes nothing
        qz.qz_kv_append_fp8_paged(dev[:, H:2 * H], dev[:, 2 * H:], i32(slots), cache)
        for i, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
            ref_append(qkv[:, (i + 1) * H:(i + 2) * H], slots, codes[i], scales[i])
            assert_same_bytes(host(s), scales[i], "scales")
            assert_same_bytes(host(c.contiguous()), codes[i], "codes")


def test_append_skips_slots_outside_the_cache():
    H, P, D = 2, 16, 64
    cache, codes, scales = new_cache(3, H, P, D)
    slots = [-1, 5, 6, -1, 3 * P, 40, -2147483648, 2147483647, 17]
    x = np.random.default_rng(0).standard_normal((len(slots), H, D)).astype(np.float32)
    qz.qz_kv_append_fp8_paged(dev_f32(x), dev_f32(x), i32(slots), cache)
    for i, (c, s) in enumerate(((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale))):
        ref_append(x, slots, codes[i], scales[i])
        assert_same_bytes(host(c), codes[i], "codes")
        assert_same_bytes(host(s), scales[i], "scales")
    qz.qz_kv_append_fp8_paged(dev_f32(x[:0]), dev_f32(x[:0]), i32([]), cache)       # nothing to write


# ------------------------------------------------------------ attention

def quantized_pages(pages, H, P, D, g, spread=0.0):
    x = torch.randn((pages, H, P, D), generator=g, device="cuda")
    x *= torch.exp(spread * torch.randn((pages, H, 1, 1), generator=g, device="cuda"))
    s = x.abs().amax(dim=(2, 3)) / torch.full((pages, H), 448.0, device="cuda")
    return (x / s[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def check_attention(lens, Hq, Hkv, D, P, causal, seed=0, q_std=1.0, spread=0.0, max_q=None, pages_extra=2, bias=0.0,
                    cache_tensors=None, page_ids=None, sm_scale=None):
    """lens: (keys, queries) per request. Compares O and lse with the formula in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, T = len(lens), sum(n for _, n in lens)
    counts = [-(-L // P) for L, _ in lens]
    blocks = max(counts + [1])
    n_pages = sum(counts) + pages_extra
    if cache_tensors is None:
        kc, ks = quantized_pages(n_pages, Hkv, P, D, g, spread)
        vc, vs = quantized_pages(n_pages, Hkv, P, D, g, spread)
        if bias:
            x = kc.view(torch.float8_e4m3fn).float() * ks[:, :, None, None] + bias * torch.randn((1, Hkv, 1, D), generator=g, device="cuda")
            ks = x.abs().amax(dim=(2, 3)) / 448.0
            kc = (x / ks[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        kc, ks, vc, vs = cache_tensors
    order = torch.randperm(n_pages, generator=g, device="cuda").tolist() if page_ids is None else page_ids
    table = torch.full((B, blocks + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
        if lens[b][0] % P:                                    # never written: NaN codes
            for x in (kc, vc):
                x[order[at - 1], :, lens[b][0] % P:] = 0x7F if b % 2 else 0xFF
    table = table.cuda()[:, :blocks]
    qkv = torch.randn((T, Hq + 2, D), generator=g, device="cuda") * q_std
    q = qkv.to(torch.bfloat16)[:, :Hq]                        # tokens further apart than dense
    cu = np.concatenate([[0], np.cumsum([n for _, n in lens])])
    mq = max([n for _, n in lens] + [1]) if max_q is None else max_q
    sm = 1 / math.sqrt(D) if sm_scale is None else sm_scale
    out = torch.full((T, Hq + 1, D), 7.0, dtype=torch.bfloat16, device="cuda")[:, 1:]
    lse = torch.full((T, Hq), 7.0, device="cuda")
    cache = qz.PagedKV(kc, vc, ks, vs)
    qz.qz_attn_fp8_paged(q, cache, table, i32([L for L, _ in lens]), i32(cu.tolist()), mq, sm, causal=causal, out=out, lse=lse)
    G = Hq // Hkv
    bad = []
    for b, (L, n) in enumerate(lens):
        pages = table[b, :counts[b]].long()
        for h in range(Hkv):
            code_k = kc[pages, h].view(torch.float8_e4m3fn).double().reshape(-1, D)[:L]
            code_v = vc[pages, h].view(torch.float8_e4m3fn).double().reshape(-1, D)[:L]
            s_k = ks[pages, h].double().repeat_interleave(P)[:L]
            s_v = vs[pages, h].double().repeat_interleave(P)[:L]
            K, V = code_k * s_k[:, None], code_v * s_v[:, None]
            i0 = np.arange(min(n, mq))
            sees = torch.from_numpy(np.arange(L)[None, :] <= (L - min(n, mq) + i0)[:, None] if causal
                                    else np.ones((len(i0), L), bool)).cuda()
            for a in range(h * G, h * G + G):
                rows = slice(int(cu[b]), int(cu[b]) + len(i0))
                qa = q[rows, a].double()
                x = (qa @ K.T * sm).masked_fill(~sees, -math.inf)
                want_lse = torch.logsumexp(x, dim=1) if L else torch.full((len(i0),), -math.inf, device="cuda", dtype=torch.float64)
                p = torch.exp(x - torch.where(torch.isinf(want_lse), 0.0, want_lse)[:, None])
                want = p @ V
                amax = qa.abs().amax(dim=1)
                dx = 2.0 ** -16 * abs(sm) * amax[:, None] * K.abs().sum(dim=1)[None] + 2.0 ** -21 * torch.where(sees, x, 0.0).abs()
                dx = torch.where(sees, dx, 0.0).amax(dim=1) if L else torch.zeros(len(i0), device="cuda", dtype=torch.float64)
                top = (p * s_v[None]).amax(dim=1) if L else dx
                ulp = torch.where(want != 0, torch.ldexp(torch.ones_like(want), torch.frexp(want)[1] - 9), 0.0)
                tol = ((2.5 * dx + 2.0 ** -8)[:, None] * (p @ V.abs())
                       + 2.0 ** -17 * top[:, None] * (sees.double() @ code_v.abs()) + ulp)
                err = (out[rows, a].double() - want).abs()
                e_lse = (lse[rows, a].double() - want_lse).abs().nan_to_num(nan=0.0)
                empty = torch.isinf(want_lse)
                ok = bool((err <= tol).all()) and bool((lse[rows, a][empty] == -math.inf).all()) \
                    and bool((e_lse[~empty] <= (dx + 2.0 ** -18 * (1 + want_lse.abs()))[~empty]).all())
                if not ok:
                    bad.append((b, a, float((err - tol).max()), float(err.max()), float(e_lse.max())))
    assert not bad, f"{len(bad)} (request, head) pairs outside the tolerance: {bad[:5]}"
    assert qz.qz_device_error() == 0
    return out, lse


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 2, 3, 8])
def test_single_tokens(D, P, G):
    check_attention([(1, 1), (0, 1), (P, 1), (P + 1, 1), (517, 1), (2 * P - 1, 1), (1000, 1)], 2 * G, 2, D, P, True, seed=G)


@pytest.mark.parametrize("G, Hkv", [(4, 8), (7, 1), (9, 2), (16, 1), (17, 1), (32, 1), (71, 1)])
def test_single_tokens_of_many_heads(G, Hkv):
    check_attention([(300, 1), (40, 1), (0, 1)], G * Hkv, Hkv, 128, 16, True, seed=G)


@pytest.mark.parametrize("n", [2, 3, 4, 5, 8, 13])
@pytest.mark.parametrize("causal", [True, False])
def test_a_few_tokens_each(n, causal):
    check_attention([(n, n), (200 + n, n), (77, n), (1, n), (0, n), (600, 1)], 8, 2, 128, 32, causal, seed=n)


@pytest.mark.parametrize("D, P, G, Hkv", [(128, 16, 4, 2), (128, 64, 1, 3), (64, 32, 2, 2), (64, 128, 5, 1), (128, 128, 8, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(D, P, G, Hkv, causal):
    check_attention([(300, 300), (129, 1), (700, 200), (64, 64), (1, 1), (0, 33), (50, 90), (257, 255)], G * Hkv, Hkv, D, P,
                    causal, seed=P)


@pytest.mark.parametrize("causal", [True, False])
def test_long_prompt_and_long_prefix(causal):
    check_attention([(2300, 1100), (5000, 40)], 4, 1, 128, 64, causal)


def test_rows_that_see_nothing():
    """Fewer keys than queries under the causal rule: the first queries are empty."""
    out, lse = check_attention([(3, 10), (40, 200), (0, 5)], 4, 2, 64, 16, True)
    assert bool((out[:7] == 0).all()) and bool((lse[:7] == -math.inf).all()) and bool((out[10:170] == 0).all())


def test_large_logits_and_uneven_scales():
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 128, 16, True, q_std=12.0, seed=3)
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 128, 16, True, spread=2.0, seed=4)
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 64, 32, False, bias=4.0, seed=5)
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 64, 32, True, q_std=1e-20, seed=6)
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 64, 32, True, sm_scale=-0.3, seed=7)
    check_attention([(900, 1), (333, 5), (400, 400)], 8, 2, 64, 32, True, sm_scale=0.0, seed=8)


def test_many_requests_and_a_long_cache():
    rng = np.random.default_rng(0)
    check_attention([(int(n), 1) for n in rng.integers(0, 400, 300)], 4, 1, 64, 16, True)
    check_attention([(40000, 1), (5, 1)], 8, 1, 128, 128, True)


def test_queries_longer_than_max_q_are_cut():
    g = check_attention([(100, 12), (30, 4)], 2, 1, 64, 16, True, max_q=8)
    assert bool((g[0][8:12] == 7.0).all()) and bool((g[1][8:12] == 7.0).all())         # not written


def test_pages_past_four_gigabytes():
    """Pages whose byte offsets need more than 32 bits."""
    P, H, D = 128, 4, 128
    n = (1 << 32) // (H * P * D) + 9
    kc = torch.zeros((n, H, P, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros((n, H, P, D), dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones((n, H), device="cuda"), torch.ones((n, H), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = [n - 1, 3, n - 2, n - 5, 0, n - 3, 7, n - 4]
    for c, s in ((kc, ks), (vc, vs)):
        x, sx = quantized_pages(len(ids), H, P, D, g)
        c[ids], s[ids] = x, sx
    check_attention([(500, 1), (400, 60)], 8, H, D, P, True, cache_tensors=(kc, ks, vc, vs), page_ids=ids)
    slots = i32([(n - 1) * P + i for i in range(5)])
    x = torch.randn((5, H, D), generator=g, device="cuda")
    cache = qz.PagedKV(kc, vc, ks, vs)
    qz.qz_kv_append_fp8_paged(x, x, slots, cache)
    back = kc[n - 1, :, :5].view(torch.float8_e4m3fn).float() * ks[n - 1][:, None, None]
    assert float((back.transpose(0, 1) - x).abs().max()) <= float(x.abs().max()) / 16


def test_entries_outside_the_cache_are_not_seen():
    """A block table entry outside the cache hides its keys; the rest of the row stands."""
    g = torch.Generator(device="cuda").manual_seed(0)
    P, D, H = 16, 64, 2
    kc, ks = quantized_pages(8, H, P, D, g)
    vc, vs = quantized_pages(8, H, P, D, g)
    cache = qz.PagedKV(kc, vc, ks, vs)
    for n in (1, 40):
        q = torch.randn((n, 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        got, _ = qz.qz_attn_fp8_paged(q, cache, i32([[3, -1, 5, 8, 1]]), i32([70]), i32([0, n]), n, 0.125, causal=False)
        want, _ = qz.qz_attn_fp8_paged(q, cache, i32([[3, 5, 1]]), i32([38]), i32([0, n]), n, 0.125, causal=False)
        assert float((got.float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
        got, lse = qz.qz_attn_fp8_paged(q, cache, i32([[-1, 9]]), i32([30]), i32([0, n]), n, 0.125, causal=False, lse=True)
        assert bool((got == 0).all()) and bool((lse == -math.inf).all())


def test_nan_in_one_request_stays_there():
    g = torch.Generator(device="cuda").manual_seed(0)
    P, D, H = 16, 64, 1
    kc, ks = quantized_pages(12, H, P, D, g)
    vc, vs = quantized_pages(12, H, P, D, g)
    cache = qz.PagedKV(kc, vc, ks, vs)
    table, kv = i32([[0, 1, 2], [3, 4, 5], [6, 7, 8]]), i32([40, 33, 48])
    for n in (1, 30):
        q = torch.randn((3 * n, 4, D), generator=g, device="cuda").to(torch.bfloat16)
        args = (cache, table, kv, i32([0, n, 2 * n, 3 * n]), n, 0.125)
        want, _ = qz.qz_attn_fp8_paged(q, *args)
        q[n:2 * n, 1, 3] = math.nan
        q[n:2 * n, 2, 3] = math.inf
        got, _ = qz.qz_attn_fp8_paged(q, *args)
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[n:2 * n, 1:3] = False
        assert bool((got[keep] == want[keep]).all())


@pytest.mark.parametrize("q_std", [1e6, 1e12, 1e25, 1e36])
def test_logits_past_the_resolution_of_fp32_stay_in_their_rows(q_std):
    """Where the rounding of a score is itself large, its row has no defined answer; the call ends and the others keep theirs."""
    g = torch.Generator(device="cuda").manual_seed(0)
    P, D, H = 16, 64, 1
    kc, ks = quantized_pages(48, H, P, D, g)
    vc, vs = quantized_pages(48, H, P, D, g)
    cache = qz.PagedKV(kc, vc, ks, vs)
    table, kv = torch.arange(48, dtype=torch.int32, device="cuda").view(3, 16), i32([256, 240, 250])
    for n in (1, 200):
        q = torch.randn((3 * n, 2, D), generator=g, device="cuda").to(torch.bfloat16)
        args = (cache, table, kv, i32([0, n, 2 * n, 3 * n]), n, 100.0)
        want, _ = qz.qz_attn_fp8_paged(q, *args)
        q[n:2 * n, 1] *= q_std
        got, _ = qz.qz_attn_fp8_paged(q, *args)
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[n:2 * n, 1] = False
        assert bool((got[keep] == want[keep]).all())
    assert qz.qz_device_error() == 0


def test_another_stream_and_reused_workspace():
    """Calls chained on a stream of their own give the same bits as alone, small and large in turn."""
    g = torch.Generator(device="cuda").manual_seed(0)
    P, D, H = 32, 128, 2
    kc, ks = quantized_pages(80, H, P, D, g)
    vc, vs = quantized_pages(80, H, P, D, g)
    cache, ws = qz.PagedKV(kc, vc, ks, vs), qz.Workspace()
    jobs = []
    for L, n in ((2000, 1), (70, 70), (900, 3), (2500, 300)):
        q = torch.randn((n, 4 * H, D), generator=g, device="cuda").to(torch.bfloat16)
        jobs.append((q, cache, torch.arange(80, dtype=torch.int32, device="cuda")[None], i32([L]), i32([0, n]), n, 0.1))
    alone = [qz.qz_attn_fp8_paged(*j)[0] for j in jobs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(3):
            got = [qz.qz_attn_fp8_paged(*j, ws=ws)[0] for j in jobs]
    st.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a, b)


def test_a_step_after_another():
    """Tables, write and attention chained without a wait: prompts, then single tokens, against attention over the
    values that the cache holds in the end."""
    P, D, Hkv, Hq, B = 16, 64, 2, 6, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    cache = qz.PagedKV.empty(40, Hkv, P, D)
    cache.k_codes.fill_(0x7F)
    cache.v_codes.fill_(0xFF)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free, head, ctx = torch.randperm(40, generator=g, device="cuda").to(torch.int32), i32([0]), i32([0, 0, 0])
    for new in ([30, 1, 77], [1, 1, 1], [1, 0, 1], [2, 16, 1], [1, 1, 1]):
        T = sum(new)
        slots, pos, cu, kv, head = qz.qz_block_tables(ctx, i32(new), table, free, head, P, T)
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        qz.qz_kv_append_fp8_paged(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], slots, cache)
        out, _ = qz.qz_attn_fp8_paged(qkv[:, :Hq], cache, table, kv, cu, max(new), 0.125)
        at = 0
        for b, n in enumerate(new):
            L = int(kv[b])
            pages = table[b, :-(-L // P)].long()
            K, V = (((c[pages].view(torch.float8_e4m3fn).double() * s[pages].double()[..., None, None]).transpose(0, 1)
                     .reshape(Hkv, -1, D)[:, :L]) for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)))
            for i in range(n):
                see = L - n + i + 1
                for a in range(Hq):
                    x = torch.softmax(K[a // 3, :see] @ qkv[at + i, a].double() * 0.125, 0)
                    err = (out[at + i, a].double() - x @ V[a // 3, :see]).abs()
                    assert float((err - 2.0 ** -7 * (x @ V[a // 3, :see].abs())).max()) <= 0
            at += n
        ctx = kv
    assert host(ctx).tolist() == [35, 19, 81] and int(head) == -(-35 // P) + -(-19 // P) + -(-81 // P)
