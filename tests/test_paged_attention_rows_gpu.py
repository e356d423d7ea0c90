"""Attention over the paged FP8 cache, where its kernels hand work and state on: many items a CTA, maxima that rise
inside a tile, unusual scales and queries. Tolerances: paged_ref.py."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
from paged_ref import check, encode, formula, page_tables

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def sums(lens):
    return [0] + np.cumsum(lens).tolist()


@pytest.mark.parametrize("D, Hkv, G, P, causal", [(128, 8, 2, 16, True), (64, 8, 4, 32, False), (128, 4, 3, 64, False),
                                                  (64, 16, 1, 128, True)])
def test_many_items(D, Hkv, G, P, causal):
    """Several items a CTA of the prefill kernel, more than 32 requests: long items whose second row tile is empty next to
    full ones, single tokens and requests without keys or tokens among them."""
    rng = np.random.default_rng(D + P)
    g = torch.Generator(device="cuda").manual_seed(P)
    n = rng.integers(1, 700, 70)
    n[::3] = rng.integers(1, 128, 24) // G + 256 // G * rng.integers(0, 3, 24) + 1            # few rows in the last tile pair
    n[4::9] = 1
    n[7::20] = 0
    past = rng.integers(0, 1500, 70)
    kv = past + n if causal else past
    kv[11::23] = 0
    kv[5] = max(n[5] - 40, 1)                                  # causal: rows that see nothing
    n, kv = n.tolist(), kv.tolist()
    items = sum(-(-x * G // 256) for x in n if x * G > 32) * Hkv
    assert items > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    table, pages = page_tables(kv, P, 3, g)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    size = torch.exp(rand(pages, Hkv, 1, 1))                   # pages of scales of their own
    cache = qz.PagedKV(*(lambda k, v: (k[0], v[0], k[1], v[1]))(encode(rand(pages, Hkv, P, D) * size.clamp(max=2)),
                                                                encode(rand(pages, Hkv, P, D) * size)))
    cu = sums(n)
    q = rand(cu[-1], Hkv * G, D).to(torch.bfloat16)
    args = (q, cache, table, i32(kv), i32(cu), max(n), D ** -0.5)
    out, lse = qz.qz_attn_fp8_paged(*args, causal=causal, lse=True)
    check(out, lse, formula(q, cache, table, kv, cu, D ** -0.5, causal))
    for _ in range(5):                                         # whichever CTA takes an item
        again, lse2 = qz.qz_attn_fp8_paged(*args, causal=causal, lse=True)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    assert qz.qz_device_error() == 0


def rising(L, step, D, H, P, g):
    """Keys whose products with the returned direction grow by `step` doublings (of 2^x) every 64 keys, and a little from key to key."""
    u = torch.where(torch.rand(D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    pages = -(-L // P)
    j = torch.arange(pages * P, device="cuda")
    a = (step * math.log(2.0) * torch.floor(j / 64.0) + torch.rand(pages * P, generator=g, device="cuda")) / D
    k = a[:, None] * u[None] + 0.01 * torch.randn((H, pages * P, D), generator=g, device="cuda")
    v = torch.randn((pages, H, P, D), generator=g, device="cuda")
    k = encode(k.reshape(H, pages, P, D).transpose(0, 1).contiguous())
    return u, k, encode(v)


@pytest.mark.parametrize("D, P, causal", [(128, 16, True), (64, 64, False), (128, 128, False)])
@pytest.mark.parametrize("step", [2.5, 6.0, 11.0])
def test_maxima_that_rise_in_every_half_of_a_tile(D, P, causal, step):
    """The stored P and O of a tile are scaled again and again; rows of other sizes rise elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(int(step * 2) + D)
    L, n, H, G = 1100, 300, 2, 3
    u, (kc, ks), (vc, vs) = rising(L, step, D, H, P, g)
    cache = qz.PagedKV(kc, vc, ks, vs)
    r = 0.3 + torch.rand((n, H * G, 1), generator=g, device="cuda")
    q = (r * u + 0.05 * torch.randn((n, H * G, D), generator=g, device="cuda")).to(torch.bfloat16)
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    out, lse = qz.qz_attn_fp8_paged(q, cache, table, i32([L]), i32([0, n]), n, 1.0, causal=causal, lse=True)
    check(out, lse, formula(q, cache, table, [L], [0, n], 1.0, causal))
    few, lse = qz.qz_attn_fp8_paged(q[:7], cache, table, i32([L]), i32([0, 7]), 7, 1.0, causal=causal, lse=True)
    check(few, lse, formula(q[:7], cache, table, [L], [0, 7], 1.0, causal))
    assert qz.qz_device_error() == 0


@pytest.mark.parametrize("D, P, causal", [(128, 16, True), (64, 64, False)])
def test_a_nan_row_leaves_rows_that_rise_alone(D, P, causal):
    """A row of NaN never finds a maximum; its neighbours in the warp raise theirs all the same."""
    g = torch.Generator(device="cuda").manual_seed(D)
    L, n, H, G = 900, 250, 1, 4
    u, (kc, ks), (vc, vs) = rising(L, 10.0, D, H, P, g)
    cache = qz.PagedKV(kc, vc, ks, vs)
    q = (u + 0.05 * torch.randn((n, H * G, D), generator=g, device="cuda")).to(torch.bfloat16)
    table = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
    for rows in (n, 5):
        args = (cache, table, i32([L]), i32([0, rows]), rows, 1.0)
        want, want_lse = qz.qz_attn_fp8_paged(q[:rows], *args, causal=causal, lse=True)
        check(want, want_lse, formula(q[:rows], cache, table, [L], [0, rows], 1.0, causal))
        bad = q[:rows].clone()
        bad[::7, 2, 5] = math.nan
        got, lse = qz.qz_attn_fp8_paged(bad, *args, causal=causal, lse=True)
        hit = torch.zeros((rows, H * G), dtype=torch.bool, device="cuda")
        hit[::7, 2] = True
        assert bool(got[hit].isnan().all()) and bool(lse[hit].isnan().all())
        assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 2.0 ** -100, 2.0 ** -79])
@pytest.mark.parametrize("where", ["first", "middle", "last", "alone"])
@pytest.mark.parametrize("n, causal", [(1, True), (6, False), (200, True), (200, False)])
def test_value_scales_down_to_zero(n, causal, where, scale):
    """Pages of zeros as a quantizer without a floor leaves them, and codes under scales too small to matter: their
    keys count in the denominator, their values as good as nothing."""
    g = torch.Generator(device="cuda").manual_seed(n)
    P, D, H, G, L = 32, 64, 2, 2, 470
    kc, ks = encode(torch.randn((15, H, P, D), generator=g, device="cuda"))
    vc, vs = encode(torch.randn((15, H, P, D), generator=g, device="cuda"))
    pages = {"first": slice(0, 5), "middle": slice(6, 9), "last": slice(11, 15), "alone": slice(0, 15)}[where]
    vs[pages, 0] = scale
    if scale == 0:
        vc[pages, 0] = 0
    cache = qz.PagedKV(kc, vc, ks, vs)
    q = torch.randn((n, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(15, dtype=torch.int32, device="cuda")[None]
    out, lse = qz.qz_attn_fp8_paged(q, cache, table, i32([L]), i32([0, n]), n, 0.125, causal=causal, lse=True)
    check(out, lse, formula(q, cache, table, [L], [0, n], 0.125, causal))


def three_requests(n, g, P=16, D=64, H=2, G=2):
    kc, ks = encode(torch.randn((12, H, P, D), generator=g, device="cuda"))
    vc, vs = encode(torch.randn((12, H, P, D), generator=g, device="cuda"))
    q = torch.randn((3 * n, H * G, D), generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    return q, qz.PagedKV(kc, vc, ks, vs), table, [60, 50, 64], [0, n, 2 * n, 3 * n]


def poisoned(run, spoil, rows, heads):
    """run() before and after spoil(): NaN in these rows and heads, every other bit as before."""
    want, want_lse = run()
    spoil()
    got, lse = run()
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[rows, heads] = True
    assert bool(got[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -1.0])
@pytest.mark.parametrize("page", [0, 2])
def test_value_scales_that_are_no_sizes(n, bad, page):
    """NaN, infinite and negative value scales are NaN in the rows that see them, in both kernels."""
    q, cache, table, kv, cu = three_requests(n, torch.Generator(device="cuda").manual_seed(n))
    run = lambda: qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), n, 0.125, causal=False, lse=True)  # noqa: E731
    poisoned(run, lambda: cache.v_scale[4 + page, :1].fill_(bad), slice(n, 2 * n), slice(0, 2))


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("page", [0, 2])
def test_key_scales_that_are_no_numbers(n, bad, page):
    """NaN and infinite key scales are NaN in the rows that see them, in both kernels."""
    q, cache, table, kv, cu = three_requests(n, torch.Generator(device="cuda").manual_seed(n))
    run = lambda: qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), n, 0.125, causal=False, lse=True)  # noqa: E731
    poisoned(run, lambda: cache.k_scale[4 + page, :1].fill_(bad), slice(n, 2 * n), slice(0, 2))


@pytest.mark.parametrize("n", [1, 60, 300])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("small", [1.0, 1e-35])
def test_key_scales_keep_their_sign(n, causal, small):
    g = torch.Generator(device="cuda").manual_seed(n)
    q, cache, table, _, cu = three_requests(n, g)
    cache.k_scale *= torch.where(torch.rand(cache.k_scale.shape, generator=g, device="cuda") < 0.5, -small, 1.0)
    kv = [60, 50, 17]
    out, lse = qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), n, 0.3, causal=causal, lse=True)
    check(out, lse, formula(q, cache, table, kv, cu, 0.3, causal))


@pytest.mark.parametrize("n", [1, 60])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_queries_that_are_no_numbers(n, bad):
    """NaN and infinite queries are NaN in their own rows, in both kernels; a row that sees no key stays 0."""
    q, cache, table, kv, cu = three_requests(n, torch.Generator(device="cuda").manual_seed(n))
    run = lambda: qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), n, 0.125, causal=True, lse=True)  # noqa: E731
    poisoned(run, lambda: q[n:2 * n, 3, 40].fill_(bad), slice(2 * n - min(n, 50), 2 * n), slice(3, 4))


def test_queries_that_are_no_numbers_alone_with_one_sign():
    """An infinite query against keys that all lie to one side: every score is infinite, the row NaN."""
    g = torch.Generator(device="cuda").manual_seed(0)
    for n in (1, 60):
        q, cache, table, kv, cu = three_requests(n, g)
        cache.k_codes.view(torch.float8_e4m3fn)[:, :, :, 7] = 2.0
        for bad in (math.inf, -math.inf):
            q[:, 1, 7] = bad
            out, lse = qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), n, 0.125, causal=False, lse=True)
            assert bool(out[:, 1].isnan().all()) and bool(lse[:, 1].isnan().all())
            assert not bool(out[:, 0].isnan().any())


@pytest.mark.parametrize("kv, n", [([256], [256]), ([5000], [256]), ([300], [40]), ([0], [50]), ([517], [1]), ([700, 3], [1, 1]),
                                   ([900, 64], [100, 1])])
def test_a_block_table_much_wider_than_the_keys(kv, n):
    """The parts that a wide table makes of the keys, most of them empty, against the formula."""
    g = torch.Generator(device="cuda").manual_seed(kv[0])
    P, D, Hkv, G = 64, 128, 2, 4
    table, pages = page_tables(kv, P, 2, g, width=32768 // P)
    k, v = (encode(torch.randn((pages, Hkv, P, D), generator=g, device="cuda")) for _ in range(2))
    cache, cu = qz.PagedKV(k[0], v[0], k[1], v[1]), sums(n)
    q = torch.randn((cu[-1], Hkv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    out, lse = qz.qz_attn_fp8_paged(q, cache, table, i32(kv), i32(cu), max(n), 0.09, lse=True)
    check(out, lse, formula(q, cache, table, kv, cu, 0.09, True))
