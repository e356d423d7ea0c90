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
