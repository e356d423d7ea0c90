"""Attention over the paged FP8 cache by its formula, in 64 bits, with the error that the kernels' arithmetic allows.

p is the softmax, sv_j the value scale of key j's page, c_j its code's value, V_j = c_j sv_j; L <= 2^13 keys:
* dx, error of a score. The prefill kernel's two E4M3 parts of q leave at most 2^-17 of the row's amax, the fp32 sums of
  D <= 128 products at most as much: 2^-16 |sm_scale| amax(q) sum_d |K_jd|. The fp32 roundings of the factor and of the
  exponent x log2(e) + log2 sv - m + 8: 2^-21 (|x| + |log2 sv| + 8).
* p's share of the error enters numerator and denominator: 2.5 dx. P is rounded to f16, 2^-11 of itself; fp32 sums of
  2^9 steps of 16 keys, each cut to 2^-23 at worst, 2^-14, and l's 2^-15: together below 2^-10 of sum_j p_j |V_j|.
* p below 2^-14 lose bits: at most 2^-25 each, twice where stored P is scaled, and the largest p is 2^7 at least:
  2^-31 max_j(p_j sv_j) sum_j |c_j|.
* a value scale of at most 2^-80 counts as 0: 448 * 2^-80 < 2^-71.
* the result is rounded once to bf16: half an ulp at most 2^-8 of the power of two below it.
* lse: dx, l's 2^-15 and 2^-20 |lse| for the logarithm and the product with ln 2.
"""
import math

import torch

F8 = torch.float8_e4m3fn


def formula(q, cache, table, kv, cu, sm, causal):
    """(O, lse, allowed error of O, of lse), fp64. table: every page that a request's keys need is in the cache."""
    T, Hq, D = q.shape
    G, P = Hq // cache.heads, cache.page_size
    want = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    tol, tol_lse = torch.zeros_like(want), torch.zeros_like(lse)
    for b in range(len(kv)):
        t0, t1, L = cu[b], cu[b + 1], kv[b]
        n = t1 - t0
        if n == 0 or L == 0:
            continue
        pages = table[b, :-(-L // P)].long()
        ck, cv = (x[pages].view(F8).double().transpose(0, 1).reshape(cache.heads, -1, D)[:, :L].repeat_interleave(G, 0)
                  for x in (cache.k_codes, cache.v_codes))
        sk, sv = (s[pages].double().T.repeat_interleave(P, 1)[:, :L].repeat_interleave(G, 0)
                  for s in (cache.k_scale, cache.v_scale))                                     # [Hq, L]
        K, V = ck * sk[..., None], cv * sv[..., None]
        rows = q[t0:t1].double().transpose(0, 1)                                               # [Hq, n, D]
        x = rows @ K.transpose(1, 2) * sm
        seen = torch.ones((n, L), dtype=torch.bool, device="cuda")
        if causal:
            seen = torch.arange(L, device="cuda")[None, :] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        some = seen.any(dim=1)
        e = 2.0 ** -16 * abs(sm) * rows.abs().amax(-1)[..., None] * K.abs().sum(-1)[:, None] \
            + 2.0 ** -21 * (x.abs() + torch.log2(sv.clamp(min=2.0 ** -80)).abs()[:, None] + 8)
        dx = torch.where(seen, e, 0.0).amax(-1)                                                # [Hq, n]
        x = torch.where(seen, x, -math.inf)
        z = torch.logsumexp(x, dim=-1)
        p = torch.where(some[:, None], torch.exp(x - torch.where(some, z, 0.0)[..., None]), 0.0)
        o = torch.where(some[:, None], torch.where(seen, p, 0.0) @ V, 0.0)
        top = (p * sv.clamp(min=2.0 ** -80)[:, None]).amax(-1)
        a = (2.5 * dx + 2.0 ** -10)[..., None] * (p @ V.abs()) + 2.0 ** -71 \
            + 2.0 ** -31 * top[..., None] * (seen.double() @ cv.abs())
        a = torch.where(some[:, None], a, 0.0)
        half_ulp = torch.ldexp(torch.ones_like(a), torch.frexp(o.abs() + a)[1] - 9)
        want[t0:t1], lse[t0:t1] = o.transpose(0, 1), torch.where(some, z, -math.inf).T
        tol[t0:t1] = torch.where(some[:, None], a + half_ulp, 0.0).transpose(0, 1)
        tol_lse[t0:t1] = (dx + 2.0 ** -15 + 2.0 ** -20 * torch.where(some, z, 0.0).abs()).T
    return want, lse, tol, tol_lse


def check(out, lse, ref):
    """Every row of out and lse is within the allowed error; rows without keys are 0 and -inf. NaN is never within."""
    want, want_lse, tol, tol_lse = ref
    bad = ~((out.double() - want).abs() <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} outputs outside the tolerance, first {bad.nonzero()[0].tolist()}"
    empty = want_lse == -math.inf
    assert bool((lse[empty] == -math.inf).all()), "lse of rows without keys"
    bad = ~((lse.double() - want_lse).abs() <= tol_lse) & ~empty
    assert not bool(bad.any()), f"{int(bad.sum())} lse outside the tolerance, first {bad.nonzero()[0].tolist()}"


def encode(x, floor=1e-12):
    """Codes and scales of pages [pages, H, P, D], one scale per (page, head)."""
    s = x.abs().amax(dim=(2, 3)).clamp(min=floor) / 448.0
    return (x / s[:, :, None, None]).clamp(-448, 448).to(F8).view(torch.uint8), s


def page_tables(kv, P, extra, generator, width=None):
    """Block tables of requests of kv keys, pages in a random order; entries behind a request's pages are -1."""
    counts = [-(-n // P) for n in kv]
    order = torch.randperm(sum(counts) + extra, generator=generator, device="cuda").to(torch.int32)
    table = torch.full((len(kv), width or max(counts + [1])), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(counts) + extra
