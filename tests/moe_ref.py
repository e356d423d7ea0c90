"""The operators of a block of experts from their definitions, in 64 bits on the host, and the bounds that
follow from the kernels' arithmetic: fp32 sums, each output rounded once."""
import math

import numpy as np
import torch

FLT_MAX = 3.4028234663852886e38
U = 2.0 ** -24                                   # half a step of fp32, relative


# ------------------------------------------------------------------ routing

def route(logits, k, sigmoid=False, renorm=True, scale=1.0, bias=None, groups=1, top_groups=1, group_best=1, n=None):
    """ids, weights, offsets, row_token, token_row as numpy; one token at a time, sorts of (key, index) pairs."""
    L = logits.double().cpu().numpy()
    T, E = L.shape
    n = T if n is None else min(max(n, 0), T)
    b = None if bias is None else bias.double().cpu().numpy()
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    size = E // groups
    for t in range(n):
        l = [(-math.inf if math.isnan(v) else min(v, FLT_MAX)) for v in L[t].tolist()]
        if sigmoid:
            p = [1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v)) for v in l]
            logp = [min(v, 0.0) - math.log1p(math.exp(-abs(v))) if v > -math.inf else -math.inf for v in l]
        else:
            m = max(max(l), -FLT_MAX)
            e = [math.exp(v - m) for v in l]
            z = math.fsum(e)
            p = [v / z if z else 0.0 for v in e]
            logp = [v - m for v in l]
        bb = [0.0] * E if b is None else [-math.inf if math.isnan(v) else min(v, FLT_MAX) for v in b.tolist()]
        key = [a + c if v > -math.inf else -math.inf for a, c, v in zip(p, bb, l)]
        there = [v > -math.inf for v in key]
        if groups > 1:
            val = []
            for g in range(groups):
                best = sorted((key[e] for e in range(g * size, g * size + size) if there[e]), reverse=True)[:group_best]
                val.append(sum(best) if best else -math.inf)
            kept = [g for g in sorted(range(groups), key=lambda g: (-val[g], g))[:top_groups] if val[g] > -math.inf]
            there = [there[e] and e // size in kept for e in range(E)]
        rank = key if b is not None else l
        top = sorted((e for e in range(E) if there[e]), key=lambda e: (-rank[e], e))[:k]
        ids[t, :len(top)] = top
        if renorm and top:
            m = max(logp[e] for e in top)
            q = [math.exp(logp[e] - m) for e in top]
            w[t, :len(top)] = [scale * v / math.fsum(q) for v in q]
        else:
            w[t, :len(top)] = [scale * p[e] for e in top]
    return (ids, w) + plan(ids, E)


def plan(ids, E):
    T, k = ids.shape
    offsets = np.zeros(E + 1, np.int64)
    row_token = np.full(T * k, -1, np.int32)
    token_row = np.full((T, k), -1, np.int32)
    r = 0
    for e in range(E):
        offsets[e] = r
        for t, j in zip(*np.nonzero(ids == e)):
            row_token[r], token_row[t, j] = t, r
            r += 1
    offsets[E] = r
    return offsets, row_token, token_row


def weight_bound(logits, w):
    """A chosen score's exponential has an argument that is rounded once (a unit per e-fold, at most 104 before it
    underflows), expf 4 units, the sum as much again and 5 more, quotient and scale 2."""
    return (2 * 104 + 4 + 4 + 5 + 2) * U * np.abs(w) + 2.0 ** -140


# ------------------------------------------------------------------ the experts' products

def quantize_blocks(w):
    """E4M3 codes (uint8) and scales of [.., N, K] in 128 x 128 blocks."""
    b = w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))                # [.., N/128, 128, K/128, 128]
    s = b.abs().amax(dim=(-3, -1)).clamp(min=1e-12)
    s = s / torch.full_like(s, 448.0)
    c = (b / s[..., :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.view(torch.uint8).reshape(w.shape).contiguous(), s.contiguous()


def quantize_rows(x):
    g = x.unflatten(-1, (-1, 128))
    s = g.abs().amax(dim=-1).clamp(min=1e-12)
    s = s / torch.full_like(s, 448.0)
    return (g / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2).contiguous(), s.contiguous()


def values(codes, scales, block=False):
    v = codes.view(torch.float8_e4m3fn).double()
    s = scales.double().repeat_interleave(128, dim=-1)
    return v * (s.repeat_interleave(128, dim=-2) if block else s)


def product(qA, sA, qW, sW, offsets, row_token=None):
    """P [rows, N] and its bound's sum of |a w|, both in 64 bits; rows of no expert NaN."""
    a, w = values(qA, sA), values(qW, sW, block=True)
    T, E, N = a.shape[0], w.shape[0], w.shape[1]
    rows = T if row_token is None else row_token.numel()
    at = torch.arange(rows, device=a.device) if row_token is None else row_token.long()
    there = (at >= 0) & (at < T)
    x = a[at.clamp(0, max(T - 1, 0))] * there[:, None] if T else torch.zeros((rows, a.shape[1]), dtype=a.dtype, device=a.device)
    x = torch.where(there[:, None], x, 0.0)
    P = torch.full((rows, N), math.nan, dtype=torch.float64, device=a.device)
    S = torch.zeros_like(P)
    off = [min(max(int(v), 0), rows) for v in offsets.tolist()]
    for e in range(E):
        lo, hi = off[e], max(off[e], off[e + 1])
        P[lo:hi] = x[lo:hi] @ w[e].T
        S[lo:hi] = x[lo:hi].abs() @ w[e].abs().T
    return P, S


def product_bound(S, K):
    """An fp32 sum of K / 32 steps of the tensor cores (32 products a step, aligned to the largest: 2^-22 of the step's
    sum of magnitudes each), then one multiplication and addition per block of 128."""
    return S * ((K // 32 + 8) * 2.0 ** -22)


def swiglu(P, B):
    """h and its bound from P = [gate | up] and P's bound B. |silu'| <= 1.1. The exponential of -g (CUDA's fast one: 2 + 1.16 |g|
    units in the last place, each two of U) reaches h by its share e^-g / (1 + e^-g) <= 1, which is next to nothing for
    positive g of any size; the fast quotient has 2 units, the sum and the product one rounding each. Where e^-g passes fp32's
    range (or the quotient's, 2^126), the sigmoid is 0 instead of less than 2^-125."""
    g, u = P.chunk(2, dim=-1)
    bg, bu = B.chunk(2, dim=-1)
    e = torch.exp(-g)
    s = g / (1 + e)
    h = s * u
    share = torch.where(torch.isinf(e), 1.0, e / (1 + e))
    rel = (2 * (2 + 1.16 * g.abs()) * share + 4 + 2) * U
    return h, 1.1 * bg * (u.abs() + bu) + s.abs() * bu + rel * h.abs() + (g * u).abs() * 2.0 ** -125


def check_codes(codes, scales, want, bound, what=""):
    """Codes and scales per 128 columns against the values they stand for, each off by at most `bound` before they are encoded."""
    R, N = want.shape
    amax = want.abs().view(R, N // 128, 128).amax(dim=-1)
    off = bound.view(R, N // 128, 128).amax(dim=-1)
    s = scales.double()
    assert bool(((s - amax.clamp(min=1e-12) / 448).abs() <= off / 448 + 4 * U * s).all()), f"{what}: scales"
    v = values(codes, scales)
    step = s.repeat_interleave(128, dim=-1) * 2.0 ** -10                    # half a step of the subnormal codes
    err = (v - want).abs()
    tol = torch.maximum(want.abs() * 2.0 ** -4, step) * (1 + 2.0 ** -12) + 2 * bound
    # the largest of a group may saturate by its scale's own rounding
    assert bool((err <= tol + 8 * U * want.abs()).all()), f"{what}: codes, worst {float((err - tol).max())}"


def check_bf16(got, want, bound, what=""):
    err = (got.double() - want).abs()
    tol = want.abs() * 2.0 ** -8 + bound * (1 + 2.0 ** -8) + 2.0 ** -133
    assert bool((err <= tol).all()), f"{what}: worst {float((err - tol).max())}"


# ------------------------------------------------------------------ the residual norm

def residual_norm(x, gamma=None, y=None, token_row=None, weights=None, alpha=1.0, gamma_y=None, eps=1e-6):
    """(r, n, bound of r, bound of n) in 64 bits."""
    x = x.double()
    T, H = x.shape
    r, br = x, torch.zeros_like(x)
    # a sum of squares in fp32: at most 32 terms a thread, 5 steps of a warp, 16 warps; half of that through the root,
    # root, quotient and two products
    rel = ((32 + 5 + 16) / 2 + 6) * U
    if y is not None:
        k = 1 if token_row is None and weights is None else (token_row if token_row is not None else weights).shape[1]
        at = torch.arange(T * k, device=x.device).view(T, k) if token_row is None else token_row.long()
        w = torch.ones((T, k), dtype=torch.float64, device=x.device) if weights is None else weights.double()
        ok = (at >= 0) & (at < y.shape[0])
        z, mag = torch.zeros_like(x), torch.zeros_like(x)
        for j in range(k):
            if y.shape[0]:
                v = w[:, j, None] * y.double()[at[:, j].clamp(0, y.shape[0] - 1)]
                v = torch.where(ok[:, j, None], v, 0.0)
                z, mag = z + v, mag + v.abs()
        bz = mag * (k * U)
        if gamma_y is not None:
            inv = 1 / torch.sqrt(z.square().mean(dim=1, keepdim=True) + eps)
            # an error of z's elements reaches the root mean square as their own mean square does
            moved = bz.square().mean(dim=1, keepdim=True).sqrt() * inv
            bz = (bz * inv + z.abs() * inv * (moved + rel)) * gamma_y.double().abs() * (1 + 1e-6)
            z = z * inv * gamma_y.double()
        r = x + alpha * z
        br = abs(alpha) * bz + (abs(alpha) * z.abs() + r.abs()) * U * 2
    if gamma is None:
        return r, None, br, None
    inv = 1 / torch.sqrt(r.square().mean(dim=1, keepdim=True) + eps)
    moved = br.square().mean(dim=1, keepdim=True).sqrt() * inv
    n = r * inv * gamma.double()
    bn = (br * inv + r.abs() * inv * (moved + rel)) * gamma.double().abs() * (1 + 1e-6)
    return r, n, br, bn
