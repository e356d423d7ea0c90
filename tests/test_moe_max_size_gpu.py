"""A block of experts on tensors of more than 2^31 elements: outputs, gathered inputs, weights, the residual stream, logits."""
import math

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref
import test_residual_rmsnorm_gpu as norm

pytestmark = pytest.mark.gpu

LIMIT = 1 << 31


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def codes_of(shape, seed):
    """E4M3 codes of either sign without NaN, up to 30 (magnitudes 0 .. 0x5F)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0, 0x60, shape, generator=g, device="cuda", dtype=torch.uint8)
    return c | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)


def offsets(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i32(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("swiglu", [False, True])
def test_outputs(swiglu):
    """Few tokens many times: each of the rows has one of tokens x experts results."""
    tokens, N, K = 29, 4096, 128
    rows = LIMIT // (N // 2 if swiglu else N) + 10007
    g = torch.Generator(device="cuda").manual_seed(1)
    qA, sA = ref.quantize_rows(torch.randn((tokens, K), generator=g, device="cuda"))
    qW, sW = ref.quantize_blocks(torch.randn((3, N, K), generator=g, device="cuda") * 0.1)
    off = offsets(0, 1000, rows - 40000, rows - 3)                # the last rows belong to nobody
    row_token = torch.randint(0, tokens, (rows,), generator=g, device="cuda").int()
    if swiglu:
        codes = torch.full((rows, N // 2), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, N // 256), 7.0, device="cuda")
        qz.qz_moe_gemm_fp8_swiglu(qA, sA, qW, sW, off, row_token, codes=codes, scales=scales)
        assert bool((codes[-3:] == 0x55).all()) and bool((scales[-3:] == 7.0).all())
        outs = (codes, scales)
    else:
        Y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        qz.qz_moe_gemm_fp8(qA, sA, qW, sW, off, row_token, Y=Y)
        assert bool((Y[-3:] == 7.0).all())
        outs = (Y,)
    # every token with every expert, against 64 bits
    every = i32(list(range(tokens)) * 3)
    P, S = ref.product(qA, sA, qW, sW, offsets(0, tokens, 2 * tokens, 3 * tokens), every)
    B = ref.product_bound(S, K)
    expert = torch.bucketize(torch.arange(rows - 3, device="cuda"), off[1:3].long(), right=True)
    which = expert * tokens + row_token[:rows - 3].long()
    first = torch.full((3 * tokens,), rows, device="cuda").scatter_reduce_(0, which, torch.arange(rows - 3, device="cuda"), "amin")
    assert int(first.max()) < rows                                # all of them occur
    if swiglu:
        h, bh = ref.swiglu(P, B)
        ref.check_codes(codes[first], scales[first], h, bh, "first rows")
    else:
        ref.check_bf16(Y[first], P, B, "first rows")
    # and the others are the same bits
    for lo in range(0, rows - 3, 1 << 16):
        hi = min(lo + (1 << 16), rows - 3)
        for out in outs:
            assert torch.equal(out[lo:hi], out[first][which[lo:hi]]), lo


def test_gathered_and_ordered_rows():
    K, N = 7168, 256
    tokens = LIMIT // K + 501
    qA, sA = codes_of((tokens, K), 2), torch.rand((tokens, K // 128), device="cuda") * 0.01
    qW, sW = codes_of((2, N, K), 3), torch.rand((2, N // 128, K // 128), device="cuda") * 0.01
    at = i32([tokens - 1, 0, tokens - 2, 299593, 299592, 5] + list(range(tokens - 300, tokens)))
    rows = at.numel()
    Y = qz.qz_moe_gemm_fp8(qA, sA, qW, sW, offsets(0, 200, rows), at)
    few = (qA[at.long()], sA[at.long()])
    P, S = ref.product(*few, qW, sW, offsets(0, 200, rows))
    ref.check_bf16(Y, P, ref.product_bound(S, K), "gathered")
    # the last rows where they lie: the others belong to nobody
    lo = tokens - 300
    Y = torch.zeros((tokens, N), dtype=torch.bfloat16, device="cuda")
    qz.qz_moe_gemm_fp8(qA, sA, qW, sW, offsets(lo, lo + 130, tokens), Y=Y)
    P, S = ref.product(qA[lo:], sA[lo:], qW, sW, offsets(0, 130, 300))
    ref.check_bf16(Y[lo:], P, ref.product_bound(S, K), "ordered")
    assert not Y[:lo].any()


@pytest.mark.parametrize("swiglu", [False, True])
def test_weights(swiglu):
    K, N, E = 4096, 2048, 260
    assert E * K * N > LIMIT
    qW, sW = codes_of((E, N, K), 4), torch.rand((E, N // 128, K // 128), device="cuda") * 0.01
    counts = torch.zeros(E, dtype=torch.int64)
    counts[[0, 100, 255, 256, 259]] = torch.tensor([3, 40, 129, 5, 70])
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    rows = int(off[-1])
    qA, sA = codes_of((rows, K), 5), torch.rand((rows, K // 128), device="cuda") * 0.01
    used = counts.nonzero()[:, 0].cuda()
    P, S = ref.product(qA, sA, qW[used], sW[used], i32([0] + off[1:][counts > 0].tolist()))
    B = ref.product_bound(S, K)
    if swiglu:
        codes, scales = qz.qz_moe_gemm_fp8_swiglu(qA, sA, qW, sW, i32(off))
        ref.check_codes(codes, scales, *ref.swiglu(P, B), "codes")
    else:
        ref.check_bf16(qz.qz_moe_gemm_fp8(qA, sA, qW, sW, i32(off)), P, B, "Y")


@pytest.mark.parametrize("k", [0, 2])
def test_residual_stream(k):
    """k = 2: each token's rows lie anywhere in a y of as many elements."""
    H = 16384
    T = LIMIT // H + 77
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    y = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16()
    rows = torch.randint(0, T, (T, 2), generator=g, device="cuda").int() if k else None
    gates = torch.rand((T, 2), generator=g, device="cuda") if k else None
    if k:
        rows[0] = i32([T - 1, T - 2])
    got = qz.qz_residual_rmsnorm(x, gamma, y, rows, gates, normed=True, fp8=True)
    at = torch.tensor([0, 1, LIMIT // H - 1, LIMIT // H, LIMIT // H + 1, T - 1], device="cuda")
    d = dict(x=x[at], gamma=gamma, y=y if k else y[at], token_row=rows[at] if k else None, weights=gates[at] if k else None)
    if k:
        pick = rows[at].long().reshape(-1)
        d.update(y=y[pick], token_row=torch.arange(2 * len(at), device="cuda").int().view(-1, 2))
    want = norm.check(d, normed=True, fp8=True)                   # against 64 bits
    for a, b in zip(want, got):
        assert torch.equal(a, b[at])
    # all others through the same call in parts that 32 bits reach
    for lo in range(0, T, T // 3 + 1):
        hi = min(lo + T // 3 + 1, T)
        part = qz.qz_residual_rmsnorm(x[lo:hi], gamma, y if k else y[lo:hi], rows[lo:hi] if k else None, gates[lo:hi] if k else None,
                                      normed=True, fp8=True)
        assert all(torch.equal(a, b[lo:hi]) for a, b in zip(part, got)), lo


def test_logits_far_apart():
    E, T, k = 24, 2100, 3
    wide = torch.empty((T, 1 << 20), device="cuda")
    assert wide.numel() > LIMIT
    logits = wide[:, 1000:1000 + E]
    logits.copy_(torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(7), device="cuda"))
    got = qz.qz_moe_route(logits, k, n_tokens=i32([T - 5]))
    want = ref.route(logits, k, n=T - 5)
    for i in (0, 2, 3, 4):
        assert bool((got[i].cpu().long() == torch.as_tensor(want[i]).long()).all())


def test_four_million_tokens():
    """Logits of more than 2^31 elements, chosen one by one: the largest, its lowest index, and rows in the order of the tokens."""
    E = 512
    T = LIMIT // E + 12345
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(8))
    ids, w, off, row_token, token_row = qz.qz_moe_route(logits, 1, scale=0.5)
    index = torch.arange(E, device="cuda")
    want = torch.cat([torch.where(c == c.amax(dim=1, keepdim=True), index, E).amin(dim=1) for c in logits.split(1 << 18)])
    assert torch.equal(ids[:, 0].long(), want)
    assert bool((w == 0.5).all())
    order = torch.sort(want, stable=True)[1]
    assert torch.equal(row_token.long(), order)
    assert torch.equal(token_row[:, 0].long()[order], torch.arange(T, device="cuda"))
    assert torch.equal(off[1:].long(), torch.bincount(want, minlength=E).cumsum(0)) and int(off[0]) == 0
    assert math.prod(logits.shape) > LIMIT
