"""Steps of few tokens, whose products share their K in clusters: captured and replayed on other routings, on two streams at
once, and against their definition whatever the number of rows."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref
from test_moe_block_gpu import ex, gen  # noqa: F401  (the example, loaded once)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 3, 8])
def test_a_captured_step_of_few_tokens(ex, T):  # noqa: F811
    block = ex.MoEBlock(gen(20))
    x, att = (torch.zeros((T, ex.HIDDEN), device="cuda").bfloat16() for _ in range(2))
    n = torch.full((1,), T, dtype=torch.int32, device="cuda")
    block(x, att, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, att, n)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    other = ex.MoEBlock(gen(21))
    for seed, tokens in ((1, T), (2, 1), (3, 0), (4, T), (1, T)):
        x.copy_(torch.randn((T, ex.HIDDEN), generator=gen(seed), device="cuda"))
        att.copy_(torch.randn((T, ex.HIDDEN), generator=gen(seed + 50), device="cuda"))
        n.fill_(tokens)
        want, beside = block(x, att, n), other(x, att)
        torch.cuda.synchronize()
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            again = other(x, att)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (seed, tokens)
        assert all(torch.equal(a, b) for a, b in zip(again, beside))
    assert qz.qz_device_error() == 0


@pytest.mark.parametrize("rows", [1, 2, 16, 31, 32, 33])
@pytest.mark.parametrize("K", [128, 384, 512, 1152, 2048, 4096])
def test_every_split_of_k(rows, K):
    """K of one to 32 blocks, also those that 2 or 4 CTAs cannot share evenly; few columns, so that there are CTAs to share it."""
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    N = 512
    qA, sA = ref.quantize_rows(torch.randn((rows, K), generator=g, device="cuda"))
    qW, sW = ref.quantize_blocks(torch.randn((3, N, K), generator=g, device="cuda") * 0.05)
    off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    P, S = ref.product(qA, sA, qW, sW, off)
    B = ref.product_bound(S, K)
    ref.check_bf16(qz.qz_moe_gemm_fp8(qA, sA, qW, sW, off), P, B, "Y")
    ref.check_codes(*qz.qz_moe_gemm_fp8_swiglu(qA, sA, qW, sW, off), *ref.swiglu(P, B), "codes")
