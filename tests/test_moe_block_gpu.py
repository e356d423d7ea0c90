"""The operators of a block of experts together, as a serving loop runs them: stage by stage against the definitions, in
graphs that are replayed on other routings, on several streams, and the example."""
import importlib.util
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def ex():
    return example()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("T, n", [(1, None), (37, None), (150, 90), (300, 0)])
def test_a_block_stage_by_stage(ex, T, n):
    """Each stage on what the stage before it gave: errors of one do not hide in the next."""
    block = ex.MoEBlock(gen(1))
    g = gen(T)
    x = torch.randn((T, ex.HIDDEN), generator=g, device="cuda").bfloat16()
    attention = torch.randn((T, ex.HIDDEN), generator=g, device="cuda").bfloat16()
    nt = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
    x1, normed, codes, scales = qz.qz_residual_rmsnorm(x, block.gamma, y=attention, normed=True, fp8=True)
    r, v, br, bv = ref.residual_norm(x, block.gamma, attention)
    ref.check_bf16(x1, r, br, "residual")
    ref.check_bf16(normed, v, bv, "norm")
    ref.check_codes(codes, scales, v, bv, "codes")
    logits = normed @ block.router
    kw = dict(bias=block.bias, groups=4, top_groups=2, group_best=2)
    ids, gates, offsets, row_token, token_row = qz.qz_moe_route(logits, ex.TOP_K, score=qz.SCORE_SIGMOID, n_tokens=nt, **kw)
    want = ref.route(logits, ex.TOP_K, sigmoid=True, n=n, **kw)
    for got, w in zip((ids, offsets, row_token, token_row), (want[0], want[2], want[3], want[4])):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    live = int(offsets[-1])
    assert live == ex.TOP_K * (T if n is None else n)
    h, hs = qz.qz_moe_gemm_fp8_swiglu(codes, scales, *block.up, offsets, row_token)
    P, S = ref.product(codes, scales, *block.up, offsets, row_token)
    want_h, bh = ref.swiglu(P[:live], ref.product_bound(S[:live], ex.HIDDEN))
    if live:
        ref.check_codes(h[:live], hs[:live], want_h, bh, "up")
    rows = qz.qz_moe_gemm_fp8(h, hs, *block.down, offsets)
    if live:
        P, S = ref.product(h, hs, *block.down, offsets)
        ref.check_bf16(rows[:live], P[:live], ref.product_bound(S[:live], ex.INNER), "down")
    out = qz.qz_residual_rmsnorm(x1, block.next_gamma, y=rows, token_row=token_row, weights=gates, normed=True, fp8=True)
    r, v, br, bv = ref.residual_norm(x1, block.next_gamma, rows, token_row, gates)
    ref.check_bf16(out[0], r, br, "residual behind the block")
    ref.check_bf16(out[1], v, bv, "next norm")
    ref.check_codes(out[2], out[3], v, bv, "next codes")
    if n is not None:                                             # padding: nothing was added
        assert torch.equal(out[0][n:], x1[n:])
    both = block(x, attention, nt)                                # and all at once, without a wait between the calls
    assert all(torch.equal(a, b) for a, b in zip(both, out))
    assert qz.qz_device_error() == 0


def test_a_captured_step_on_other_routings(ex):
    block = ex.MoEBlock(gen(2))
    T = 48
    x, att = (torch.zeros((T, ex.HIDDEN), device="cuda").bfloat16() for _ in range(2))
    n = torch.full((1,), T, dtype=torch.int32, device="cuda")
    block(x, att, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, att, n)
    for seed, tokens in ((1, 48), (2, 1), (3, 0), (4, 33), (1, 48)):
        g = gen(seed)
        x.copy_(torch.randn((T, ex.HIDDEN), generator=g, device="cuda"))
        att.copy_(torch.randn((T, ex.HIDDEN), generator=g, device="cuda"))
        n.fill_(tokens)
        graph.replay()
        torch.cuda.synchronize()
        want = block(x, att, n)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (seed, tokens)


def test_steps_behind_one_another_and_on_two_streams(ex):
    """Blocks whose calls follow one another without a wait, on two streams at once with a workspace each."""
    blocks = [ex.MoEBlock(gen(3)), ex.MoEBlock(gen(4))]
    T = 500
    xs = [torch.randn((T, ex.HIDDEN), generator=gen(5 + i), device="cuda").bfloat16() for i in range(2)]
    atts = [torch.randn((T, ex.HIDDEN), generator=gen(7 + i), device="cuda").bfloat16() for i in range(2)]

    def chain(b, x, att):
        for _ in range(4):
            x = b(x, att)[0]
        return x

    want = [chain(b, x, a) for b, x, a in zip(blocks, xs, atts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = chain(blocks[i], xs[i], atts[i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert qz.qz_device_error() == 0


def test_calls_on_a_given_stream_allocate_on_it(ex):
    """The current stream is behind with writes to memory that it has freed; calls on another stream must not get it."""
    block = ex.MoEBlock(gen(9))
    T = 300
    x = torch.randn((T, ex.HIDDEN), generator=gen(1), device="cuda").bfloat16()
    logits = torch.randn((T, ex.EXPERTS), generator=gen(2), device="cuda")
    codes, scales, _ = qz.qz_quantize_fp8(x, qz.FP8_GROUP_1x128)
    side = torch.cuda.Stream()

    def run(stream):
        r = qz.qz_moe_route(logits, ex.TOP_K, stream=stream)
        h = qz.qz_moe_gemm_fp8_swiglu(codes, scales, *block.up, r[2], r[3], stream=stream)
        y = qz.qz_moe_gemm_fp8(*h, *block.down, r[2], stream=stream)
        return (*r, *h, y, *qz.qz_residual_rmsnorm(x, block.gamma, y=y, token_row=r[4], weights=r[1], normed=True, fp8=True, stream=stream))

    want = run(None)
    torch.cuda.synchronize()
    sizes = [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(20_000_000)                                 # the current stream falls behind
    for s in sizes * 3:
        torch.empty(s, dtype=torch.uint8, device="cuda").fill_(0xEE)
    got = run(side)
    side.synchronize()
    same = [torch.equal(a, b) for a, b in zip(got, want)]
    torch.cuda.synchronize()
    assert all(same) and all(torch.equal(a, b) for a, b in zip(got, want)), same


def test_one_route_for_many_experts_with_few_tokens_each():
    """512 experts, most without rows, and the products over their rows."""
    E, T, K, N, k = 512, 40, 256, 256, 6
    g = gen(11)
    logits = torch.randn((T, E), generator=g, device="cuda")
    _, _, offsets, row_token, _ = qz.qz_moe_route(logits, k)
    qA, sA = ref.quantize_rows(torch.randn((T, K), generator=g, device="cuda"))
    qW, sW = ref.quantize_blocks(torch.randn((E, N, K), generator=g, device="cuda") * 0.1)
    P, S = ref.product(qA, sA, qW, sW, offsets, row_token)
    ref.check_bf16(qz.qz_moe_gemm_fp8(qA, sA, qW, sW, offsets, row_token), P, ref.product_bound(S, K))


def test_the_example_runs():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py")], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "decode steps" in out.stdout
