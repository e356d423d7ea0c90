"""A block of experts of a decoder served in FP8.

    python examples/moe_block.py

Runs the library's calls as a serving loop makes them, without a count on the host: the residual norm in
front of the block (qz_residual_rmsnorm: bf16 for the router's product, FP8 codes for the experts'), the
routing (qz_moe_route), the experts' products (qz_moe_gemm_fp8_swiglu, qz_moe_gemm_fp8), and the norm of
the next block, which gathers the experts' rows by their gates into the residual. The decode step is
captured into a CUDA graph once and replayed on other tokens and routings. Random weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_linear_quantizers_gb300 as qz  # noqa: E402

HIDDEN, INNER, EXPERTS, TOP_K = 1024, 512, 32, 4


def quantize_experts(w):
    """[experts, N, K] into E4M3 codes and a scale per 128 x 128 block: the experts' rows are one tall matrix."""
    E, N, K = w.shape
    codes, scales, _ = qz.qz_quantize_fp8(w.reshape(E * N, K), qz.FP8_BLOCK_128x128)
    return codes.view(E, N, K), scales.view(E, N // 128, K // 128)


class MoEBlock:
    def __init__(self, generator=None):
        rnd = lambda *s: torch.randn(s, generator=generator, device="cuda")  # noqa: E731
        self.gamma = (1 + 0.1 * rnd(HIDDEN)).bfloat16()
        self.next_gamma = (1 + 0.1 * rnd(HIDDEN)).bfloat16()
        self.router = (rnd(HIDDEN, EXPERTS) * HIDDEN ** -0.5).bfloat16()
        self.bias = 0.01 * rnd(EXPERTS)
        self.up = quantize_experts(rnd(EXPERTS, 2 * INNER, HIDDEN) * HIDDEN ** -0.5)
        self.down = quantize_experts(rnd(EXPERTS, HIDDEN, INNER) * INNER ** -0.5)
        self.ws = qz.Workspace()

    def __call__(self, x, attention, n_tokens=None):
        """x [tokens, hidden]: the residual stream; attention: what the block before it adds; n_tokens: how many of a
        padded step's rows are tokens. Returns the residual stream behind the block, and its norm and codes."""
        x, normed, codes, scales = qz.qz_residual_rmsnorm(x, self.gamma, y=attention, normed=True, fp8=True)
        logits = normed @ self.router
        _, gates, offsets, row_token, token_row = qz.qz_moe_route(logits, TOP_K, score=qz.SCORE_SIGMOID, bias=self.bias,
                                                                  groups=4, top_groups=2, group_best=2, n_tokens=n_tokens, ws=self.ws)
        h = qz.qz_moe_gemm_fp8_swiglu(codes, scales, *self.up, offsets, row_token)
        rows = qz.qz_moe_gemm_fp8(*h, *self.down, offsets)
        return qz.qz_residual_rmsnorm(x, self.next_gamma, y=rows, token_row=token_row, weights=gates, normed=True, fp8=True)


def main():
    torch.manual_seed(0)
    block = MoEBlock()
    prompt = torch.randn((700, HIDDEN), device="cuda").bfloat16()
    out = block(prompt, torch.randn_like(prompt))
    # a decode step of at most 16 tokens, captured once
    x, attention = torch.zeros((16, HIDDEN), device="cuda").bfloat16(), torch.zeros((16, HIDDEN), device="cuda").bfloat16()
    n = torch.full((1,), 16, dtype=torch.int32, device="cuda")
    block(x, attention, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = block(x, attention, n)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for tokens in (16, 3, 9):
        x.copy_(torch.randn_like(x))
        attention.copy_(torch.randn_like(x))
        n.fill_(tokens)
        start.record()
        graph.replay()
        end.record()
    torch.cuda.synchronize()
    assert qz.qz_device_error() == 0
    assert all(bool(torch.isfinite(t.float()).all()) for t in (out[0], out[1], step[0], step[1]))
    print(f"prompt of {prompt.shape[0]} tokens, then decode steps of up to {x.shape[0]}: last step {start.elapsed_time(end) * 1e3:.0f} us")


if __name__ == "__main__":
    main()
