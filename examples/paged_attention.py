"""One attention layer of a decoder served on a paged FP8 KV cache.

    python examples/paged_attention.py

Runs the library's calls as a serving loop makes them, step after step without a wait on the host:
block tables and slot maps from the requests' lengths (qz_block_tables), the INT4 q, k, v
projections (qz_gemm_w4a16), the write of the new tokens (qz_kv_append_fp8_paged), attention over
the cache (qz_attn_fp8_paged) and the output projection. Sizes are those of the Qwen3-0.6B linear
set: 16 query heads on 8 KV heads of 128, hidden size 1024; random weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_linear_quantizers_gb300 as qz  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM = 1024, 16, 8, 128
W4A16_TOKENS = 64                                    # tokens that one W4A16 call takes


class Linear:
    """An INT4 linear layer [K, N]: bf16 tokens in and out."""

    def __init__(self, w):
        self.qweight, self.scale, _ = qz.qz_quantize_int4_g128(w)
        self.n = w.shape[1]

    def __call__(self, x):
        y = torch.empty((x.shape[0], self.n), dtype=torch.bfloat16, device=x.device)
        for t in range(0, x.shape[0], W4A16_TOKENS):
            qz.qz_gemm_w4a16(x[t:t + W4A16_TOKENS], self.qweight, self.scale, Y=y[t:t + W4A16_TOKENS])
        return y


class Requests:
    """The requests' side of the cache: lengths, block table and free pages, all on the GPU."""

    def __init__(self, count, max_tokens, pages, page_size):
        self.page_size = page_size
        self.table = torch.full((count, -(-max_tokens // page_size)), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda").to(torch.int32)
        self.head = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(count, dtype=torch.int32, device="cuda")

    def step(self, new):
        """Room for `new` tokens of each request; once per step, for all layers."""
        lens = torch.tensor(new, dtype=torch.int32).cuda()
        slots, positions, cu, self.lens, self.head = qz.qz_block_tables(
            self.lens, lens, self.table, self.free, self.head, self.page_size, sum(new))
        return slots, positions, cu, max(new)


class AttentionLayer:
    def __init__(self, pages, page_size, generator=None):
        w = lambda k, n: torch.randn((k, n), generator=generator, device="cuda") * 0.02  # noqa: E731
        self.qkv = Linear(w(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM))
        self.o = Linear(w(HEADS * DIM, HIDDEN))
        self.cache = qz.PagedKV.empty(pages, KV_HEADS, page_size, DIM)
        self.ws = qz.Workspace()

    def __call__(self, x, requests, step):
        slots, _, cu, max_new = step
        qkv = self.qkv(x).view(-1, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split((HEADS, KV_HEADS, KV_HEADS), dim=1)          # slices: the calls take their strides
        qz.qz_kv_append_fp8_paged(k, v, slots, self.cache)
        out, _ = qz.qz_attn_fp8_paged(q, self.cache, requests.table, requests.lens, cu, max_new, DIM ** -0.5, ws=self.ws)
        return self.o(out.view(-1, HEADS * DIM))


def main():
    torch.manual_seed(0)
    prompts, page_size, tokens = [700, 33, 1, 256], 16, 20
    most = max(prompts) + tokens
    pages = sum(-(-(n + tokens) // page_size) for n in prompts)
    requests = Requests(len(prompts), most, pages, page_size)
    layer = AttentionLayer(pages, page_size)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for new in [prompts] + [[1] * len(prompts)] * tokens:
        x = torch.randn((sum(new), HIDDEN), device="cuda").to(torch.bfloat16)
        start.record()
        y = layer(x, requests, requests.step(new))
        end.record()
    torch.cuda.synchronize()
    assert qz.qz_device_error() == 0 and bool(torch.isfinite(y.float()).all())
    print(f"{len(prompts)} requests, lengths {requests.lens.tolist()}, {int(requests.head)} of {pages} pages used; "
          f"last step {start.elapsed_time(end) * 1e3:.0f} us")


if __name__ == "__main__":
    main()
