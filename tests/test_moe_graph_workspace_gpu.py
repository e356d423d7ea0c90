"""A captured routing after its workspace has grown: its replays write into memory that is still the workspace's."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
from test_moe_route_gpu import check, gen

pytestmark = pytest.mark.gpu


def test_a_captured_step_after_its_workspace_grew():
    ws, E, k = qz.Workspace(), 256, 8
    small, large = (torch.randn((T, E), generator=gen(T), device="cuda") for T in (77, 9000))
    qz.qz_moe_route(small, k, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = qz.qz_moe_route(small, k, ws=ws)
    first = ws.buf.numel()
    want = [t.clone() for t in qz.qz_moe_route(large, k, ws=ws)]
    assert ws.buf.numel() > first
    others = [torch.full((first,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(64)]   # would take what was freed
    for seed in (1, 2):
        small.copy_(torch.randn(small.shape, generator=gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 0x5A).all()) for t in others)
        assert all(torch.equal(a, b) for a, b in zip(step, check(small, k)))
        assert all(torch.equal(a, b) for a, b in zip(want, qz.qz_moe_route(large, k, ws=ws)))
