"""A Workspace that grows keeps the buffers that captured graphs may hold (CPU)."""
import weakref

import torch

import bit_quantized_linear_quantizers_gb300 as qz


def test_what_a_workspace_outgrows_stays_allocated():
    ws = qz.Workspace(torch.device("cpu"))
    held, sizes = [], []
    for n in (300, 301, 5000, 40, 5001, 1 << 20):
        buf = ws.get(n)
        assert buf.numel() >= n
        held.append(weakref.ref(buf))
        sizes.append(buf.numel())
        del buf
    assert all(r() is not None for r in held)
    assert sum(b.numel() for b in ws.outgrown) < ws.buf.numel()
    assert sizes == sorted(sizes)
    lost = held[0]
    del ws
    assert lost() is None                                         # and no longer than it lives
