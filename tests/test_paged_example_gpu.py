"""The attention-layer example, prompts and then single tokens, against the same layer in 64 bits over the values
that its cache and its INT4 weights stand for. The layer rounds to bf16 three times (q, k and v, the
attention's output, the result: 2^-9 each) and keeps at least 8 bits of the probabilities, each an independent
error of the sums behind it, so the result is off by well under 2^-6 of its norm."""
import os
import sys

import pytest
import torch

from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def weight(lin, k):
    """The values of an INT4 layer's weight [K, N]."""
    shifts = torch.arange(0, 32, 4, device="cuda")
    q = (lin.qweight[:, None, :].long() >> shifts[None, :, None]) & 15
    q = torch.where(q > 7, q - 16, q).reshape(k, -1).double()
    return q * lin.scale.double().repeat_interleave(128, dim=0)


def test_layer_over_steps():
    import paged_attention as ex
    import bit_quantized_linear_quantizers_gb300 as qz
    g = torch.Generator(device="cuda").manual_seed(0)
    prompts, P = [70, 1, 200], 16
    pages = sum(-(-(n + 4) // P) for n in prompts)
    req, layer = ex.Requests(len(prompts), 204, pages, P), ex.AttentionLayer(pages, P, g)
    wq, wo = weight(layer.qkv, ex.HIDDEN), weight(layer.o, ex.HEADS * ex.DIM)
    for new in (prompts, [1, 1, 1], [1, 0, 2], [2, 3, 1]):
        x = torch.randn((sum(new), ex.HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        y = layer(x, req, req.step(new))
        q = (x.double() @ wq)[:, :ex.HEADS * ex.DIM].view(-1, ex.HEADS, ex.DIM)
        c, rows, at = layer.cache, [], 0
        for b, n in enumerate(new):
            L = int(req.lens[b])
            ids = req.table[b, :-(-L // P)].long()
            K, V = (((codes[ids].view(torch.float8_e4m3fn).double() * s[ids].double()[..., None, None]).transpose(0, 1)
                     .reshape(ex.KV_HEADS, -1, ex.DIM)[:, :L].repeat_interleave(ex.HEADS // ex.KV_HEADS, dim=0))
                    for codes, s in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)))
            s = torch.einsum("nhd,hld->hnl", q[at:at + n], K) * ex.DIM ** -0.5
            hide = torch.arange(L, device="cuda")[None] > (L - n + torch.arange(n, device="cuda"))[:, None]
            p = torch.softmax(s.masked_fill(hide, float("-inf")), dim=-1)
            rows.append(torch.einsum("hnl,hld->nhd", p, V).reshape(n, ex.HEADS * ex.DIM))
            at += n
        want = torch.cat(rows) @ wo
        assert float((y.double() - want).norm() / want.norm()) < 2.0 ** -6
    assert req.lens.tolist() == [74, 5, 204] and int(req.head) == pages - sum(
        -(-(n + 4) // P) - -(-m // P) for n, m in zip(prompts, req.lens.tolist()))
    assert qz.qz_device_error() == 0


def test_example_runs(capsys):
    import paged_attention as ex
    ex.main()
    assert "4 requests, lengths [720, 53, 21, 276]" in capsys.readouterr().out
