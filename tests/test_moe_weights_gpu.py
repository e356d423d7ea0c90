"""The routing's weights against 64 bits, with bounds that go by each weight's own arithmetic, in half units of fp32.

expf: 2 units in the last place (4 half units); a difference of logits is rounded once, which moves its exponential by that
many half units as it has e-folds; a sum over 32 lanes 5, a quotient 1 (the fast one of a plain sigmoid 4), the scale 1.
"""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("E, k", [(8, 2), (64, 8), (256, 8), (512, 16)])
@pytest.mark.parametrize("spread", [0.01, 2.0, 20.0])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("renorm", [True, False])
def test_weights_are_as_exact_as_their_arithmetic(E, k, spread, sigmoid, renorm):
    g = torch.Generator(device="cuda").manual_seed(E + k)
    logits = spread * torch.randn((500, E), generator=g, device="cuda")
    ids, w = qz.qz_moe_route(logits, k, score=qz.SCORE_SIGMOID if sigmoid else qz.SCORE_SOFTMAX, renormalize=renorm, scale=0.7)[:2]
    l = logits.double()
    c = l.gather(1, ids.long())
    scale = float(torch.tensor(0.7, dtype=torch.float32))
    if not sigmoid:
        over = c if renorm else l                                 # what the sum is over
        d, do = over.amax(dim=1, keepdim=True) - c, over.amax(dim=1, keepdim=True) - over
        p = torch.softmax(over, dim=1)
        want = torch.exp(-d) / torch.exp(-do).sum(dim=1, keepdim=True)
        adds = 5 if renorm else 5 + E // 32
        bound = (d + 4) + (p * (do + 4)).sum(dim=1, keepdim=True) + adds + 2
    elif renorm:
        m = c.amax(dim=1, keepdim=True).clamp(max=0.0)
        q = torch.where(c >= 0, torch.sigmoid(c), torch.exp(c - m) * torch.sigmoid(-c))
        want = q / q.sum(dim=1, keepdim=True)
        each = torch.where(c >= 0, 4.0, (m - c) + 8.0)
        bound = each + (want * each).sum(dim=1, keepdim=True) + 5 + 2
    else:
        want, bound = torch.sigmoid(c), torch.full_like(c, 10.0)
    want = want * scale
    off = ((w.double() - want).abs() - 2.0 ** -148) / want / U
    assert bool((off <= bound * 1.001).all()), float((off / bound).max())
