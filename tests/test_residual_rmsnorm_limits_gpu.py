"""The residual norm of rows with infinities, and of no rows."""
import math

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gather", [False, True])
def test_a_row_with_infinities_is_zero_but_in_their_places(dt, gather):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((6, 384), generator=g, device="cuda").to(dt)
    y = torch.randn((6, 384), generator=g, device="cuda").bfloat16()
    gamma = torch.ones(384, device="cuda", dtype=dt)
    x[1, 5], x[2, 300] = math.inf, -math.inf
    y[4, 130] = math.inf
    x[5, 7], y[5, 7] = math.inf, -math.inf                       # their sum is NaN
    rows = torch.arange(6, device="cuda").int().view(6, 1) if gather else None
    r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, y, rows, normed=True, fp8=True)
    for t, c in ((1, 5), (2, 300), (4, 130)):
        there = torch.arange(384, device="cuda") == c
        assert math.isinf(float(r[t, c])) and math.isnan(float(n[t, c])) and not n[t, ~there].any()
        assert int(codes[t, c]) & 0x7F == 0x7F and not (codes[t, ~there] & 0x7F).any()
        assert bool((scales[t] == torch.tensor(1e-12, device="cuda") / torch.tensor(448.0, device="cuda")).all())
    assert bool(torch.isnan(n[5].float()).all())
    assert bool(torch.isfinite(n[[0, 3]].float()).all()) and bool(n[[0, 3]].any(dim=1).all())


def test_no_rows():
    x, gamma = torch.empty((0, 256), device="cuda"), torch.ones(256, device="cuda")
    for kw in (dict(), dict(y=torch.empty((0, 256), device="cuda").bfloat16())):
        r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, normed=True, fp8=True, **kw)
        assert r.shape == n.shape == codes.shape == (0, 256) and scales.shape == (0, 2)
