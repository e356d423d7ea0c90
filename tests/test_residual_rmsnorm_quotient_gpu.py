"""The norm's quotient: r / root is formed as one, so that rows of equal magnitudes give exactly gamma."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

pytestmark = pytest.mark.gpu

H = 1024
VALUES = [1, 3, 41, 47, 49, 55, 61, 83, 97, 107, 109, 115, 121, 123, 127]    # their squares' sums are exact: 127^2 * 1024 < 2^24


def rows(dt):
    g = torch.Generator(device="cuda").manual_seed(1)
    sign = torch.where(torch.rand((len(VALUES), H), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    v = torch.tensor(VALUES, dtype=torch.float32, device="cuda")[:, None] * sign
    return v.to(dt), sign, (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dt)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gather", [True, False])
def test_rows_of_equal_magnitudes_give_gamma(dt, gather):
    x, sign, gamma = rows(dt)
    kw = {}
    if gather:                                                    # the form of a CTA per row: a block that adds nothing
        kw = dict(y=torch.empty((0, H), device="cuda").bfloat16(), token_row=torch.full((len(VALUES), 2), -1, device="cuda").int())
    r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, eps=1e-30, normed=True, fp8=True, **kw)
    want = sign * gamma.float()
    c, s, _ = qz.qz_quantize_fp8(want, qz.FP8_GROUP_1x128)
    assert torch.equal(r, x) and torch.equal(n, want.bfloat16())
    assert torch.equal(codes, c) and torch.equal(scales, s)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_and_so_behind_the_block(dt):
    y, sign, gamma_y = rows(torch.bfloat16)
    gamma_y = gamma_y.to(dt)
    x = torch.zeros((len(VALUES), H), dtype=dt, device="cuda")
    r = qz.qz_residual_rmsnorm(x, y=y, gamma_y=gamma_y, eps=1e-30)[0]
    assert torch.equal(r, (sign * gamma_y.float()).to(dt))
