"""The gate of the experts' products, h = g u / (1 + exp(-g)), seen through the fp32 scales of its codes."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                                    # half a step of fp32, relative


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_gates_of_any_size_are_as_exact_as_small_ones(sign):
    """One product a row, exact by its powers of two: g = sign x, u = 2^100 x. All 128 columns of a row are alike, so that the
    scale is h / 448.
    In half steps: 2^t 4 (2 units in the last place), the correction of its exponent 1, 1 + exp 1, its reciprocal 2, and a
    rounding each of g times it, of u times that and of the scale: 11, to first order (1 % for the rest)."""
    x = torch.cat([torch.linspace(0.01, 87.0, 4001, device="cuda"), torch.tensor([2.0 ** -20, 1.0, 2.0, 64.0], device="cuda")])
    T, K = x.numel(), 128
    qA = torch.zeros((T, K), dtype=torch.uint8, device="cuda")
    qA[:, 0] = 0x38                                               # 1.0
    qW = torch.zeros((1, 256, K), dtype=torch.uint8, device="cuda")
    qW[0, :128, 0] = 0x38 if sign > 0 else 0xB8
    qW[0, 128:, 0] = 0x38
    sW = torch.tensor([1.0, 2.0 ** 100], device="cuda").view(1, 2, 1)
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    codes, scales = qz.qz_moe_gemm_fp8_swiglu(qA, x.view(T, 1), qW, sW, offsets)
    g = x.double() * sign
    want = (g * (x.double() * 2.0 ** 100) / (1 + torch.exp(-g))).abs() / 448
    off = ((scales[:, 0].double() - want).abs() / want / U).max().item()
    assert off <= 11 * 1.01, off
    assert bool((codes == (0x7E if sign > 0 else 0xFE)).all())    # each is the largest of its group


def test_gates_past_the_range_of_exp():
    """exp(-g) beyond fp32 on either side, gates near fp32's limit, infinities and NaN."""
    inf, nan = float("inf"), float("nan")
    v = [-89.0, -127.0, -1e4, -2.4e38, -3.4e38, 89.0, 129.0, 1e4, inf, -inf, nan]
    x = torch.tensor(v, device="cuda")
    T, K = len(v), 128
    qA = torch.zeros((T, K), dtype=torch.uint8, device="cuda")
    qA[:, 0] = 0x38
    qW = torch.zeros((1, 256, K), dtype=torch.uint8, device="cuda")
    qW[0, :, 0] = 0x38
    sW = torch.tensor([1.0, 2.0 ** -30], device="cuda").view(1, 2, 1)
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    codes, scales = qz.qz_moe_gemm_fp8_swiglu(qA, x.view(T, 1), qW, sW, offsets)
    least = (torch.tensor(1e-12, device="cuda") / torch.tensor(448.0, device="cuda")).item()
    assert scales[:5, 0].tolist() == [least] * 5 and not (codes[:5] & 0x7F).any()
    want = (x[5:8].double() ** 2 * 2.0 ** -30 / 448)
    assert bool(((scales[5:8, 0].double() - want).abs() <= 4 * U * want).all())
    assert not torch.isfinite(scales[8, 0]) and bool(((codes[8:] & 0x7F) == 0x7F).all())
