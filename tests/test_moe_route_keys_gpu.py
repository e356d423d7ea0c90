"""Group scores whose keys cancel: what 32 bits leave of a sum is off by the roundings of its keys, however small it is."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
from test_moe_route_gpu import check, gen

pytestmark = pytest.mark.gpu


def test_two_groups_whose_biases_cancel():
    """Sums of 1.0000060 and 1.0000035; the keys near 100 are rounded by up to 4e-6."""
    logits = torch.tensor([[1.2e-5, 1.2e-5, 1.8e-5, -4e-6]], device="cuda")
    bias = torch.tensor([100.0, -100.0, 100.0, -100.0], device="cuda")
    ids = qz.qz_moe_route(logits, 2, score=qz.SCORE_SIGMOID, bias=bias, groups=2, top_groups=1, group_best=2)[0]
    assert ids.tolist() == [[0, 1]]


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("big", [16.0, 100.0, 1000.0, 1e6])
@pytest.mark.parametrize("raised", [1, 3])
@pytest.mark.parametrize("T", [7, 200])
def test_group_keys_that_cancel(sigmoid, big, raised, T):
    """Every group has keys near +big and near -big, and all sums lie within a few roundings of them: of one raised key a group
    the sum is what is left of both, and which of the others is its second best is as close."""
    g = gen(int(big) + raised)
    E, groups = 64, 8
    bias = torch.full((E,), -big, device="cuda")
    bias.view(groups, -1)[:, 2:2 + raised] = big
    spread = big * 2.0 ** -22 * (1 if sigmoid else 64)            # a softmax of 64 has slopes of 1/64
    logits = 0.3 + spread * torch.randn((T, E), generator=g, device="cuda")
    for top in (1, 3, 7):
        check(logits, 6, sigmoid, bias=bias, groups=groups, top_groups=top, group_best=2)
    one = bias.clone()
    one.view(groups, -1)[::2] = 0.0                               # and groups of small keys beside them
    check(logits, 6, sigmoid, bias=one, groups=groups, top_groups=3, group_best=2)


@pytest.mark.parametrize("big", [100.0, 1e6, 2.0 ** 127])
def test_groups_of_few_open_experts_beside_large_keys(big):
    """A group's score is the one open key where there is one alone; others' keys do not make it less exact."""
    g = gen(5)
    logits = torch.randn((150, 64), generator=g, device="cuda")
    logits.view(150, 8, 8)[:, ::3, 1:] = -float("inf")
    bias = 0.1 * torch.randn(64, generator=g, device="cuda")
    bias.view(8, 8)[1, :2] = torch.tensor([big, -big], device="cuda")
    bias.view(8, 8)[4, :3] = -big
    for top in (2, 4):
        check(logits, 4, sigmoid=True, bias=bias, groups=8, top_groups=top, group_best=2)
        check(logits, 4, sigmoid=True, bias=bias, groups=8, top_groups=top, group_best=1)


@pytest.mark.parametrize("E, G, T", [(378, 7, 16), (378, 27, 700), (403, 13, 15), (403, 31, 40), (377, 13, 50), (379, 1, 50), (512, 32, 33)])
def test_sizes_around_the_default_limit_of_shared_memory(E, G, T):
    """16 warps' counts and keys of 378 experts are 48 KB, which with the kernel's own arrays is more than a launch has without asking."""
    g = gen(E + T)
    logits = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    check(logits, 6, sigmoid=True, bias=bias, groups=G, top_groups=min(G, 3), group_best=2)
    check(logits, 6, groups=G, top_groups=min(G, 3), group_best=2)
