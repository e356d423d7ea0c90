"""Routing of tokens to experts against its definition in 64 bits: ids and the plan of the rows exactly."""
import math

import numpy as np
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref

pytestmark = pytest.mark.gpu


def check(logits, k, sigmoid=False, renorm=True, scale=1.0, bias=None, groups=1, top_groups=1, group_best=1, n=None, **kw):
    nt = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
    got = qz.qz_moe_route(logits, k, score=qz.SCORE_SIGMOID if sigmoid else qz.SCORE_SOFTMAX, renormalize=renorm, scale=scale,
                          bias=bias, groups=groups, top_groups=top_groups, group_best=group_best, n_tokens=nt, **kw)
    want = ref.route(logits, k, sigmoid, renorm, scale, bias, groups, top_groups, group_best, n)
    ids, w, off, row_token, token_row = [x.cpu().numpy() for x in got]
    np.testing.assert_array_equal(ids, want[0])
    np.testing.assert_array_equal(off, want[2])
    np.testing.assert_array_equal(row_token, want[3])
    np.testing.assert_array_equal(token_row, want[4])
    assert np.all(np.abs(w - want[1]) <= ref.weight_bound(logits, want[1])), np.abs(w - want[1]).max()
    return got


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("T", [1, 2, 17, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("E, k", [(8, 2), (60, 4), (64, 8), (128, 8), (256, 8), (257, 16), (512, 6)])
def test_softmax_without_bias(T, E, k):
    g = gen(T * 1000 + E)
    dt = torch.float32 if (T + E) % 2 else torch.bfloat16
    check((torch.randn((T, E), generator=g, device="cuda") * 2).to(dt), k, renorm=bool(T % 2), scale=1.5)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("E, k, G, top, best", [(256, 8, 8, 4, 2), (160, 6, 8, 3, 1), (60, 4, 4, 2, 2), (384, 8, 1, 1, 1),
                                                (64, 8, 32, 5, 2), (32, 3, 32, 3, 1), (512, 16, 16, 16, 2), (9, 9, 3, 3, 2)])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("T", [5, 333])
def test_bias_and_groups(sigmoid, E, k, G, top, best, biased, T):
    g = gen(E * 7 + T)
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    logits = torch.randn((T, E), generator=g, device="cuda") * 1.5
    check(logits, k, sigmoid, renorm=T == 5, scale=2.5, bias=bias, groups=G, top_groups=top, group_best=best)
    check(logits.bfloat16(), k, sigmoid, renorm=T != 5, bias=bias, groups=G, top_groups=top, group_best=best)


def test_ties_go_to_the_lowest_index():
    logits = torch.zeros((70, 96), device="cuda")
    check(logits, 5)
    check(logits, 5, sigmoid=True, bias=torch.zeros(96, device="cuda"))
    check(logits, 5, sigmoid=True, groups=8, top_groups=3, group_best=2)
    check(logits, 7, bias=torch.full((96,), -0.5, device="cuda"), groups=8, top_groups=3, group_best=2)
    g = gen(1)
    coarse = torch.randint(-2, 3, (500, 128), generator=g, device="cuda").float()
    check(coarse, 8)
    check(coarse, 8, sigmoid=True, bias=torch.randint(0, 2, (128,), generator=g, device="cuda") * 0.25, groups=8, top_groups=3, group_best=2)
    zero = torch.where(torch.rand((64, 40), generator=g, device="cuda") < 0.5, 0.0, -0.0)
    check(zero, 6)


def test_keys_that_32_bits_cannot_tell_apart():
    """Biases that cancel the scores to a few units in the last place, and differ from one another in 64 bits."""
    g = gen(2)
    T, E = 400, 64
    row = torch.randn(E, generator=g, device="cuda")
    bias = (0.75 - torch.sigmoid(row.double())).float()           # every key is 0.75 within a rounding of fp32
    check(row.expand(T, E).contiguous(), 8, sigmoid=True, bias=bias)
    check(row.expand(T, E).contiguous(), 8, sigmoid=True, bias=bias, groups=8, top_groups=2, group_best=2)
    check(row.expand(T, E).contiguous(), 8, sigmoid=True, bias=bias, groups=16, top_groups=5, group_best=1)
    p = torch.softmax(row.double(), 0)
    check(row.expand(T, E).contiguous(), 8, bias=(0.5 - p).float(), groups=4, top_groups=2, group_best=2)
    check(row.expand(T, E).contiguous(), 8, bias=(0.5 - p).float())


def test_masked_logits_and_biases():
    g = gen(3)
    T, E, k = 150, 72, 6
    logits = torch.randn((T, E), generator=g, device="cuda")
    u = torch.rand((T, E), generator=g, device="cuda")
    logits = torch.where(u < 0.3, -math.inf, logits)
    logits = torch.where(u > 0.95, math.nan, logits)
    logits = torch.where((u > 0.5) & (u < 0.52), torch.finfo(torch.float32).min, logits)
    logits[3] = -math.inf                                         # nothing open at all
    logits[4] = math.nan
    logits[5] = torch.finfo(torch.float32).min                    # everything open
    logits[6, 1:] = -math.inf                                     # one expert
    logits[7, 10:] = -math.inf
    bias = torch.randn(E, generator=g, device="cuda") * 0.2
    bias[5], bias[9] = -math.inf, math.nan
    for sigmoid in (False, True):
        for renorm in (False, True):
            check(logits, k, sigmoid, renorm)
            check(logits, k, sigmoid, renorm, bias=bias)
            check(logits, k, sigmoid, renorm, bias=bias, groups=8, top_groups=2, group_best=2)
            check(logits, k, sigmoid, renorm, groups=9, top_groups=3, group_best=1)
    logits[8, 4] = math.inf                                       # the largest finite value
    logits[9, :3] = math.inf
    bias[7] = math.inf
    check(logits, k)
    check(logits, k, sigmoid=True, bias=bias)


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("big", [math.inf, torch.finfo(torch.float32).max, 2.0 ** 127])
@pytest.mark.parametrize("T", [3, 200])
def test_group_scores_past_the_range_of_fp32(sigmoid, big, T):
    """Two keys of a group whose sum is infinite in 32 bits: more such groups than are kept, as many, fewer; and the
    same below zero, where the group stays open."""
    g = gen(8)
    logits = torch.randn((T, 64), generator=g, device="cuda")
    for n in (1, 2, 3, 8):
        for sign in (1.0, -1.0) if math.isfinite(big) else (1.0,):
            bias = torch.zeros(64, device="cuda")
            bias.view(8, 8)[8 - n:, 2:4] = sign * big
            check(logits, 4, sigmoid, bias=bias, groups=8, top_groups=2, group_best=2)
            bias.view(8, 8)[8 - n:] = sign * big
            check(logits, 6, sigmoid, bias=bias, groups=8, top_groups=2, group_best=2)
    bias = torch.zeros(64, device="cuda")
    bias.view(8, 8)[:, 0] = big                                   # one such key a group: in 64 bits too, all sums are the same
    check(logits, 4, sigmoid, bias=bias, groups=8, top_groups=2, group_best=2)


def test_scores_that_underflow_keep_their_ratios():
    g = gen(4)
    logits = torch.randn((40, 32), generator=g, device="cuda") - 300.0
    check(logits, 4, sigmoid=True)
    check(logits, 4, sigmoid=True, renorm=False)
    wide = torch.randn((40, 32), generator=g, device="cuda") * 60
    check(wide, 8)
    check(wide, 8, sigmoid=True)


@pytest.mark.parametrize("T, n", [(10, 0), (10, 10), (10, 99), (10, -3), (77, 64), (600, 129), (600, 0)])
def test_padded_steps(T, n):
    g = gen(T + n)
    check(torch.randn((T, 64), generator=g, device="cuda"), 4, n=n)


def test_no_tokens():
    got = qz.qz_moe_route(torch.empty((0, 24), device="cuda"), 3)
    assert got[0].shape == (0, 3) and got[2].tolist() == [0] * 25


def test_strided_logits_and_given_outputs():
    g = gen(6)
    wide = torch.randn((45, 200), generator=g, device="cuda")
    out = dict(ids=torch.empty((45, 4), dtype=torch.int32, device="cuda"), weights=torch.empty((45, 4), device="cuda"),
               offsets=torch.empty(97, dtype=torch.int32, device="cuda"), row_token=torch.empty(180, dtype=torch.int32, device="cuda"),
               token_row=torch.empty((45, 4), dtype=torch.int32, device="cuda"))
    got = check(wide[:, 3:99], 4, **out)
    assert got[0] is out["ids"] and got[4] is out["token_row"]
    check(wide.bfloat16()[:, 1:98], 4)


def test_the_same_plan_on_every_call():
    g = gen(7)
    logits = torch.randn((5000, 256), generator=g, device="cuda")
    a = qz.qz_moe_route(logits, 8, ws=qz.Workspace())
    for _ in range(3):
        b = qz.qz_moe_route(logits, 8)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    np.testing.assert_array_equal(a[3].cpu().numpy(), ref.plan(a[0].cpu().numpy(), 256)[1])


@pytest.mark.parametrize("T", [1, 15, 16, 17, 33])
def test_smallest_and_largest_shapes(T):
    """One expert, every expert chosen, groups of one, groups that are no power of two, 512 experts."""
    g = gen(9 + T)

    def rand(*s):
        return torch.randn(s, generator=g, device="cuda")

    check(rand(T, 1), 1)
    check(rand(T, 16), 16)
    check(rand(T, 2), 1, sigmoid=True, bias=rand(2))
    check(rand(T, 32), 1, groups=32, top_groups=32)
    check(rand(T, 33), 3, groups=11, top_groups=2, group_best=2)
    check(rand(T, 34), 5, sigmoid=True, bias=0.01 * rand(34), groups=17, top_groups=3, group_best=2)
    check(rand(T, 512), 16, sigmoid=True, renorm=False, groups=2, top_groups=1)
    check(rand(T, 512), 16, sigmoid=True, bias=0.1 * rand(512), groups=32, top_groups=1, group_best=2)
