"""The residual norm around a block against its definition in 64 bits."""
import math

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref

pytestmark = pytest.mark.gpu


def data(T, H, k, dt, seed, rows=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = rnd(T, H)
    x[:, ::37] *= 25
    n = T * max(k, 1) if rows is None else rows
    return dict(x=x.to(dt), gamma=(1 + 0.2 * rnd(H)).to(dt), y=rnd(n, H).bfloat16(), gamma_y=(1 + 0.2 * rnd(H)).to(dt),
                token_row=torch.randint(-1, n + 2, (T, k), generator=g, device="cuda").int() if k else None,
                weights=torch.rand((T, k), generator=g, device="cuda") if k else None)


def check(d, alpha=1.0, eps=1e-6, **out):
    x = d["x"].clone()
    got = qz.qz_residual_rmsnorm(d["x"], d.get("gamma"), y=d.get("y"), token_row=d.get("token_row"), weights=d.get("weights"),
                                 alpha=alpha, gamma_y=d.get("gamma_y"), eps=eps, **out)
    r, n, br, bn = ref.residual_norm(x, d.get("gamma"), d.get("y"), d.get("token_row"), d.get("weights"), alpha, d.get("gamma_y"), eps)
    if got[0] is not None:
        if x.dtype == torch.float32:
            assert bool(((got[0].double() - r).abs() <= br + U32 * r.abs()).all())
        else:
            ref.check_bf16(got[0], r, br, "r")
    if got[1] is not None:
        ref.check_bf16(got[1], n, bn, "n")
    if got[2] is not None:
        ref.check_codes(got[2], got[3], n, bn, "codes")
    return got


U32 = 2.0 ** -24


@pytest.mark.parametrize("T, H", [(1, 128), (3, 256), (2, 896), (17, 2048), (5, 4096), (1, 4224), (2, 8192), (3, 8320), (2, 16384)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [0, 1, 3, 8])
@pytest.mark.parametrize("post", [True, False])
def test_all_outputs(T, H, dt, k, post):
    d = data(T, H, k, dt, T * H + k)
    if not post:
        d["gamma_y"] = None
    check(d, alpha=0.37 if post else 1.0, normed=True, fp8=True)


@pytest.mark.parametrize("H", [8, 16, 24, 200, 1000, 4104, 16376])
def test_odd_hidden_sizes_without_codes(H):
    check(data(3, H, 2, torch.bfloat16, H), normed=True)
    d = data(3, H, 0, torch.float32, H)
    d["gamma_y"] = None
    check(d, normed=True)


def test_each_output_alone():
    d = data(9, 512, 2, torch.bfloat16, 5)
    full = check(d, normed=True, fp8=True)
    assert torch.equal(check(d)[0], full[0])
    assert torch.equal(check(d, out=None, normed=True)[1], full[1])
    c = check(d, out=None, fp8=True)
    assert torch.equal(c[2], full[2]) and torch.equal(c[3], full[3]) and c[0] is None and c[1] is None
    only = dict(d, gamma=None)
    assert torch.equal(check(only)[0], full[0])
    plain = dict(x=d["x"], gamma=d["gamma"])                    # no block: a norm alone
    assert torch.equal(check(plain, normed=True)[0], d["x"])


def test_in_place_and_strides():
    g = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((31, 3, 640), generator=g, device="cuda").bfloat16()
    d = data(31, 640, 0, torch.bfloat16, 8)
    d["x"] = wide[:, 1]
    want = check(d, normed=True, fp8=True)
    before = wide.clone()
    got = check(d, normed=True, fp8=True, out=wide[:, 1])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(wide[:, 0], before[:, 0]) and torch.equal(wide[:, 2], before[:, 2])
    ywide = torch.randn((31, 1288), generator=g, device="cuda").bfloat16()
    d["y"] = ywide[:, 8:648]
    check(d, normed=True)


def test_rows_that_are_not_there():
    d = data(6, 256, 4, torch.float32, 11)
    d["token_row"][:] = -1
    d["gamma_y"] = None
    got = check(d, normed=True, fp8=True)
    assert torch.equal(got[0], d["x"])                          # nothing was added
    d["gamma_y"] = d["gamma"]
    assert torch.equal(check(d)[0], d["x"])                     # nor from a norm of nothing
    d = data(6, 256, 2, torch.bfloat16, 12, rows=1)
    d["token_row"] = torch.tensor([[0, 0], [0, 1], [-1, 0], [2147483647, -2147483648], [0, 0], [1, 1]], dtype=torch.int32, device="cuda")
    check(d, normed=True)
    d["y"] = d["y"][:0]
    d["gamma_y"] = None
    assert torch.equal(check(d)[0], d["x"])


def test_rows_of_zeros_tiny_and_large_values():
    d = data(4, 512, 0, torch.float32, 13)
    d["gamma_y"] = None
    d["x"][0], d["y"][0] = 0, 0
    d["x"][1] *= 1e-20
    d["y"][1] = 0
    d["x"][2] *= 1e15
    got = check(d, normed=True, fp8=True, eps=1e-12)
    assert not got[2][0].any() and bool((got[3][0] == torch.tensor(1e-12, device="cuda") / torch.tensor(448.0, device="cuda")).all())


def test_a_sum_of_squares_past_the_range_gives_zeros():
    d = data(3, 256, 0, torch.float32, 15)
    d["gamma_y"] = None
    d["x"][1] *= 1e25                                            # squares past 3.4e38
    for y in (d["y"], None):
        got = qz.qz_residual_rmsnorm(d["x"], d["gamma"], y, normed=True, fp8=True)
        assert not got[1][1].any() and not (got[2][1] & 0x7F).any()
        assert bool(torch.isfinite(got[1].float()).all()) and bool(got[1][0].any())


def test_nan_and_infinities_stay_in_their_row():
    d = data(8, 256, 2, torch.bfloat16, 14)
    d["token_row"] = torch.arange(16, dtype=torch.int32, device="cuda").view(8, 2)
    clean = qz.qz_residual_rmsnorm(d["x"], d["gamma"], d["y"], d["token_row"], d["weights"], normed=True, fp8=True)
    d["x"][1, 3] = math.nan
    d["x"][2, 5] = math.inf
    d["y"][7, 9] = -math.inf                                     # token 3
    d["weights"][4, 1] = math.nan
    got = qz.qz_residual_rmsnorm(d["x"], d["gamma"], d["y"], d["token_row"], d["weights"], normed=True, fp8=True)
    for a, b in zip(clean, got):
        assert torch.equal(a[[0, 5, 6, 7]], b[[0, 5, 6, 7]])
    assert bool(torch.isnan(got[1][[1, 4]].float()).all()) and bool(torch.isnan(got[1][2, 5]).item()) and bool(torch.isnan(got[1][3, 9]).item())


def test_codes_are_the_quantizers():
    """What the norm encodes is what qz_quantize_fp8 makes of the same fp32 row: gamma of 1 and an exact norm."""
    x = torch.where(torch.rand((5, 1024), device="cuda") < 0.5, 1.0, -1.0) * 2.0
    x = torch.cat([x, -x], dim=1)
    gamma = torch.randn(2048, device="cuda")
    _, _, codes, scales = qz.qz_residual_rmsnorm(x, gamma, eps=1e-30, fp8=True)
    n = torch.sign(x) * gamma                                    # mean of squares 4, root 2: exact
    c, s, _ = qz.qz_quantize_fp8(n, qz.FP8_GROUP_1x128)
    assert torch.equal(codes, c) and torch.equal(scales, s)
