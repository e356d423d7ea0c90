"""The experts' products over ragged rows against their definition in 64 bits."""
import math

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz
import moe_ref as ref

pytestmark = pytest.mark.gpu


def data(counts, tokens, N, K, seed, gather=True, tail=0):
    """Experts with the given row counts, rows in any order of the tokens; `tail` rows of no expert behind them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    rows = sum(counts) + tail
    x = rnd(tokens if gather else rows, K)
    x[:, ::41] *= 20
    qA, sA = ref.quantize_rows(x)
    qW, sW = ref.quantize_blocks(rnd(len(counts), N, K) * 0.05)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    rt = torch.randint(0, tokens, (rows,), generator=g, device="cuda").int() if gather else None
    return dict(qA=qA, sA=sA, qW=qW, sW=sW, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), row_token=rt)


def check(d, which="both"):
    K = d["qA"].shape[1]
    P, S = ref.product(**d)
    B = ref.product_bound(S, K)
    there = ~torch.isnan(P[:, 0])
    rows, N = P.shape
    if which != "swiglu":
        Y = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
        qz.qz_moe_gemm_fp8(d["qA"], d["sA"], d["qW"], d["sW"], d["offsets"], d["row_token"], Y=Y)
        ref.check_bf16(Y[there], P[there], B[there], "Y")
        assert bool((Y[~there] == 7.0).all())
    if which != "plain" and N % 256 == 0:
        codes = torch.full((rows, N // 2), 0x55, dtype=torch.uint8, device="cuda")
        scales = torch.full((rows, N // 256), 7.0, device="cuda")
        qz.qz_moe_gemm_fp8_swiglu(d["qA"], d["sA"], d["qW"], d["sW"], d["offsets"], d["row_token"], codes=codes, scales=scales)
        h, bh = ref.swiglu(P[there], B[there])
        ref.check_codes(codes[there], scales[there], h, bh, "swiglu")
        assert bool((codes[~there] == 0x55).all()) and bool((scales[~there] == 7.0).all())
    assert qz.qz_device_error() == 0


@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [5, 0, 17, 1], [128, 127, 129, 1], [0, 0, 0], [300], [2] * 40,
                                    [1, 200, 3, 64, 31, 33, 0, 260]])
@pytest.mark.parametrize("N, K", [(128, 128), (256, 256), (768, 640), (1280, 1152)])
def test_ragged_rows(counts, N, K):
    check(data(counts, 23, N, K, sum(counts) + N))
    check(data(counts, 23, N, K, sum(counts) + N, gather=False))


def test_rows_of_no_expert_are_not_written():
    check(data([3, 0, 130], 50, 512, 384, 1, tail=9))
    d = data([40, 50], 50, 256, 256, 2, gather=False, tail=100)
    d["offsets"] = torch.tensor([5, 60, 130], dtype=torch.int32, device="cuda")     # nor rows before the first
    check(d)


def test_offsets_outside_the_rows_are_cut_off():
    d = data([10, 20, 30], 16, 256, 128, 3)
    d["offsets"] = torch.tensor([-7, 15, 40, 1000], dtype=torch.int32, device="cuda")
    check(d)
    d["offsets"] = torch.tensor([-2147483648, -5, 70, 2147483647], dtype=torch.int32, device="cuda")
    check(d)


def test_tokens_that_are_not_there_are_rows_of_zeros():
    d = data([70, 6], 12, 512, 256, 4)
    d["row_token"][::3] = -1
    d["row_token"][1::7] = 12
    d["row_token"][5], d["row_token"][6] = 2147483647, -2147483648
    check(d)
    d["qA"], d["sA"] = d["qA"][:0], d["sA"][:0]
    check(d)


def test_one_token_many_times_and_experts_without_rows():
    d = data([1] * 8 + [0] * 100 + [3], 1, 512, 512, 5)
    check(d)


def test_the_same_bits_on_every_call_and_alone():
    """A row's result depends on its own inputs alone: not on the rows beside it, nor on the call."""
    d = data([200, 3, 77, 1, 0, 9], 64, 768, 896, 6)
    Y = qz.qz_moe_gemm_fp8(**d)
    H = qz.qz_moe_gemm_fp8_swiglu(**d)
    for _ in range(3):
        assert torch.equal(qz.qz_moe_gemm_fp8(**d), Y)
        assert all(torch.equal(a, b) for a, b in zip(qz.qz_moe_gemm_fp8_swiglu(**d), H))


def test_nan_reaches_its_own_row_alone():
    d = data([40, 50], 90, 256, 384, 7, gather=False)
    Y, (codes, scales) = qz.qz_moe_gemm_fp8(**d), qz.qz_moe_gemm_fp8_swiglu(**d)
    d["qA"][3, 200] = 0x7F
    d["sA"][45, 1] = math.nan
    Y2, (codes2, scales2) = qz.qz_moe_gemm_fp8(**d), qz.qz_moe_gemm_fp8_swiglu(**d)
    rest = [r for r in range(90) if r not in (3, 45)]
    assert torch.equal(Y[rest], Y2[rest]) and torch.equal(codes[rest], codes2[rest]) and torch.equal(scales[rest], scales2[rest])
    assert bool(torch.isnan(Y2[[3, 45]].float()).all())
    assert bool(((codes2[[3, 45]] & 0x7F) == 0x7F).all())


def test_large_and_saturating_gates():
    d = data([33], 33, 512, 256, 8, gather=False)
    d["sA"] *= 300.0                                             # gates of either sign far past exp's range
    check(d, "swiglu")
    d["sA"] *= 0
    check(d)


def test_agrees_with_the_single_product():
    """One expert with 256 rows is qz_gemm_fp8_block's problem."""
    d = data([256], 256, 512, 1024, 9, gather=False)
    Y = qz.qz_moe_gemm_fp8(**d)
    want = qz.qz_gemm_fp8_block(d["qA"], d["sA"], d["qW"][0], d["sW"][0])
    P, S = ref.product(**d)
    B = 2 * ref.product_bound(S, 1024)
    assert bool(((Y.double() - want.double()).abs() <= B + P.abs() * 2.0 ** -7).all())
