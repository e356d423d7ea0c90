"""The refusals of a block of experts, on the CPU: host validation behind the C ABI (every call carries an invalid
argument or nothing to do, so none can launch) and the binding's own checks."""
import ctypes

import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz

FAKE = ctypes.c_void_p(0x10000)        # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
NULL = None
INF, NAN = float("inf"), float("nan")


def routing(**kw):
    r = dict(experts=64, top_k=8, score=0, renormalize=1, scale=1.0, groups=8, top_groups=4, group_best=2)
    r.update(kw)
    return ctypes.byref(qz._MoeRouting(**r))


@pytest.mark.parametrize("kw, want", [
    (dict(experts=0), 1), (dict(experts=520), 2), (dict(top_k=0), 1), (dict(top_k=17, top_groups=8), 2), (dict(top_k=16, groups=16, top_groups=3), 2),
    (dict(score=2), 1), (dict(renormalize=2), 1), (dict(scale=INF), 1), (dict(scale=NAN), 1), (dict(groups=0), 1), (dict(groups=7), 2),
    (dict(groups=64, top_groups=8, group_best=1), 2), (dict(top_groups=0), 1), (dict(top_groups=9), 1), (dict(group_best=0), 1), (dict(group_best=3), 1),
    (dict(experts=32, groups=32, top_groups=32, group_best=2), 2)])
def test_routing_validation(kw, want):
    f = qz.lib.qz_moe_route
    assert f(FAKE, 0, 4, 512, NULL, NULL, routing(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, NULL, 0, NULL) == want


def test_route_arguments():
    f = qz.lib.qz_moe_route
    ok = [FAKE, 0, 4, 64, FAKE, FAKE, routing(), FAKE, FAKE, FAKE, FAKE, FAKE, NULL, 0, NULL]
    for i, v, want in [(0, NULL, 1), (0, ODD, 3), (1, 2, 1), (2, -1, 1), (2, 1 << 31, 2), (2, 1 << 28, 2), (3, 63, 1), (4, ODD, 3),
                       (5, ODD, 3), (6, None, 1), (7, NULL, 1), (7, ODD, 3), (8, NULL, 1), (8, ODD, 3), (9, NULL, 1), (9, ODD, 3),
                       (10, NULL, 1), (10, ODD, 3), (11, NULL, 1), (11, ODD, 3), (2, 100000, 7)]:
        a = list(ok)
        a[i] = v
        assert f(*a) == want, (i, v)
    need = qz.qz_workspace_size(qz.OP_MOE_ROUTE, 100000, 64, 8)
    assert need > 0
    a = list(ok)
    a[2], a[12], a[13] = 100000, FAKE, need - 1
    assert f(*a) == 7
    a[12], a[13] = ctypes.c_void_p(0x10008), need
    assert f(*a) == 7
    assert qz.qz_workspace_size(qz.OP_MOE_ROUTE, -1, 64, 8) == 0
    assert qz.qz_workspace_size(qz.OP_MOE_ROUTE, 1 << 40, 64, 8) == 0


def test_route_workspace_of_sizes_that_the_call_rejects():
    for tokens in (0, 1, 16, 17, 100000, (1 << 31) - 1):
        for experts in (-(1 << 40), -1, 0, 513, 1 << 40):
            assert qz.qz_workspace_size(qz.OP_MOE_ROUTE, tokens, experts, 1) == 0
    assert qz.qz_workspace_size(qz.OP_MOE_ROUTE, (1 << 31) - 1, 512, 1) <= 304 * 512 * 4


@pytest.mark.parametrize("swiglu", [False, True])
def test_expert_product_validation(swiglu):
    f = qz.lib.qz_moe_gemm_fp8_swiglu if swiglu else qz.lib.qz_moe_gemm_fp8
    # qA, sA, tokens, row_token, rows, offsets, experts, qW, sW, outputs, N or I, K, stream
    out = [FAKE, FAKE] if swiglu else [FAKE]
    ok = [FAKE, FAKE, 16, FAKE, 32, FAKE, 8, FAKE, FAKE] + out + [256, 512, NULL]
    n, k = len(ok) - 3, len(ok) - 2
    bad = [(0, NULL, 1), (0, ODD, 3), (1, NULL, 1), (1, ODD, 3), (2, -1, 1), (2, 1 << 31, 2), (3, ODD, 3), (4, -1, 1), (4, 1 << 31, 2), (5, NULL, 1),
           (5, ODD, 3), (6, 0, 1), (6, 513, 2), (7, NULL, 1), (7, ODD, 3), (8, NULL, 1), (8, ODD, 3), (9, NULL, 1), (9, ODD, 3),
           (n, 0, 1), (n, 64, 2), (n, 1 << 29, 2), (k, 0, 1), (k, 192, 2)]
    if swiglu:
        bad += [(10, NULL, 1), (10, ODD, 3), (n, 1 << 30, 2), (n, -128, 1)]
    for i, v, want in bad:
        a = list(ok)
        a[i] = v
        assert f(*a) == want, (i, v)
    a = list(ok)
    a[4] = 0                                                     # no rows: nothing to do
    assert f(*a) == 0


def block(**kw):
    b = dict(y=0x10000, rows=64, ldy=512, k=2, token_row=0x10000, weights=0x10000, alpha=1.0, gamma=0x10000)
    b.update(kw)
    return ctypes.byref(qz._BlockOutput(**b))


def test_residual_norm_validation():
    f = qz.lib.qz_residual_rmsnorm
    # x, dtype, tokens, hidden, ldx, block, x_out, ldo, gamma, eps, normed, codes, scales, stream
    ok = [FAKE, 1, 4, 512, 512, block(), FAKE, 512, FAKE, 1e-6, FAKE, FAKE, FAKE, NULL]
    for i, v, want in [(0, NULL, 1), (0, ODD, 3), (1, 2, 1), (2, -1, 1), (2, 1 << 31, 2), (3, 0, 1), (3, 504, 2), (3, 500, 2), (3, 16512, 2), (4, 511, 1),
                       (4, 513, 3), (6, ODD, 3), (7, 511, 1), (7, 516, 3), (8, NULL, 1), (8, ODD, 3), (9, 0.0, 1), (9, -1.0, 1),
                       (9, NAN, 1), (9, INF, 1), (10, ODD, 3), (11, NULL, 1), (11, ODD, 3), (12, NULL, 1), (12, ODD, 3)]:
        a = list(ok)
        a[i] = v
        assert f(*a) == want, (i, v)
    for kw, want in [(dict(k=0), 1), (dict(k=17), 2), (dict(rows=-1), 1), (dict(rows=1 << 31), 2), (dict(y=0), 1), (dict(ldy=511), 1), (dict(ldy=516), 3),
                     (dict(alpha=NAN), 1), (dict(alpha=INF), 1), (dict(y=0x10008), 3), (dict(gamma=0x10008), 3), (dict(token_row=0x10002), 3),
                     (dict(weights=0x10002), 3), (dict(token_row=0, rows=7), 1)]:
        a = list(ok)
        a[5] = block(**kw)
        assert f(*a) == want, kw
    a = list(ok)
    a[6] = a[10] = a[11] = a[12] = NULL                          # no output at all
    assert f(*a) == 1
    a = list(ok)
    a[2] = 0                                                     # no tokens: nothing to do
    assert f(*a) == 0


@pytest.fixture
def on_device0(monkeypatch):
    monkeypatch.setattr(qz, "_device", lambda: 0)


def test_wrappers_refuse_host_tensors(on_device0):
    with pytest.raises(ValueError, match="logits: .*on cpu"):
        qz.qz_moe_route(torch.zeros((4, 8)), 2)
    qA, sA = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    qW, sW = torch.zeros((2, 256, 256), dtype=torch.uint8), torch.zeros((2, 2, 2))
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="qA: .*on cpu"):
        qz.qz_moe_gemm_fp8(qA, sA, qW, sW, off)
    with pytest.raises(ValueError, match="qA: .*on cpu"):
        qz.qz_moe_gemm_fp8_swiglu(qA, sA, qW, sW, off)
    with pytest.raises(ValueError, match="x: .*on cpu"):
        qz.qz_residual_rmsnorm(torch.zeros((2, 128)), torch.zeros(128))


def test_wrappers_refuse_wrong_shapes_and_types(monkeypatch):
    monkeypatch.setattr(qz, "_device", lambda: -1)               # host tensors pass the check of the device
    with pytest.raises(TypeError):
        qz.qz_moe_route(torch.zeros((4, 8), dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="bias"):
        qz.qz_moe_route(torch.zeros((4, 8)), 2, bias=torch.zeros(7))
    with pytest.raises(ValueError, match="n_tokens"):
        qz.qz_moe_route(torch.zeros((4, 8)), 2, n_tokens=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="row_token"):
        qz.qz_moe_route(torch.zeros((4, 8)), 2, row_token=torch.zeros(7, dtype=torch.int32))
    qA, sA = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2))
    qW, sW = torch.zeros((2, 256, 256), dtype=torch.uint8), torch.zeros((2, 2, 2))
    off = torch.zeros(3, dtype=torch.int32)
    for bad in (dict(qA=qA[:, :128]), dict(sA=sA[:, :1]), dict(qW=qW[0]), dict(sW=sW[:1]), dict(offsets=off[:2]), dict(offsets=off.long()),
                dict(row_token=torch.zeros(4)), dict(Y=torch.zeros((4, 256)))):
        with pytest.raises(ValueError):
            qz.qz_moe_gemm_fp8(**{**dict(qA=qA, sA=sA, qW=qW, sW=sW, offsets=off), **bad})
    with pytest.raises(ValueError, match="codes"):
        qz.qz_moe_gemm_fp8_swiglu(qA, sA, qW, sW, off, codes=torch.zeros((4, 256), dtype=torch.uint8))
    x = torch.zeros((3, 128))
    for bad in (dict(y=torch.zeros((3, 128))), dict(y=torch.zeros((3, 64), dtype=torch.bfloat16)), dict(token_row=torch.zeros((3, 2), dtype=torch.int32)),
                dict(gamma=torch.zeros(128, dtype=torch.bfloat16)), dict(out=torch.zeros((2, 128))), dict(out=torch.zeros((3, 128)).bfloat16()),
                dict(normed=torch.zeros((3, 128))), dict(gamma_y=torch.zeros(128)),
                dict(y=torch.zeros((6, 128), dtype=torch.bfloat16), token_row=torch.zeros((2, 2), dtype=torch.int32))):
        with pytest.raises(ValueError):
            qz.qz_residual_rmsnorm(**{**dict(x=x, gamma=torch.zeros(128)), **bad})
