"""The residual norm's choice of outputs in the binding (CPU: no tokens, so that nothing is launched)."""
import pytest
import torch

import bit_quantized_linear_quantizers_gb300 as qz


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(qz, "_device", lambda: -1)
    monkeypatch.setattr(qz, "_raw_stream", lambda stream, dev: 0)


@pytest.mark.parametrize("no", [None, False])
def test_outputs_that_are_left_out(no):
    x, gamma = torch.zeros((0, 256)), torch.ones(256)
    r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, out=no, normed=True, fp8=no)
    assert r is None and n.shape == (0, 256) and codes is None and scales is None
    r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, normed=no, fp8=True)
    assert r.shape == (0, 256) and n is None and codes.shape == (0, 256) and scales.shape == (0, 2)
    r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, out=no, normed=no, fp8=no)
    assert r is None and n is None and codes is None and scales is None


def test_no_tokens():
    """A tensor of no elements has a null pointer: that is no missing argument."""
    f = qz.lib.qz_residual_rmsnorm
    assert f(None, 1, 0, 512, 512, None, None, 512, None, 1e-6, None, None, None, None) == 0
    assert f(None, 1, 1, 512, 512, None, None, 512, None, 1e-6, None, None, None, None) == 1
    assert f(None, 1, 0, 500, 512, None, None, 512, None, 1e-6, None, None, None, None) == 2    # sizes are checked all the same
    x, gamma = torch.zeros((0, 256), dtype=torch.bfloat16), torch.ones(256).bfloat16()
    rows, gates = torch.zeros((0, 3), dtype=torch.int32), torch.zeros((0, 3))
    for kw in (dict(), dict(y=x), dict(y=torch.zeros((7, 256)).bfloat16(), token_row=rows, weights=gates), dict(y=x, token_row=rows, gamma_y=gamma)):
        r, n, codes, scales = qz.qz_residual_rmsnorm(x, gamma, normed=True, fp8=True, **kw)
        assert r.shape == n.shape == codes.shape == (0, 256) and scales.shape == (0, 2)
