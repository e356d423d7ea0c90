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
    with pytest.raises(qz.QZError):
        qz.qz_residual_rmsnorm(x, gamma, out=no, normed=no, fp8=no)
