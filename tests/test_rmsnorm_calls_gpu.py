"""Calls of the root-mean-square norm that ask for less than all of it, and weights that are no
ordinary numbers."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("h", [96, 2051, 9999, 16384, 20000, 20003, 32768])
def test_backward_of_nothing(dev, h, dtype):
    """Neither gradient asked for: no kernel runs, whatever the row's length."""
    x = torch.randn(5, h, device=dev).to(dtype)
    g = torch.randn(5, h, device=dev).to(dtype)
    w = torch.ones(h, device=dev, dtype=dtype)
    _, _, rstd = lce.rmsnorm_fwd(x, w, eps=EPS)
    torch.cuda.synchronize()
    lce.lce_timing_enable(True)
    try:
        lce.lce_timing_read()
        assert lce.rmsnorm_bwd(g, x, rstd, grad_x=False) == (None, None)
        assert lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=x, grad_x=False,
                               grad_weight=False) == (None, None)
        assert lce.lce_timing_read() == []
    finally:
        lce.lce_timing_enable(False)
    # one of the two is as it was
    dx, dw = lce.rmsnorm_bwd(g, x, rstd, w)
    assert torch.equal(lce.rmsnorm_bwd(g, x, rstd, w, grad_weight=False)[0], dx)
    assert torch.equal(lce.rmsnorm_bwd(g, x, rstd, w, grad_x=False)[1], dw)
