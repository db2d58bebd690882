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


@pytest.mark.parametrize("h", [48, 1000, 4096, 20003])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_special_weights(dev, h, dtype):
    """Weights that are infinite, NaN, zero, or so large that some results overflow: y is s · rstd ·
    weight of the definition in 64 bits, rounded to its type. Finite results: the tolerance of
    test_rmsnorm_gpu.py, 36 roundings of 2^-24 for rstd and the products, and half a step."""
    gen = torch.Generator().manual_seed(h)
    x = (torch.randn(7, h, generator=gen) * 2).to(dtype)
    x[3, ::5] = 0
    w = 1 + 0.2 * torch.randn(h, generator=gen)
    inf, big = float("inf"), torch.finfo(dtype).max
    for k, value in enumerate((inf, -inf, float("nan"), 0.0, big, -big)):
        w[k::40] = value
    x, w = x.to(dev), w.to(dtype).to(dev)
    for weight in (w, w.float()):
        y, _, _ = lce.rmsnorm_fwd(x, weight, eps=EPS)
        sd = x.double()
        exact = sd * ((sd * sd).mean(1, keepdim=True) + EPS).rsqrt() * weight.double()
        nan = torch.isnan(exact)
        assert torch.equal(torch.isnan(y), nan)
        # beside the largest number either side of the overflow is right
        near = (exact.abs() / big - 1).abs() < 2 * torch.finfo(dtype).eps
        far = exact.abs() > big
        some = ~nan & ~near
        assert torch.equal(y[some & far], torch.copysign(torch.full_like(y, inf),
                                                         exact.to(y.dtype))[some & far])
        few = some & ~far
        f = torch.finfo(dtype)
        half = torch.clamp(exact.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)
        err = (y.double() - exact).abs()
        assert (err[few] <= (1.01 * (36 * 2.0 ** -24 * exact.abs() + half))[few]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("h", [7, 128, 2051, 4096, 20003])
def test_rstd_of_the_8_bit_form(dev, h, dtype):
    """The statistics beside 8-bit rows are those of the 16-bit form, and serve the backward."""
    x = (torch.randn(33, h, device=dev) * 2).to(dtype)
    r = torch.randn(33, h, device=dev).to(dtype)
    w, g = torch.rand(h, device=dev).to(dtype) + 0.5, torch.randn(33, h, device=dev).to(dtype)
    for scale in (None, torch.float32):
        q, c, s, rstd = lce.rmsnorm_fp8_fwd(x, w, r, eps=EPS, scale_dtype=scale, return_rstd=True)
        _, total, stats = lce.rmsnorm_fwd(x, w, r, eps=EPS)
        assert torch.equal(s, total) and torch.equal(rstd, stats)
        plain = lce.rmsnorm_fp8_fwd(x, w, r, eps=EPS, scale_dtype=scale)
        assert len(plain) == 3
        for a, b in zip(plain[:2], (q, c)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(lce.rmsnorm_bwd(g, s, rstd, w), lce.rmsnorm_bwd(g, total, stats, w)):
            assert torch.equal(a, b)
    *_, rstd = lce.rmsnorm_fp8_fwd(x[:0], w, return_rstd=True)
    assert rstd.shape == (0,)
