"""Layer norm forward and backward against their definitions in fp64.

Tolerances to first order, u = 2^-24. A row sum is added over at most 32 elements of a lane, 6
shuffle steps and 16 wavefronts: D = 56 roundings cover it and its division by h. The bounds
below follow each value through the formula; rounding to the output's type adds half a step."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
D = 56
EPS = 1e-5
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTHS = [1, 2, 7, 64, 511, 512, 513, 1024, 1025, 2048, 2051, 4096, 4097, 8192, 9999, 16384, 16385,
          32768]


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def half_step(dtype, exact):
    f = torch.finfo(dtype)
    return torch.clamp(exact.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def inputs(n, h, dtype, pdtype, dev, seed=0, offset=0.0):
    gen = torch.Generator().manual_seed(seed + 31 * n + h)
    x = (torch.randn(n, h, generator=gen) * 2 + offset).to(dtype).to(dev)
    w = (1 + 0.2 * torch.randn(h, generator=gen)).to(pdtype).to(dev)
    b = (0.3 * torch.randn(h, generator=gen)).to(pdtype).to(dev)
    g = torch.randn(n, h, generator=gen).to(dtype).to(dev)
    return x, w, b, g


def check_forward(x, w, b, y, mean, rstd, eps=EPS):
    xd = x.double()
    h = x.shape[1]
    w = torch.ones(h, device=x.device) if w is None else w
    b = torch.zeros(h, device=x.device) if b is None else b
    mu = xd.mean(1, keepdim=True)
    c = xd - mu
    var = (c * c).mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    exact = c * r * w.double() + b.double()
    dmu = D * U * xd.abs().mean(1, keepdim=True)
    dc = dmu + U * c.abs()
    dvar = (D + 4) * U * var + 2 * (c.abs() * dc).mean(1, keepdim=True) + (dc * dc).mean(1, keepdim=True)
    rel_r = 0.5 * dvar / (var + eps) + 5 * U
    size = c.abs() * r * w.double().abs()
    tol = (dc * r * w.double().abs() + size * (rel_r + 4 * U) + 2 * U * (size + b.double().abs())
           + half_step(y.dtype, exact))
    # second-order terms: where the variance is all rounding error the first-order bound of r
    # is taken twice
    err = (y.double() - exact).abs()
    assert (err <= 1.1 * tol).all(), ((err - tol).max(), err.max())
    if mean is not None:
        assert ((mean.double() - mu[:, 0]).abs() <= dmu[:, 0]).all()
        assert ((rstd.double() / r[:, 0] - 1).abs() <= 1.1 * rel_r[:, 0]).all()


@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward(dev, h, dtype):
    for n, pdtype in ((1, dtype), (9, torch.float32), (130, dtype)):
        x, w, b, _ = inputs(n, h, dtype, pdtype, dev)
        y, mean, rstd = lce.layernorm_fwd(x, w, b, eps=EPS)
        assert y.dtype == dtype
        check_forward(x, w, b, y, mean, rstd)


def test_forward_many_rows_and_offset(dev):
    """More rows than the grid deals at once, and a mean far larger than the deviation."""
    x, w, b, _ = inputs(40000, 96, torch.float32, torch.float32, dev, offset=50.0)
    check_forward(x, w, b, *lce.layernorm_fwd(x, w, b, eps=EPS))
    x, w, b, _ = inputs(5001, 4096, torch.bfloat16, torch.bfloat16, dev, offset=-3.0)
    check_forward(x, w, b, *lce.layernorm_fwd(x, w, b, eps=EPS))


def test_forward_past_the_caches(dev):
    """More than 512 MiB of rows: non-temporal loads and stores, and offsets past 2^31 bytes."""
    for dtype, n, h in ((torch.float32, 17000, 4096), (torch.bfloat16, 140000, 8192)):
        x, w, b, _ = inputs(64, h, dtype, dtype, dev)
        many = x.repeat(n // 64 + 1, 1)[:n]
        y, mean, rstd = lce.layernorm_fwd(many, w, b, eps=EPS)
        check_forward(x, w, b, y[:64], mean[:64], rstd[:64])
        whole = n // 64 * 64
        assert torch.equal(y[:whole].view(-1, 64, h), y[:64].expand(n // 64, 64, h))
        assert torch.equal(y[whole:], y[:n - whole])
        assert torch.equal(mean[:whole].view(-1, 64), mean[:64].expand(n // 64, 64))


def test_forward_without_parameters_strided_and_in_place(dev):
    for dtype in DTYPES:
        x, w, b, _ = inputs(37, 300, dtype, dtype, dev)
        check_forward(x, None, None, *lce.layernorm_fwd(x, eps=EPS))
        check_forward(x, w, None, *lce.layernorm_fwd(x, w, eps=EPS))
        check_forward(x, None, b, *lce.layernorm_fwd(x, None, b, eps=EPS))
        y, mean, rstd = lce.layernorm_fwd(x, w, b, eps=EPS, return_stats=False)
        assert mean is None and rstd is None
        xs = x[:, 1:250]
        buf = torch.full((37, 260), 7.0, dtype=dtype, device=dev)
        out = buf[:, 5:254]
        _, mean, rstd = lce.layernorm_fwd(xs, w[1:250], b[1:250], eps=EPS, out=out)
        check_forward(xs, w[1:250], b[1:250], out, mean, rstd)
        assert (buf[:, :5] == 7).all() and (buf[:, 254:] == 7).all()
        z = x.clone()
        assert lce.layernorm_fwd(z, w, b, eps=EPS, out=z)[0] is z
        assert torch.equal(z, y)


def test_rows_do_not_touch_each_other(dev):
    """A row of NaN or infinity stays its own; a constant row gives the bias."""
    for h in (100, 3000, 9000):
        x, w, b, _ = inputs(6, h, torch.float32, torch.float32, dev)
        want = lce.layernorm_fwd(x, w, b)[0]
        x[1], x[3, 0], x[4] = float("nan"), float("inf"), 2.5
        got = lce.layernorm_fwd(x, w, b)[0]
        for i in (0, 2, 5):
            assert torch.equal(got[i], want[i])
        assert got[1].isnan().all() and got[3].isnan().all()
        assert torch.equal(got[4], b)


def check_backward(x, g, mean, rstd, w, gx, gw, gb, old=None):
    n, h = x.shape
    wd = torch.ones(h, device=x.device, dtype=torch.float64) if w is None else w.double()
    r, gd = rstd.double()[:, None], g.double()
    xh = (x.double() - mean.double()[:, None]) * r
    u = gd * wd
    m1, m2 = u.mean(1, keepdim=True), (u * xh).mean(1, keepdim=True)
    if gx is not None:
        exact = r * (u - m1 - xh * m2)
        tol = r * U * (6 * u.abs() + (D + 6) * u.abs().mean(1, keepdim=True)
                       + (D + 12) * xh.abs() * (u * xh).abs().mean(1, keepdim=True))
        err = (gx.double() - exact).abs()
        assert (err <= tol + half_step(gx.dtype, exact)).all(), err.max()
    for got, terms, k in ((gw, gd * xh, 0), (gb, gd, 1)):
        if got is None:
            continue
        exact, size = terms.sum(0), terms.abs().sum(0)
        if old is not None:
            exact, size = exact + old[k].double(), size + old[k].double().abs()
        tol = (n + 6) * U * size + half_step(got.dtype, exact)
        err = (got.double() - exact).abs()
        assert (err <= tol).all(), (k, (err - tol).max())


def stats(x):
    xd = x.double()
    return xd.mean(1).float(), (xd.var(1, unbiased=False) + EPS).rsqrt().float()


@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward(dev, h, dtype):
    for n, pdtype in ((1, dtype), (11, torch.float32), (300, dtype)):
        x, w, _, g = inputs(n, h, dtype, pdtype, dev, seed=1)
        mean, rstd = stats(x)
        gx, gw, gb = lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True)
        assert gx.dtype == dtype and gw.dtype == pdtype and gb.dtype == pdtype
        check_backward(x, g, mean, rstd, w, gx, gw, gb)


def test_backward_many_rows_repeats_bit_for_bit(dev):
    x, w, _, g = inputs(5001, 1500, torch.bfloat16, torch.bfloat16, dev, seed=2)
    mean, rstd = stats(x)
    first = lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True)
    check_backward(x, g, mean, rstd, w, *first)
    again = lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_backward_outputs_accumulate_strides_in_place(dev):
    for dtype in DTYPES:
        x, w, _, g = inputs(90, 200, dtype, dtype, dev, seed=3)
        mean, rstd = stats(x)
        ref = lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True)
        gx, gw, gb = lce.layernorm_bwd(g, x, mean, rstd, w, grad_x=False, grad_weight=False,
                                       grad_bias=True)
        assert gx is None and gw is None and torch.equal(gb, ref[2])
        gx, gw, gb = lce.layernorm_bwd(g, x, mean, rstd, w, grad_weight=False)
        assert gw is None and gb is None and torch.equal(gx, ref[0])
        check_backward(x, g, mean, rstd, None, *lce.layernorm_bwd(g, x, mean, rstd))
        old = (torch.randn(200, device=dev), torch.randn(200, device=dev))
        gw, gb = old[0].clone(), old[1].clone()
        lce.layernorm_bwd(g, x, mean, rstd, w, grad_weight=gw, grad_bias=gb, accumulate=True)
        check_backward(x, g, mean, rstd, w, None, gw, gb, old)
        xs, gs = x[:, 3:180], g[:, 7:184]
        buf = torch.full((90, 190), 4.0, dtype=dtype, device=dev)
        out = buf[:, 1:178]
        lce.layernorm_bwd(gs, xs, mean, rstd, w[:177], grad_x=out)
        check_backward(xs, gs, mean, rstd, w[:177], out, None, None)
        assert (buf[:, :1] == 4).all() and (buf[:, 178:] == 4).all()
        z = g.clone()
        assert lce.layernorm_bwd(z, x, mean, rstd, w, grad_x=z)[0] is z
        assert torch.equal(z, ref[0])


def test_empty_batch(dev):
    x = torch.empty(0, 40, device=dev)
    w = torch.ones(40, device=dev)
    y, mean, rstd = lce.layernorm_fwd(x, w, w)
    assert y.shape == (0, 40) and mean.shape == (0,)
    gx, gw, gb = lce.layernorm_bwd(x, x, mean, rstd, w, grad_bias=True)
    assert gx.shape == (0, 40) and not gw.any() and not gb.any()
    keep = w.clone()
    lce.layernorm_bwd(x, x, mean, rstd, w, grad_weight=keep, accumulate=True)
    assert torch.equal(keep, w)


def test_gradients_against_differences(dev):
    """Central differences of f = Σ c · y in fp32 inputs, taken in fp64 of the kernel's outputs:
    a step of 2^-6 leaves a third-order term below 1e-3 of the value here and fp32 rounding of
    f's terms over twice the step."""
    gen = torch.Generator().manual_seed(9)
    n, h, t = 5, 130, 2.0 ** -6
    x = torch.randn(n, h, generator=gen).to(dev)
    w, b = torch.randn(h, generator=gen).to(dev), torch.randn(h, generator=gen).to(dev)
    c, d = torch.randn(n, h, generator=gen).to(dev), torch.randn(n, h, generator=gen).to(dev)
    dw = torch.randn(h, generator=gen).to(dev)
    f = lambda x_, w_: (lce.layernorm_fwd(x_, w_, b)[0].double() * c.double()).sum()  # noqa: E731
    _, mean, rstd = lce.layernorm_fwd(x, w, b)
    gx, gw, gb = lce.layernorm_bwd(c, x, mean, rstd, w, grad_bias=True)
    noise = 40 * U * (c.double().abs() * (3 * w.double().abs() + b.double().abs())).sum() / t
    for step, want in (((f(x + t * d, w) - f(x - t * d, w)) / (2 * t), (gx.double() * d).sum()),
                       ((f(x, w + t * dw) - f(x, w - t * dw)) / (2 * t), (gw.double() * dw).sum())):
        # third-order term: t²/6 · f''' with |f'''| at most a few times Σ|c w d³|
        third = t * t * (c.double().abs() * w.double().abs() * (1 + d.double().abs()) ** 3).sum()
        assert (step - want).abs() <= noise + third
    assert ((gb.double() - c.double().sum(0)).abs() <= 8 * U * c.double().abs().sum(0)).all()


def test_rows_past_4_gib(dev):
    """Rows whose bytes start past 2^32 are normalised, in place, as the same rows by themselves,
    and so is their gradient."""
    n, h, last = 600001, 4096, 70
    x = torch.zeros(n, h, dtype=torch.bfloat16, device=dev)
    x[-last:] = torch.randn(last, h, device=dev).to(torch.bfloat16)
    w = torch.randn(h, device=dev).to(torch.bfloat16)
    tail = x[-last:].clone()
    y, mean, rstd = lce.layernorm_fwd(tail, w)
    g = torch.randn(last, h, device=dev).to(torch.bfloat16)
    gx, gw, _ = lce.layernorm_bwd(g, tail, mean, rstd, w)
    got, m, r = lce.layernorm_fwd(x, w, out=x)
    assert torch.equal(got[-last:], y) and not got[:-last].any()
    assert torch.equal(m[-last:], mean) and torch.equal(r[-last:], rstd)
    x[-last:] = tail
    x[:-last] = 0
    big = torch.zeros_like(x)
    big[-last:] = g
    bx, bw, _ = lce.layernorm_bwd(big, x, m, r, w, grad_x=big)
    assert torch.equal(bx[-last:], gx) and not bx[:-last].any()
    # two fp32 sums of the same terms (at most `last` that are not 0), each rounded to bf16
    size = (g.float() * ((tail.float() - mean[:, None]) * rstd[:, None])).abs().sum(0)
    assert ((bw.float() - gw.float()).abs() <= 2.0 ** -7 * gw.float().abs()
            + 4 * last * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("h", [1000, 12288, 12289, 20011])
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_of_long_rows_in_place_and_in_parts(dev, h, dtype):
    """The parameter sums of the longest rows read the gradient that the rows' own pass overwrites
    in place; each output alone equals its part of the whole."""
    x, w, _, g = inputs(333, h, dtype, dtype, dev, seed=6)
    mean, rstd = stats(x)
    ref = lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True)
    check_backward(x, g, mean, rstd, w, *ref)
    z = g.clone()
    got = lce.layernorm_bwd(z, x, mean, rstd, w, grad_x=z, grad_bias=True)
    assert got[0] is z and all(torch.equal(a, b) for a, b in zip(got, ref))
    gx, gw, gb = lce.layernorm_bwd(g, x, mean, rstd, w, grad_weight=False)
    assert gw is None and gb is None and torch.equal(gx, ref[0])
    gx, gw, gb = lce.layernorm_bwd(g, x, mean, rstd, w, grad_x=False)
    assert gx is None and gb is None and torch.equal(gw, ref[1])
    old = (torch.randn(h, device=dev), torch.randn(h, device=dev))
    gw, gb = old[0].clone(), old[1].clone()
    need = lce.layernorm_workspace_size(333, h)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    lce.layernorm_bwd(g, x, mean, rstd, w, grad_weight=gw, grad_bias=gb, accumulate=True,
                      workspace=ws[:need])
    check_backward(x, g, mean, rstd, w, None, gw, gb, old)
    assert (ws[need:] == 0xFF).all()


def test_backward_of_short_rows_fills_the_partial_rows(dev):
    x, w, _, g = inputs(9000, 130, torch.float32, torch.float32, dev, seed=7)
    mean, rstd = stats(x)
    check_backward(x, g, mean, rstd, w, *lce.layernorm_bwd(g, x, mean, rstd, w, grad_bias=True))
