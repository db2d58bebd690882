"""Root-mean-square norm of a sum, 16- and 8-bit outputs, and its gradients, against their
definitions in fp64.

Tolerances to first order, u = 2^-24. A row sum is added over at most 32 elements of a lane, 6
lane exchanges and 16 wavefronts: D = 56 roundings cover it, its division by h and eps. The bounds
below follow each value through the formula; rounding to the output's type adds half a step."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce
from linear_cross_entropy_masked_amd.autograd import (RMSNorm, TiedHead, add_rms_norm,
                                                      linear_cross_entropy_pieces, rms_norm)

from _fp8 import E4M3, E8M0, block_max, check_scales, half_step_e4m3, spread
from _helpers import gpu_device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
D = 56
EPS = 1e-6
REL = 0.5 * (D + 4) * U + 6 * U  # of y: the root of the mean, its reciprocal, two products
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTHS = [1, 3, 7, 8, 64, 127, 129, 511, 512, 513, 1024, 1028, 2048, 2051, 4096, 4097, 8192, 9999,
          16384, 16385, 32768]


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def half_step(dtype, exact):
    f = torch.finfo(dtype)
    return torch.clamp(exact.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def inputs(n, h, dtype, pdtype, dev, seed=0):
    gen = torch.Generator().manual_seed(seed + 31 * n + h)
    x = (torch.randn(n, h, generator=gen) * 2).to(dtype).to(dev)
    r = torch.randn(n, h, generator=gen).to(dtype).to(dev)
    w = (1 + 0.2 * torch.randn(h, generator=gen)).to(pdtype).to(dev)
    g = torch.randn(n, h, generator=gen).to(dtype).to(dev)
    return x, r, w, g


def sum_of(x, r):
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def exact_norm(s, w, eps=EPS):
    sd = s.double()
    rstd = ((sd * sd).mean(1, keepdim=True) + eps).rsqrt()
    return sd * rstd * (1.0 if w is None else w.double()), rstd[:, 0]


def check_forward(x, r, w, y, s, rstd, eps=EPS):
    assert torch.equal(s, sum_of(x, r))
    exact, er = exact_norm(s, w, eps)
    err = (y.double() - exact).abs()
    tol = REL * exact.abs() + half_step(y.dtype, exact)
    assert (err <= 1.01 * tol).all(), (err - tol).max()
    if rstd is not None:
        assert ((rstd.double() / er - 1).abs() <= REL).all()


@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_forward(dev, h, dtype):
    for n, pdtype, add in ((1, dtype, True), (9, torch.float32, False), (130, dtype, True)):
        x, r, w, _ = inputs(n, h, dtype, pdtype, dev)
        y, s, rstd = lce.rmsnorm_fwd(x, w, r if add else None, eps=EPS)
        assert y.dtype == dtype and (add or s is x)
        check_forward(x, r if add else None, w, y, s, rstd)


def test_forward_many_rows(dev):
    """More rows than the grid deals at once; rows past the caches (streamed)."""
    x, r, w, _ = inputs(40000, 96, torch.float32, torch.float32, dev)
    check_forward(x, r, w, *lce.rmsnorm_fwd(x, w, r, eps=EPS))
    x, r, w, _ = inputs(5000, 16384, torch.bfloat16, torch.bfloat16, dev)
    check_forward(x, r, w, *lce.rmsnorm_fwd(x, w, r, eps=EPS))


@pytest.mark.parametrize("h", [100, 512, 2051])
def test_forward_strides_and_places(dev, h):
    """Rows inside wider ones, and every place that the sum and the result may share."""
    bigs = [torch.randn(11, h + extra, device=dev).bfloat16() for extra in (9, 5)]
    x, r = bigs[0][:, 3:3 + h], bigs[1][:, 4:4 + h]
    w = torch.rand(h, device=dev).bfloat16()
    y, s, rstd = lce.rmsnorm_fwd(x, w, r, eps=EPS)
    check_forward(x, r, w, y, s, rstd)
    y0, s0 = y.clone(), s.clone()
    for place in ("sum in residual", "sum in x", "y in x", "y in residual", "y in x, sum in r"):
        wide = [t.clone() for t in bigs]
        xx, rr = wide[0][:, 3:3 + h], wide[1][:, 4:4 + h]
        kw = {"sum in residual": dict(residual_out=rr), "sum in x": dict(residual_out=xx),
              "y in x": dict(out=xx), "y in residual": dict(out=rr),
              "y in x, sum in r": dict(out=xx, residual_out=rr)}[place]
        y, s, _ = lce.rmsnorm_fwd(xx, w, rr, eps=EPS, **kw)
        assert torch.equal(y, y0) and torch.equal(s, s0), place
        for name, t in kw.items():
            assert (y if name == "out" else s).data_ptr() == t.data_ptr()
        for big, now, lo in zip(bigs, wide, (3, 4)):  # the columns beside the rows
            assert torch.equal(now[:, :lo], big[:, :lo]), place
            assert torch.equal(now[:, lo + h:], big[:, lo + h:]), place
    y, s, rstd = lce.rmsnorm_fwd(x, None, None, eps=EPS, return_rstd=False)
    assert rstd is None
    check_forward(x, None, None, y, s, None)


def test_forward_special_values(dev):
    x = torch.zeros(5, 300, device=dev)
    x[1] = 1e-30
    x[2, 7] = float("inf")
    x[3, 7] = float("nan")
    x[4] = 3.0
    y, _, rstd = lce.rmsnorm_fwd(x, eps=1e-6)
    assert (y[0] == 0).all() and abs(rstd[0].item() - 1000.0) < 1e-3
    assert torch.isfinite(y[1]).all() and torch.isnan(y[2, 7]) and (y[2, 8:] == 0).all()
    assert torch.isnan(y[3]).all()
    assert ((y[4] - 1).abs() < 1e-6).all()
    y, _, rstd = lce.rmsnorm_fwd(x[:1], eps=0.0)  # 0 / 0
    assert torch.isinf(rstd).all() and torch.isnan(y).all()
    for n in (0, 1):
        y, s, rstd = lce.rmsnorm_fwd(x[:n], None, x[:n])
        assert y.shape == s.shape == (n, 300) and rstd.shape == (n,)


# ---------------------------------------------------------------- 8 bits

def check_fp8(y, q, c):
    """q and c against 64-bit y that the kernel knows to a relative error of REL."""
    n, h = y.shape
    check_scales(c, block_max(y, 1), REL)
    cs = spread(c, 1, n, h)
    v = y / cs
    tol = half_step_e4m3(v.abs() * (1 + 1e-6)) + (REL + U) * v.abs()
    err = (q.double() - v).abs()
    assert (err <= tol).all(), (err - tol).max()
    top = block_max(q.double(), 1)
    assert (top <= 448).all()
    if c.dtype == torch.float32:  # the largest of a block is the largest e4m3 number
        assert (top[block_max(y, 1) > 1e-30] == 448).all()


@pytest.mark.parametrize("scale", [E8M0, torch.float32])
@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_fp8_forward(dev, h, dtype, scale):
    for n, pdtype, add in ((1, dtype, True), (19, torch.float32, False), (130, dtype, True)):
        x, r, w, _ = inputs(n, h, dtype, pdtype, dev)
        r = r if add else None
        q, c, s = lce.rmsnorm_fp8_fwd(x, w, r, eps=EPS, scale_dtype=scale)
        assert q.dtype == E4M3 and c.dtype == scale and c.shape == (-(-h // 128), n)
        assert torch.equal(s, sum_of(x, r))
        check_fp8(exact_norm(s, w)[0], q, c)


@pytest.mark.parametrize("h", [4096, 8200, 32768])
@pytest.mark.parametrize("dtype", DTYPES)
def test_fp8_scales_beside_powers_of_two(dev, h, dtype):
    """Blocks whose largest y / 448 lies within a few fp32 steps of a power of two get the scale of
    the definition. The rows are whole numbers, so that their sums of squares are exact."""
    gen = torch.Generator().manual_seed(h)
    x = torch.randint(-2, 3, (40, h), generator=gen).double()
    at = torch.arange(0, h, 128) + torch.randint(0, 128 if h % 128 == 0 else 8, (-(-h // 128),),
                                                 generator=gen)
    x[:, at] = torch.randint(3, 8, (40, len(at)), generator=gen).double()
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + torch.tensor(EPS).double())
    for row in range(0, 40, 4):
        w = torch.zeros(h)
        steps = torch.randint(-3, 4, (len(at),), generator=gen).double() * 2.0 ** -23
        scale = 2.0 ** torch.randint(-12, 3, (len(at),), generator=gen).double()
        w[at] = (448 * scale / (x * r)[row, at] * (1 + steps)).float()
        q, c, _ = lce.rmsnorm_fp8_fwd(x.to(dtype).to(dev), w.to(dev), eps=EPS)
        top = torch.nn.functional.pad((x * r * w.double()).abs(), (0, -h % 128)).view(40, -1, 128)
        exact = (top.amax(-1) / 448).float().double()
        assert torch.equal(c.view(torch.uint8).t().cpu().double(),
                           torch.ceil(torch.log2(exact)) + 127)


def test_fp8_is_the_quantised_norm(dev):
    """In fp32 rows nothing is rounded between: the 8-bit form is the quantiser of the norm."""
    x, r, w, _ = inputs(37, 1000, torch.float32, torch.float32, dev)
    y, s, _ = lce.rmsnorm_fwd(x, w, r, eps=EPS)
    for scale in (E8M0, torch.float32):
        q, c, s8 = lce.rmsnorm_fp8_fwd(x, w, r, eps=EPS, scale_dtype=scale)
        q2, c2 = lce.fp8_quantize(y, scale_dtype=scale)
        assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8))
        assert torch.equal(c.view(torch.uint8), c2.view(torch.uint8))
        assert torch.equal(s, s8)


def test_fp8_places(dev):
    """Given outputs with strides of their own; nothing beside them is touched."""
    h, n = 300, 21
    x, r, w, _ = inputs(n, h, torch.bfloat16, torch.bfloat16, dev)
    q0, c0, s0 = lce.rmsnorm_fp8_fwd(x, w, r, scale_dtype=torch.float32)
    q = torch.full((n, h + 9), 1.0, device=dev).to(E4M3)
    c = torch.full((3, n + 4), -7.0, device=dev)
    rr = r.clone()
    q1, c1, s1 = lce.rmsnorm_fp8_fwd(x, w, rr, out=q[:, 5:5 + h], scales=c[:, 2:2 + n],
                                     residual_out=rr)
    assert torch.equal(q1.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(c1, c0)
    assert torch.equal(rr, s0) and s1 is rr
    assert (q[:, :5].float() == 1).all() and (q[:, 5 + h:].float() == 1).all()
    assert (c[:, :2] == -7).all() and (c[:, 2 + n:] == -7).all()


@pytest.mark.parametrize("scale", [E8M0, torch.float32])
def test_fp8_special_values(dev, scale):
    """Blocks of zeros, of the smallest numbers, and with a NaN or infinity."""
    x = torch.zeros(4, 384, device=dev)
    x[1, :128], x[1, 128:256] = 1.0, 1e-42
    x[2, 5], x[2, 200] = 1.0, float("nan")
    x[3, 0], x[3, 300] = 2.0, float("inf")
    q, c = lce.fp8_quantize(x, scale_dtype=scale)
    cs = spread(c, 1, 4, 384)
    assert (q[0].float() == 0).all() and (cs[0] == 2.0 ** -126).all()
    assert (cs[1, 128:] == 2.0 ** -126).all()
    assert ((q[1].double() * cs[1] - x[1].double()).abs()[128:] <= 2.0 ** -136).all()
    bad = torch.zeros(4, 384, dtype=torch.bool, device=dev)
    bad[2, 128:256] = bad[3, 256:] = True
    assert torch.equal(torch.isnan(q.float()), bad) and torch.equal(torch.isnan(cs), bad)


# ---------------------------------------------------------------- gradients

def check_backward(g, x, rstd, w, gs, dx, dw, base=None):
    n, h = x.shape
    gd, xd, rs = g.double(), x.double(), rstd.double()[:, None]
    wd = torch.ones(h, dtype=torch.float64, device=x.device) if w is None else w.double()
    xh, u = xd * rs, gd * wd
    mean = (u * xh).mean(1, keepdim=True)
    size = (u * xh).abs().mean(1, keepdim=True)
    if dx is not None:
        exact = rs * (u - xh * mean) + (0 if gs is None else gs.double())
        inner = rs * (u.abs() + (xh * mean).abs())
        tol = 5 * U * inner + rs * xh.abs() * (D + 6) * U * size + half_step(dx.dtype, exact)
        if gs is not None:
            tol = tol + U * (inner + gs.double().abs())
        err = (dx.double() - exact).abs()
        assert (err <= 1.01 * tol).all(), (err - tol).max()
    if dw is not None:
        exact = (gd * xh).sum(0) + (0 if base is None else base.double())
        # each row's term carries two roundings; the rows are added in chains of at most n + 16
        tol = (n + 18) * U * (gd * xh).abs().sum(0) + half_step(dw.dtype, exact)
        if base is not None:
            tol = tol + U * base.double().abs()
        err = (dw.double() - exact).abs()
        assert (err <= 1.01 * tol).all(), (err - tol).max()


@pytest.mark.parametrize("h", WIDTHS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_backward(dev, h, dtype):
    for n, pdtype, add in ((1, dtype, True), (9, torch.float32, False), (700, dtype, True)):
        if n * h > 3e6:
            n = 130
        x, r, w, g = inputs(n, h, dtype, pdtype, dev)
        _, _, rstd = lce.rmsnorm_fwd(x, w, eps=EPS)
        dx, dw = lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=r if add else None)
        assert dx.dtype == dtype and dw.dtype == pdtype
        check_backward(g, x, rstd, w, r if add else None, dx, dw)
        again = lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=r if add else None)
        assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


@pytest.mark.parametrize("h", [96, 2051, 20000, 20003])
def test_backward_outputs(dev, h):
    """In place, accumulated, skipped, empty; an fp32 gradient of a 16-bit weight; one tensor as
    both upstream gradients."""
    x, r, w, g = inputs(33, h, torch.bfloat16, torch.bfloat16, dev)
    _, _, rstd = lce.rmsnorm_fwd(x, w, eps=EPS)
    dx, dw = lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=r)
    for place in (0, 1):
        g2, r2 = g.clone(), r.clone()
        got, _ = lce.rmsnorm_bwd(g2, x, rstd, w, grad_residual=r2, grad_x=(g2, r2)[place])
        assert got is (g2, r2)[place] and torch.equal(got, dx)
        assert torch.equal((r2, g2)[place], (r, g)[place])
    base = torch.randn(h, device=dev)
    buf = base.clone()
    none, got = lce.rmsnorm_bwd(g, x, rstd, w, grad_x=False, grad_weight=buf, accumulate=True)
    assert none is None and got is buf
    check_backward(g, x, rstd, w, None, None, buf, base)
    got, none = lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=r, grad_weight=False)
    assert none is None and torch.equal(got, dx)
    got, none = lce.rmsnorm_bwd(g, x, rstd)  # no weight: no gradient of one
    assert none is None
    check_backward(g, x, rstd, None, None, got, None)
    got, _ = lce.rmsnorm_bwd(g, x, rstd, w, grad_residual=g)
    check_backward(g, x, rstd, w, g, got, None)
    _, zero = lce.rmsnorm_bwd(g[:0], x[:0], rstd[:0], w)
    assert (zero == 0).all()
    was = buf.clone()
    lce.rmsnorm_bwd(g[:0], x[:0], rstd[:0], w, grad_weight=buf, accumulate=True)
    assert torch.equal(buf, was)


def test_backward_against_differences(dev):
    """The gradients as the slope of the forward along random directions, in 64 bits by central
    differences (error of the difference ~ step^2 = 1e-8 of the third derivative)."""
    x, r, w, c = inputs(6, 200, torch.float32, torch.float32, dev)
    cs = torch.randn_like(c)  # the sum's own use
    s = sum_of(x, r)
    _, _, rstd = lce.rmsnorm_fwd(s, w, eps=EPS)
    dx, dw = lce.rmsnorm_bwd(c, s, rstd, w, grad_residual=cs)

    def value(sd, wd):
        y = sd * ((sd * sd).mean(1, keepdim=True) + EPS).rsqrt() * wd
        return (y * c.double()).sum() + (sd * cs.double()).sum()
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        ds = torch.randn(6, 200, generator=gen, dtype=torch.float64).to(dev)
        dwd = torch.randn(200, generator=gen, dtype=torch.float64).to(dev)
        t = 1e-4
        slope = (value(s.double() + t * ds, w.double() + t * dwd)
                 - value(s.double() - t * ds, w.double() - t * dwd)) / (2 * t)
        got = (dx.double() * ds).sum() + (dw.double() * dwd).sum()
        size = (dx.double() * ds).abs().sum() + (dw.double() * dwd).abs().sum()
        assert (got - slope).abs() <= 1e-5 * size


# ---------------------------------------------------------------- autograd

def test_autograd(dev):
    """add_rms_norm: both results used, gradients of x, residual and weight, any leading shape and
    a broadcast upstream gradient."""
    x, r, w, _ = inputs(24, 160, torch.float32, torch.float32, dev)
    leaves = [t.clone().view(2, 12, 160).requires_grad_() if t.dim() == 2
              else t.clone().requires_grad_() for t in (x, r, w)]
    y, s = add_rms_norm(*leaves[:2], leaves[2], eps=EPS)
    assert y.shape == s.shape == (2, 12, 160)
    (y.sum() + (s * s).sum()).backward()
    ref = [t.detach().double().requires_grad_() for t in leaves]
    sd = ref[0] + ref[1]
    yd = sd * ((sd * sd).mean(-1, keepdim=True) + EPS).rsqrt() * ref[2]
    (yd.sum() + (sd * sd).sum()).backward()
    for a, b in zip(leaves, ref):
        assert (a.grad.double() - b.grad).abs().max() <= 2e-5 * b.grad.abs().max()
    # one result unused, and no residual
    for use in (0, 1):
        t = [u.detach().clone().requires_grad_() for u in leaves]
        out = add_rms_norm(t[0], t[1], t[2], eps=EPS)[use]
        out.sum().backward()
        if use == 1:
            assert (t[0].grad == 1).all() and (t[1].grad == 1).all()
            assert t[2].grad is None or (t[2].grad == 0).all()
        else:
            assert torch.equal(t[0].grad, t[1].grad)
    t = leaves[0].detach().clone().requires_grad_()
    rms_norm(t, leaves[2].detach(), eps=EPS).sum().backward()
    assert torch.isfinite(t.grad).all()


def test_module_and_tied_head(dev):
    """RMSNorm in a bf16 model, and a tied head on it: loss and gradients against 64 bits."""
    torch.manual_seed(0)
    norm = RMSNorm(128, device=dev, dtype=torch.bfloat16)
    x = torch.randn(5, 7, 128, device=dev).bfloat16()
    y = norm(x)
    check_forward(x.view(-1, 128), None, norm.weight.detach(), y.detach().view(-1, 128),
                  x.view(-1, 128), None, norm.eps)
    y, s = norm(x, x)
    assert torch.equal(s, x + x)
    head = TiedHead(1000, 128, rms=True, device=dev)
    assert head.norm.bias is None
    tokens = torch.randint(0, 1000, (3, 9), device=dev)
    e = head.embed(tokens)
    loss = head(e, tokens, residual=e)
    loss.backward()
    w = head.weight.detach().double().requires_grad_()
    ed = w[tokens]
    sd = 2 * ed
    yd = sd * ((sd * sd).mean(-1, keepdim=True) + head.norm.eps).rsqrt()
    ref = torch.nn.functional.cross_entropy((yd @ w.t()).view(-1, 1000), tokens.view(-1))
    ref.backward()
    assert (loss.double() - ref).abs() <= 2e-3 * ref
    err = (head.weight.grad.double() - w.grad).norm() / w.grad.norm()
    assert err <= 2e-2  # bf16 operands and sums of two bf16 gradients
    # the same as the parts
    parts = linear_cross_entropy_pieces(rms_norm(e + e, head.norm.weight, eps=head.norm.eps),
                                        head.weight, tokens, reduction="mean")
    assert torch.equal(parts, loss)


def test_graph_and_streams(dev):
    """A captured step replayed on other inputs, with eager work between; and a call on a side
    stream."""
    x, r, w, g = inputs(64, 1000, torch.bfloat16, torch.bfloat16, dev)

    def step():
        y, s, rstd = lce.rmsnorm_fwd(x, w, r, eps=EPS)
        q, c, _ = lce.rmsnorm_fp8_fwd(x, w, r, eps=EPS)
        return (y, s, q.view(torch.uint8), c.view(torch.uint8),
                *lce.rmsnorm_bwd(g, s, rstd, w, grad_residual=r))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(on_side, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        x.copy_(torch.randn(64, 1000, generator=torch.Generator().manual_seed(seed)))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, eager):
            assert torch.equal(a, b)
