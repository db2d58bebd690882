"""Embedding lookup and its gradient against their definitions in fp64.

Tolerances, u = 2^-24: the lookup is one fp32 product and one rounding to the table's type; a
gradient element is a sum of m fp32 terms in some order (at most m roundings of partial sums,
each at most Σ|g|), one product and one rounding."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
IGN = -100


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def half_step(dtype, exact):
    """Half a step of dtype at |exact|: relative for normal numbers, absolute below them."""
    f = torch.finfo(dtype)
    return torch.clamp(exact.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def draw_tokens(gen, n, v, dev, ignored=0.1, bad=0.0):
    """Tokens as in text: token r in proportion to 1 / (r + 1)."""
    u = torch.rand(n, generator=gen, dtype=torch.float64)
    t = (torch.exp(u * torch.log(torch.tensor(v + 1.0, dtype=torch.float64))) - 1).long()
    t = t.clamp(0, v - 1)
    t[torch.rand(n, generator=gen) < ignored] = IGN
    if bad:
        m = torch.rand(n, generator=gen) < bad
        t[m] = torch.where(torch.rand(int(m.sum()), generator=gen) < 0.5, v, -7)
    return t.to(torch.int32).to(dev)


def valid(tok, v):
    return (tok >= 0) & (tok < v) & (tok != IGN)


def check_lookup(w, tok, scale, out):
    v = w.shape[0]
    ok = valid(tok, v)
    exact = w.double()[tok.long().clamp(0, v - 1)] * float(torch.tensor(scale, dtype=torch.float32))
    exact = torch.where(ok[:, None], exact, torch.zeros_like(exact))
    err = (out.double() - exact).abs()
    tol = half_step(w.dtype, exact) + U32 * exact.abs()
    assert (err <= tol).all(), err.max()
    assert not out[~ok].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,v,h", [(1, 1, 1), (1, 1000, 4096), (5, 7, 3), (300, 100, 257),
                                   (257, 513, 1000), (1000, 50, 8), (33, 11, 8200), (64, 9, 20011)])
def test_lookup(dev, dtype, n, v, h):
    gen = torch.Generator().manual_seed(n * 7 + v + h)
    w = torch.randn(v, h, generator=gen).to(dtype).to(dev)
    tok = draw_tokens(gen, n, v, dev, bad=0.05)
    status = torch.full((), -1, dtype=torch.int32, device=dev)
    out = lce.embed_fwd(w, tok, scale=1.7, status=status)
    check_lookup(w, tok, 1.7, out)
    is_bad = bool(((tok != IGN) & ~valid(tok, v)).any())
    assert status.item() == (lce.LCE_STATUS_BAD_TOKEN if is_bad else 0)


def test_lookup_of_strided_and_misaligned_rows(dev):
    gen = torch.Generator().manual_seed(3)
    for dtype in DTYPES:
        w = torch.randn(40, 131, generator=gen).to(dtype).to(dev)[:, 1:100]
        tok = draw_tokens(gen, 77, 40, dev)
        buf = torch.full((77, 120), 5.0, dtype=dtype, device=dev)
        out = buf[:, 3:102]
        assert lce.embed_fwd(w, tok, scale=0.5, out=out) is out
        check_lookup(w, tok, 0.5, out)
        assert (buf[:, :3] == 5).all() and (buf[:, 102:] == 5).all()


def test_int64_tokens_and_other_ignore_index(dev):
    w = torch.randn(10, 16, device=dev)
    tok = torch.tensor([3, 0, 2 ** 33 + 3, -100, 9], device=dev)
    status = torch.zeros((), dtype=torch.int32, device=dev)
    out = lce.embed_fwd(w, tok, ignore_index=0, status=status)
    assert torch.equal(out[0], w[3]) and torch.equal(out[4], w[9])
    assert not out[1:4].any() and status.item() == lce.LCE_STATUS_BAD_TOKEN


def check_grad(g, tok, v, scale, got, old=None):
    n, h = g.shape
    ok = valid(tok, v)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    t = tok.long()[ok]
    gd = g.double()[ok]
    exact = torch.zeros(v, h, dtype=torch.float64, device=g.device).index_add_(0, t, gd) * s32
    size = torch.zeros_like(exact).index_add_(0, t, gd.abs()) * abs(s32)
    m = torch.zeros(v, dtype=torch.float64, device=g.device).index_add_(
        0, t, torch.ones(len(t), dtype=torch.float64, device=g.device))
    if old is not None:
        exact = exact + old.double()
        size = size + old.double().abs()
    tol = (m[:, None] + 2) * U32 * size + half_step(got.dtype, exact)
    err = (got.double() - exact).abs()
    assert (err <= tol).all(), ((err - tol).max(), err.max())
    untouched = m == 0
    if old is None:
        assert not got[untouched].any()
    else:
        assert torch.equal(got[untouched], old[untouched])


CASES = [(1, 1, 1, 0.0), (1, 5000, 64, 0.0), (7, 3, 5, 0.2), (64, 1000, 256, 0.1),
         (500, 40, 2049, 0.1), (2049, 300, 72, 0.3), (8192, 500, 32, 0.1), (8193, 4000, 40, 0.05),
         (20000, 65, 16, 0.0), (150000, 3000, 8, 0.1), (6000, 2, 1024, 0.5)]


@pytest.mark.parametrize("n,v,h,ignored", CASES)
@pytest.mark.parametrize("dtype,wide", [(torch.bfloat16, True), (torch.bfloat16, False),
                                        (torch.float16, True), (torch.float16, False),
                                        (torch.float32, True)])
def test_gradient(dev, n, v, h, ignored, dtype, wide):
    gen = torch.Generator().manual_seed(n + v + h)
    g = torch.randn(n, h, generator=gen).to(dtype).to(dev)
    tok = draw_tokens(gen, n, v, dev, ignored, bad=0.02 if n > 100 else 0.0)
    g[~valid(tok, v)] = float("nan")  # rows without a token are not read
    out_dtype = torch.float32 if wide else dtype
    # fp16 sums of thousands of rows stay in range under this scale
    scale = 0.01
    got = lce.embed_bwd(g, tok, v, scale=scale, dtype=out_dtype)
    assert got.dtype == out_dtype and got.shape == (v, h)
    check_grad(g, tok, v, scale, got)
    again = lce.embed_bwd(g, tok, v, scale=scale, dtype=out_dtype)
    assert torch.equal(got, again)
    old = torch.randn(v, h, generator=gen).to(out_dtype).to(dev)
    buf = old.clone()
    assert lce.embed_bwd(g, tok, v, scale=scale, grad_weight=buf, accumulate=True) is buf
    check_grad(g, tok, v, scale, buf, old)


@pytest.mark.parametrize("n", [3, 5000, 70000])
def test_gradient_of_one_token_and_of_none(dev, n):
    """Every row names the same token (its sum crosses every chunk), or no row names one."""
    g = torch.randn(n, 96, device=dev)
    tok = torch.full((n,), 4, dtype=torch.int32, device=dev)
    got = lce.embed_bwd(g, tok, 9)
    check_grad(g, tok, 9, 1.0, got)
    none = lce.embed_bwd(g, torch.full_like(tok, IGN), 9)
    assert not none.any()
    buf = torch.ones(9, 96, device=dev)
    lce.embed_bwd(g, torch.full_like(tok, IGN), 9, grad_weight=buf, accumulate=True)
    assert (buf == 1).all()


def test_gradient_with_a_vocabulary_past_32_bit_keys(dev):
    """(v + 1) · 2048 past 2^32: the sort's keys are 64-bit."""
    n, v = 9000, 2200001
    gen = torch.Generator().manual_seed(5)
    g = torch.randn(n, 8, generator=gen).to(dev)
    tok = torch.randint(0, v, (n,), generator=gen, dtype=torch.int32).to(dev)
    tok[::3] = v - 1
    check_grad(g, tok, v, 1.0, lce.embed_bwd(g, tok, v))


def test_gradient_of_strided_rows(dev):
    gen = torch.Generator().manual_seed(6)
    for dtype in DTYPES:
        g = torch.randn(300, 90, generator=gen).to(dtype).to(dev)[:, 1:70]
        tok = draw_tokens(gen, 300, 50, dev)
        buf = torch.full((50, 80), 3.0, device=dev)
        lce.embed_bwd(g, tok, 50, grad_weight=buf[:, 5:74])
        check_grad(g, tok, 50, 1.0, buf[:, 5:74])
        assert (buf[:, :5] == 3).all() and (buf[:, 74:] == 3).all()


def test_empty_batch(dev):
    w = torch.randn(6, 8, device=dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    assert lce.embed_fwd(w, none).shape == (0, 8)
    g = torch.empty(0, 8, device=dev)
    assert not lce.embed_bwd(g, none, 6).any()
    buf = w.clone()
    lce.embed_bwd(g, none, 6, grad_weight=buf, accumulate=True)
    assert torch.equal(buf, w)


def test_gradient_against_differences(dev):
    """d/dW of f(W) = Σ c · out is linear in W: one step of W in a direction moves f by the
    gradient's product with it, exactly up to fp32 rounding."""
    gen = torch.Generator().manual_seed(8)
    w = torch.randn(30, 24, generator=gen).to(dev)
    c = torch.randn(200, 24, generator=gen).to(dev)
    tok = draw_tokens(gen, 200, 30, dev)
    d = torch.randn(30, 24, generator=gen).to(dev)
    grad = lce.embed_bwd(c, tok, 30, scale=3.0)
    f = lambda t: (lce.embed_fwd(t, tok, scale=3.0).double() * c.double()).sum()  # noqa: E731
    step = (f(w + d) - f(w - d)) / 2
    want = (grad.double() * d.double()).sum()
    # each output carries two fp32 roundings of values up to 3 · (|w| + |d|)
    tol = 8 * U32 * (3 * (w.abs() + d.abs()).double()[tok.long().clamp(min=0)]
                     * c.double().abs()).sum()
    assert (step - want).abs() <= tol


def test_a_table_past_4_gib(dev):
    """Rows whose bytes start past 2^32, looked up and added into."""
    n, v, h = 3000, 1200003, 2048
    w = torch.zeros(v, h, dtype=torch.bfloat16, device=dev)
    gen = torch.Generator().manual_seed(9)
    tok = (v - 1 - torch.randint(0, 900, (n,), generator=gen)).to(torch.int32).to(dev)
    tok[:1000] = torch.randint(0, v, (1000,), generator=gen, dtype=torch.int32).to(dev)
    rows = tok.unique().long()
    w[rows] = torch.randn(len(rows), h, generator=gen).to(torch.bfloat16).to(dev)
    assert torch.equal(lce.embed_fwd(w, tok), w[tok.long()])
    g = torch.randn(n, h, generator=gen).to(torch.bfloat16).to(dev)
    w.fill_(1.0)
    lce.embed_bwd(g, tok, v, grad_weight=w)
    small = torch.searchsorted(rows, tok.long()).to(torch.int32)
    check_grad(g, small, len(rows), 1.0, w[rows])
    w[rows] = 0
    assert not w.any()
