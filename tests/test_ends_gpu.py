"""The embedding, layer norm and vocabulary-piece operators as a training step uses them together:
through autograd, on a tied table, under HIP graph capture and on another stream. Each result is
held to the chain of the binding's calls, which test_embed_gpu.py, test_layernorm_gpu.py and
test_pieces_gpu.py hold to fp64."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce
from linear_cross_entropy_masked_amd import autograd as ag

from _helpers import gpu_device

pytestmark = pytest.mark.gpu
IGN = -100
B, U = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def batch(dev, n, v, seed=0, ignored=0.2):
    gen = torch.Generator().manual_seed(seed)
    tok = torch.randint(0, v, (n,), generator=gen)
    lab = torch.randint(0, v, (n,), generator=gen)
    lab[torch.rand(n, generator=gen) < ignored] = IGN
    tok[torch.rand(n, generator=gen) < 0.05] = IGN
    return tok.to(dev), lab.to(dev)


def bf16(dev, *shape, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * std).to(torch.bfloat16).to(dev)


def test_embedding_autograd(dev):
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        w = torch.randn(50, 72, device=dev).to(dtype).requires_grad_()
        tok, _ = batch(dev, 60, 50)
        tok = tok.view(4, 15)
        out = ag.embedding(tok, w, scale=2.0)
        assert out.shape == (4, 15, 72) and out.dtype == dtype
        assert torch.equal(out.view(60, 72), lce.embed_fwd(w.detach(), tok.view(-1), scale=2.0))
        g = torch.randn(4, 15, 72, device=dev).to(dtype)
        out.backward(g)
        assert w.grad.dtype == dtype
        assert torch.equal(w.grad, lce.embed_bwd(g.view(60, 72), tok.view(-1), 50, scale=2.0))
        buf = torch.ones(50, 72, device=dev)
        w.grad = None
        ag.embedding(tok, w, scale=2.0, weight_grad_buffer=buf).backward(g)
        want = torch.ones(50, 72, device=dev)
        lce.embed_bwd(g.view(60, 72), tok.view(-1), 50, scale=2.0, grad_weight=want, accumulate=True)
        assert w.grad is None and torch.equal(buf, want)
        # a broadcast upstream gradient
        (ag.embedding(tok, w).sum() * 3).backward()
        ones = torch.full((60, 72), 3.0, device=dev, dtype=dtype)
        assert torch.equal(w.grad, lce.embed_bwd(ones, tok.view(-1), 50))
    with pytest.raises(ValueError, match="weight_grad_buffer"):
        ag.embedding(tok, w, weight_grad_buffer=torch.zeros(50, 71, device=dev))


def test_layer_norm_autograd(dev):
    x = torch.randn(3, 7, 130, device=dev, requires_grad=True)
    m = ag.LayerNorm(130, device=dev)
    with torch.no_grad():
        m.weight.normal_()
        m.bias.normal_()
    y = m(x)
    g = torch.randn_like(y)
    y.backward(g)
    flat = x.detach().view(21, 130)
    ref, mean, rstd = lce.layernorm_fwd(flat, m.weight.detach(), m.bias.detach())
    assert torch.equal(y.detach().view(21, 130), ref)
    gx, gw, gb = lce.layernorm_bwd(g.view(21, 130), flat, mean, rstd, m.weight.detach(),
                                   grad_bias=True)
    assert torch.equal(x.grad.view(21, 130), gx)
    assert torch.equal(m.weight.grad, gw) and torch.equal(m.bias.grad, gb)
    # no parameters, a transposed input, a broadcast gradient
    x2 = torch.randn(40, 16, device=dev).t().requires_grad_()
    ag.layer_norm(x2).sum().backward()
    _, mean, rstd = lce.layernorm_fwd(x2.detach().contiguous())
    want, _, _ = lce.layernorm_bwd(torch.ones(16, 40, device=dev), x2.detach().contiguous(), mean,
                                   rstd)
    assert torch.equal(x2.grad, want)
    # only the bias asks for a gradient
    xb = torch.randn(5, 130, device=dev)
    b = torch.zeros(130, device=dev, requires_grad=True)
    ag.layer_norm(xb, None, b).backward(torch.ones(5, 130, device=dev))
    assert (b.grad == 5).all()
    with pytest.raises(RuntimeError):
        z = torch.randn(2, 130, device=dev, requires_grad=True)
        (gz,) = torch.autograd.grad(ag.layer_norm(z).sum(), z, create_graph=True)
        gz.sum().backward()


@pytest.mark.parametrize("reduction", ["sum", "mean", "none"])
@pytest.mark.parametrize("many", [False, True])
def test_piece_loss_autograd(dev, reduction, many):
    n, h, sizes = 90, 64, [300, 77]
    _, lab = batch(dev, n, 377)
    hid = bf16(dev, 6, 15, h).requires_grad_()
    ws = [bf16(dev, s, h, seed=s, std=0.2).requires_grad_() for s in sizes]
    bs = [torch.randn(s, device=dev, requires_grad=True) for s in sizes]
    wt, bt = (ws, bs) if many else (ws[0], bs[0])
    if not many:
        lab = torch.where(lab >= 300, torch.full_like(lab, IGN), lab)
    mask = torch.rand(6, 15, device=dev) < 0.8
    out = ag.linear_cross_entropy_pieces(hid, wt, lab.view(6, 15), bt, mask=mask,
                                         reduction=reduction, piece_size=128)
    folded = torch.where(mask.view(-1), lab, torch.full_like(lab, IGN))
    det = (lambda t: [x.detach() for x in t]) if many else (lambda t: t.detach())
    t = None if reduction == "mean" else 1
    flat = hid.detach().view(n, h)
    loss, lse, rows = lce.flce_pieces_fwd(flat, det(wt), folded, det(bt), num_label_tokens=t,
                                          return_rows=True)
    if reduction == "none":
        assert out.shape == (6, 15) and torch.equal(out.detach().view(-1), rows)
        g = torch.randn(6, 15, device=dev)
        kw = dict(grad_rows=g.view(-1))
    else:
        assert torch.equal(out.detach(), loss)
        g = torch.tensor(1.5, device=dev)
        kw = dict(grad_output=g, num_label_tokens=t)
    out.backward(g)
    gh, gw, gb = lce.flce_pieces_bwd(flat, det(wt), folded, lse, det(bt), piece_size=128, **kw)
    assert torch.equal(hid.grad.view(n, h), gh)
    for k, (w, b) in enumerate(zip(ws, bs)):
        if not many and k == 1:
            assert w.grad is None
            continue
        assert torch.equal(w.grad, gw[k] if many else gw)
        assert torch.equal(b.grad, gb[k] if many else gb)


def test_piece_loss_frozen_tensors_and_buffers(dev):
    n, h = 70, 128
    _, lab = batch(dev, n, 400)
    hid = bf16(dev, n, h).requires_grad_()
    base, new = bf16(dev, 300, h, seed=1, std=0.1), bf16(dev, 100, h, seed=2, std=0.1)
    new.requires_grad_()  # tokens added to a frozen vocabulary
    loss = ag.linear_cross_entropy_pieces(hid, [base, new], lab, reduction="mean")
    loss.backward()
    _, lse, _ = lce.flce_pieces_fwd(hid.detach(), [base, new.detach()], lab)
    gh, gw, _ = lce.flce_pieces_bwd(hid.detach(), [base, new.detach()], lab, lse)
    assert base.grad is None and torch.equal(new.grad, gw[1]) and torch.equal(hid.grad, gh)
    base.requires_grad_()
    new.grad = None
    bias = [torch.randn(300, device=dev, requires_grad=True),
            torch.randn(100, device=dev, requires_grad=True)]
    bufs = [torch.ones(300, h, device=dev), torch.ones(100, h, device=dev).to(torch.bfloat16)]
    ag.linear_cross_entropy_pieces(hid, [base, new], lab, bias, reduction="mean",
                                   weight_grad_buffer=bufs).backward()
    assert base.grad is None and new.grad is None
    db = [b.detach() for b in bias]
    _, lse, _ = lce.flce_pieces_fwd(hid.detach(), [base.detach(), new.detach()], lab, db)
    want = [torch.ones(300, h, device=dev), torch.ones(100, h, device=dev).to(torch.bfloat16)]
    _, _, gb = lce.flce_pieces_bwd(hid.detach(), [base.detach(), new.detach()], lab, lse, db,
                                   grad_weight=want,
                                   grad_bias=[torch.zeros(300, device=dev),
                                              torch.zeros(100, device=dev)], accumulate=True)
    for k in range(2):
        assert torch.equal(bufs[k], want[k]) and torch.equal(bias[k].grad, gb[k])
    with pytest.raises(ValueError, match="buffers"):
        ag.linear_cross_entropy_pieces(hid, [base, new], lab, weight_grad_buffer=bufs[0])


def test_norm_and_loss_in_one(dev):
    """The joined function gives the two functions' results, without keeping the normalised
    states."""
    n, h, v = 130, 192, 500
    _, lab = batch(dev, n, v)
    mod = ag.LinearCrossEntropyPieces(reduction="mean")
    res = []
    for joined in (False, True):
        x = bf16(dev, n, h, seed=4).requires_grad_()
        nw, nb = bf16(dev, h, seed=5).requires_grad_(), bf16(dev, h, seed=6).requires_grad_()
        w = bf16(dev, v, h, seed=7, std=0.1).requires_grad_()
        if joined:
            loss = ag.norm_linear_cross_entropy(x, nw, nb, w, lab, reduction="mean")
        else:
            loss = mod(ag.layer_norm(x, nw, nb), w, lab)
        loss.backward()
        res.append((loss.detach(), x.grad, nw.grad, nb.grad, w.grad))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def step_of_calls(table, nw, nb, tok, lab, scale, buffer):
    """One training step of a model that is nothing but its two ends, as calls of the binding."""
    x = lce.embed_fwd(table, tok, scale=scale)
    y, mean, rstd = lce.layernorm_fwd(x, nw, nb)
    loss, lse, rows = lce.flce_pieces_fwd(y, table, lab, return_rows=True)
    gy, _, _ = lce.flce_pieces_bwd(y, table, lab, lse, grad_weight=buffer, accumulate=True)
    gx, gnw, gnb = lce.layernorm_bwd(gy, x, mean, rstd, nw, grad_bias=True)
    lce.embed_bwd(gx, tok, table.shape[0], scale=scale, grad_weight=buffer, accumulate=True)
    return loss, rows, gnw, gnb, buffer


@pytest.mark.parametrize("n,v,h", [(3, 70, 64), (300, 1000, 256), (1025, 777, 72)])
def test_tied_head_step(dev, n, v, h):
    tok, lab = batch(dev, n, v, seed=n)
    head = ag.TiedHead(v, h, scale=3.0, main_grad=True, device=dev)
    x = head.embed(tok)
    loss = head(x, lab)
    loss.backward()
    assert head.weight.grad is None
    buf = torch.zeros(v, h, device=dev)
    nw, nb = head.norm.weight.detach(), head.norm.bias.detach()
    want = step_of_calls(head.weight.detach(), nw, nb, tok, lab, 3.0, buf)
    assert torch.equal(loss.detach(), want[0])
    assert torch.equal(head.norm.weight.grad, want[2])
    assert torch.equal(head.norm.bias.grad, want[3])
    assert torch.equal(head.main_grad, want[4])
    # without the fp32 buffer autograd adds two bf16 gradients: three roundings to bf16 of
    # without the fp32 buffer autograd adds two bf16 gradients: each part is rounded (B of it at
    # most), then their sum (B of at most 1 + B of the parts' sizes)
    plain = ag.TiedHead(v, h, scale=3.0, device=dev)
    with torch.no_grad():
        plain.weight.copy_(head.weight)
    plain(plain.embed(tok), lab).backward()
    part = torch.zeros(v, h, device=dev)
    x0 = lce.embed_fwd(head.weight.detach(), tok, scale=3.0)
    y0, mean, rstd = lce.layernorm_fwd(x0, nw, nb)
    _, lse, _ = lce.flce_pieces_fwd(y0, head.weight.detach(), lab)
    lce.flce_pieces_bwd(y0, head.weight.detach(), lab, lse, grad_weight=part)
    size = part.abs() + (head.main_grad - part).abs()
    err = (plain.weight.grad.float() - head.main_grad).abs()
    assert (err <= 2 * B * (1 + 2 * B) * size + 1e-30).all()


def test_step_against_fp64_autograd(dev):
    """The whole step against plain fp64 autograd of the same model. The kernels round the hidden
    states, their normalised form and both hidden gradients to bf16: four relative errors of at
    most 2^-8 each along the chain, which a norm-wise bound of 2^-5 leaves room for."""
    n, v, h = 200, 300, 128
    tok, lab = batch(dev, n, v, seed=11)
    head = ag.TiedHead(v, h, scale=2.0, main_grad=True, device=dev)
    loss = head(head.embed(tok), lab)
    loss.backward()
    w = head.weight.detach().double().cpu().requires_grad_()
    ok = (tok >= 0).cpu()
    x = torch.where(ok[:, None], w[tok.cpu().clamp(min=0)] * 2.0, 0.0)
    c = x - x.mean(1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5)
    z = y @ w.t()
    keep = (lab >= 0).cpu()
    rows = torch.logsumexp(z, 1) - z.gather(1, lab.cpu().clamp(min=0)[:, None])[:, 0]
    ref = rows[keep].mean()
    ref.backward()
    assert abs(loss.item() - ref.item()) <= 2.0 ** -5 * abs(ref.item())
    d = (head.main_grad.double().cpu() - w.grad).norm() / w.grad.norm()
    assert d <= 2.0 ** -5


def test_graph_replays(dev):
    """The chain of calls captured once and replayed with eager work between the replays; every
    replay is the eager result bit for bit."""
    n, v, h = 300, 700, 128
    table, nw, nb = bf16(dev, v, h, std=0.05), bf16(dev, h, seed=1), bf16(dev, h, seed=2)
    tok, lab = batch(dev, n, v, seed=5)
    tok, lab = tok.to(torch.int32), lab.to(torch.int32)
    buf = torch.zeros(v, h, device=dev)

    def run():
        buf.zero_()
        return step_of_calls(table, nw, nb, tok, lab, 2.0, buf)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(4):
        t2, l2 = batch(dev, n, v, seed=50 + k, ignored=0.2 + 0.2 * k)
        tok.copy_(t2)
        lab.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        junk = torch.randn(1 << 20, device=dev).sum()  # the program's own work in between
        want = step_of_calls(table, nw, nb, tok, lab, 2.0, torch.zeros(v, h, device=dev))
        torch.cuda.synchronize()
        assert junk.isfinite()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), k


def test_two_streams_at_once(dev):
    """Two steps in flight on two streams do not share scratch memory."""
    n, v, h = 500, 900, 256
    table, nw, nb = bf16(dev, v, h, std=0.05), bf16(dev, h, seed=1), bf16(dev, h, seed=2)
    data = [batch(dev, n, v, seed=s) for s in (1, 2)]
    want = [step_of_calls(table, nw, nb, *d, 2.0, torch.zeros(v, h, device=dev)) for d in data]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for d, s in zip(data, streams):
            with torch.cuda.stream(s):
                got.append(step_of_calls(table, nw, nb, *d, 2.0, torch.zeros(v, h, device=dev)))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[k % 2])), k


@pytest.mark.parametrize("which", [0, 1])
def test_piece_loss_with_a_bias_on_one_piece(dev, which):
    """A bias of zeros adds nothing: pieces without one give the same loss and gradients, and the
    one that has a bias gets its gradient."""
    sizes = [300, 70]
    _, lab = batch(dev, 90, sum(sizes))
    b = torch.linspace(-1, 1, sizes[which], device=dev)

    def run(mixed):
        hid = bf16(dev, 90, 64, seed=1).requires_grad_()
        ws = [bf16(dev, v, 64, seed=2 + k, std=0.3).requires_grad_() for k, v in enumerate(sizes)]
        bs = [None if mixed else torch.zeros(v, device=dev) for v in sizes]
        bs[which] = b.clone().requires_grad_()
        loss = ag.linear_cross_entropy_pieces(hid, ws, lab, bs)
        loss.backward()
        return [loss.detach(), hid.grad, *(w.grad for w in ws), bs[which].grad]
    for got, want in zip(run(True), run(False)):
        assert torch.equal(got, want)
    hid, ws = bf16(dev, 90, 64, seed=1), [bf16(dev, v, 64, seed=2 + k) for k, v in enumerate(sizes)]
    bs = [None, None]
    bs[which] = b
    _, lse, _ = lce.flce_pieces_fwd(hid, ws, lab, bs)
    _, _, gbs = lce.flce_pieces_bwd(hid, ws, lab, lse, bs)
    assert gbs[1 - which] is None and gbs[which].shape == b.shape


def test_layer_norm_with_a_bias_alone(dev):
    """An fp32 bias beside bf16 rows and no weight: its gradient is not rounded to bf16."""
    x = bf16(dev, 400, 96, seed=3)
    b = torch.zeros(96, device=dev, requires_grad=True)
    g = bf16(dev, 400, 96, seed=4)
    ag.layer_norm(x, None, b).backward(g)
    assert b.grad.dtype == torch.float32
    exact = g.double().sum(0)
    assert ((b.grad.double() - exact).abs() <= 401 * U * g.double().abs().sum(0)).all()
    w = bf16(dev, 300, 96, seed=5, std=0.1)
    _, lab = batch(dev, 400, 300)
    b.grad = None
    ag.norm_linear_cross_entropy(x, None, b, w, lab).backward()
    y, _, _ = lce.layernorm_fwd(x, None, b.detach())
    _, lse, _ = lce.flce_pieces_fwd(y, w, lab)
    gy, _, _ = lce.flce_pieces_bwd(y, w, lab, lse, num_label_tokens=1, grad_weight=False)
    exact = gy.double().sum(0)
    assert ((b.grad.double() - exact).abs() <= 401 * U * gy.double().abs().sum(0)).all()


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("frozen", [False, True])
def test_a_buffer_for_one_of_two_weights(dev, which, frozen):
    """The weight with a buffer has its gradient added there, as with a buffer for both; the other
    one gets its own in .grad, as without buffers (none where it is frozen)."""
    n, h, sizes = 90, 64, [300, 77]
    _, lab = batch(dev, n, sum(sizes))

    def run(joined, buffers, freeze=False):
        x = bf16(dev, n, h, seed=1).requires_grad_()
        ws = [bf16(dev, v, h, seed=2 + k, std=0.3).requires_grad_(k == which or not freeze)
              for k, v in enumerate(sizes)]
        bs = [torch.zeros(v, device=dev, requires_grad=True) for v in sizes]
        if joined:
            loss = ag.norm_linear_cross_entropy(x, None, None, ws, lab, bs,
                                                weight_grad_buffer=buffers)
        else:
            loss = ag.linear_cross_entropy_pieces(x, ws, lab, bs, weight_grad_buffer=buffers)
        loss.backward()
        return x.grad, [w.grad for w in ws], [b.grad for b in bs]
    for joined in (False, True):
        both = [torch.zeros(v, h, device=dev) for v in sizes]
        run(joined, both)
        gx, gws, gbs = run(joined, None)
        one = [None, None]
        one[which] = torch.zeros(sizes[which], h, device=dev)
        gx2, gws2, gbs2 = run(joined, one, frozen)
        assert gws2[which] is None and torch.equal(one[which], both[which])
        assert gws2[1 - which] is None if frozen else torch.equal(gws2[1 - which], gws[1 - which])
        assert torch.equal(gx2, gx) and all(torch.equal(a, b) for a, b in zip(gbs2, gbs))
