"""The label element and the per-row coefficients of the loss in pieces of the vocabulary, held
tighter than test_pieces_gpu.py holds them.

Tolerances, u = 2^-24 and b = 2^-8 as there: a logit gradient d = p - [v = y] carries its fp32 error
p·(dz + dlse + 2^-16) + 2u, and every element but the label's also half a bf16 step, b·|d|, of the
matrix operand. The label's keeps its fp32 value: what the operand's rounding leaves of it is itself
an fp32 number, added with the same factors. Coefficient, scale and their products are 4 roundings
more; the products are fp32 sums of exact products, of the operand and of what it left, n (or v) +
8 additions each. What the operand left of the labels, at most b·|d|·|hidden| a row, is summed for
each class and goes into its weight gradient in bf16: b of that."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce
from linear_cross_entropy_masked_amd import autograd as ag

from _helpers import gpu_device
from test_pieces_gpu import B, IGN, U, make, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def raised(hid, w, lab, by):
    """Hidden states whose label logit is `by` higher."""
    y = lab.long().clamp(min=0)
    wy = w[y].double()
    up = hid.double() + by * wy / (wy * wy).sum(1, keepdim=True)
    return torch.where((lab >= 0)[:, None], up.to(torch.bfloat16), hid)


class Sharp:
    """Gradients in fp64 and their bounds with an exact label element."""

    def __init__(self, hid, w, b, lab, t=None, rows=None):
        n, h = hid.shape
        v = w.shape[0]
        self.keep = keep = lab >= 0
        hd = torch.where(keep[:, None], hid, torch.zeros_like(hid)).double()
        wd = w.double()
        z = hd @ wd.t()
        dz = (h + 2) * U * (hd.abs() @ wd.abs().t())
        if b is not None:
            z = z + b.double()
        dz = dz + 2 * U * z.abs()
        y = lab.long().clamp(0, v - 1)[:, None]
        lse = torch.logsumexp(z, 1)
        dlse = dz.max(1).values + 2.0 ** -16 + 2 * U * lse.abs()
        self.lse = torch.where(keep, lse, torch.zeros_like(lse))
        t = int(keep.sum()) if t is None else t
        c = torch.full_like(lse, 1.0 / t) if rows is None else rows.double()
        c = torch.where(keep, c, torch.zeros_like(lse))[:, None]
        p = (z - lse[:, None]).exp()
        ed = (p * (dz + dlse[:, None] + 2.0 ** -16) + 2 * U) * c.abs()
        d = p.scatter_add(1, y, torch.full_like(y, -1, dtype=p.dtype)) * c
        operand = B * d.abs()
        operand.scatter_(1, y, 0.0)
        eb = ed + operand + 4 * U * d.abs()
        self.gh, self.gw = d @ wd, d.t() @ hd
        self.dgh = eb @ wd.abs() + (2 * v + 16) * U * (d.abs() @ wd.abs())
        label = (d.abs().gather(1, y) * hd.abs())[keep]
        self.dgw = (eb.t() @ hd.abs() + (2 * n + 16) * U * (d.abs().t() @ hd.abs())
                    + B * B * (1 + B) * torch.zeros_like(self.gw).index_add_(0, y[keep, 0], label))


# few tiles; products apart and together; a split hidden gradient and one that is not; more than one
# run of the label sort; rows numbered in a launch of their own; hidden sizes off 64
SHAPES = [(3, 64, 500), (40, 72, 3000), (300, 200, 2000), (300, 1032, 4097), (700, 1024, 5003),
          (2500, 256, 9001), (9001, 64, 520), (300, 4096, 66000)]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("by", [0.0, 8.0])
def test_label_element(dev, n, h, v, by):
    """Weight gradients in both types, fp32 ones accumulated, and the fp32 hidden gradient carried
    between pieces. A third of the rows share one label."""
    hid, w, b, lab = make(dev, n, h, v, bias=by == 0.0)
    lab[::3] = torch.where(lab[::3] >= 0, torch.full_like(lab[::3], v - 1), lab[::3])
    hid = raised(hid, w, lab, by)
    e = Sharp(hid, w, b, lab)
    lse = e.lse.float()
    gw, acc = torch.empty(v, h, device=dev), torch.full((n, h), 9.0, device=dev)
    lce.flce_piece_bwd(hid, w, lab, lse, b, v_start=0, vocab=v, first=True, last=False,
                       hidden_acc=acc, grad_weight=gw)
    near(gw, e.gw, e.dgw, "grad_weight")
    near(acc, e.gh, e.dgh, "hidden_acc")
    assert not acc[~e.keep].any()
    old = torch.randn(v, h, device=dev)
    buf = old.clone()
    gh, _, _ = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=buf, grad_bias=False,
                                   accumulate=True, piece_size=max(1, v // 3))
    near(gh, e.gh, e.dgh + 8 * U * e.gh.abs(), "grad_hidden")
    near(buf, e.gw + old.double(), e.dgw + 4 * U * (e.gw.abs() + old.double().abs()), "accumulated")
    alone = torch.empty(v, h, device=dev)
    lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_hidden=False, grad_weight=alone, grad_bias=False)
    near(alone, e.gw, e.dgw, "grad_weight alone")
    for piece in (None, max(1, v // 3)):
        _, gw, _ = lce.flce_pieces_bwd(hid, w, lab, lse, b, piece_size=piece)
        near(gw, e.gw, e.dgw, "bf16 grad_weight")


@pytest.mark.parametrize("by", [0.0, 6.0, 12.0])
def test_fp32_weight_gradient_norm_wise(dev, by):
    """The library's 1e-4 for fp32 weight gradients. Independent roundings of the elements off the
    label leave 8e-4 (the rms relative error of a bf16 rounding) times sqrt(e^{1.5^2} / v), 1.4e-5
    here; a label element rounded to bf16 leaves up to 2e-3."""
    n, h, v = 1024, 768, 32777
    hid, w, b, lab = make(dev, n, h, v, masked=0.0)
    hid = raised(hid, w, lab, by)
    e = Sharp(hid, w, b, lab)
    gw = torch.empty(v, h, device=dev)
    lce.flce_pieces_bwd(hid, w, lab, e.lse.float(), b, grad_weight=gw, grad_bias=False)
    assert float((gw.double() - e.gw).norm() / e.gw.norm()) <= 1e-4
    near(gw, e.gw, e.dgw, "grad_weight")


@pytest.mark.parametrize("n,h,v", [(40, 72, 3000), (300, 1032, 4097), (9001, 64, 520)])
def test_label_element_with_row_gradients(dev, n, h, v):
    hid, w, b, lab = make(dev, n, h, v)
    g = torch.randn(n, device=dev)
    g[2] = 0.0
    g[lab == IGN] = float("nan")
    e = Sharp(hid, w, b, lab, rows=g)
    gw = torch.empty(v, h, device=dev)
    gh, _, _ = lce.flce_pieces_bwd(hid, w, lab, e.lse.float(), b, grad_rows=g, grad_weight=gw)
    near(gw, e.gw, e.dgw, "grad_weight")
    near(gh, e.gh, e.dgh, "grad_hidden")
    _, gw, _ = lce.flce_pieces_bwd(hid, w, lab, e.lse.float(), b, grad_rows=g, grad_hidden=False)
    near(gw, e.gw, e.dgw, "bf16 grad_weight")


@pytest.mark.parametrize("n,h,v,piece", [(12, 64, 900, None), (1003, 256, 4000, None),
                                         (1003, 256, 4000, 1500), (9001, 64, 520, None)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_equal_row_gradients_are_the_summed_loss(dev, n, h, v, piece, dtype):
    """Row gradients that are all 1 / T are the mean loss, bit for bit: the common factor stays out
    of the bf16 operand, where it would be rounded the same way in every label element. What rows
    without a label have for a coefficient does not count."""
    hid, w, b, lab = make(dev, n, h, v)
    g = torch.full((n,), 1.0 / 1003, device=dev)
    g[lab == IGN] = 7.0
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    res = []
    for kw in (dict(grad_rows=g), dict(num_label_tokens=1003)):
        gw = torch.empty(v, h, dtype=dtype, device=dev)
        res.append(lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=gw, piece_size=piece, **kw))
    for got, want in zip(*res):
        assert torch.equal(got, want)


def test_mean_of_the_row_terms_is_the_mean_loss(dev):
    n, h, v = 1003, 128, 700
    hid, w, _, lab = make(dev, n, h, v, bias=False)
    res = []
    for reduction in ("none", "sum"):
        x, wt = hid.clone().requires_grad_(), w.clone().requires_grad_()
        out = ag.linear_cross_entropy_pieces(x, wt, lab, reduction=reduction,
                                             num_label_tokens=n if reduction == "sum" else None)
        out.mean().backward()
        res.append((x.grad, wt.grad))
    for got, want in zip(*res):
        assert torch.equal(got, want)


def test_row_gradients_of_zero_and_of_infinity(dev):
    """All zeros give zeros; an infinite coefficient reaches its own row of the hidden gradient, and
    the other rows keep theirs."""
    n, h, v = 100, 64, 700
    hid, w, b, lab = make(dev, n, h, v)
    lab[5], lab[6] = 3, 4
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    for out in lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=torch.zeros(n, device=dev)):
        assert not out.any()
    g = torch.randn(n, device=dev)
    want, _, _ = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g)
    for value in (float("inf"), float("nan")):
        g2 = g.clone()
        g2[5] = value
        ref = g.clone()
        ref[5] = 0.0
        got, _, _ = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g2)
        want, _, _ = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=ref)
        others = torch.arange(n, device=dev) != 5
        assert torch.equal(got[others], want[others])
        assert not got[5].isfinite().any()


@pytest.mark.parametrize("n,h,v", [(70, 64, 600), (300, 1032, 4097)])
def test_the_hidden_gradient_in_fp32(dev, n, h, v):
    """Without grad_hidden, hidden_acc holds all pieces after the last, of several or of one."""
    hid, w, b, lab = make(dev, n, h, v)
    e = Sharp(hid, w, b, lab)
    for parts in ([v], [v - 100, 100], [100, v - 200, 100]):
        acc = torch.full((n, h), float("nan"), device=dev)
        at = 0
        for k, (ws, bs) in enumerate(zip(w.split(parts), b.split(parts))):
            lce.flce_piece_bwd(hid, ws, lab, e.lse.float(), bs, v_start=at, vocab=v, first=k == 0,
                               last=k == len(parts) - 1, hidden_acc=acc)
            at += len(ws)
        near(acc, e.gh, e.dgh + 4 * U * e.gh.abs(), "hidden_acc")
        assert not acc[~e.keep].any()
    # with grad_hidden the last piece goes there alone
    acc, gh = torch.empty(n, h, device=dev), torch.empty(n, h, dtype=torch.bfloat16, device=dev)
    lce.flce_piece_bwd(hid, w[:-100], lab, e.lse.float(), b[:-100], v_start=0, vocab=v, first=True,
                       last=False, hidden_acc=acc, grad_hidden=gh)
    before = acc.clone()
    lce.flce_piece_bwd(hid, w[-100:], lab, e.lse.float(), b[-100:], v_start=v - 100, vocab=v,
                       first=False, last=True, hidden_acc=acc, grad_hidden=gh)
    assert torch.equal(acc, before)
    near(gh, e.gh, e.dgh + 4 * U * e.gh.abs(), "grad_hidden")


@pytest.mark.parametrize("n", [300, 9001])
def test_replays_with_other_labels(dev, n):
    """Fresh gradients in both types and row gradients, captured and replayed with other labels and
    coefficients and eager work between: what one replay notes of its labels is gone in the next."""
    h, v = 128, 700
    hid, w, b, lab = make(dev, n, h, v)
    g = torch.randn(n, device=dev)
    lse = Sharp(hid, w, b, lab).lse.float()

    def run():
        gw = torch.empty(v, h, device=dev)
        return (*lce.flce_pieces_bwd(hid, w, lab, lse, b),
                *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g, grad_weight=gw))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(4):
        lab.copy_(torch.randint(0, v if k % 2 else 40, (n,), device=dev, dtype=torch.int32))
        lab[k::5] = IGN
        g.copy_(torch.randn(n, device=dev))
        lse.copy_(torch.logsumexp(hid.float() @ w.float().t() + b, 1))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        junk = torch.randn(1 << 20, device=dev).sum()
        want = run()
        torch.cuda.synchronize()
        assert junk.isfinite() and all(torch.equal(x, y) for x, y in zip(got, want)), k
