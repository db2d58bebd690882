"""Per-row coefficients of the loss in pieces of the vocabulary."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce
from linear_cross_entropy_masked_amd import autograd as ag

from _helpers import gpu_device
from test_pieces_gpu import IGN, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


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
