"""A decoding step behind the last layer as it is used: residual and norm in 8 bits, logits in 8
bits, selection and reordering, from a tied head that trains in 16 bits.

The 8-bit operands are what the library's quantiser makes of them (tested by itself), so the logits
are compared with the exact product of the same 8-bit values."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce
from linear_cross_entropy_masked_amd.autograd import TiedHead
from linear_cross_entropy_masked_amd.serving import Fp8Head

from _fp8 import spread
from _helpers import gpu_device
from test_beam_gpu import check_step
from test_fp8_gpu import check_product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


@pytest.fixture(scope="module")
def head(dev):
    torch.manual_seed(3)
    h = TiedHead(3001, 256, rms=True, device=dev)
    torch.nn.init.normal_(h.weight, std=0.1)
    torch.nn.init.normal_(h.norm.weight, 1.0, 0.1)
    return h


@pytest.mark.parametrize("scale", [None, torch.float32])
@pytest.mark.parametrize("batch,beams", [(1, 4), (30, 8)])
def test_step(dev, head, batch, beams, scale):
    served = Fp8Head.of(head, scale_dtype=scale, logits_dtype=torch.float32)
    x = torch.randn(batch, beams, 256, device=dev).bfloat16()
    r = torch.randn(batch, beams, 256, device=dev).bfloat16()
    z, s = served(x, r)
    assert z.shape == (batch, beams, 3001) and torch.equal(s, x + r)
    q, c, _ = lce.rmsnorm_fp8_fwd(x.view(-1, 256), head.norm.weight, r.view(-1, 256),
                                  eps=head.norm.eps, scale_dtype=served.scales.dtype)
    check_product(z.view(-1, 3001), q, c, served.weight, served.scales)
    # 8 bits beside 16: each operand is off by at most 1/16, independently over 256 columns
    full = torch.nn.functional.linear(
        torch.nn.functional.rms_norm(s.float(), (256,), head.norm.weight.float(), head.norm.eps),
        head.weight.float())
    assert (z - full).norm() / full.norm() <= 2 / 16
    scores = torch.randn(batch, beams, device=dev) - 5
    history = torch.randint(0, 3001, (batch, beams, 9), device=dev)
    before = history.clone()
    got = served.step(x, scores, r, states=[history], eos=7)
    check_step(z, scores, beams, None, 7, got=got)
    assert torch.equal(history, torch.gather(before, 1, got[1].long()[..., None].expand(-1, -1, 9)))


def test_bias_bans_tokens(dev, head):
    bias = torch.zeros(3001, device=dev)
    bias[5:] = float("-inf")
    served = Fp8Head(head.weight, head.norm.weight, bias, eps=head.norm.eps)
    x = torch.randn(2, 3, 256, device=dev).bfloat16()
    best, parents, tokens, _ = served.step(x, torch.zeros(2, 3, device=dev), num=20)
    assert (tokens[:, :15] < 5).all() and (tokens[:, 15:] == -100).all()
    assert (parents[:, 15:] == -1).all() and (best[:, 15:] == float("-inf")).all()
    assert (head.embed(tokens)[:, 15:] == 0).all()  # no token: a zero row


def test_a_captured_step(dev, head):
    """The whole step as one graph, replayed on other hidden states."""
    served = Fp8Head.of(head)
    x = torch.randn(2, 4, 256, device=dev).bfloat16()
    r = torch.randn(2, 4, 256, device=dev).bfloat16()
    scores = torch.zeros(2, 4, device=dev)

    def step():
        return served.step(x, scores, r, eos=1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        x.copy_(torch.randn(2, 4, 256, generator=torch.Generator().manual_seed(seed)))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(held, eager):
            assert torch.equal(p, q)


def test_refusals(dev, head):
    with pytest.raises(ValueError, match="rms"):
        Fp8Head.of(TiedHead(64, 32, device=dev))
    with pytest.raises(ValueError, match="16"):
        Fp8Head(torch.zeros(64, 40, device=dev))
    with pytest.raises(ValueError, match="rms"):
        x = torch.zeros(2, 32, device=dev).bfloat16()
        TiedHead(64, 32, device=dev)(x, torch.zeros(2, dtype=torch.long, device=dev), residual=x)
