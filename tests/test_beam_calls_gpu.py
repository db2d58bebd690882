"""States of a beam search that lie in one another's gaps, reordered in place and into one another."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def follow(x, parents):
    at = torch.arange(len(x), device=x.device)[:, None]
    rows = x[at, parents.long().clamp(min=0)]
    keep = ((parents >= 0) & (parents < x.shape[1])).view(*parents.shape, *([1] * (x.dim() - 2)))
    return torch.where(keep, rows, torch.zeros((), dtype=x.dtype, device=x.device))


# keys and values [batch, beams, 2, length, dim]; with heads outside; runs of odd bytes
@pytest.mark.parametrize("shape,dim,dtype", [
    ((3, 4, 2, 50, 32), 2, torch.bfloat16), ((2, 8, 2, 5, 40, 64), 2, torch.bfloat16),
    ((2, 5, 3, 7, 11), 2, torch.uint8), ((2, 4, 6, 2, 9, 16), 3, torch.float16),
    ((1, 16, 2, 20000), 2, torch.float32), ((4, 3, 40, 2), 3, torch.int32)])
def test_interlaced_states(dev, shape, dim, dtype):
    whole = torch.randint(0, 200, shape, device=dev).to(dtype)
    batch, beams = shape[:2]
    parents = torch.randint(0, beams, (batch, beams), device=dev, dtype=torch.int32)
    parents[0, 0] = -1
    parents[-1] = torch.arange(beams, device=dev)
    expect = follow(whole, parents)
    # in place: both parts, then one of them
    for some in (range(shape[dim]), range(1, shape[dim])):
        now = whole.clone()
        states = [now.select(dim, k) for k in some]
        got = lce.beam_reorder(states, parents, out=states)
        assert all(a is b for a, b in zip(got, states))
        for k in range(shape[dim]):
            ref = expect if k in some else whole
            assert torch.equal(now.select(dim, k), ref.select(dim, k))
    # from one part into another, and all into another tensor's
    now = whole.clone()
    lce.beam_reorder([now.select(dim, 0)], parents, out=[now.select(dim, 1)])
    assert torch.equal(now.select(dim, 1), expect.select(dim, 0))
    assert torch.equal(now.select(dim, 0), whole.select(dim, 0))
    into = torch.zeros_like(whole)
    lce.beam_reorder([whole.select(dim, k) for k in range(shape[dim])], parents,
                     out=[into.select(dim, k) for k in range(shape[dim])])
    assert torch.equal(into, expect)


def test_shared_bytes_are_refused(dev):
    x = torch.zeros(2, 4, 2, 10, 8, device=dev)
    parents = torch.zeros(2, 4, dtype=torch.int32, device=dev)
    for states in ([x[:, :, 0], x], [x[:, :, 0], x[:, :, 0]], [x[:, :, 0, :6], x[:, :, 0, 5:]]):
        with pytest.raises(lce.LceError):
            lce.beam_reorder(states, parents, out=states)
    with pytest.raises(lce.LceError):
        lce.beam_reorder([x[:, :, 0, :6]], parents, out=[x[:, :, 0, 4:]])


def test_step_with_caches_in_one_tensor(dev):
    """Fp8Head.step, captured and not, with keys and values of a layer in one tensor."""
    from linear_cross_entropy_masked_amd.serving import Fp8Head
    torch.manual_seed(0)
    head = Fp8Head(torch.randn(500, 64, device=dev).bfloat16())
    x = torch.randn(2, 4, 64, device=dev).bfloat16()
    scores = torch.randn(2, 4, device=dev)
    cache = torch.randn(2, 4, 2, 30, 16, device=dev).bfloat16()
    now = cache.clone()
    states = [now[:, :, 0], now[:, :, 1]]
    _, parents, _, _ = head.step(x, scores, states=states)
    assert torch.equal(now, follow(cache, parents))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = head.step(x, scores, states=states)
    for seed in range(3):
        x.copy_(torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(seed)))
        now.copy_(cache)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(now, follow(cache, held[1]))
