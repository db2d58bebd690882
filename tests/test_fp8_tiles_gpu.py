"""The 8-bit product's large tiles (256 x 256), at sizes that its rule sends there, with the choice of
kernel asserted by name: a later change of the rule that leaves a test of them without its kernel
fails it. Tolerances as in test_fp8_gpu.py."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _fp8 import E4M3, E8M0, spread
from _helpers import gpu_device
from test_fp8_gpu import check_product, operands

pytestmark = pytest.mark.gpu

SCALES = [E8M0, torch.float32]


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def named(call):
    """What a call returns and the names of the kernels that it launched."""
    torch.cuda.synchronize()
    lce.lce_timing_enable(True)
    try:
        lce.lce_timing_read()
        out = call()
        torch.cuda.synchronize()
        return out, {name for name, _, _ in lce.lce_timing_read()}
    finally:
        lce.lce_timing_enable(False)


# 256 large tiles, whole and ragged on both sides; one to six slices in a ring of two, last blocks of
# 16 to 128 columns; a second round of tiles
SHAPES = [(4096, 4096, 16), (4096, 4096, 128), (4096, 4096, 272), (3850, 4095, 656),
          (3841, 3969, 384), (4095, 3850, 144), (7937, 8191, 528)]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(dev, m, n, k, scale):
    a, ca, b, cb = operands(m, n, k, scale, dev)
    for bias in (None, torch.randn(n, device=dev)):
        out, names = named(lambda: lce.fp8_matmul(a, ca, b, cb, bias))
        assert names == {"fp8_matmul_large"} and out.dtype == torch.bfloat16
        check_product(out, a, ca, b, cb, bias)
        assert torch.equal(out, lce.fp8_matmul(a, ca, b, cb, bias))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("m,n,k", [(4096, 4096, 272), (3850, 4095, 1040)])
def test_product_of_whole_numbers_is_exact(dev, m, n, k, scale):
    """Small whole numbers and scales: a product is at most 64 and a grid of 2^-13 of that holds
    whole numbers, every sum is one below 2^24, so the result is rounded once, to bf16."""
    gen = torch.Generator().manual_seed(m)
    a = torch.randint(-8, 9, (m, k), generator=gen).float().to(dev).to(E4M3)
    b = torch.randint(-8, 9, (n, k), generator=gen).float().to(dev).to(E4M3)
    kb, nb = -(-k // 128), -(-n // 128)
    ca = torch.exp2(torch.randint(0, 3, (kb, m), generator=gen).float()).to(dev)
    cb = torch.exp2(torch.randint(0, 3, (nb, kb), generator=gen).float()).to(dev)
    if scale == E8M0:
        ca, cb = ((c.log2() + 127).to(torch.uint8).view(E8M0) for c in (ca, cb))
    bias = torch.randint(-5, 6, (n,), generator=gen).float().to(dev)
    out, names = named(lambda: lce.fp8_matmul(a, ca, b, cb, bias))
    assert names == {"fp8_matmul_large"}
    exact = (a.double() * spread(ca, 1, m, k)) @ (b.double() * spread(cb, 128, n, k)).t() + bias
    assert torch.equal(out, exact.float().bfloat16())


@pytest.mark.parametrize("scale", SCALES)
def test_product_strides_and_special_values(dev, scale):
    """Operands, scales and result inside wider ones, what lies beside them NaN; a NaN row, a NaN
    block of columns, rows of zeros, infinite biases."""
    m, n, k = 3850, 4095, 400
    a, ca, b, cb = operands(m, n, k, scale, dev)

    def inside(t, left, right, below):
        shape = (t.shape[0] + below, left + t.shape[1] + right)
        if t.dtype == torch.float32:
            wide = torch.full(shape, float("nan"), device=dev)
            view = wide[:t.shape[0], left:left + t.shape[1]]
            view.copy_(t)
            return view
        wide = torch.full(shape, 0xff if t.dtype == E8M0 else 0x7f, device=dev, dtype=torch.uint8)
        view = wide[:t.shape[0], left:left + t.shape[1]]
        view.copy_(t.view(torch.uint8))
        return view.view(t.dtype)
    ref = lce.fp8_matmul(a, ca, b, cb)
    wide = torch.full((m + 2, n + 7), float("nan"), device=dev, dtype=torch.bfloat16)
    view = wide[:m, 3:3 + n]
    args = inside(a, 16, 32, 3), inside(ca, 1, 2, 2), inside(b, 32, 16, 5), inside(cb, 3, 1, 1)
    got, names = named(lambda: lce.fp8_matmul(*args, out=view))
    assert names == {"fp8_matmul_large"} and got is view and torch.equal(view, ref)
    assert torch.isnan(wide[m:]).all() and torch.isnan(wide[:, :3]).all()
    assert torch.isnan(wide[:, 3 + n:]).all()
    a8, ca8, cb8 = (t.view(torch.uint8).clone() if t.dtype != torch.float32 else t.clone()
                    for t in (a, ca, cb))
    a8[4] = 0
    nan = 255 if scale == E8M0 else float("nan")
    ca8[1, 2000], cb8[5, 0] = nan, nan
    bias = torch.zeros(n, device=dev)
    bias[7], bias[4000] = float("-inf"), float("inf")
    out, names = named(lambda: lce.fp8_matmul(a8.view(E4M3), ca8.view(scale), b, cb8.view(scale),
                                              bias))
    assert names == {"fp8_matmul_large"}
    expect = torch.zeros(m, n, dtype=torch.bool, device=dev)
    expect[2000], expect[:, 640:768] = True, True
    assert torch.equal(torch.isnan(out), expect)
    assert torch.equal(torch.isinf(out), (torch.isinf(bias)[None] & ~expect))
    ordinary = ~torch.isinf(bias) & ~expect[0]
    assert (out[4][ordinary] == 0).all()
    keep = torch.arange(m, device=dev) != 2000
    keep[4] = False
    assert torch.equal(out[keep][:, ordinary], ref[keep][:, ordinary])


def test_graph(dev):
    """Large tiles captured, replayed on other inputs with eager work between."""
    x = torch.randn(3850, 656, device=dev)
    w, cw = lce.fp8_quantize(torch.randn(4095, 656, device=dev), block_rows=128)

    def step():
        a, ca = lce.fp8_quantize(x)
        return lce.fp8_matmul(a, ca, w, cw)
    _, names = named(step)
    assert "fp8_matmul_large" in names
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on_side, step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(3):
        x.copy_(torch.randn(3850, 656, generator=torch.Generator().manual_seed(seed)))
        eager = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, eager)
