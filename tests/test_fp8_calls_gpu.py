"""Products of 8-bit blocks whose scales lie far apart, and the ways that a product can be asked
for."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _fp8 import E4M3, E8M0
from _helpers import gpu_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def by_blocks(ad, ca, bd, cb, n):
    """sum_b ca cb (sum over block b), the block's sum and its scaling in fp64."""
    out = torch.zeros(ad.shape[0], n, dtype=torch.float64, device=ad.device)
    for b in range(0, ad.shape[1], 128):
        t = ad[:, b:b + 128] @ bd[:, b:b + 128].t()
        out += t * ca[b // 128][:, None] * cb[:, b // 128].repeat_interleave(128)[:n][None]
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n,k", [(7, 256, 256), (40, 256, 256), (80, 512, 1040), (300, 256, 256),
                                   (300, 256, 1040), (4096, 4096, 256)])
def test_scales_whose_product_leaves_fp32(dev, m, n, k, dtype):
    """Powers of two that multiply past fp32 on either side, around sums that bring the result back:
    zeros under 2^140, 2^-18 under 2^140, 2^24.6 under 2^-150. The results are sums of equal products
    but for one far smaller, so their error is the output's half step (and 2^-20 for the rest)."""
    a = torch.zeros(m, k, device=dev)
    byte = torch.full((-(-k // 128), m), 127, dtype=torch.uint8, device=dev)
    kind = torch.arange(m, device=dev) % 5
    a[kind == 1, 5] = 2.0 ** -9
    a[kind == 2, :128] = 448.0
    a[kind == 3, :128] = 1.0
    a[kind == 4, :128] = 448.0
    byte[0] = torch.tensor([227, 227, 37, 127, 0], dtype=torch.uint8, device=dev)[kind]
    b = torch.full((n, k), 448.0, device=dev)
    first = torch.arange(n, device=dev) // 128 % 2 == 0
    b[first, 5] = 2.0 ** -9
    cb = torch.full((n // 128, -(-k // 128)), 127, dtype=torch.uint8, device=dev)
    cb[0::2, 0], cb[1::2, 0] = 127 + 40, 127 - 60
    a8, b8, ca8, cb8 = a.to(E4M3), b.to(E4M3), byte.view(E8M0), cb.view(E8M0)
    out = lce.fp8_matmul(a8, ca8, b8, cb8, dtype=dtype).double()
    exact = by_blocks(a.double(), torch.exp2(byte.double() - 127), b.double(),
                      torch.exp2(cb.double() - 127), n)
    tiny = 2.0 ** -126
    rel = torch.finfo(dtype).eps / 2 + 2.0 ** -20
    ordinary = exact.abs() >= tiny
    assert ordinary[2, 128] and ordinary[1, 0] and not ordinary[0].any()
    assert ((out - exact).abs() <= rel * exact.abs())[ordinary].all()
    assert (out[~ordinary].abs() <= tiny).all() and (out[0] == 0).all()
    # and NaN scales among them
    byte[0, 2] = 255
    out = lce.fp8_matmul(a8, ca8, b8, cb8, dtype=dtype)
    assert torch.isnan(out[2]).all() and not torch.isnan(out[:2]).any()


def cancelling(m, n, k, dev):
    """Whole numbers under scales of 1: six ordinary columns of each eight beside two large ones that
    cancel, in the first 80 eights. No partial sum, in whatever order, reaches 2^24 (80 · 448^2 and
    64 k), so that sums in fp32 are exact."""
    gen = torch.Generator().manual_seed(m + n + k)
    a = torch.randint(-8, 9, (m, k), generator=gen).float()
    b = torch.randint(-8, 9, (n, k), generator=gen).float()
    a[:, 0:640:8], a[:, 1:640:8] = 448.0, -448.0
    b[:, 0:640:8] = b[:, 1:640:8] = 448.0
    ca = torch.full((-(-k // 128), m), 127, dtype=torch.uint8)
    cb = torch.full((-(-n // 128), -(-k // 128)), 127, dtype=torch.uint8)
    return (a.to(dev).to(E4M3), ca.to(dev).view(E8M0), b.to(dev).to(E4M3), cb.to(dev).view(E8M0))


@pytest.mark.parametrize("scale", [E8M0, torch.float32])
@pytest.mark.parametrize("m,n,k", [(9, 300, 272), (64, 129, 1040), (65, 130, 16), (65, 300, 1040),
                                   (300, 1003, 272), (1003, 2051, 640), (3850, 4095, 656)])
def test_precise(dev, m, n, k, scale):
    """bf16 results of fp32 sums, whatever the rows: those of cancelling() are exact and rounded
    once. Without it they are within what is documented: 2^-10 of the product of the largest
    magnitudes of each eight columns."""
    a, ca, b, cb = cancelling(m, n, k, dev)
    if scale == torch.float32:
        ca, cb = torch.ones(ca.shape, device=dev), torch.ones(cb.shape, device=dev)
    bias = torch.randint(-9, 10, (n,), device=dev).float()
    exact = a.double() @ b.double().t() + bias.double()
    out = lce.fp8_matmul(a, ca, b, cb, bias, precise=True)
    assert torch.equal(out, exact.float().bfloat16())
    fast = lce.fp8_matmul(a, ca, b, cb, bias)
    if m <= 64:
        assert torch.equal(fast, out)
    else:
        a8, b8 = (torch.nn.functional.pad(t.double().abs(), (0, -k % 8)).view(len(t), -1, 8).amax(-1)
                  for t in (a, b))
        tol = 2.0 ** -10 * (a8 @ b8.t()) + exact.abs() * 2.0 ** -8
        assert ((fast.double() - exact).abs() <= 1.01 * tol).all()
    for dtype in (torch.float16, torch.float32):  # nothing to choose
        plain, asked = (lce.fp8_matmul(a, ca, b, cb, bias, dtype=dtype, precise=p)
                        for p in (False, True))
        assert torch.equal(plain, asked) and torch.equal(plain, exact.to(dtype))


def test_precise_into_graph_and_head(dev):
    from linear_cross_entropy_masked_amd.serving import Fp8Head
    a, ca, b, cb = cancelling(300, 700, 1040, dev)
    out = torch.empty(300, 707, device=dev, dtype=torch.bfloat16)[:, 3:703]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lce.fp8_matmul(a, ca, b, cb, out=out, precise=True)
    ref = lce.fp8_matmul(a, ca, b, cb, dtype=torch.float32).bfloat16()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    torch.manual_seed(0)
    w, x = torch.randn(700, 256, device=dev).bfloat16(), torch.randn(100, 256, device=dev).bfloat16()
    z, _ = Fp8Head(w, precise=True)(x)
    fp32, _ = Fp8Head(w, logits_dtype=torch.float32)(x)
    assert z.dtype == torch.bfloat16 and torch.equal(z, fp32.bfloat16())


@pytest.mark.parametrize("scale", [None, torch.float32])
def test_head_in_a_cast_model(dev, scale):
    """A model around a head that is cast to the type of its hidden states answers as before."""
    from linear_cross_entropy_masked_amd.serving import Fp8Head
    torch.manual_seed(0)
    w, nw = torch.randn(700, 256, device=dev), torch.rand(256, device=dev) + 0.5
    model = torch.nn.ModuleDict({"head": Fp8Head(w, nw.bfloat16().float(),
                                                 torch.randn(700, device=dev), scale_dtype=scale)})
    x = torch.randn(20, 256, device=dev).bfloat16()
    before, _ = model["head"](x)
    after, _ = model.to(torch.bfloat16)["head"](x)
    assert torch.equal(before, after) and model["head"].norm_weight.dtype == torch.bfloat16
    assert torch.equal(model.cpu().to(dev)["head"](x)[0], before)


@pytest.mark.parametrize("m,n,k", [(13, 256, 128), (52, 200, 272), (130, 256, 128),
                                   (300, 300, 1040)])
def test_large_scales_over_sums_that_cancel(dev, m, n, k):
    """Products of 448^2 that cancel within a block, all 128 of them in pairs but two of 0 and 2^-18,
    under scales up to 2^145: fp32 holds the block's sum in any order (126 · 448^2 < 2^25), so the
    scale may not meet the products before they are added where it would carry them past fp32, and
    nothing is NaN. Exact is 2^-18 times the scale, but beside 448^2 fp32 has steps of 2^-6, so the
    sum of 128 products is off by up to 2 (128 + 8) 2^-24 of the sum of their magnitudes, 410; times
    the scale that is finite up to 2^118."""
    powers = torch.tensor([0, 60, 90, 100, 102, 103, 104, 110, 111, 118, 125, 140, 145], device=dev)
    e = powers[torch.arange(m, device=dev) % len(powers)]
    a = torch.zeros(m, k, device=dev)
    a[:, 0:126:2], a[:, 1:126:2] = 448.0, -448.0
    a[:, 127] = 2.0 ** -9
    b = torch.full((n, k), 448.0, device=dev)
    b[:, 127] = 2.0 ** -9
    ca = torch.full((-(-k // 128), m), 127, dtype=torch.uint8, device=dev)
    ca[0] = (e - 40 + 127).to(torch.uint8)
    cb = torch.full((-(-n // 128), -(-k // 128)), 127, dtype=torch.uint8, device=dev)
    cb[:, 0] = 127 + 40
    args = a.to(E4M3), ca.view(E8M0), b.to(E4M3), cb.view(E8M0)
    exact = torch.exp2(e.double() - 18)[:, None].expand(m, n)
    for dtype in (torch.float32, torch.bfloat16):
        out = lce.fp8_matmul(*args, dtype=dtype, precise=True)
        assert not torch.isnan(out).any(), e[torch.isnan(out).any(1)].unique()
        tol = 2 * 136 * 2.0 ** -24 * 126 * 448.0 ** 2 * torch.exp2(e.double())[:, None]
        near = (out.double() - exact).abs() <= tol + exact * torch.finfo(dtype).eps
        assert near[e <= 118].all()
