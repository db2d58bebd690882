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
