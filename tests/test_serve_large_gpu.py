"""Tensors of more than 4 GiB through the root-mean-square norm, 8-bit product and beam search
entry points: offsets past 32 bits. What lies behind them is compared with a call on a copy of it
(rows are independent of one another, bit for bit) or with whole numbers."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device
from test_beam_gpu import check_step, follow

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def random_rows(n, h, dev, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return torch.empty(n, h, device=dev, dtype=torch.bfloat16).normal_(generator=gen)


def test_norm_and_quantiser(dev):
    n, h = 262151, 8200
    x = random_rows(n, h, dev, 1)
    assert x.numel() * 2 > 1 << 32
    w = random_rows(1, h, dev, 2)[0]
    tail = slice(n - 9, n)
    y, s, rstd = lce.rmsnorm_fwd(x, w, x)
    y0, s0, rstd0 = lce.rmsnorm_fwd(x[tail].clone(), w, x[tail].clone())
    assert torch.equal(y[tail], y0) and torch.equal(s[tail], s0) and torch.equal(rstd[tail], rstd0)
    del y
    dx, _ = lce.rmsnorm_bwd(x, s, rstd, w, grad_residual=s)
    dx0, _ = lce.rmsnorm_bwd(x[tail].clone(), s0, rstd0, w, grad_residual=s0)
    assert torch.equal(dx[tail], dx0)
    del dx, s
    q, c, s = lce.rmsnorm_fp8_fwd(x, w, x)
    q0, c0, _ = lce.rmsnorm_fp8_fwd(x[tail].clone(), w, x[tail].clone())
    assert torch.equal(q[tail].view(torch.uint8), q0.view(torch.uint8))
    assert torch.equal(c[:, tail].contiguous().view(torch.uint8), c0.view(torch.uint8))
    del q, s
    for rows in (1, 128):
        q, c = lce.fp8_quantize(x, block_rows=rows)
        lo = n - n % 128
        q0, c0 = lce.fp8_quantize(x[lo:].clone(), block_rows=rows)
        assert torch.equal(q[lo:].view(torch.uint8), q0.view(torch.uint8))
        got = c[:, lo:].contiguous() if rows == 1 else c[lo // 128:]
        assert torch.equal(got.view(torch.uint8), c0.view(torch.uint8))


@pytest.mark.parametrize("m", [5, 40, 200, 20003])
def test_product(dev, m):
    """Operands in rows 4 MiB apart, and an output of more than 4 GiB for the most rows."""
    n, k, ld = (1100, 400, 1 << 22) if m < 1000 else (128256, 16, 16)
    gen = torch.Generator(device=dev).manual_seed(m)

    def whole(rows):
        return torch.randint(-2, 3, (rows, k), generator=gen, device=dev).float()
    a, b = whole(m), whole(n)
    wide = torch.empty(n * ld, dtype=torch.uint8, device=dev).view(E4M3).view(n, ld)
    wide[:, :k] = b.to(E4M3)
    blocks = -(-k // 128)
    ca = torch.ones(blocks, m, device=dev)
    cb = torch.ones(-(-n // 128), blocks, device=dev)
    out = lce.fp8_matmul(a.to(E4M3), ca, wide[:, :k], cb, dtype=torch.float32 if m < 1000 else None)
    assert m < 1000 or out.numel() * 2 > 1 << 32
    # sums of at most 400 products of whole numbers up to 2: exact, in bf16 up to 256
    for lo in (0, max(0, m - 300)):
        assert torch.equal(out[lo:lo + 300].float(), a[lo:lo + 300] @ b.t())
    if m < 1000:  # the left operand's rows, and the output's
        far = torch.empty(m * ld, dtype=torch.uint8, device=dev).view(E4M3).view(m, ld)
        far[:, :k] = a.to(E4M3)
        to = torch.empty(m, 1 << 23, device=dev)
        lce.fp8_matmul(far[:, :k], ca, wide[:, :k], cb, out=to[:, :n])
        assert torch.equal(to[:, :n], out)


def test_beam_step(dev):
    b, k, v = 1030, 16, 131077
    z = random_rows(b * k, v, dev, 3).view(b, k, v)
    assert z.numel() * 2 > 1 << 32
    s = torch.randn(b, k, device=dev)
    got = lce.beam_step(z, s, num=9, eos=4)
    check_step(z[-1:], s[-1:], 9, eos=4, got=tuple(t[-1:] for t in got))


def test_beam_reorder(dev):
    """Runs, beams and entries that start past 4 GiB, out of place and in place."""
    gen = torch.Generator().manual_seed(4)
    p = torch.randint(-1, 4, (2, 4), generator=gen, dtype=torch.int32).to(dev)
    p[1, 3] = 2
    x = torch.empty(2, 4, 600_000_003, dtype=torch.uint8, device=dev)
    x[:, :, -5000:] = torch.randint(0, 255, (2, 4, 5000), device=dev, dtype=torch.uint8)
    x[:, :, :5000] = torch.randint(0, 255, (2, 4, 5000), device=dev, dtype=torch.uint8)
    heads = torch.empty(2, 4, 3, 2 ** 28 + 7, dtype=torch.int16, device=dev)[:, :, :, :999]
    heads.copy_(torch.randint(-9, 9, heads.shape, device=dev, dtype=torch.int16))
    ends = torch.cat((x[:, :, :5000], x[:, :, -5000:]), 2)
    want, want_heads = follow(ends, p), follow(heads, p)
    got, got_heads = lce.beam_reorder([x, heads], p)
    assert torch.equal(torch.cat((got[:, :, :5000], got[:, :, -5000:]), 2), want)
    assert torch.equal(got_heads, want_heads)
    del got
    lce.beam_reorder([x, heads], p, out=[x, heads])
    assert torch.equal(torch.cat((x[:, :, :5000], x[:, :, -5000:]), 2), want)
    assert torch.equal(heads, want_heads)
