"""8-bit blocks in fp64, from their definition: values and scales of e4m3 in blocks of 128."""
import torch

E4M3 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
LEAST = 2.0 ** -126


def half_step_e4m3(v):
    """Half the distance between neighbouring e4m3 numbers at |v| (4 significant bits, steps of
    2^-9 at least)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def scale_values(c):
    """Scales as fp64 numbers."""
    if c.dtype == torch.float32:
        return c.double()
    bits = c.view(torch.uint8)
    v = torch.exp2(bits.double() - 127)
    return torch.where(bits == 255, torch.full_like(v, float("nan")), v)


def spread(c, block_rows, n, h):
    """Scales as one fp64 value per element: block-major for rows, row-major for squares."""
    c = scale_values(c)
    if block_rows == 1:
        return c.t().repeat_interleave(128, 1)[:, :h]
    return c.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :h]


def block_max(y, block_rows):
    """The largest magnitude of each block, laid out as its scale is."""
    n, h = y.shape
    rows = 1 if block_rows == 1 else 128
    p = torch.nn.functional.pad(y.abs(), (0, -h % 128, 0, -n % rows))
    m = p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128).amax((1, 3))
    return m.t() if block_rows == 1 else m


def check_scales(c, top, rel):
    """c against the definition from the blocks' largest magnitudes, which are known to a relative
    error of `rel`; the division by 448 rounds once (2^-24)."""
    exact = (top / 448).clamp(min=LEAST)
    got = scale_values(c)
    rel = rel + 2.0 ** -24
    if c.dtype == torch.float32:
        assert ((got / exact - 1).abs() <= rel * 1.01).all()
    else:
        lo, hi = (torch.exp2(torch.ceil(torch.log2((exact * (1 + s * rel)).clamp(min=LEAST))))
                  for s in (-1.01, 1.01))
        assert ((got == lo) | (got == hi)).all()
