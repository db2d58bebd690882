"""Linear cross entropy in pieces of the vocabulary against its definition in fp64.

Tolerances, u = 2^-24 (fp32) and b = 2^-8 (half a bf16 step, relative). A logit is an fp32 sum of
h exact products in some order: off by at most dz = (h + 2)·u·Σ|hidden·w| + 2u|z|. The logsumexp
is off by at most the largest dz of its row, the rounding of its exponents (2u·|z − max|, at most
2^-17 here), of at most 90 added positive terms (90u < 2^-17) and of the result; together 2^-16
and 2u·|lse| bound it. A logit gradient d = p − [v = y] then carries p·(dz + dlse + 2^-16) and
its bf16 rounding b·|d|; the products add an fp32 sum of exact products and round once."""
import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu

U, B = 2.0 ** -24, 2.0 ** -8
IGN = -100


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def make(dev, n, h, v, masked=0.2, bias=True, sigma=1.5, seed=0):
    gen = torch.Generator().manual_seed(seed + 7 * n + 3 * h + v)
    hid = torch.randn(n, h, generator=gen).to(torch.bfloat16).to(dev)
    w = (torch.randn(v, h, generator=gen) * sigma / h ** 0.5).to(torch.bfloat16).to(dev)
    b = (torch.randn(v, generator=gen) * 0.5).to(dev) if bias else None
    lab = torch.randint(0, v, (n,), generator=gen)
    lab[torch.rand(n, generator=gen) < masked] = IGN
    return hid, w, b, lab.to(torch.int32).to(dev)


class Exact:
    def __init__(self, hid, w, b, lab, t=None, g=1.0, rows=None):
        n, h = hid.shape
        v = w.shape[0]
        keep = (lab != IGN) & (lab >= 0) & (lab < v)
        self.keep = keep
        hd = torch.where(keep[:, None], hid, torch.zeros_like(hid)).double()
        wd = w.double()
        z = hd @ wd.t()
        dz = (h + 2) * U * (hd.abs() @ wd.abs().t())
        if b is not None:
            z = z + b.double()
        dz = dz + 2 * U * torch.where(z.isinf(), 0.0, z.abs())
        y = lab.long().clamp(0, v - 1)[:, None]
        lse = torch.logsumexp(z, 1)
        live = torch.where(z.isinf(), torch.zeros_like(dz), dz)
        self.dlse = live.max(1).values + 2.0 ** -16 + 2 * U * lse.abs()
        zy = z.gather(1, y)[:, 0]
        zero = torch.zeros_like(lse)
        self.lse = torch.where(keep, lse, zero)
        self.rows = torch.where(keep, lse - zy, zero)
        self.drows = torch.where(keep, self.dlse + dz.gather(1, y)[:, 0] + 2 * U * self.rows.abs(),
                                 zero)
        t = int(keep.sum()) if t is None else t
        self.loss = float(self.rows.sum()) / t if t else 0.0
        self.dloss = (float(self.drows.sum()) / t if t else 0.0) + 2 * U * abs(self.loss)
        p = (z - lse[:, None]).exp()
        one = torch.zeros_like(p).scatter_(1, y, 1.0)
        c = (g / t if t else 0.0) * torch.ones_like(lse) if rows is None else rows.double()
        c = torch.where(keep, c, zero)[:, None]
        d = p - one
        ed = (p * (live + self.dlse[:, None] + 2.0 ** -16) + 2 * U) * c.abs()
        d = d * c
        eb = ed + (B + 3 * U) * d.abs()
        self.gh, self.gw, self.gb = d @ wd, d.t() @ hd, d.sum(0)
        self.dgh = eb @ wd.abs() + (v + 8) * U * (d.abs() @ wd.abs())
        self.dgw = eb.t() @ hd.abs() + (n + 8) * U * (d.abs().t() @ hd.abs())
        self.dgb = ed.sum(0) + (n + 8) * U * d.abs().sum(0)


def half(dtype, x):
    f = torch.finfo(dtype)
    return torch.clamp(x.abs() * (f.eps / 2), min=f.smallest_normal * f.eps / 2)


def near(got, exact, tol, what):
    err = (got.double() - exact).abs()
    tol = tol + half(got.dtype, exact.abs() + tol)
    assert (err <= tol).all(), f"{what}: {float((err - tol).max()):.3g} past the bound"


def check_fwd(e, loss, lse, rows):
    assert abs(float(loss) - e.loss) <= e.dloss
    near(lse, e.lse, torch.where(e.keep, e.dlse, torch.zeros_like(e.dlse)), "lse")
    near(rows, e.rows, e.drows, "rows")
    assert not lse[~e.keep].any() and not rows[~e.keep].any()


def check_bwd(e, gh, gw, gb):
    if gh is not None:
        near(gh, e.gh, e.dgh, "grad_hidden")
        assert not gh[~e.keep].any()
    if gw is not None:
        near(gw, e.gw, e.dgw, "grad_weight")
    if gb is not None:
        near(gb, e.gb, e.dgb, "grad_bias")


SHAPES = [(1, 8, 1), (1, 64, 3000), (3, 40, 255), (16, 768, 1000), (17, 72, 257), (33, 200, 64),
          (32, 136, 301), (64, 4096, 500), (65, 64, 1001), (128, 72, 900),
          (130, 136, 4), (255, 1032, 700), (256, 256, 256),
          (300, 768, 5003), (1000, 64, 129), (600, 2048, 2300)]


@pytest.mark.parametrize("n,h,v", SHAPES)
@pytest.mark.parametrize("bias", [True, False])
def test_forward_and_backward(dev, n, h, v, bias):
    hid, w, b, lab = make(dev, n, h, v, bias=bias)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    e = Exact(hid, w, b, lab)
    check_fwd(e, loss, lse, rows)
    gh, gw, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b)
    assert gw.dtype == torch.bfloat16 and gh.dtype == torch.bfloat16
    assert (gb is None) == (b is None)
    check_bwd(e, gh, gw, gb)


@pytest.mark.parametrize("n,h,sizes,piece", [(5, 64, [100, 1, 300], None), (70, 72, [513, 7, 64], 50),
                                             (300, 256, [1000], 257), (500, 128, [3000, 500], 1024),
                                             (64, 64, [64, 64, 65], 1)])
def test_weight_in_pieces(dev, n, h, sizes, piece):
    """A weight in several tensors, each taken in several pieces, against the whole."""
    v = sum(sizes)
    hid, w, b, lab = make(dev, n, h, v)
    ws, bs = list(w.split(sizes)), list(b.split(sizes))
    loss, lse, rows = lce.flce_pieces_fwd(hid, ws, lab, bs, return_rows=True)
    e = Exact(hid, w, b, lab)
    check_fwd(e, loss, lse, rows)
    gh, gw, gb = lce.flce_pieces_bwd(hid, ws, lab, lse, bs, piece_size=piece)
    assert [tuple(t.shape) for t in gw] == [(s, h) for s in sizes]
    check_bwd(e, gh, torch.cat(gw), torch.cat(gb))
    one = lce.flce_pieces_bwd(hid, w, lab, lse, b, piece_size=max(1, v // 3))
    check_bwd(e, *one)


def test_pieces_in_any_order_and_states_that_combine(dev):
    """The pieces of a state may come in any order, and two states over disjoint pieces combine
    as the header says."""
    n, h, sizes = 200, 64, [300, 111, 700]
    hid, w, b, lab = make(dev, n, h, sum(sizes))
    e = Exact(hid, w, b, lab)
    ws, bs = w.split(sizes), b.split(sizes)
    at = [0, 300, 411]
    v = sum(sizes)
    state = torch.empty(3, n, device=dev)
    for k, i in enumerate((2, 0, 1)):
        lce.flce_piece_fwd(hid, ws[i], lab, state, bs[i], v_start=at[i], vocab=v, first=k == 0)
    check_fwd(e, *lce.flce_piece_loss(state, lab, vocab=v, return_rows=True))
    one, two = torch.empty(3, n, device=dev), torch.empty(3, n, device=dev)
    lce.flce_piece_fwd(hid, ws[0], lab, one, bs[0], v_start=0, vocab=v, first=True)
    lce.flce_piece_fwd(hid, ws[1], lab, two, bs[1], v_start=300, vocab=v, first=True)
    lce.flce_piece_fwd(hid, ws[2], lab, two, bs[2], v_start=411, vocab=v, first=False)
    m = torch.maximum(one[0], two[0])
    s = one[1] * (one[0] - m).exp() + two[1] * (two[0] - m).exp()
    both = torch.stack([m, s, one[2] + two[2]])
    assert torch.isneginf(both[0][~e.keep]).all()
    check_fwd(e, *lce.flce_piece_loss(both, lab, vocab=v, return_rows=True))
    # partial hidden gradients of the two shards add to the whole
    lse = e.lse.float()
    parts = []
    for i in range(3):
        acc = torch.full((n, h), 9.0, device=dev)
        gw = torch.empty(sizes[i], h, device=dev)
        lce.flce_piece_bwd(hid, ws[i], lab, lse, bs[i], v_start=at[i], vocab=v, first=True,
                           last=False, hidden_acc=acc, grad_weight=gw)
        near(gw, e.gw[at[i]:at[i] + sizes[i]], e.dgw[at[i]:at[i] + sizes[i]], "grad_weight")
        parts.append(acc)
    near(parts[0] + parts[1] + parts[2], e.gh, e.dgh + 4 * U * e.gh.abs(), "hidden_acc")


@pytest.mark.parametrize("n", [7, 64, 200, 700])
def test_rows_without_a_label(dev, n):
    """Masked rows may hold anything, and all rows may be masked."""
    h, v = 136, 600
    hid, w, b, lab = make(dev, n, h, v, masked=0.5)
    lab[0], lab[-1] = IGN, IGN
    lab[n // 2] = 17
    hid[lab == IGN] = float("nan")
    hid[0] = float("inf")
    e = Exact(hid, w, b, lab)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b))
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, piece_size=100))
    none = torch.full_like(lab, IGN)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, none, b, return_rows=True)
    assert loss.item() == 0 and not lse.any() and not rows.any()
    for out in lce.flce_pieces_bwd(hid, w, none, lse, b, piece_size=256):
        assert not out.any()


def test_bad_labels_and_other_ignore_index(dev):
    n, h, v = 90, 64, 300
    hid, w, b, lab = make(dev, n, h, v, masked=0.0)
    status = torch.full((), -1, dtype=torch.int32, device=dev)
    lce.flce_pieces_fwd(hid, w, lab, b, status=status)
    assert status.item() == 0
    lab[3], lab[50], lab[60] = v, -1, 2 ** 31 - 1
    e = Exact(hid, w, b, lab)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True, status=status)
    assert status.item() == lce.LCE_STATUS_BAD_LABEL
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b))
    big = torch.cat([lab] * 60)
    st2 = torch.full((), -1, dtype=torch.int32, device=dev)
    got = lce.flce_pieces_fwd(torch.cat([hid] * 60), w, big, b, return_rows=True, status=st2)
    assert st2.item() == lce.LCE_STATUS_BAD_LABEL
    assert abs(float(got[0]) - e.loss) <= e.dloss
    near(got[2], e.rows.repeat(60), e.drows.repeat(60), "rows")
    # ignore_index may be a class
    lab = torch.randint(0, v, (n,), device=dev, dtype=torch.int32)
    lab[:40] = 5
    other = torch.where(lab == 5, torch.full_like(lab, IGN), lab)
    e = Exact(hid, w, b, other)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True, ignore_index=5)
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, ignore_index=5))


@pytest.mark.parametrize("n", [20, 300])
def test_classes_masked_by_the_bias(dev, n):
    """Whole tiles and a whole piece whose bias is minus infinity."""
    h, v = 64, 1500
    hid, w, b, lab = make(dev, n, h, v)
    b[:700] = float("-inf")
    b[900] = float("-inf")
    lab[lab >= 0] = lab[lab >= 0] % 500 + 950
    e = Exact(hid, w, b, lab)
    ws, bs = w.split([600, 900]), b.split([600, 900])
    for wt, bt in ((w, b), (ws, bs)):
        loss, lse, rows = lce.flce_pieces_fwd(hid, wt, lab, bt, return_rows=True)
        check_fwd(e, loss, lse, rows)
        gh, gw, gb = lce.flce_pieces_bwd(hid, wt, lab, lse, bt)
        cat = (lambda t: torch.cat(list(t))) if wt is ws else (lambda t: t)
        check_bwd(e, gh, cat(gw), cat(gb))
        assert not cat(gw)[:700].any() and not cat(gb)[:700].any()


@pytest.mark.parametrize("n", [20, 100, 300])
def test_every_class_masked(dev, n):
    """A bias of minus infinity throughout: the logsumexp is minus infinity, whichever kernel ran;
    and one that leaves a single class gives that class's logit."""
    hid, w, b, lab = make(dev, n, 64, 900, masked=0.0)
    b[:] = float("-inf")
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    assert torch.isneginf(lse).all()
    b[700] = 0.25
    lab[:] = 700
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    assert float(loss) == 0 and not rows.any()
    near(lse, hid.double() @ w[700].double() + 0.25,
         67 * U * (hid.double().abs() @ w[700].double().abs()) + 2 * U, "lse")
    gh, gw, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b)
    # the two forward kernels and the backward's product add a logit in different orders
    off = float((67 * U * (hid.double().abs() @ w[700].double().abs())).max()) * 2 + 4 * U
    assert (gw[:700] == 0).all() and (gw[701:] == 0).all()
    assert float(gb.abs().max()) <= 2 * off


@pytest.mark.parametrize("n", [12, 400])
def test_row_gradients(dev, n):
    """Each row's term with its own upstream gradient, among them 0."""
    h, v = 192, 900
    hid, w, b, lab = make(dev, n, h, v)
    g = torch.randn(n, device=dev)
    g[1] = 0.0
    e = Exact(hid, w, b, lab, rows=g)
    lse = e.lse.float()
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g))
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g, piece_size=256))


def test_normalisers_upstream_gradient_and_accumulate(dev):
    n, h, v = 150, 128, 777
    hid, w, b, lab = make(dev, n, h, v)
    gout = torch.tensor(-2.5, device=dev)
    for t in (1, 37, 0):
        e = Exact(hid, w, b, lab, t=t, g=-2.5)
        loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, num_label_tokens=t, return_rows=True)
        check_fwd(e, loss, lse, rows)
        check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, num_label_tokens=t,
                                          grad_output=gout))
    e = Exact(hid, w, b, lab)
    for dtype in (torch.float32, torch.bfloat16):
        old = torch.randn(v, h, device=dev).to(dtype)
        oldb = torch.randn(v, device=dev)
        gw, gb = old.clone(), oldb.clone()
        gh, got, gotb = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=gw, grad_bias=gb,
                                            accumulate=True, piece_size=300)
        assert got is gw and gotb is gb
        near(gw, e.gw + old.double(), e.dgw + 2 * U * (e.gw.abs() + old.double().abs()), "acc")
        near(gb, e.gb + oldb.double(), e.dgb + 2 * U * (e.gb.abs() + oldb.double().abs()), "acc")
    gw = torch.full((v, h), 3.0, device=dev)  # fp32, overwritten
    gh, got, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_hidden=False, grad_weight=gw,
                                      grad_bias=False)
    assert gh is None and gb is None
    check_bwd(e, None, gw, None)
    gh, gw, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=False, piece_size=300)
    assert gw is None
    check_bwd(e, gh, None, gb)


def test_peaked_rows(dev):
    """Rows whose label the model all but knows, and rows whose largest logit is far above."""
    n, h, v = 300, 256, 1000
    hid, w, b, lab = make(dev, n, h, v, sigma=8.0)
    y = lab.long().clamp(min=0)
    b2 = b.clone()
    b2[y[::7]] += 25.0
    e = Exact(hid, w, b2, lab)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b2, return_rows=True)
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b2))


@pytest.mark.parametrize("n,h,v", [(260, 64, 32777), (1003, 72, 32769), (2048, 64, 32784),
                                   (300, 200, 32785)])
@pytest.mark.parametrize("bias", [True, False])
def test_classes_past_a_multiple_of_the_tile(dev, n, h, v, bias):
    """A last tile of few classes, with labels and the largest bias among them."""
    hid, w, b, lab = make(dev, n, h, v, bias=bias)
    lab[::9] = torch.arange(len(lab[::9]), device=dev, dtype=torch.int32) % (v % 256) + v // 256 * 256
    if bias:
        b[v - 1] = 3.0
    e = Exact(hid, w, b, lab)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b))
    g = torch.randn(n, device=dev)
    check_bwd(Exact(hid, w, b, lab, rows=g),
              *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_rows=g))


def test_long_batches(dev):
    """Past 8192 rows the labelled rows are numbered in a launch of their own."""
    for masked in (0.3, 0.97):
        hid, w, b, lab = make(dev, 9001, 64, 520, masked=masked)
        hid[lab == IGN] = float("nan")
        e = Exact(hid, w, b, lab)
        loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
        check_fwd(e, loss, lse, rows)
        check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b))
        check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, piece_size=256))


def test_few_labelled_rows_take_more_splits(dev):
    """Many row tiles in the launch, few rows that count: the hidden gradient's contraction is cut
    into more ranges, in the memory that was asked for."""
    n, h, v = 1500, 64, 20000
    hid, w, b, lab = make(dev, n, h, v, masked=0.9)
    e = Exact(hid, w, b, lab)
    loss, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    need = lce.flce_piece_bwd_workspace_size(n, h, v)
    ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    gh = torch.empty(n, h, dtype=torch.bfloat16, device=dev)
    lce.flce_piece_bwd(hid, w, lab, lse, b, v_start=0, vocab=v, first=True, last=True,
                       grad_hidden=gh, workspace=ws[:need])
    assert (ws[need:] == 0xFF).all()
    near(gh, e.gh, e.dgh, "grad_hidden")
    assert not gh[~e.keep].any()


def test_a_piece_past_4_gib(dev):
    """Logit gradients of one piece past 2^32 bytes: the same weight gradient, bit for bit, as in
    pieces of a tenth, and the hidden gradient within its rounding."""
    n, h, v = 17000, 64, 128256
    hid, w, b, lab = make(dev, n, h, v, bias=False)
    assert lce.flce_piece_bwd_workspace_size(n, h, v) > 2 ** 32
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab)
    gh, gw, _ = lce.flce_pieces_bwd(hid, w, lab, lse, piece_size=v)
    gh2, gw2, _ = lce.flce_pieces_bwd(hid, w, lab, lse, piece_size=12800)
    assert torch.equal(gw, gw2)
    # two bf16 roundings, and fp32 sums of v products of which the label's is the largest
    size = (w.float().abs().max() * 2 / int((lab != IGN).sum())).item()
    assert ((gh.float() - gh2.float()).abs() <= 2 * B * gh.float().abs() + v * U * size).all()


def test_agrees_with_the_loss_by_chunks_of_rows(dev):
    n, h, v = 700, 256, 3001
    hid, w, b, lab = make(dev, n, h, v)
    loss, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    loss2, lse2 = lce.flce_fwd(hid, w, lab, b, chunk_size=256)
    e = Exact(hid, w, b, lab)
    assert abs(float(loss) - float(loss2)) <= 2 * e.dloss
    assert ((lse - lse2).abs().double() <= 2 * e.dlse).all()


def test_empty_batch(dev):
    w = torch.randn(50, 64, device=dev).to(torch.bfloat16)
    b = torch.randn(50, device=dev)
    hid = torch.empty(0, 64, dtype=torch.bfloat16, device=dev)
    lab = torch.empty(0, dtype=torch.int32, device=dev)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    assert loss.item() == 0 and lse.shape == (0,) and rows.shape == (0,)
    gh, gw, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b)
    assert gh.shape == (0, 64) and not gw.any() and not gb.any()
    gw = torch.ones(50, 64, device=dev)
    lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=gw, grad_bias=False, accumulate=True)
    assert (gw == 1).all()


def test_results_repeat_bit_for_bit_and_workspaces_are_respected(dev):
    """Twice the same bits, from workspaces of exactly the size asked for, full of NaN, with
    guard bytes behind them that stay."""
    n, h, v = 330, 200, 1300
    hid, w, b, lab = make(dev, n, h, v)

    def guarded(nbytes):
        t = torch.full((nbytes + 4096,), 0xFF, dtype=torch.uint8, device=dev)
        return t, t[:nbytes]

    outs = []
    for _ in range(2):
        f, fw = guarded(lce.flce_piece_fwd_workspace_size(n, h, v))
        l, lw = guarded(lce.flce_piece_loss_workspace_size(n))
        k, kw = guarded(lce.flce_piece_bwd_workspace_size(n, h, v))
        state = torch.full((3, n), float("nan"), device=dev)
        lce.flce_piece_fwd(hid, w, lab, state, b, v_start=0, vocab=v, first=True, workspace=fw)
        loss, lse, rows = lce.flce_piece_loss(state, lab, vocab=v, return_rows=True, workspace=lw)
        gh = torch.full((n, h), float("nan"), dtype=torch.bfloat16, device=dev)
        gw = torch.full((v, h), float("nan"), device=dev)
        gb = torch.full((v,), float("nan"), device=dev)
        lce.flce_piece_bwd(hid, w, lab, lse, b, v_start=0, vocab=v, first=True, last=True,
                           grad_hidden=gh, grad_weight=gw, grad_bias=gb, workspace=kw)
        for whole, ws in ((f, fw), (l, lw), (k, kw)):
            assert (whole[ws.numel():] == 0xFF).all()
        outs.append((loss, lse, rows, gh, gw, gb))
    check_fwd(Exact(hid, w, b, lab), *outs[0][:3])
    check_bwd(Exact(hid, w, b, lab), *outs[0][3:])
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_gradients_against_differences(dev):
    """Central differences of the kernels' own loss along one direction of the hidden states and
    one of the bias. The step is a power of two that bf16 inputs hold exactly."""
    n, h, v = 40, 64, 300
    hid, w, b, lab = make(dev, n, h, v)
    hid = (hid.float() * 8).round().div(8).to(torch.bfloat16)  # multiples of 1/8 up to 4
    hid = hid.clamp(-3.75, 3.75)
    d = torch.randint(-1, 2, (n, h), device=dev).to(torch.bfloat16)
    t = 2.0 ** -5  # 1/8 multiples below 4 plus 1/32: 7 bits

    def f(x, bb):
        return float(lce.flce_pieces_fwd(x, w, lab, bb, num_label_tokens=1)[0])

    e = Exact(hid, w, b, lab, t=1)
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    gh, _, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b, num_label_tokens=1)
    up, down = hid + (t * d.float()).to(torch.bfloat16), hid - (t * d.float()).to(torch.bfloat16)
    assert torch.equal((up.float() - down.float()), 2 * t * d.float())
    # third differences of a row's lse along a direction are at most 4 · (half the range of its
    # logit changes)^3; the fp32 noise of f is its bound over the step
    move = (d.double() @ w.double().t()).abs().max(1).values
    for step, want, tol in (((f(up, b) - f(down, b)) / (2 * t), (gh.double() * d.double()).sum(),
                             float((e.dgh + B * e.gh.abs()).sum()) + float((move ** 3).sum()) * t * t),
                            ((f(hid, b + t) - f(hid, b - t)) / (2 * t), gb.double().sum(),
                             float(e.dgb.sum()))):
        assert abs(step - float(want)) <= tol + 2 * e.dloss / t
    db = torch.randn(v, device=dev)
    step = (f(hid, b + t * db) - f(hid, b - t * db)) / (2 * t)
    third = float(db.abs().max()) ** 3 * n * t * t
    assert abs(step - float((gb.double() * db).sum())) <= 2 * e.dloss / t + third + float((e.dgb * db.abs()).sum())


@pytest.mark.parametrize("n", [20, 40, 300])
def test_a_weight_past_4_gib(dev, n):
    """Classes whose weight rows start past 2^32 bytes, through each of the logits kernels: the
    terms against fp64, the gradients of one piece against those of four."""
    h, v = 4096, 600011
    gen = torch.Generator().manual_seed(n)
    hid = torch.randn(n, h, generator=gen).to(torch.bfloat16).to(dev)
    w = torch.randn(v, h, device=dev, dtype=torch.bfloat16).mul_(2.0 ** -6)
    lab = (v - 1 - torch.randint(0, 50000, (n,), generator=gen)).to(torch.int32).to(dev)
    lab[3] = IGN
    _, lse, rows = lce.flce_pieces_fwd(hid, w, lab, return_rows=True)
    hd = hid.double()
    z, dz = [], []
    for lo in range(0, v, 50000):
        wd = w[lo:lo + 50000].double()
        z.append(hd @ wd.t())
        dz.append((h + 2) * U * (hd.abs() @ wd.abs().t()) + 2 * U * z[-1].abs())
    z, dz = torch.cat(z, 1), torch.cat(dz, 1)
    keep = lab != IGN
    exact = torch.where(keep, torch.logsumexp(z, 1), torch.zeros_like(z[:, 0]))
    dlse = dz.max(1).values + 2.0 ** -16 + 2 * U * exact.abs()
    near(lse, exact, dlse, "lse")
    y = lab.long().clamp(min=0)[:, None]
    terms = torch.where(keep, exact - z.gather(1, y)[:, 0], torch.zeros_like(exact))
    near(rows, terms, dlse + dz.gather(1, y)[:, 0] + 2 * U * terms.abs(), "rows")
    del z, dz
    gh, gw, _ = lce.flce_pieces_bwd(hid, w, lab, lse, piece_size=v)
    gh2, gw2, _ = lce.flce_pieces_bwd(hid, w, lab, lse, piece_size=150003)
    assert torch.equal(gw, gw2)
    # two bf16 roundings, and fp32 sums of v products of which the label's is the largest
    size = (w.float().abs().max() * 2 / int(keep.sum())).item()
    assert ((gh.float() - gh2.float()).abs() <= 2 * B * gh.float().abs() + v * U * size).all()
    assert gw[lab[keep].long()].any(1).all()


# on either side of the sizes at which the products change their tiles: 128 x 128 ones up to 256
# of them, else 128 rows up to 128 and 256 past that; the two gradient products apart or together
EDGES = [(129, 64, 16384), (129, 64, 16385), (40, 72, 32768), (40, 72, 32769), (128, 136, 33001),
         (8192, 64, 512), (8193, 64, 512), (300, 1000, 4096), (300, 1032, 4097), (700, 1024, 5003)]


@pytest.mark.parametrize("n,h,v", EDGES)
@pytest.mark.parametrize("masked", [0.1, 0.9])
def test_tile_choices(dev, n, h, v, masked):
    hid, w, b, lab = make(dev, n, h, v, masked=masked)
    loss, lse, rows = lce.flce_pieces_fwd(hid, w, lab, b, return_rows=True)
    e = Exact(hid, w, b, lab)
    check_fwd(e, loss, lse, rows)
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b))
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_hidden=False))
    check_bwd(e, *lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=False))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,h,v", [(300, 1032, 4097), (100, 256, 2000)])
def test_both_gradient_products_accumulate(dev, n, h, v, dtype):
    """Weight gradients in fp32 and added to what is there, with the hidden gradient or without."""
    hid, w, b, lab = make(dev, n, h, v)
    _, lse, _ = lce.flce_pieces_fwd(hid, w, lab, b)
    e = Exact(hid, w, b, lab)
    fresh = torch.empty(v, h, dtype=dtype, device=dev)
    gh, _, gb = lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_weight=fresh)
    check_bwd(e, gh, fresh, gb)
    for hidden in (True, False):
        old = torch.randn(v, h, device=dev).to(dtype)
        buf, bias = old.clone(), torch.zeros(v, device=dev)
        lce.flce_pieces_bwd(hid, w, lab, lse, b, grad_hidden=hidden, grad_weight=buf,
                            grad_bias=bias, accumulate=True)
        # one fp32 addition more, and the sum's rounding to the buffer's type
        near(buf, e.gw + old.double(), e.dgw + U * (e.gw.abs() + old.double().abs()), "grad_weight")
        near(bias, e.gb, e.dgb, "grad_bias")
    none = torch.full_like(lab, IGN)
    gh, gw, gb = lce.flce_pieces_bwd(hid, w, none, torch.zeros_like(lse), b)
    assert not gh.any() and not gw.any() and not gb.any()
