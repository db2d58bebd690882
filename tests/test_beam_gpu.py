"""Beam search's selection and the reordering of states against plain definitions.

A score is score_j + (z − lse_j). The library's lse: exponentials to a few u = 2^-24 of a rounded
argument (2u per unit of distance from the maximum, which weighted by the probabilities is at most
the entropy, below 13 for 2^18 classes) and sums of at most 60 roundings: 100 u in all, so a
returned score is within 100 u and half an fp32 step of the exact one. Which candidates are taken
is checked without a tolerance where it can be (within a beam: the largest logits, ties to the
lower token) and to twice that bound between beams."""
import math

import pytest
import torch

import linear_cross_entropy_masked_amd as lce

from _helpers import gpu_device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def check_step(logits, scores, num, finished=None, eos=None, got=None, ignore_index=-100):
    if got is None:
        got = lce.beam_step(logits, scores, num=num, finished=finished, eos=eos,
                            ignore_index=ignore_index)
    best, parents, tokens, done = (None if t is None else t.cpu() for t in got)
    b, k, v = logits.shape
    z = logits.cpu().double() + 0.0
    s = scores.cpu().double()
    fin = torch.zeros(b, k, dtype=torch.bool) if finished is None else finished.cpu()
    assert best.shape == parents.shape == tokens.shape == (b, num)
    for i in range(b):
        cand = []  # exact scores of each beam's candidates, best first, with their tokens
        for j in range(k):
            row, acc = z[i, j], s[i, j].item()
            bad = bool(torch.isnan(row).any() or (row == INF).any())
            if math.isnan(acc) or acc == INF or acc == -INF:
                cand.append(([], []))
            elif fin[i, j]:
                cand.append(([acc], [eos]))
            elif bad or not (row > -INF).any():
                cand.append(([], []))
            else:
                order = torch.sort(row, descending=True, stable=True).indices[:num]
                order = order[row[order] > -INF]
                # z − lse = (z − max) − log Σ exp(z − max): max + log Σ would lose the log beside a
                # maximum above 2^53
                far = row - row.max()
                logp = far[order] - far.exp().sum().log()
                cand.append(((acc + logp).tolist(), order.tolist()))
        flat = sorted((x for c in cand for x in c[0]), reverse=True)
        n = min(num, len(flat))
        taken = [0] * k
        for r in range(num):
            if r >= n:
                assert best[i, r] == -INF and parents[i, r] == -1
                assert tokens[i, r] == ignore_index and (done is None or not done[i, r])
                continue
            j = int(parents[i, r])
            at = taken[j]
            taken[j] += 1
            assert tokens[i, r] == cand[j][1][at], (i, r, j)  # the beam's next one, no other
            exact = cand[j][0][at]
            tol = 100 * U + abs(exact) * U + 1e-300
            assert abs(best[i, r].item() - exact) <= tol, (i, r)
            assert abs(exact - flat[r]) <= 2 * 100 * U + 1e-12 * abs(exact), (i, r)
            if r:
                assert best[i, r] <= best[i, r - 1]
            if done is not None:
                assert bool(done[i, r]) == bool(fin[i, j] or tokens[i, r] == eos)
    return got


def data(b, k, v, dtype, dev, seed=0, std=2.5):
    gen = torch.Generator().manual_seed(seed + b + 3 * k + 7 * v)
    z = (torch.randn(b, k, v, generator=gen) * std).to(dtype).to(dev)
    s = (torch.randn(b, k, generator=gen) - 20).to(dev)
    return z, s


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("b,k,v,num", [
    (1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 64), (1, 4, 2047, 4), (3, 5, 2049, 10), (2, 4, 4096, 8),
    (1, 4, 32777, 4), (5, 8, 9999, 16), (2, 16, 5000, 32), (1, 64, 700, 64), (2, 2, 50257, 64),
    (40, 8, 128256, 16), (200, 5, 8200, 10), (7, 12, 100003, 24), (1, 1, 262144, 64)])
def test_step(dev, b, k, v, num, dtype):
    """One to many slices, every slice length, one to 64 beams and candidates."""
    z, s = data(b, k, v, dtype, dev)
    check_step(z, s, num)


@pytest.mark.parametrize("v,num", [(40, 8), (5000, 16), (20000, 64)])
def test_step_finished(dev, v, num):
    z, s = data(6, 8, v, torch.bfloat16, dev)
    gen = torch.Generator().manual_seed(1)
    fin = torch.rand(6, 8, generator=gen) < 0.4
    fin[0], fin[1] = True, False
    s[0, 3] = -INF  # finished, but no beam at all
    z[2, :, 3] += 12  # eos is likely
    check_step(z, s, num, fin.to(dev), 3)
    check_step(z, s, num, None, 3)


def test_step_ties(dev):
    """Rows of few different values, or one: more ties than the ranked lists hold."""
    for v, num in ((100, 16), (3000, 5), (9000, 64), (70000, 32)):
        for values in (1, 2, 5):
            gen = torch.Generator().manual_seed(v + values)
            z = torch.randint(0, values, (2, 3, v), generator=gen).to(torch.bfloat16).to(dev)
            z[0, 1] = z[0, 0]  # two equal beams: the same score, the lower beam first
            s = torch.full((2, 3), -1.5, device=dev)
            s[1, 2] = 0.0
            check_step(z, s, num)
    z = torch.zeros(1, 2, 500, device=dev)
    z[0, 0, 1::2] = -0.0  # the same number
    got = check_step(z, torch.zeros(1, 2, device=dev), 6)
    assert got[1].tolist() == [[0] * 6] and got[2].tolist() == [[0, 1, 2, 3, 4, 5]]


def test_step_in_unkind_orders(dev):
    """Rising, falling and clustered rows: the best logits all in a few threads' registers."""
    for v in (2048, 8192, 40000):
        up = torch.arange(v, dtype=torch.float32, device=dev) * 1e-3
        z = torch.stack([up, up.flip(0), torch.where(torch.arange(v, device=dev) % 2048 < 64,
                                                     up + 30, up)])[None]
        for num in (3, 32, 64):
            check_step(z, torch.zeros(1, 3, device=dev), num)
        many = z.expand(90, 3, v).contiguous()  # longer slices
        check_step(many[:, :, :], torch.zeros(90, 3, device=dev), 32)


def test_step_masks(dev):
    """Banned classes, rows with one class or none left, the lowest numbers of a type, beams
    without a score."""
    z, s = data(8, 4, 3000, torch.float32, dev)
    z[0, :, 5:] = -INF
    z[1, 0] = -INF
    z[2] = -INF
    z[3, 1, :] = -INF
    z[3, 1, 2999] = 4.0
    z[4, 2, 7:] = torch.finfo(torch.float32).min
    s[5] = torch.tensor([0.0, -INF, -INF, -INF], device=dev)  # the first step of a search
    s[6, 1] = -1e9
    z[7, :, ::2] = -1e30
    check_step(z, s, 8)
    check_step(z[..., :3].contiguous(), s, 16)
    low = torch.full((1, 2, 50), torch.finfo(torch.bfloat16).min, device=dev).bfloat16()
    check_step(low, torch.zeros(1, 2, device=dev), 5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("base", [2.0 ** 25, -3e9, 3e9, 1e12, -1e30, 1e30, -8e37, 2e38])
def test_step_large_logits(dev, dtype, base):
    """Rows far from zero: a score is what lies between the logits, however large they are."""
    v, num = 5000, 6
    z = torch.full((1, 2, v), base, device=dev).to(dtype)
    step = 2.0 ** (math.frexp(base)[1] - 1) * torch.finfo(dtype).eps
    z[0, 0, 7::9] -= 3 * step  # one to all of the next lower values, as the type has them
    z[0, 1, 11] += 5 * step
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    s = torch.tensor([[-1.5, -2.0]], device=dev)
    best, parents, tokens, _ = lce.beam_step(z, s, num=num, status=status)
    assert status.item() == 0
    d = z.cpu().double()
    d = d - d.amax(-1, keepdim=True)
    exact = s.cpu().double()[..., None] + (d - torch.log(torch.exp(d).sum(-1, keepdim=True)))
    want = exact.flatten().sort(descending=True).values[:num]
    got = exact[0, parents[0].long().cpu(), tokens[0].long().cpu()]
    for r in range(num):
        tol = 100 * U + abs(want[r].item()) * U
        assert abs(got[r] - want[r]) <= 2 * tol and abs(best[0, r].item() - got[r]) <= tol, r


def test_step_finished_without_a_score(dev):
    """A finished beam whose score is no number has no candidate and is reported."""
    z, s = data(2, 3, 100, torch.bfloat16, dev)
    fin = torch.tensor([[False, True, False], [True, False, False]], device=dev)
    for bad in (float("nan"), INF):
        t = s.clone()
        t[0, 1] = bad
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        got = lce.beam_step(z, t, num=5, finished=fin, eos=3, status=status)
        check_step(z, t, 5, fin, 3, got=got)
        assert status.item() == lce.LCE_STATUS_BAD_LOGITS


def test_step_bad_logits(dev):
    """A NaN or plus infinity takes its beam out and is reported, wherever it is."""
    z, s = data(6, 3, 20000, torch.float32, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lce.beam_step(z, s, status=status)
    assert status.item() == 0
    z[0, 1, 0] = float("nan")
    z[1, 2, 19999] = INF
    z[2, 0, :] = -INF
    z[2, 0, 7777] = float("nan")
    z[3] = float("nan")
    s[4, 1] = float("nan")
    s[5, 0] = INF
    for i in range(6):
        status.zero_()
        got = lce.beam_step(z[i:i + 1], s[i:i + 1], num=6, status=status)
        check_step(z[i:i + 1], s[i:i + 1], 6, got=got)
        assert status.item() == lce.LCE_STATUS_BAD_LOGITS
    # whatever a finished beam's logits are
    fin = torch.zeros(6, 3, dtype=torch.bool, device=dev)
    fin[0, 1] = True
    status.zero_()
    check_step(z[:1], s[:1], 6, fin[:1], 4,
               got=lce.beam_step(z[:1], s[:1], num=6, finished=fin[:1], eos=4, status=status))
    assert status.item() == 0


def test_step_strides(dev):
    """Logits inside wider rows, at odd offsets, and in strides that have to be copied."""
    z, s = data(3, 4, 5001, torch.bfloat16, dev)
    ref = lce.beam_step(z, s)
    wide = torch.full((3, 4, 5010), INF, device=dev).bfloat16()
    wide[..., 3:5004] = z
    gap = torch.zeros(3, 6, 5001, device=dev).bfloat16()
    gap[:, 1:5] = z
    for view in (wide[..., 3:5004], gap[:, 1:5], z.transpose(0, 1).contiguous().transpose(0, 1)):
        for p, q in zip(ref[:3], lce.beam_step(view, s.t().contiguous().t())):
            assert torch.equal(p, q)
    for same in (z[:1, :1].expand(1, 4, 5001), z[:, :1].expand(3, 4, 5001),
                 z[:1, :1].expand(3, 1, 5001), z[:1, :1].expand(3, 4, 5001)):
        t = s[:same.shape[0], :same.shape[1]]
        for p, q in zip(lce.beam_step(same.contiguous(), t)[:3], lce.beam_step(same, t)):
            assert torch.equal(p, q)
    one = lce.beam_step(wide[1:2, 2:3, 3:5004], s[1:2, 2:3], num=4)
    check_step(z[1:2, 2:3].contiguous(), s[1:2, 2:3], 4, got=one)
    empty = lce.beam_step(z[:0], s[:0], num=4, eos=1)
    assert [t.shape for t in empty] == [(0, 4)] * 4


def test_step_is_log_softmax_for_one_beam(dev):
    """num = 1 of one beam is the argmax, its score the log-probability of the loss layer."""
    z, _ = data(9, 1, 30000, torch.bfloat16, dev)
    best, _, tokens, _ = lce.beam_step(z, torch.zeros(9, 1, device=dev))
    assert torch.equal(tokens[:, 0].long(), z[:, 0].float().argmax(-1))
    rows, _ = lce.ce_rows_fwd(z[:, 0], tokens[:, 0])
    assert ((best[:, 0] + rows).abs() <= 200 * U + rows.abs() * 4 * U).all()


# ---------------------------------------------------------------- states

def follow(x, parents):
    at = torch.arange(len(x), device=x.device)[:, None]
    y = x[at, parents.long().clamp(0, x.shape[1] - 1)]
    ok = ((parents >= 0) & (parents < x.shape[1])).view(*parents.shape, *[1] * (x.dim() - 2))
    return torch.where(ok, y, torch.zeros((), dtype=x.dtype, device=x.device))


def parents_of(b, beams, slots, dev, seed=0):
    gen = torch.Generator().manual_seed(seed + b + beams + slots)
    return torch.randint(-1, beams + 1, (b, slots), generator=gen, dtype=torch.int32).to(dev)


@pytest.mark.parametrize("b,beams,slots,rest,dtype", [
    (1, 1, 1, (), torch.int32), (3, 4, 4, (), torch.bool), (2, 4, 8, (5,), torch.int32),
    (5, 3, 2, (7, 3), torch.bfloat16), (2, 8, 8, (1000, 33), torch.float32),
    (1, 64, 64, (129,), torch.float64), (4, 5, 5, (3, 4099), torch.uint8),
    (2, 2, 2, (40000,), torch.bfloat16), (3, 16, 16, (2, 3, 4, 5), torch.int64)])
def test_reorder(dev, b, beams, slots, rest, dtype):
    x = torch.randint(0, 2 if dtype == torch.bool else 100, (b, beams, *rest), device=dev).to(dtype)
    p = parents_of(b, beams, slots, dev)
    got, = lce.beam_reorder([x], p)
    assert torch.equal(got, follow(x, p))
    if slots == beams:
        y = x.clone()
        same, = lce.beam_reorder([y], p, out=[y])
        assert same is y and torch.equal(y, got)


def test_reorder_many_states(dev):
    """More states than a launch holds, of all sizes and types, in one call."""
    p = parents_of(3, 6, 6, dev)
    shapes = [(3, 6, *r) for r in ((), (1,), (50, 7), (3, 1000), (0,), (17000,))] * 4
    kinds = [torch.int32, torch.bfloat16, torch.uint8, torch.float32]
    states = [torch.randint(0, 99, s, device=dev).to(kinds[i % 4]) for i, s in enumerate(shapes)]
    want = [follow(x, p) for x in states]
    for x, y in zip(lce.beam_reorder(states, p), want):
        assert torch.equal(x, y)
    lce.beam_reorder(states, p, out=states)
    for x, y in zip(states, want):
        assert torch.equal(x, y)
    assert lce.beam_reorder([], p) == []
    twice = lce.beam_reorder([states[2], states[2]], p)  # the same state into two places
    assert torch.equal(twice[0], twice[1])


def test_reorder_strided_caches(dev):
    """Caches with room behind what is used: only that moves; beams at other dimensions."""
    p = parents_of(2, 4, 4, dev)
    cache = torch.randn(2, 4, 6, 90, 16, device=dev).bfloat16()  # heads, length, dim
    used = cache[:, :, :, :37]
    want, rest = follow(used, p), cache[:, :, :, 37:].clone()
    got, = lce.beam_reorder([used], p)
    assert torch.equal(got, want)
    lce.beam_reorder([used], p, out=[used])
    assert torch.equal(used, want) and torch.equal(cache[:, :, :, 37:], rest)
    odd = torch.randn(2, 4, 50, 33, device=dev)[:, :, 1:42, 3:30]  # runs of 27 numbers
    out = torch.zeros(2, 4, 41, 27, device=dev)
    lce.beam_reorder([odd], p, out=[out])
    assert torch.equal(out, follow(odd, p))
    layers = torch.randn(5, 2, 4, 19, device=dev)  # beams behind the layers
    view = layers.permute(1, 2, 0, 3)
    want = follow(view, p)
    lce.beam_reorder([view], p, out=[view])
    assert torch.equal(view, want)
    with pytest.raises(ValueError, match="runs"):
        lce.beam_reorder([layers.permute(1, 2, 3, 0)], p)
    with pytest.raises((ValueError, lce.LceError)):
        lce.beam_reorder([cache], p, out=[cache.flip(0)[:, :, :, :1].expand_as(cache)])


def test_a_search(dev):
    """A whole search on a fixed table of next-token logits, histories and a cache following their
    beams: the same hypotheses as an exhaustive one in 64 bits."""
    v, beams, steps, eos = 6, 4, 5, 0
    gen = torch.Generator().manual_seed(5)
    table = (torch.randn(v, v, generator=gen) * 2).to(dev)  # logits after each token
    scores = torch.tensor([[0.0] + [-INF] * (beams - 1)], device=dev)
    tokens = torch.full((1, beams), 1, dtype=torch.int32, device=dev)
    finished = torch.zeros(1, beams, dtype=torch.bool, device=dev)
    history = torch.zeros(1, beams, steps, dtype=torch.int32, device=dev)
    trace = torch.zeros(1, beams, 3, device=dev)  # a state that depends on the whole path
    for t in range(steps):
        logits = table[tokens.clamp(min=0).long()]
        scores, parents, tokens, finished = lce.beam_step(logits, scores, finished=finished,
                                                          eos=eos)
        lce.beam_reorder([history, trace], parents, out=[history, trace])
        history[:, :, t] = tokens
        trace[:] = trace * 2 + tokens[..., None]
    logp = torch.log_softmax(table.double().cpu(), -1)
    paths = [((), 0.0)]
    for t in range(steps):
        nxt = []
        for path, s in paths:
            last = path[-1] if path else 1
            if path and eos in path:
                nxt.append((path + (eos,), s))
            else:
                nxt += [(path + (w,), s + logp[last, w].item()) for w in range(v)]
        paths = sorted(nxt, key=lambda p: -p[1])[:beams]
    assert [tuple(h) for h in history[0].tolist()] == [p for p, _ in paths]
    for s, (_, want) in zip(scores[0].tolist(), paths):
        assert abs(s - want) <= steps * (100 * U + abs(want) * U)
    for row, (path, _) in zip(trace[0].tolist(), paths):
        assert row == [float(sum(w << (steps - 1 - i) for i, w in enumerate(path)))] * 3


def test_graph_and_streams(dev):
    """Selection and reordering captured together and replayed on other logits; two captured steps
    that alternate."""
    z, s = data(4, 4, 9000, torch.bfloat16, dev)
    state = torch.randn(4, 4, 700, device=dev)

    def step():
        best, parents, tokens, done = lce.beam_step(z, s, num=4, eos=2)
        return best, parents, tokens, done, *lce.beam_reorder([state], parents)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    for p, q in zip(on_side, step()):
        assert torch.equal(p, q)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        graphs.append((graph, held))
    for seed in range(4):
        z.copy_(data(4, 4, 9000, torch.bfloat16, dev, seed + 50)[0])
        eager = step()
        graph, held = graphs[seed % 2]
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(held, eager):
            assert torch.equal(p, q)
