"""Measured cases of the operators at the two ends of a language model: the embedding lookup and
its gradient, layer norm forward and backward, and the linear cross entropy taken in pieces of
the vocabulary, forward and backward.

Each case can be computed in a plain form (elementary torch operations in 32 bits) or, with
``own`` set, by this package's kernels; ``exact`` computes the same outputs in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # the token of each of 32 sequences that are being decoded, at an 8B model's table
        {"name": "embed_decode", "op": "embed", "n": 32, "v": 128256, "h": 4096, "dtype": "bf16",
         "masked": 0.0, "scale": 64.0},
        # one training batch's lookup, a few rows being padding
        {"name": "embed_batch", "op": "embed", "n": 8192, "v": 128256, "h": 4096, "dtype": "bf16",
         "masked": 0.05, "scale": 64.0},
        # gradient of a small model's table, into fp32 main gradients, odd vocabulary
        {"name": "embed_grad_small", "op": "embed_grad", "n": 2048, "v": 32777, "h": 768,
         "dtype": "bf16", "grad": "fp32", "masked": 0.05, "scale": 1.0},
        # gradient of an 8B model's table over a long batch
        {"name": "embed_grad_large", "op": "embed_grad", "n": 32768, "v": 128256, "h": 4096,
         "dtype": "bf16", "grad": "bf16", "masked": 0.05, "scale": 64.0},
        # the final norm of 8 tokens being decoded
        {"name": "norm_decode", "op": "norm", "n": 8, "h": 4096, "dtype": "bf16"},
        # the final norm of a long-context batch
        {"name": "norm_long", "op": "norm", "n": 32768, "h": 8192, "dtype": "bf16"},
        # its gradient at the 8B head's batch
        {"name": "norm_grad", "op": "norm_grad", "n": 8192, "h": 4096, "dtype": "bf16"},
        # its gradient with an odd number of rows and columns
        {"name": "norm_grad_odd", "op": "norm_grad", "n": 4099, "h": 2051, "dtype": "fp16"},
        # log-probabilities of 16 given tokens under an 8B model's head
        {"name": "loss_score", "op": "loss", "n": 16, "v": 128256, "h": 4096, "bias": False,
         "masked": 0.0},
        # evaluation loss of a ragged batch, small model with a bias, odd vocabulary
        {"name": "loss_eval", "op": "loss", "n": 1003, "v": 32777, "h": 768, "bias": True,
         "masked": 0.1},
        # fine-tuning step of the small model: half of the rows are prompt and carry no label
        {"name": "loss_train_small", "op": "loss_grad", "n": 2048, "v": 32777, "h": 768,
         "bias": True, "masked": 0.5},
        # training step at the 8B head's batch
        {"name": "loss_train_large", "op": "loss_grad", "n": 8192, "v": 128256, "h": 4096,
         "bias": False, "masked": 0.05},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "loss", "loss_grad"])
    if op in ("embed", "embed_grad"):
        h = _log(rng, 64, 8192)
        v = _log(rng, 500, min(262144, 128256 * 4096 // h))
        n = _log(rng, 1, min(65536, 32768 * 4096 // h))
        case = {"op": op, "n": n, "v": v, "h": h, "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "masked": rng.choice([0.0, 0.05, 0.3]), "scale": rng.choice([1.0, h ** 0.5])}
        if op == "embed_grad":
            case["grad"] = rng.choice(["fp32", case["dtype"]])
        return case
    if op in ("norm", "norm_grad"):
        h = _log(rng, 64, 16384)
        return {"op": op, "n": _log(rng, 1, 8192 * 4096 // h), "h": h,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    h = 8 * _log(rng, 8, 512)
    v = _log(rng, 1000, 128256)
    n = _log(rng, 1, 8192)
    return {"op": op, "n": n, "v": v, "h": h, "bias": rng.choice([True, False]),
            "masked": rng.choice([0.0, 0.05, 0.5])}


def _tokens(g, n, v, masked):
    """Token numbers with the frequencies of text (the r-th most frequent one in proportion to
    1 / r, spread over the vocabulary); a share of the rows carries none."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.exp(u * math.log(v + 1.0)).long().sub_(1).clamp_(0, v - 1)
    tok = (rank * 7919 + 13) % v
    if masked:
        drop = torch.rand(n, generator=g, device="cuda") < masked
        drop[0] = False
        tok = torch.where(drop, torch.full_like(tok, IGNORE), tok)
    return tok.to(torch.int32)


def _normal(g, shape, std, dtype):
    x = torch.empty(shape, device="cuda", dtype=dtype)
    return x.normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"op": case["op"], "n": case["n"], "h": case["h"]}
    op, n, h = case["op"], case["n"], case["h"]
    if op in ("embed", "embed_grad"):
        dt = DTYPES[case["dtype"]]
        s["v"], s["scale"] = case["v"], case["scale"]
        s["tokens"] = _tokens(g, n, case["v"], case["masked"])
        if op == "embed":
            s["weight"] = _normal(g, (case["v"], h), 0.02, dt)
        else:
            s["grad"] = _normal(g, (n, h), 1e-3, dt)
            s["grad_dtype"] = DTYPES[case["grad"]]
    elif op in ("norm", "norm_grad"):
        dt = DTYPES[case["dtype"]]
        # hidden states: a few columns are far larger than the others
        x = _normal(g, (n, h), 1.0, torch.float32)
        x[:, :: max(1, h // 7)] *= 8.0
        s["x"] = (x + 0.1).to(dt)
        s["weight"] = (1.0 + _normal(g, (h,), 0.1, torch.float32)).to(dt)
        s["bias"] = _normal(g, (h,), 0.1, dt)
        if op == "norm_grad":
            s["grad"] = _normal(g, (n, h), 1e-2, dt)
            xf = s["x"].double()  # what the forward pass has kept
            s["mean"] = xf.mean(-1).float()
            s["rstd"] = (xf.var(-1, unbiased=False) + EPS).rsqrt().float()
    else:
        s["hidden"] = _normal(g, (n, h), 1.0, torch.bfloat16)
        s["weight"] = _normal(g, (case["v"], h), 1.3 / math.sqrt(h), torch.bfloat16)
        s["bias"] = _normal(g, (case["v"],), 0.2, torch.float32) if case["bias"] else None
        s["labels"] = _tokens(g, n, case["v"], case["masked"])
    return s


def _run_own(s):
    import linear_cross_entropy_masked_amd as lce
    op = s["op"]
    if op == "embed":
        return lce.embed_fwd(s["weight"], s["tokens"], scale=s["scale"])
    if op == "embed_grad":
        return lce.embed_bwd(s["grad"], s["tokens"], s["v"], scale=s["scale"],
                             dtype=s["grad_dtype"])
    if op == "norm":
        return lce.layernorm_fwd(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_grad":
        return lce.layernorm_bwd(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"],
                                 grad_bias=True)
    loss, lse, rows = lce.flce_pieces_fwd(s["hidden"], s["weight"], s["labels"], s["bias"],
                                          return_rows=True)
    if op == "loss":
        return loss, lse, rows
    gh, gw, gb = lce.flce_pieces_bwd(s["hidden"], s["weight"], s["labels"], lse, s["bias"])
    return loss, lse, rows, gh, gw, gb


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op == "embed":
        tok = s["tokens"].long()
        keep = (tok >= 0)[:, None]
        rows = s["weight"][tok.clamp(min=0)].float() * s["scale"]
        return torch.where(keep, rows, torch.zeros_like(rows)).to(s["weight"].dtype)
    if op == "embed_grad":
        tok = s["tokens"].long()
        g = torch.where((tok >= 0)[:, None], s["grad"].float(), 0.0)
        w = torch.zeros(s["v"], s["h"], device=g.device, dtype=torch.float32)
        w.index_add_(0, tok.clamp(min=0), g)
        return (w * s["scale"]).to(s["grad_dtype"])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(-1)
        c = x - mean[:, None]
        rstd = ((c * c).mean(-1) + EPS).rsqrt()
        y = c * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return y.to(s["x"].dtype), mean, rstd
    if op == "norm_grad":
        g, dt = s["grad"].float(), s["x"].dtype
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        u = g * s["weight"].float()
        dx = (u - u.mean(-1, keepdim=True) - xhat * (u * xhat).mean(-1, keepdim=True))
        dx = dx * s["rstd"][:, None]
        return dx.to(dt), (g * xhat).sum(0).to(dt), g.sum(0).to(dt)
    hid, wt, lab = s["hidden"].float(), s["weight"].float(), s["labels"].long()
    z = hid @ wt.t()
    if s["bias"] is not None:
        z = z + s["bias"]
    keep = lab >= 0
    y = lab.clamp(min=0)
    top = z.max(-1).values
    lse = torch.where(keep, (z - top[:, None]).exp().sum(-1).log() + top, 0.0)
    rows = torch.where(keep, lse - z.gather(1, y[:, None])[:, 0], 0.0)
    count = keep.sum()
    loss = (rows.double().sum() / count).float()
    if op == "loss":
        return loss, lse, rows
    d = (z - lse[:, None]).exp()
    d.scatter_add_(1, y[:, None], torch.full_like(d[:, :1], -1.0))
    d = torch.where(keep[:, None], d / count, 0.0)
    gh = (d @ wt).to(torch.bfloat16)
    gw = (d.t() @ hid).to(torch.bfloat16)
    return loss, lse, rows, gh, gw, (d.sum(0) if s["bias"] is not None else None)


def work(case):
    op, n, h = case["op"], case["n"], case["h"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op in ("embed", "embed_grad"):
        b, v = size[case["dtype"]], case["v"]
        kept = n * (1.0 - case["masked"])
        if op == "embed":
            return {"bytes": 4 * n + kept * h * b + n * h * b, "flops": kept * h}
        return {"bytes": 4 * n + kept * h * b + v * h * size[case["grad"]], "flops": kept * h}
    if op == "norm":
        b = size[case["dtype"]]
        return {"bytes": 2 * n * h * b + 2 * h * b + 8 * n, "flops": 8 * n * h}
    if op == "norm_grad":
        b = size[case["dtype"]]
        return {"bytes": 3 * n * h * b + 3 * h * b + 8 * n, "flops": 14 * n * h}
    v, kept = case["v"], n * (1.0 - case["masked"])
    once = 2 * kept * h + 2 * v * h + (4 * v if case["bias"] else 0) + 12 * n
    if op == "loss":
        return {"bytes": once, "flops": 2 * kept * h * v}
    return {"bytes": once + 2 * n * h + 2 * v * h + (4 * v if case["bias"] else 0),
            "flops": 6 * kept * h * v}


def exact(case, seed):
    s = prepare(case, seed)
    op, h = s["op"], s["h"]
    f64 = torch.float64
    if op == "embed":
        tok = s["tokens"].tolist()
        out = torch.zeros(len(tok), h, device="cuda", dtype=f64)
        at = torch.tensor([i for i, t in enumerate(tok) if t >= 0], device="cuda")
        of = torch.tensor([t for t in tok if t >= 0], device="cuda")
        if len(at):
            out[at] = s["weight"].index_select(0, of).to(f64) * s["scale"]
        return out
    if op == "embed_grad":
        # rows put in the order of their tokens; a token's rows are then one range of a
        # running sum
        tok = s["tokens"]
        order = torch.argsort(tok, stable=True)
        order = order[tok[order] >= 0]
        t = tok[order]
        out = torch.zeros(s["v"], h, device="cuda", dtype=f64)
        if len(t):
            which, count = torch.unique_consecutive(t, return_counts=True)
            end = torch.cumsum(count, 0)
            for lo in range(0, h, 512):
                cols = slice(lo, min(h, lo + 512))
                run_sum = torch.cumsum(s["grad"][order][:, cols].to(f64), 0)
                upto = run_sum[end - 1]
                out[which.long(), cols] = s["scale"] * torch.diff(
                    upto, dim=0, prepend=torch.zeros_like(upto[:1]))
        return out
    if op == "norm":
        x = s["x"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["bias"].to(f64), (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None],
                          s["weight"].to(f64))
        return y, mean, rstd
    if op == "norm_grad":
        # the three sums of the gradient's formula, taken as inner products over the columns
        x, g, w = s["x"].to(f64), s["grad"].to(f64), s["weight"].to(f64)
        r, mu = s["rstd"].to(f64), s["mean"].to(f64)
        a = g @ w / h
        b = torch.einsum("nh,nh,h->n", g, x, w) / h - mu * a  # mean of u · (x − mean)
        dx = r[:, None] * (g * w - a[:, None]) - (r ** 3 * b)[:, None] * (x - mu[:, None])
        dw = (x * g).t() @ r - g.t() @ (mu * r)
        return dx, dw, g.sum(0)
    hid = s["hidden"].to(f64).requires_grad_(op == "loss_grad")
    wt = s["weight"].to(f64).requires_grad_(op == "loss_grad")
    bias = None if s["bias"] is None else s["bias"].to(f64).requires_grad_(op == "loss_grad")
    lab = s["labels"].long()
    at = torch.nonzero(lab >= 0)[:, 0]
    z = torch.nn.functional.linear(hid[at], wt, bias)
    part = torch.logsumexp(z, dim=1)
    term = part - z.gather(1, lab[at][:, None]).squeeze(1)
    total = term.mean()
    lse = torch.zeros(len(lab), device="cuda", dtype=f64).index_copy(0, at, part.detach())
    rows = torch.zeros(len(lab), device="cuda", dtype=f64).index_copy(0, at, term.detach())
    out = (total.detach(), lse, rows)
    if op == "loss":
        return out
    total.backward()
    return out + (hid.grad, wt.grad, None if bias is None else bias.grad)
