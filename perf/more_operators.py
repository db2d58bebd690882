"""Measured cases of the operators behind a model's last layer: root-mean-square norm with the
residual's addition (16- and 8-bit outputs, gradients), the matrix product in 8-bit floating point
with a scale for each block of 128, and beam search's selection with the reordering of states.

Each case can be computed in a plain form (elementary torch operations in 32 bits, the scores of a
beam search in 64) or, with ``own`` set, by this package's kernels; ``exact`` computes the same
outputs in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
FP8 = torch.float8_e4m3fn
E8M0 = torch.float8_e8m0fnu
EPS = 1e-6
LARGEST = 448.0  # of e4m3
LEAST = 2.0 ** -126  # the smallest scale


def listed():
    return [
        # the final norm of 8 tokens being decoded, the last layer's output added to the stream
        {"name": "norm_decode", "op": "norm", "n": 8, "h": 4096, "dtype": "bf16",
         "residual": True},
        # the same for 32 tokens in front of a head in 8 bits
        {"name": "norm8_decode", "op": "norm8", "n": 32, "h": 4096, "dtype": "bf16",
         "residual": True, "scale": "pow2"},
        # a long-context batch on its way into 8-bit products
        {"name": "norm8_long", "op": "norm8", "n": 32768, "h": 8192, "dtype": "bf16",
         "residual": True, "scale": "pow2"},
        # gradient of the norm at the 8B head's batch, with the stream's own gradient
        {"name": "norm_grad", "op": "norm_grad", "n": 8192, "h": 4096, "dtype": "bf16",
         "residual": True},
        # its gradient with an odd number of rows and columns
        {"name": "norm_grad_odd", "op": "norm_grad", "n": 4099, "h": 2051, "dtype": "fp16",
         "residual": False},
        # logits of 16 tokens being decoded under an 8B model's head held in 8 bits
        {"name": "product_decode", "op": "product", "m": 16, "n": 128256, "k": 4096,
         "scale": "pow2", "out": "fp32", "bias": False, "from": "fp8"},
        # logits of a ragged batch, small model with a bias, odd vocabulary, scales of any value
        {"name": "product_odd", "op": "product", "m": 1003, "n": 32777, "k": 768,
         "scale": "fp32", "out": "bf16", "bias": True, "from": "fp8"},
        # a square projection of a prompt of 2048 tokens whose activations come in 16 bits
        {"name": "product_project", "op": "product", "m": 2048, "n": 4096, "k": 4096,
         "scale": "fp32", "out": "bf16", "bias": False, "from": "bf16"},
        # logits of every position of the 8B head's batch
        {"name": "product_large", "op": "product", "m": 8192, "n": 128256, "k": 4096,
         "scale": "pow2", "out": "bf16", "bias": False, "from": "fp8"},
        # one sentence being translated with 4 beams, small vocabulary, some beams done
        {"name": "beam_small", "op": "beam", "b": 1, "k": 4, "v": 32777, "num": 4,
         "dtype": "bf16", "done": True},
        # 32 sentences with 8 beams each, twice as many candidates as beams
        {"name": "beam_large", "op": "beam", "b": 32, "k": 8, "v": 128256, "num": 16,
         "dtype": "bf16", "done": False},
        # the caches of four layers (keys and values of 1000 tokens) follow their beams
        {"name": "beam_states", "op": "states", "b": 16, "k": 8, "t": 1000, "w": 1024,
         "count": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "norm_grad", "product", "beam", "states"])
    if op in ("norm", "norm8", "norm_grad"):
        h = _log(rng, 64, 16384)
        case = {"op": op, "n": _log(rng, 1, 8192 * 4096 // h), "h": h,
                "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "residual": rng.choice([True, False])}
        if op == "norm8":
            case["scale"] = rng.choice(["pow2", "fp32"])
        return case
    if op == "product":
        k = 16 * _log(rng, 4, 512)
        n = _log(rng, 100, 128256)
        m = _log(rng, 1, min(8192, 8192 * 4096 // k))
        return {"op": op, "m": m, "n": n, "k": k, "scale": rng.choice(["pow2", "fp32"]),
                "out": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.choice([True, False]),
                "from": rng.choice(["fp8", "bf16"])}
    if op == "beam":
        k = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        v = _log(rng, 500, 262144)
        b = _log(rng, 1, min(64, max(1, 32 * 8 * 128256 // (k * v))))
        return {"op": op, "b": b, "k": k, "v": v, "num": rng.choice([k, 2 * k]),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "done": rng.choice([True, False])}
    k = rng.choice([2, 3, 4, 5, 8, 12, 16])
    w = _log(rng, 1, 1024)
    count = rng.choice([1, 2, 8])
    t = _log(rng, 1, 2000)
    dtype = rng.choice(["bf16", "fp32", "int32"])
    most = 2 * 10 ** 9 // (k * w * count * t * SIZES.get(dtype, 4))
    b = _log(rng, 1, max(1, min(64, most)))
    return {"op": op, "b": b, "k": k, "t": t, "w": w, "count": count, "dtype": dtype}


def _normal(g, shape, std, dtype):
    x = torch.empty(shape, device="cuda", dtype=dtype)
    return x.normal_(0.0, std, generator=g)


def _scales_of(largest, kind):
    """The scales of blocks from their largest magnitudes (32 bits)."""
    c = (largest / torch.full_like(largest, LARGEST)).clamp(min=LEAST)
    if kind == "pow2":
        m, e = torch.frexp(c)  # c = m * 2^e with 0.5 <= m < 1
        c = torch.ldexp(torch.ones_like(c), e - (m == 0.5).int())
    return torch.where(torch.isfinite(largest), c, float("nan"))


def _to_blocks(x):
    """[n, h] as [n, blocks, 128], zeros behind the last column."""
    n, h = x.shape
    return torch.nn.functional.pad(x, (0, -h % 128)).view(n, -1, 128)


def _quantise(y, kind):
    """Rows of 32-bit values in 8 bits: (e4m3 [n, h], 32-bit scales [blocks, n])."""
    b = _to_blocks(y)
    c = _scales_of(b.abs().amax(-1), kind)
    q = (b / c[:, :, None]).clamp(-LARGEST, LARGEST).reshape(len(y), -1)[:, :y.shape[1]]
    return q.to(FP8), c.t().contiguous()


def _scale_bits(c, kind):
    """32-bit scales as they are held: powers of two by their exponent."""
    if kind == "fp32":
        return c
    return (torch.frexp(c)[1] + 126).to(torch.uint8).view(E8M0)


def _scale_values(c):
    return c if c.dtype == torch.float32 else torch.ldexp(
        torch.ones(c.shape, device=c.device), c.view(torch.uint8).int() - 127)


def _scales_out(c, kind):
    """A power of two as the number that it is, whichever way it is held."""
    return _scale_bits(c, kind) if kind == "pow2" else c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm8", "norm_grad"):
        n, h, dt = case["n"], case["h"], DTYPES[case["dtype"]]
        # hidden states: a few columns are far larger than the others
        x = _normal(g, (n, h), 1.0, torch.float32)
        x[:, :: max(1, h // 7)] *= 8.0
        s["x"] = x.to(dt)
        s["add"] = _normal(g, (n, h), 0.5, dt) if case["residual"] else None
        s["weight"] = (1.0 + _normal(g, (h,), 0.1, torch.float32)).to(dt)
        if op == "norm_grad":  # x is the sum that the forward has kept; add the stream's gradient
            s["grad"] = _normal(g, (n, h), 1e-2, dt)
            s["add"] = _normal(g, (n, h), 1e-2, dt) if case["residual"] else None
            s["rstd"] = ((s["x"].double() ** 2).mean(-1) + EPS).rsqrt().float()
    elif op == "product":
        m, n, k, kind = case["m"], case["n"], case["k"], case["scale"]
        x = _normal(g, (m, k), 1.0, torch.float32)
        x[:, :: max(1, k // 7)] *= 8.0
        if case["from"] == "fp8":
            s["a"], c = _quantise(x, kind)
            s["ca"] = _scale_bits(c, kind)
        else:
            s["x"] = x.to(torch.bfloat16)
        # the weight, laid out once: blocks of 128 x 128 share a scale
        w = _normal(g, (n, k), 1.3 / math.sqrt(k), torch.bfloat16)
        s["b"] = torch.empty((n, k), device="cuda", dtype=FP8)
        s["cb"] = []
        for lo in range(0, n, 16384):
            part = _to_blocks(w[lo:lo + 16384].float())
            rows = torch.nn.functional.pad(part.abs().amax(-1), (0, 0, 0, -len(part) % 128))
            c = _scales_of(rows.view(-1, 128, part.shape[1]).amax(1), kind)
            q = part / c.repeat_interleave(128, 0)[:len(part), :, None]
            s["b"][lo:lo + 16384] = q.reshape(len(part), -1)[:, :k].to(FP8)
            s["cb"].append(_scale_bits(c, kind))
        s["cb"] = torch.cat([c.view(torch.uint8) for c in s["cb"]]).view(s["cb"][0].dtype)
        s["bias"] = _normal(g, (n,), 0.2, torch.float32) if case["bias"] else None
        s["out_dtype"] = DTYPES[case["out"]]
    elif op == "beam":
        b, k, v = case["b"], case["k"], case["v"]
        s["logits"] = _normal(g, (b, k, v), 2.5, DTYPES[case["dtype"]])
        s["scores"] = _normal(g, (b, k), 1.0, torch.float32).sub_(20.0)
        s["done"] = None
        if case["done"]:
            s["done"] = torch.rand(b, k, generator=g, device="cuda") < 0.2
        s["eos"] = 2
        s["history"] = torch.randint(0, v, (b, k, 40), generator=g, device="cuda",
                                     dtype=torch.int32)
    else:
        b, k = case["b"], case["k"]
        shape = (b, k, case["t"], case["w"])
        if case["dtype"] == "int32":
            s["states"] = [torch.randint(0, 50000, shape, generator=g, device="cuda",
                                         dtype=torch.int32) for _ in range(case["count"])]
        else:
            s["states"] = [_normal(g, shape, 1.0, DTYPES[case["dtype"]])
                           for _ in range(case["count"])]
        s["into"] = [torch.empty_like(x) for x in s["states"]]
        s["parents"] = torch.randint(0, k, (b, k), generator=g, device="cuda", dtype=torch.int32)
    return s


def _run_own(s):
    import linear_cross_entropy_masked_amd as lce
    op = s["op"]
    if op == "norm":
        y, total, rstd = lce.rmsnorm_fwd(s["x"], s["weight"], s["add"], eps=EPS)
        return y, (total if s["residual"] else None), rstd
    if op == "norm8":
        held = E8M0 if s["scale"] == "pow2" else torch.float32
        q, c, total = lce.rmsnorm_fp8_fwd(s["x"], s["weight"], s["add"], eps=EPS,
                                          scale_dtype=held)
        return q, c, (total if s["residual"] else None)
    if op == "norm_grad":
        return lce.rmsnorm_bwd(s["grad"], s["x"], s["rstd"], s["weight"],
                               grad_residual=s["add"])
    if op == "product":
        if s["from"] == "fp8":
            return lce.fp8_matmul(s["a"], s["ca"], s["b"], s["cb"], s["bias"],
                                  dtype=s["out_dtype"])
        a, ca = lce.fp8_quantize(s["x"], scale_dtype=s["cb"].dtype)
        return lce.fp8_matmul(a, ca, s["b"], s["cb"], s["bias"], dtype=s["out_dtype"]), a, ca
    if op == "beam":
        scores, parents, tokens, done = lce.beam_step(s["logits"], s["scores"], num=s["num"],
                                                      finished=s["done"], eos=s["eos"])
        history, = lce.beam_reorder([s["history"]], parents)
        return scores, parents, tokens, done, history
    return lce.beam_reorder(s["states"], s["parents"], out=s["into"])


def run(state):
    if own:
        return _run_own(state)
    s, op = state, state["op"]
    if op in ("norm", "norm8"):
        total = s["x"]
        if s["add"] is not None:
            total = (s["x"].float() + s["add"].float()).to(s["x"].dtype)
        t = total.float()
        rstd = ((t * t).mean(-1) + EPS).rsqrt()
        y = t * rstd[:, None] * s["weight"].float()
        kept = total if s["residual"] else None
        if op == "norm":
            return y.to(total.dtype), kept, rstd
        q, c = _quantise(y, s["scale"])
        return q, _scales_out(c, s["scale"]), kept
    if op == "norm_grad":
        g, dt = s["grad"].float(), s["x"].dtype
        xhat = s["x"].float() * s["rstd"][:, None]
        u = g * s["weight"].float()
        dx = (u - xhat * (u * xhat).mean(-1, keepdim=True)) * s["rstd"][:, None]
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return dx.to(dt), (g * xhat).sum(0).to(dt)
    if op == "product":
        if s["from"] == "fp8":
            a, ca = s["a"], s["ca"]
        else:
            a, ca = _quantise(s["x"].float(), s["scale"])
            ca = _scale_bits(ca, s["scale"])
        m, n, k = s["m"], s["n"], s["k"]
        af = a.float() * _scale_values(ca).t().repeat_interleave(128, 1)[:, :k]
        cb = _scale_values(s["cb"]).repeat_interleave(128, 1)[:, :k]
        bf = s["b"].float() * cb.repeat_interleave(128, 0)[:n]
        z = af @ bf.t()
        if s["bias"] is not None:
            z = z + s["bias"]
        z = z.to(s["out_dtype"])
        return z if s["from"] == "fp8" else (z, a, ca)
    if op == "beam":
        z, num = s["logits"], s["num"]
        b, k, v = z.shape
        few = min(num, v)
        # the best of each beam, equal logits in the order of their tokens
        order = torch.sort(z, dim=-1, descending=True, stable=True).indices[..., :few]
        zd = z.double()
        top = zd.amax(-1, keepdim=True)
        lse = (zd - top).exp().sum(-1, keepdim=True).log() + top
        cand = s["scores"].double()[..., None] + (zd.gather(-1, order) - lse)
        if s["done"] is not None:  # a beam that is done goes on as it is
            alone = torch.full_like(cand, -math.inf)
            alone[..., 0] = s["scores"].double()
            cand = torch.where(s["done"][..., None], alone, cand)
            order = torch.where(s["done"][..., None], s["eos"], order)
        best = torch.sort(cand.reshape(b, k * few), dim=-1, descending=True, stable=True)
        at = best.indices[:, :num]
        scores = best.values[:, :num]
        none = scores == -math.inf
        parents = torch.where(none, -1, at // few)
        tokens = torch.where(none, IGNORE, order.reshape(b, k * few).gather(1, at))
        done = tokens == s["eos"]
        if s["done"] is not None:
            done = done | (s["done"].gather(1, parents.clamp(min=0)) & ~none)
        history = _follow(s["history"], parents)
        return scores.float(), parents.int(), tokens.int(), done, history
    return [_follow(x, s["parents"]) for x in s["states"]]


def _follow(x, parents):
    """State j of each batch entry is that of beam parents[j], zeros where there is none."""
    at = torch.arange(len(x), device=x.device)[:, None]
    rows = x[at, parents.long().clamp(min=0)]
    keep = (parents >= 0).view(*parents.shape, *([1] * (x.dim() - 2)))
    return torch.where(keep, rows, torch.zeros((), dtype=x.dtype, device=x.device))


def work(case):
    op = case["op"]
    if op in ("norm", "norm8", "norm_grad"):
        n, h, el = case["n"], case["h"], SIZES[case["dtype"]]
        add = 1 if case["residual"] else 0
        if op == "norm":
            return {"bytes": n * h * el * (2 + 2 * add) + h * el + 4 * n, "flops": 5 * n * h}
        if op == "norm8":
            return {"bytes": n * h * (el * (1 + 2 * add) + 1) + h * el + n * h / 128,
                    "flops": 8 * n * h}
        return {"bytes": n * h * el * (3 + add) + 2 * h * el + 4 * n, "flops": 11 * n * h}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        sc = 1 if case["scale"] == "pow2" else 4
        moved = m * k + n * k + m * n * SIZES[case["out"]] + sc * m * k / 128
        moved += sc * n * k / 128 ** 2
        if case["from"] == "bf16":
            moved += 2 * m * k
        return {"bytes": moved + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "beam":
        rows = case["b"] * case["k"]
        return {"bytes": rows * case["v"] * SIZES[case["dtype"]] + 4 * rows
                + case["b"] * case["num"] * (13 + 2 * 4 * 40), "flops": 4 * rows * case["v"]}
    el = 4 if case["dtype"] == "int32" else SIZES[case["dtype"]]
    # on average a share of 1 - (1 - 1/k)^k of the beams is read
    k = case["k"]
    size = case["b"] * k * case["t"] * case["w"] * case["count"] * el
    return {"bytes": size * (2 - (1 - 1 / k) ** k) + 4 * case["b"] * k, "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    op, f64 = s["op"], torch.float64
    if op in ("norm", "norm8"):
        kept = s["x"]
        total = s["x"].to(f64)
        if s["add"] is not None:
            total = torch.add(total, s["add"].to(f64))
            kept = total.to(s["x"].dtype)  # what is held, and normalised
        t = kept.to(f64)
        size = torch.linalg.vector_norm(t, dim=1)
        rstd = 1.0 / torch.sqrt(size ** 2 / case["h"] + EPS)
        y = torch.einsum("nh,n,h->nh", t, rstd, s["weight"].to(f64))
        if op == "norm":
            return y, (total if case["residual"] else None), rstd
        q, c = _blocks_exact(y, case["scale"])
        return q, c, (total if case["residual"] else None)
    if op == "norm_grad":
        # the gradient as the projection of u = g · w across the row
        x, g, w = s["x"].to(f64), s["grad"].to(f64), s["weight"].to(f64)
        r = s["rstd"].to(f64)
        along = torch.einsum("nh,nh,h->n", g, x, w) * r ** 3 / case["h"]
        dx = torch.addcmul(g * torch.outer(r, w), x, along[:, None], value=-1.0)
        if s["add"] is not None:
            dx += s["add"].to(f64)
        return dx, torch.mv((g * x).t(), r)
    if op == "product":
        kind, k, n = case["scale"], case["k"], case["n"]
        if case["from"] == "fp8":
            a, ca = s["a"].to(f64), _scale_values(s["ca"]).to(f64)
        else:
            a, ca = _blocks_exact(s["x"].to(f64), kind)
        cb = _scale_values(s["cb"]).to(f64)
        rows = torch.arange(n, device="cuda") // 128
        out = torch.zeros(case["m"], n, device="cuda", dtype=f64)
        for lo in range(0, k, 1024):  # eight blocks at a time
            hi = min(k, lo + 1024)
            of = torch.arange(lo, hi, device="cuda") // 128
            left = a[:, lo:hi] * ca[of].t()
            right = s["b"][:, lo:hi].to(f64) * cb[rows][:, of]
            out.addmm_(left, right.t())
        if s["bias"] is not None:
            out += s["bias"].to(f64)
        return out if case["from"] == "fp8" else (out, a, ca)
    if op == "beam":
        logp = torch.log_softmax(s["logits"].to(f64), -1)
        b, k, v = logp.shape
        scores = s["scores"].to(f64)
        cand = logp + scores[..., None]
        if s["done"] is not None:
            rows = s["done"].nonzero()
            cand[rows[:, 0], rows[:, 1]] = -math.inf
            cand[rows[:, 0], rows[:, 1], s["eos"]] = scores[rows[:, 0], rows[:, 1]]
        best = torch.topk(cand.view(b, -1), case["num"], dim=1).values
        return best, None, None, None, None
    if case["dtype"] == "int32":
        return None
    at = (torch.arange(case["b"], device="cuda")[:, None] * case["k"] + s["parents"]).view(-1)
    return [x.flatten(0, 1).index_select(0, at).view_as(x) for x in s["states"]]


def _blocks_exact(y, kind):
    """Blocks of 128 in 8 bits from 64-bit values: (values [n, h], scales [blocks, n])."""
    n, h = y.shape
    q = torch.empty_like(y)
    scales = []
    for lo in range(0, h, 128):
        part = y[:, lo:lo + 128]
        c = torch.maximum(part.abs().max(dim=1).values / LARGEST,
                          torch.full((), LEAST, device=y.device, dtype=y.dtype))
        if kind == "pow2":
            c = torch.exp2(torch.ceil(torch.log2(c)))
        c = c.to(torch.float32).to(y.dtype)  # held in 32 bits, and so is the quotient
        v = (part / c[:, None]).to(torch.float32).to(y.dtype)
        # three bits behind the leading one, in steps of 2^-9 at least
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, lo:lo + 128] = torch.round(v / step) * step
        scales.append(c)
    return q, torch.stack(scales)
