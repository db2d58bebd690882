"""PyTorch autograd functions over the library's C-ABI calls.

Argument marshalling only: every step of the loss and its gradients runs in the library's
kernels; this module picks the calls, folds a label mask into ignore_index, flattens leading
dimensions, and keeps what the backward needs.

Behaviour follows NeMo Automodel PR #2996 (the masked CE loss with a chunk_size):
  * the forward keeps only the original-dtype logits, the labels and the fp32 lse [n] for
    the backward, which rebuilds the softmax from them (commit messages 1 and 4);
  * writing the gradient into the logits storage is opt-in and keyword-only
    (``inplace_grad=True``; default False, the logits are left intact), the backward is
    once-differentiable, so a double backward raises, and after an in-place backward the
    logits' version counter is bumped, so any other autograd user of the logits fails loudly
    instead of reading the gradient as logits; a second backward through the same graph
    (``retain_graph=True``) raises too, since the logits are gone (seventh commit message:
    the keyword-only opt-in, the once-differentiable backward and the retain_graph hazard);
  * ``reduction``: "sum" is the method's sum over labelled rows, divided by
    ``num_label_tokens`` when it is given; "mean" divides by the number of labelled rows
    (counted on the device); "none" returns the per-row terms (0 for rows without a label).

The fused linear CE function uses the split calls (``flce_fwd`` in the forward, ``flce_bwd``
in the backward): nothing of size [V, H] lives from the forward to the backward (Liger-Kernel
issue #533, feature pitch), and the upstream gradient stays on the device.

``linear_cross_entropy_pieces`` is the same loss over a weight in pieces of the vocabulary, with
per-row terms as well. ``embedding`` and ``layer_norm`` are the model's other end of a tied table
and the norm in front of the head; ``norm_linear_cross_entropy`` joins norm and loss without
keeping the normalised hidden states, and ``TiedHead`` holds one table for both ends.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import (ce_chunked_bwd, ce_chunked_bwd_inplace, ce_chunked_fwd, ce_rows_bwd, ce_rows_fwd,
               embed_bwd, embed_fwd, flce_bwd, flce_fwd, flce_pieces_bwd, flce_pieces_fwd,
               layernorm_bwd, layernorm_fwd)

REDUCTIONS = ("sum", "mean", "none")


def _check_reduction(reduction, num_label_tokens, allowed=REDUCTIONS):
    if reduction not in allowed:
        raise ValueError(f"reduction must be one of {allowed}, got {reduction!r}")
    if num_label_tokens is not None and reduction != "sum":
        raise ValueError("num_label_tokens divides the summed loss: use it with reduction='sum'")


def _normaliser(reduction, num_label_tokens):
    """The library's T: the sum is divided by T; -1 asks for the device count of labelled rows."""
    if reduction == "mean":
        return -1
    return 1 if num_label_tokens is None else int(num_label_tokens)


def _flat_labels(labels, mask, n, ignore_index):
    if labels.numel() != n:
        raise ValueError(f"labels has {labels.numel()} entries, expected {n}")
    labels = labels.reshape(n)
    if mask is not None:
        if mask.numel() != n:
            raise ValueError(f"mask has {mask.numel()} entries, expected {n}")
        mask = mask.reshape(n)
        labels = torch.where(mask.to(torch.bool), labels,
                             torch.full_like(labels, ignore_index))
    return labels


class _MaskedCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, ignore_index, chunk_size, count, reduction, inplace_grad):
        if reduction == "none":
            out, lse = ce_rows_fwd(logits, labels, ignore_index=ignore_index,
                                   chunk_size=chunk_size)
        else:
            out, lse = ce_chunked_fwd(logits, labels, ignore_index=ignore_index,
                                      chunk_size=chunk_size, num_label_tokens=count)
        ctx.save_for_backward(logits, labels, lse)
        ctx.cfg = (ignore_index, chunk_size, count, reduction, inplace_grad)
        ctx.spent = False
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        ignore_index, chunk_size, count, reduction, inplace = ctx.cfg
        if inplace and ctx.spent:
            raise RuntimeError(
                "masked CE with inplace_grad=True: the logits were overwritten by the first "
                "backward; a second backward through this graph (retain_graph=True) cannot run")
        logits, labels, lse = ctx.saved_tensors
        if g.dtype != torch.float32:
            g = g.to(torch.float32)
        if reduction == "none":
            grad = ce_rows_bwd(logits, labels, g.contiguous(), inplace=inplace,
                               ignore_index=ignore_index, chunk_size=chunk_size, lse=lse)
        elif inplace:
            grad = ce_chunked_bwd_inplace(logits, labels, ignore_index=ignore_index,
                                          chunk_size=chunk_size, num_label_tokens=count,
                                          grad_output=g, lse=lse)
        else:
            grad = ce_chunked_bwd(logits, labels, ignore_index=ignore_index,
                                  chunk_size=chunk_size, num_label_tokens=count,
                                  grad_output=g, lse=lse)
        if inplace:
            ctx.spent = True
            torch.autograd.graph.increment_version(logits)
        return grad, None, None, None, None, None, None


def masked_cross_entropy(logits, labels, *, mask=None, ignore_index: int = -100,
                         chunk_size: int = 1024, num_label_tokens: int | None = None,
                         reduction: str = "sum", inplace_grad: bool = False):
    """Masked CE over bf16 logits [..., V] with int labels [...]: a 0-d fp32 loss ("sum",
    "mean") or fp32 per-row terms of the leading shape ("none"). ``mask`` (same leading
    shape, nonzero = keep) is folded into the labels as ignore_index."""
    _check_reduction(reduction, num_label_tokens)
    if logits.dim() < 1:
        raise ValueError("logits must have a vocabulary dimension")
    lead = logits.shape[:-1]
    v = logits.shape[-1]
    flat = logits.view(-1, v)  # a view (never a copy), so an in-place gradient lands in logits
    n = flat.shape[0]
    lab = _flat_labels(labels, mask, n, ignore_index)
    out = _MaskedCE.apply(flat, lab, int(ignore_index), int(chunk_size),
                          _normaliser(reduction, num_label_tokens), reduction, bool(inplace_grad))
    return out.view(lead) if reduction == "none" else out


class MaskedCrossEntropy(torch.nn.Module):
    """Module form of :func:`masked_cross_entropy` (the constructor arguments of the masked CE
    loss in NeMo Automodel PR #2996: chunk_size, and inplace_grad keyword-only, default
    False)."""

    def __init__(self, *, ignore_index: int = -100, chunk_size: int = 1024,
                 reduction: str = "sum", inplace_grad: bool = False):
        super().__init__()
        _check_reduction(reduction, None)
        self.ignore_index = ignore_index
        self.chunk_size = chunk_size
        self.reduction = reduction
        self.inplace_grad = inplace_grad

    def forward(self, logits, labels, mask=None, num_label_tokens=None):
        return masked_cross_entropy(logits, labels, mask=mask, ignore_index=self.ignore_index,
                                    chunk_size=self.chunk_size,
                                    num_label_tokens=num_label_tokens,
                                    reduction=self.reduction, inplace_grad=self.inplace_grad)


class _LinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, bias, labels, ignore_index, chunk_size, count, grad_buffer):
        loss, lse = flce_fwd(hidden, weight, labels, bias, ignore_index=ignore_index,
                             chunk_size=chunk_size, num_label_tokens=count)
        ctx.save_for_backward(hidden, weight, bias, labels, lse)
        ctx.cfg = (ignore_index, chunk_size, count, grad_buffer)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        ignore_index, chunk_size, count, grad_buffer = ctx.cfg
        hidden, weight, bias, labels, lse = ctx.saved_tensors
        if g.dtype != torch.float32:
            g = g.to(torch.float32)
        need_h, need_w, need_b = ctx.needs_input_grad[:3]
        need_b = bool(need_b and bias is not None)
        to_buffer = grad_buffer is not None and need_w
        # each output: True = allocate, False = not computed, a tensor = written (or, with
        # accumulate, added) in place. The accumulate flag covers grad_bias too, so with the
        # weight buffer the bias gradient is added into a zeroed tensor of its own.
        gb_spec = need_b
        if to_buffer and need_b:
            gb_spec = torch.zeros(bias.shape[0], dtype=torch.float32, device=bias.device)
        gh, gw, gb = flce_bwd(
            hidden, weight, labels, lse, bias, ignore_index=ignore_index, chunk_size=chunk_size,
            num_label_tokens=count, grad_output=g, accumulate=to_buffer,
            grad_hidden=bool(need_h), grad_weight=grad_buffer if to_buffer else bool(need_w),
            grad_bias=gb_spec)
        return (gh if need_h else None,
                None if (to_buffer or not need_w) else gw,
                gb if need_b else None,
                None, None, None, None, None)


def linear_cross_entropy(hidden, weight, labels, bias=None, *, mask=None,
                         ignore_index: int = -100, chunk_size: int = 1024,
                         num_label_tokens: int | None = None, reduction: str = "sum",
                         weight_grad_buffer=None):
    """Fused linear CE: loss of logits = hidden · weightᵀ (+ bias) without materialising them.
    hidden bf16 [..., H], weight bf16 [V, H], bias fp32 [V] or None, labels [...].

    The weight gradient is computed into an fp32 accumulator; autograd hands it to ``weight``
    in the weight's dtype. With ``weight_grad_buffer`` (fp32 [V, H]) it is instead added into
    that buffer and ``weight.grad`` is left alone (an fp32 main-gradient, or tied embeddings).
    reduction: "sum" or "mean" (per-row terms are not offered for the fused layer)."""
    _check_reduction(reduction, num_label_tokens, allowed=("sum", "mean"))
    if weight_grad_buffer is not None:
        if (weight_grad_buffer.dtype != torch.float32
                or tuple(weight_grad_buffer.shape) != tuple(weight.shape)
                or not weight_grad_buffer.is_contiguous()):
            raise ValueError("weight_grad_buffer must be a contiguous fp32 tensor of the "
                             "weight's shape")
    h = hidden.shape[-1]
    flat = hidden.reshape(-1, h)
    n = flat.shape[0]
    lab = _flat_labels(labels, mask, n, ignore_index)
    return _LinearCE.apply(flat, weight, bias, lab, int(ignore_index), int(chunk_size),
                           _normaliser(reduction, num_label_tokens), weight_grad_buffer)


class LinearCrossEntropy(torch.nn.Module):
    """Module form of :func:`linear_cross_entropy` (the weight and bias are passed in, as with
    a tied lm_head)."""

    def __init__(self, *, ignore_index: int = -100, chunk_size: int = 1024,
                 reduction: str = "sum"):
        super().__init__()
        _check_reduction(reduction, None, allowed=("sum", "mean"))
        self.ignore_index = ignore_index
        self.chunk_size = chunk_size
        self.reduction = reduction

    def forward(self, hidden, weight, labels, bias=None, mask=None, num_label_tokens=None,
                weight_grad_buffer=None):
        return linear_cross_entropy(hidden, weight, labels, bias, mask=mask,
                                    ignore_index=self.ignore_index, chunk_size=self.chunk_size,
                                    num_label_tokens=num_label_tokens, reduction=self.reduction,
                                    weight_grad_buffer=weight_grad_buffer)


def ce_chunked(logits, labels, *, mask=None, ignore_index: int = -100, chunk_size: int = 1024,
               num_label_tokens: int | None = None, inplace_grad: bool = False):
    """The masked CE loss under the name and defaults of the library's interface: the sum over
    labelled rows divided by T = num_label_tokens, or by the number of labelled rows (counted
    on the device) when it is None; gradient out of place unless inplace_grad=True."""
    if num_label_tokens is None:
        return masked_cross_entropy(logits, labels, mask=mask, ignore_index=ignore_index,
                                    chunk_size=chunk_size, reduction="mean",
                                    inplace_grad=inplace_grad)
    return masked_cross_entropy(logits, labels, mask=mask, ignore_index=ignore_index,
                                chunk_size=chunk_size, num_label_tokens=num_label_tokens,
                                reduction="sum", inplace_grad=inplace_grad)


def flce(hidden, weight, labels, bias=None, *, mask=None, ignore_index: int = -100,
         chunk_size: int = 1024, num_label_tokens: int | None = None, recompute: bool = True,
         weight_grad_buffer=None):
    """The fused linear CE loss under the name and defaults of the library's interface (T as in
    :func:`ce_chunked`). Under autograd the backward always rebuilds the logits from the saved
    lse (nothing of size [N, V] or [V, H] lives between forward and backward), i.e. the
    recomputing schedule; ``recompute=False`` (keep the fp32 slice, one logits product fewer)
    is the fused call ``flce_fwd_bwd`` when the upstream gradient is known, not an autograd
    schedule, and is refused here."""
    if not recompute:
        raise ValueError("flce under autograd always recomputes; call flce_fwd_bwd for the "
                         "stored-slice schedule")
    reduction = "mean" if num_label_tokens is None else "sum"
    return linear_cross_entropy(hidden, weight, labels, bias, mask=mask,
                                ignore_index=ignore_index, chunk_size=chunk_size,
                                num_label_tokens=num_label_tokens, reduction=reduction,
                                weight_grad_buffer=weight_grad_buffer)


# ---------------------------------------------------------------- embedding and layer norm

def _rows(t):
    """A 2-d tensor whose rows the kernels can walk: contiguous ones that do not share memory
    (an upstream gradient may be a broadcast)."""
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        return t.contiguous()
    return t


def _check_buffer(buffer, weight, dtypes=(torch.float32,)):
    if buffer is not None and (buffer.dtype not in dtypes
                               or tuple(buffer.shape) != tuple(weight.shape)
                               or not buffer.is_contiguous()):
        raise ValueError("weight_grad_buffer must be a contiguous tensor of the weight's shape, "
                         f"of type {' or '.join(str(d) for d in dtypes)}")


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, scale, ignore_index, grad_buffer):
        ctx.save_for_backward(tokens)
        ctx.cfg = (weight.shape[0], weight.dtype, scale, ignore_index, grad_buffer)
        return embed_fwd(_rows(weight), tokens, scale=scale, ignore_index=ignore_index)

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        (tokens,) = ctx.saved_tensors
        v, dtype, scale, ignore_index, buffer = ctx.cfg
        if buffer is not None:
            embed_bwd(_rows(g), tokens, v, scale=scale, ignore_index=ignore_index,
                      grad_weight=buffer, accumulate=True)
            return None, None, None, None, None
        grad = embed_bwd(_rows(g), tokens, v, scale=scale, ignore_index=ignore_index, dtype=dtype)
        return grad, None, None, None, None


def embedding(tokens, weight, *, scale: float = 1.0, ignore_index: int = -100,
              weight_grad_buffer=None):
    """scale · weight[tokens]: tokens [...] (int32 or int64), weight [V, H] in bf16, fp16 or fp32;
    zero rows without a gradient where the token is ``ignore_index`` or outside the table.

    With ``weight_grad_buffer`` (fp32 [V, H]) the table's gradient is added into that buffer and
    ``weight.grad`` is left alone, as in :func:`linear_cross_entropy`: a table tied to the head
    gives both functions the same buffer."""
    _check_buffer(weight_grad_buffer, weight)
    out = _Embedding.apply(weight, tokens.reshape(-1), float(scale), int(ignore_index),
                           weight_grad_buffer)
    return out.view(*tokens.shape, weight.shape[1])


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        x = _rows(x)
        y, mean, rstd = layernorm_fwd(x, weight, bias, eps=eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad[:3]
        gx, gw, gb = _layernorm_grads(g, x, mean, rstd, weight, need_x, need_w,
                                      ctx.bias_dtype if need_b else None, False)
        return gx, gw, gb, None


def _layernorm_grads(g, x, mean, rstd, weight, need_x, need_w, bias_dtype, in_place):
    """bias_dtype: None where the bias needs no gradient (a bias without a weight may be fp32
    beside 16-bit x)."""
    g = _rows(g)
    gb = bias_dtype is not None and torch.empty(x.shape[1], dtype=bias_dtype, device=x.device)
    return layernorm_bwd(g, x, mean, rstd, weight, grad_x=g if need_x and in_place else need_x,
                         grad_weight=need_w, grad_bias=gb)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., H] in bf16, fp16 or fp32; weight and bias [H]
    of x's type or fp32 (one type for both), or None."""
    h = x.shape[-1]
    return _LayerNorm.apply(x.reshape(-1, h), weight, bias, float(eps)).view(x.shape)


class LayerNorm(torch.nn.Module):
    """Module form of :func:`layer_norm` with the parameters of torch.nn.LayerNorm over one
    dimension."""

    def __init__(self, hidden: int, eps: float = 1e-5, *, bias: bool = True, device=None,
                 dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(hidden, device=device, dtype=dtype))
        self.bias = (torch.nn.Parameter(torch.zeros(hidden, device=device, dtype=dtype))
                     if bias else None)

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, eps=self.eps)


# ---------------------------------------------------------------- loss in pieces of the vocabulary

def _piece_grads(hidden, weights, biases, labels, lse, g, cfg, need_h, need_w, need_b):
    """(grad_hidden, [grad per weight], [grad per bias]) with cfg as _LinearCEPieces keeps it."""
    ignore_index, count, per_row, piece_size, buffers = cfg
    if g.dtype != torch.float32:
        g = g.to(torch.float32)
    if buffers is None:
        buffers = [None] * len(weights)
    into = [b is not None for b in buffers]  # a weight without a buffer gets its gradient as ever
    gws = [None] * len(weights)
    gbs = [None] * len(weights)
    for k, (w, need) in enumerate(zip(weights, need_w)):
        if need:
            gws[k] = buffers[k] if into[k] else torch.empty_like(
                w, memory_format=torch.contiguous_format)
    for k, (b, need) in enumerate(zip(biases, need_b)):
        if need:  # accumulating covers the bias too: beside a buffer its gradient is added to zeros
            make = torch.zeros_like if into[k] else torch.empty_like
            gbs[k] = make(b, memory_format=torch.contiguous_format)
    gh, _, _ = flce_pieces_bwd(
        hidden, weights, labels, lse, _any(biases), piece_size=piece_size,
        ignore_index=ignore_index, num_label_tokens=count, accumulate=into,
        grad_output=None if per_row else g, grad_rows=g.contiguous() if per_row else None,
        grad_hidden=bool(need_h), grad_weight=gws, grad_bias=_any(gbs) or False)
    return gh, [None if b else w for b, w in zip(into, gws)], gbs


class _LinearCEPieces(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, labels, cfg, pieces, *tensors):
        weights, biases = list(tensors[:pieces]), list(tensors[pieces:])
        ignore_index, count, per_row, _, _ = cfg
        loss, lse, rows = flce_pieces_fwd(
            hidden, weights, labels, _any(biases),
            ignore_index=ignore_index, num_label_tokens=count, return_rows=per_row)
        ctx.save_for_backward(hidden, labels, lse, *tensors)
        ctx.cfg, ctx.pieces = cfg, pieces
        return rows if per_row else loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        hidden, labels, lse, *tensors = ctx.saved_tensors
        k = ctx.pieces
        need = ctx.needs_input_grad
        gh, gws, gbs = _piece_grads(hidden, tensors[:k], tensors[k:], labels, lse, g, ctx.cfg,
                                    need[0], need[4:4 + k], need[4 + k:])
        return gh, None, None, None, *gws, *gbs


def _any(tensors):
    """The list, None where it holds nothing."""
    return tensors if any(t is not None for t in tensors) else None


def _piece_inputs(weight, bias, buffer):
    weights = list(weight) if isinstance(weight, (list, tuple)) else [weight]
    if not weights:
        raise ValueError("weight holds no pieces")
    biases = ([None] * len(weights) if bias is None
              else list(bias) if isinstance(bias, (list, tuple)) else [bias])
    if len(biases) != len(weights):
        raise ValueError(f"{len(weights)} weight pieces but {len(biases)} biases")
    buffers = None
    if buffer is not None:
        buffers = list(buffer) if isinstance(buffer, (list, tuple)) else [buffer]
        if len(buffers) != len(weights):
            raise ValueError(f"{len(weights)} weight pieces but {len(buffers)} buffers")
        for b, w in zip(buffers, weights):
            _check_buffer(b, w, (torch.float32, torch.bfloat16))
    return weights, biases, buffers


def linear_cross_entropy_pieces(hidden, weight, labels, bias=None, *, mask=None,
                                ignore_index: int = -100, num_label_tokens: int | None = None,
                                reduction: str = "sum", piece_size: int | None = None,
                                weight_grad_buffer=None):
    """:func:`linear_cross_entropy` over a weight in pieces of the vocabulary: one bf16 [V, H]
    tensor or a sequence of them holding consecutive classes (a base vocabulary and tokens added
    to it), with fp32 biases likewise (any of them None) or None. The backward takes
    ``piece_size`` classes at a time (default: so that their bf16 logit gradients stay within
    512 MiB, but at least 4096, 8 KiB a row) and leaves each weight's gradient in the weight's own type, without an fp32 [V, H]
    accumulator.

    reduction: "sum", "mean" or "none" (the per-row terms, 0 for rows without a label; minus a
    term is the log-probability of the row's label, with its gradient). Rows without a label take
    no part in any product. ``weight_grad_buffer`` (fp32 or bf16, a sequence where weight is one):
    the gradients are added into it and ``weight.grad`` is left alone; a weight whose entry in a
    sequence is None gets its gradient in ``weight.grad``."""
    _check_reduction(reduction, num_label_tokens)
    weights, biases, buffers = _piece_inputs(weight, bias, weight_grad_buffer)
    h = hidden.shape[-1]
    flat = hidden.reshape(-1, h)
    lab = _flat_labels(labels, mask, flat.shape[0], ignore_index)
    per_row = reduction == "none"
    cfg = (int(ignore_index), _normaliser(reduction, num_label_tokens), per_row, piece_size,
           buffers)
    out = _LinearCEPieces.apply(flat, lab, cfg, len(weights), *weights, *biases)
    return out.view(hidden.shape[:-1]) if per_row else out


class LinearCrossEntropyPieces(torch.nn.Module):
    """Module form of :func:`linear_cross_entropy_pieces` (weight and bias are passed in)."""

    def __init__(self, *, ignore_index: int = -100, reduction: str = "sum",
                 piece_size: int | None = None):
        super().__init__()
        _check_reduction(reduction, None)
        self.ignore_index = ignore_index
        self.reduction = reduction
        self.piece_size = piece_size

    def forward(self, hidden, weight, labels, bias=None, mask=None, num_label_tokens=None,
                weight_grad_buffer=None):
        return linear_cross_entropy_pieces(
            hidden, weight, labels, bias, mask=mask, ignore_index=self.ignore_index,
            num_label_tokens=num_label_tokens, reduction=self.reduction,
            piece_size=self.piece_size, weight_grad_buffer=weight_grad_buffer)


class _NormLinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_weight, norm_bias, labels, eps, cfg, pieces, *tensors):
        weights, biases = list(tensors[:pieces]), list(tensors[pieces:])
        ignore_index, count, per_row, _, _ = cfg
        x = _rows(x)
        y, mean, rstd = layernorm_fwd(x, norm_weight, norm_bias, eps=eps)
        loss, lse, rows = flce_pieces_fwd(
            y, weights, labels, _any(biases),
            ignore_index=ignore_index, num_label_tokens=count, return_rows=per_row)
        ctx.save_for_backward(x, norm_weight, norm_bias, mean, rstd, labels, lse, *tensors)
        ctx.cfg, ctx.pieces, ctx.eps = cfg, pieces, eps
        return rows if per_row else loss

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, nw, nb, mean, rstd, labels, lse, *tensors = ctx.saved_tensors
        k = ctx.pieces
        need = ctx.needs_input_grad
        norm_grads = any(need[:3])
        y, _, _ = layernorm_fwd(x, nw, nb, eps=ctx.eps, return_stats=False)
        gy, gws, gbs = _piece_grads(y, tensors[:k], tensors[k:], labels, lse, g, ctx.cfg,
                                    norm_grads, need[7:7 + k], need[7 + k:])
        del y
        gx = gnw = gnb = None
        if norm_grads:
            gx, gnw, gnb = _layernorm_grads(gy, x, mean, rstd, nw, need[0], need[1],
                                            nb.dtype if need[2] else None, True)
        return gx, gnw, gnb, None, None, None, None, *gws, *gbs


def norm_linear_cross_entropy(x, norm_weight, norm_bias, weight, labels, bias=None, *,
                              eps: float = 1e-5, mask=None, ignore_index: int = -100,
                              num_label_tokens: int | None = None, reduction: str = "sum",
                              piece_size: int | None = None, weight_grad_buffer=None):
    """:func:`layer_norm` of bf16 x [..., H], then :func:`linear_cross_entropy_pieces` of the
    result. Between forward and backward only x (which the model holds anyway) and three fp32
    values a row are kept: the backward normalises x again, and its hidden gradient becomes x's
    in place. A row without a label adds nothing to any gradient as long as its x is finite."""
    _check_reduction(reduction, num_label_tokens)
    weights, biases, buffers = _piece_inputs(weight, bias, weight_grad_buffer)
    flat = x.reshape(-1, x.shape[-1])
    lab = _flat_labels(labels, mask, flat.shape[0], ignore_index)
    per_row = reduction == "none"
    cfg = (int(ignore_index), _normaliser(reduction, num_label_tokens), per_row, piece_size,
           buffers)
    out = _NormLinearCE.apply(flat, norm_weight, norm_bias, lab, float(eps), cfg, len(weights),
                              *weights, *biases)
    return out.view(x.shape[:-1]) if per_row else out


class TiedHead(torch.nn.Module):
    """Both ends of a language model on one bf16 table [V, H]: ``embed`` looks tokens up,
    ``forward`` is the final norm and the loss against the same table (Liger-Kernel issue #941:
    lm_head.weight shared with embed_tokens). ``main_grad`` (fp32 [V, H], zeros, on request)
    collects both gradients of the table without a rounding between them, and ``weight.grad``
    stays None; without it autograd adds the two in bf16."""

    def __init__(self, vocab: int, hidden: int, *, scale: float = 1.0, eps: float = 1e-5,
                 ignore_index: int = -100, main_grad: bool = False, device=None):
        super().__init__()
        self.scale, self.ignore_index = scale, ignore_index
        self.weight = torch.nn.Parameter(
            torch.empty(vocab, hidden, device=device, dtype=torch.bfloat16))
        torch.nn.init.normal_(self.weight, std=0.02)
        self.norm = LayerNorm(hidden, eps, device=device, dtype=torch.bfloat16)
        self.register_buffer(
            "main_grad", torch.zeros(vocab, hidden, device=device, dtype=torch.float32)
            if main_grad else None, persistent=False)

    def embed(self, tokens):
        return embedding(tokens, self.weight, scale=self.scale, ignore_index=self.ignore_index,
                         weight_grad_buffer=self.main_grad)

    def forward(self, x, labels, mask=None, num_label_tokens=None, reduction: str = "mean"):
        return norm_linear_cross_entropy(
            x, self.norm.weight, self.norm.bias, self.weight, labels, eps=self.norm.eps,
            mask=mask, ignore_index=self.ignore_index, num_label_tokens=num_label_tokens,
            reduction=reduction, weight_grad_buffer=self.main_grad)
