"""The last step of a model that is served: its final norm and head in 8 bits, and beam search.

Argument marshalling only, over the library's calls (``rmsnorm_fp8_fwd``, ``fp8_matmul``,
``beam_step``, ``beam_reorder``); nothing here has gradients. Training keeps the weights in 16 bits
(``autograd.TiedHead``), and a head is laid out once for serving.
"""
from __future__ import annotations

import torch

from . import beam_reorder, beam_step, fp8_matmul, fp8_quantize, rmsnorm_fp8_fwd

__all__ = ["Fp8Head", "beam_reorder", "beam_step"]

_INTEGERS = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}  # by bytes


class Fp8Head(torch.nn.Module):
    """A final root-mean-square norm and a head [V, H] in 8 bits with a scale per 128 x 128 block
    (powers of two, or any number with ``scale_dtype=torch.float32``). ``weight`` in bf16, fp16 or
    fp32, H a multiple of 16; ``norm_weight`` [H] of the hidden states' type or fp32, or None;
    ``bias`` fp32 [V] or None (minus infinity bans a token). ``precise``: bf16 logits of more than 64
    rows from fp32 sums, as all others are (see :func:`fp8_matmul`). A cast of the module, or of a
    model that holds it, reaches ``norm_weight`` alone."""

    precise = False  # of a head that was pickled without it

    def __init__(self, weight, norm_weight=None, bias=None, *, eps: float = 1e-6,
                 scale_dtype=None, logits_dtype=torch.bfloat16, precise: bool = False):
        super().__init__()
        if weight.dim() != 2 or weight.shape[1] % 16:
            raise ValueError("weight must be [V, H] with H a multiple of 16, got "
                             f"{tuple(weight.shape)}")
        self.eps, self.logits_dtype, self.precise = eps, logits_dtype, precise
        q, scales = fp8_quantize(weight.detach().contiguous(), block_rows=128,
                                 scale_dtype=scale_dtype)
        self.register_buffer("weight", q)
        self.register_buffer("scales", scales)
        self.register_buffer("norm_weight", None if norm_weight is None
                             else norm_weight.detach().clone())
        self.register_buffer("bias", None if bias is None else bias.detach().clone())

    def _apply(self, fn, *args, **kw):
        """Moves are a module's; a cast, of this module or of a model around it, is for what follows
        the hidden states' type and leaves the 8-bit weight, its scales and the fp32 bias as they
        are. torch takes 8-bit numbers and exponent bytes for floating point, so they pass as
        integers."""
        held = {}
        for name in ("weight", "scales", "bias"):
            t = self._buffers[name]
            if t is not None:
                as_bits = t.view(_INTEGERS[t.element_size()])
                held[name], self._buffers[name] = (t.dtype, as_bits), as_bits
        try:
            return super()._apply(fn, *args, **kw)
        finally:
            for name, (dtype, as_bits) in held.items():
                t = self._buffers[name]
                if t.dtype != as_bits.dtype:  # Module.type casts integers as well
                    t = as_bits.to(t.device)
                self._buffers[name] = t.view(dtype)

    @classmethod
    def of(cls, head, **kw):
        """The serving form of an ``autograd.TiedHead(rms=True)``."""
        from .autograd import RMSNorm
        if not isinstance(head.norm, RMSNorm):
            raise ValueError("only a head with rms=True has an 8-bit form")
        return cls(head.weight, head.norm.weight, eps=head.norm.eps, **kw)

    @torch.no_grad()
    def forward(self, x, residual=None):
        """Logits [..., V] of hidden states [..., H] (of x + residual), and that sum: (logits, s)."""
        h = x.shape[-1]
        flat = x.reshape(-1, h)
        add = None if residual is None else residual.reshape(-1, h)
        q, c, s = rmsnorm_fp8_fwd(flat, self.norm_weight, add, eps=self.eps,
                                  scale_dtype=self.scales.dtype)
        z = fp8_matmul(q, c, self.weight, self.scales, self.bias, dtype=self.logits_dtype,
                       precise=self.precise)
        return z.view(*x.shape[:-1], z.shape[1]), s.view(x.shape)

    @torch.no_grad()
    def step(self, x, scores, residual=None, *, states=None, num=None, finished=None, eos=None,
             status=None):
        """One step of a beam search behind the last layer: x [batch, beams, H] -> what
        :func:`beam_step` returns. ``states`` (as many candidates as beams): tensors [batch, beams,
        ...] that are put in the order of their beams, in place."""
        z, _ = self(x, residual)
        got = beam_step(z, scores, num=num, finished=finished, eos=eos, status=status)
        if states:
            beam_reorder(states, got[1], out=states)
        return got
