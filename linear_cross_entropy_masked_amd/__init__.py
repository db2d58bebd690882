"""Thin Python binding of liblce_masked.so (the C-ABI in include/lce_masked.h).

Argument marshalling only: this module checks dtypes/devices, allocates outputs and the
workspace through PyTorch (device memory and streams are all PyTorch provides here), and
calls the C entry points of the same names on the current HIP stream. Every step of the loss
runs in the library's HIP kernels; there is no CPU or PyTorch fallback, and importing a
function whose library is missing raises.

Entry points (same names as the C ABI):
    ce_chunked_fwd, ce_chunked_bwd, ce_chunked_bwd_inplace, flce_fwd_bwd, flce_fwd, flce_bwd,
    flce_piece_fwd, flce_piece_loss, flce_piece_bwd, embed_fwd, embed_bwd, layernorm_fwd,
    layernorm_bwd,
    ce_chunked_workspace_size, flce_workspace_size, embed_workspace_size,
    layernorm_workspace_size, flce_piece_{fwd,loss,bwd}_workspace_size, lce_status_str
and over all pieces of a vocabulary: flce_pieces_fwd, flce_pieces_bwd
"""
from __future__ import annotations

import ctypes
import functools
import os

__all__ = [
    "LceError", "library_path", "load_library",
    "ce_chunked_workspace_size", "ce_chunked_fwd", "ce_chunked_bwd", "ce_chunked_bwd_inplace",
    "ce_chunked_fwd_bwd_inplace", "ce_chunked_fwd_bwd_inplace_noalloc", "ce_rows_fwd",
    "ce_rows_bwd", "LCE_NOALLOC_MAX_ROWS",
    "flce_workspace_size", "flce_fwd_bwd", "flce_fwd", "flce_bwd", "lce_status_str",
    "flce_status_str",
    "FLCE_RECOMPUTE", "FLCE_ACCUMULATE", "LCE_STATUS_BAD_LABEL",
    "flce_pieces_fwd", "flce_pieces_bwd", "flce_piece_fwd", "flce_piece_loss", "flce_piece_bwd",
    "flce_piece_fwd_workspace_size", "flce_piece_loss_workspace_size",
    "flce_piece_bwd_workspace_size", "FLCE_PIECE_FIRST", "FLCE_PIECE_LAST",
    "FLCE_PIECE_ACCUMULATE",
    "embed_fwd", "embed_workspace_size", "embed_bwd", "EMBED_ACCUMULATE", "LCE_STATUS_BAD_TOKEN",
    "layernorm_fwd", "layernorm_workspace_size", "layernorm_bwd", "LAYERNORM_ACCUMULATE",
    "LAYERNORM_MAX_H",
    "lce_timing_enable", "lce_timing_read",
]

FLCE_RECOMPUTE = 1
FLCE_ACCUMULATE = 2
LCE_STATUS_BAD_LABEL = 1
LCE_STATUS_BAD_TOKEN = 1
FLCE_PIECE_FIRST = 1
FLCE_PIECE_LAST = 2
FLCE_PIECE_ACCUMULATE = 4
EMBED_ACCUMULATE = 1
LAYERNORM_ACCUMULATE = 1
LAYERNORM_MAX_H = 32768
LCE_NOALLOC_MAX_ROWS = 1 << 20  # rows the allocation-free CE step's static scratch holds

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class LceError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed with status {code}: {lce_status_str(code)}")
        self.code = code


def library_path() -> str:
    return os.environ.get("LCE_MASKED_LIB", os.path.join(_PKG, "liblce_masked.so"))


def load_library() -> ctypes.CDLL:
    """Load (once) and return the C-ABI library; raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -m linear_cross_entropy_masked_amd.build` "
            "(the HIP library is the only implementation; there is no fallback)")
    lib = ctypes.CDLL(path)
    i64, i32, u32, sz, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_void_p
    f32, dt = ctypes.c_float, ctypes.c_int
    psz = ctypes.POINTER(ctypes.c_size_t)
    sigs = {
        "lce_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "flce_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "ce_chunked_workspace_size": (ctypes.c_int, [i64, i64, i64, psz]),
        "ce_chunked_fwd": (ctypes.c_int, [vp, i64, i64, i64, vp, i32, i64, i64, vp, vp, vp, vp, sz, vp]),
        "ce_chunked_bwd": (ctypes.c_int, [vp, i64, i64, i64, vp, i64, vp, i32, i64, i64, vp, vp, vp, vp, sz, vp]),
        "ce_chunked_bwd_inplace": (ctypes.c_int, [vp, i64, i64, i64, vp, i32, i64, i64, vp, vp, vp, vp, sz, vp]),
        "ce_chunked_fwd_bwd_inplace": (ctypes.c_int, [vp, i64, i64, i64, vp, i32, i64, i64, vp, vp, vp,
                                                      vp, vp, sz, vp]),
        "ce_chunked_fwd_bwd_inplace_noalloc": (ctypes.c_int, [vp, i64, i64, i64, vp, i32, i64, i64,
                                                              vp, vp, vp, vp, vp]),
        "ce_rows_fwd": (ctypes.c_int, [vp, i64, i64, i64, vp, i32, i64, vp, vp, vp, vp, sz, vp]),
        "ce_rows_bwd": (ctypes.c_int, [vp, i64, i64, i64, vp, i64, vp, i32, i64, vp, vp, vp, vp, sz,
                                       vp]),
        "flce_workspace_size": (ctypes.c_int, [i64, i64, i64, i64, u32, psz]),
        "flce_fwd_bwd": (ctypes.c_int, [vp, vp, vp, vp, i64, i64, i64, i32, i64, i64, u32, vp, vp, vp,
                                        vp, vp, vp, vp, vp, sz, vp]),
        "flce_fwd": (ctypes.c_int, [vp, vp, vp, vp, i64, i64, i64, i32, i64, i64, vp, vp, vp, vp,
                                    sz, vp]),
        "flce_bwd": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, i64, i64, i32, i64, i64, u32, vp, vp,
                                    vp, vp, vp, vp, sz, vp]),
        "flce_piece_fwd_workspace_size": (ctypes.c_int, [i64, i64, i64, psz]),
        "flce_piece_loss_workspace_size": (ctypes.c_int, [i64, psz]),
        "flce_piece_bwd_workspace_size": (ctypes.c_int, [i64, i64, i64, psz]),
        "flce_piece_fwd": (ctypes.c_int, [vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, u32, vp, vp,
                                          sz, vp]),
        "flce_piece_loss": (ctypes.c_int, [vp, vp, i64, i64, i32, i64, vp, vp, vp, vp, vp, sz, vp]),
        "flce_piece_bwd": (ctypes.c_int, [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i32, i64, u32,
                                          vp, vp, vp, vp, vp, dt, vp, vp, sz, vp]),
        "embed_fwd": (ctypes.c_int, [vp, dt, i64, i64, i64, vp, i64, i32, f32, vp, i64, vp, vp]),
        "embed_workspace_size": (ctypes.c_int, [i64, i64, i64, psz]),
        "embed_bwd": (ctypes.c_int, [vp, dt, i64, vp, i64, i64, i64, i32, f32, u32, vp, dt, i64, vp,
                                     vp, sz, vp]),
        "layernorm_fwd": (ctypes.c_int, [vp, dt, i64, i64, i64, vp, vp, dt, f32, vp, i64, vp, vp,
                                         vp]),
        "layernorm_workspace_size": (ctypes.c_int, [i64, i64, psz]),
        "layernorm_bwd": (ctypes.c_int, [vp, dt, i64, vp, i64, vp, vp, vp, dt, i64, i64, u32, vp,
                                         i64, vp, vp, dt, vp, sz, vp]),
        "lce_timing_enable": (ctypes.c_int, [ctypes.c_int]),
        "lce_timing_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                           ctypes.POINTER(ctypes.c_double),
                                           ctypes.POINTER(ctypes.c_longlong),
                                           ctypes.POINTER(ctypes.c_int)]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _LIB = lib
    return lib


def lce_status_str(code: int) -> str:
    return load_library().lce_status_str(int(code)).decode()


def flce_status_str(code: int) -> str:
    return load_library().flce_status_str(int(code)).decode()


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise LceError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require(t, name, dtype, dims, device=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimension(s), got shape {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _labels_i32(labels, n, device, ignore_index=-100):
    """int32 labels for the C ABI. An int64 label outside the int32 range is not a vocabulary
    index: it becomes a negative value other than ignore_index, so the library flags it
    (LCE_STATUS_BAD_LABEL) and treats the row as unlabelled instead of wrapping it onto a
    class."""
    import torch
    _require(labels, "labels", None, 1, device)
    if labels.shape[0] != n:
        raise ValueError(f"labels has {labels.shape[0]} entries, expected {n}")
    if labels.dtype == torch.int64:
        bad = -1 if int(ignore_index) != -1 else -2
        wide = (labels > 2 ** 31 - 1) | (labels < -(2 ** 31))
        labels = torch.where(wide, torch.full_like(labels, bad), labels).to(torch.int32)
    elif labels.dtype != torch.int32:
        raise TypeError("labels must be int32 or int64")
    return labels.contiguous()


def _require_lse(lse, n, device):
    import torch
    _require(lse, "lse", torch.float32, 1, device)
    if lse.shape[0] != n or (n > 1 and lse.stride(0) != 1):
        raise ValueError(f"lse must be a contiguous float32 [{n}] tensor, got shape "
                         f"{tuple(lse.shape)} stride {tuple(lse.stride())}")


def _workspace(nbytes, device, workspace=None):
    import torch
    if workspace is not None:
        if workspace.device != device or workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace must hold at least {nbytes} bytes on {device}")
        return workspace
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def _count_arg(num_label_tokens):
    return -1 if num_label_tokens is None else int(num_label_tokens)


def ce_chunked_workspace_size(n: int, v: int, chunk_size: int) -> int:
    out = ctypes.c_size_t()
    _check("ce_chunked_workspace_size",
           load_library().ce_chunked_workspace_size(n, v, chunk_size, ctypes.byref(out)))
    return out.value


def flce_workspace_size(n: int, h: int, v: int, chunk_size: int, flags: int = 0) -> int:
    out = ctypes.c_size_t()
    _check("flce_workspace_size",
           load_library().flce_workspace_size(n, h, v, chunk_size, flags, ctypes.byref(out)))
    return out.value


def _logits_2d(logits):
    import torch
    _require(logits, "logits", torch.bfloat16, 2)
    n, v = logits.shape
    if n == 0 or v == 0:
        return n, v, v
    if logits.stride(1) != 1 and v > 1:
        raise ValueError("logits rows must be contiguous (stride(1) == 1)")
    return n, v, (logits.stride(0) if n > 1 else v)


def ce_chunked_fwd(logits, labels, *, ignore_index: int = -100, chunk_size: int = 1024,
                   num_label_tokens: int | None = None, return_lse: bool = True,
                   status=None, workspace=None):
    """Sum-reduced masked CE forward. Returns (loss fp32 0-d tensor, lse fp32 [n] or None)."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    nbytes = ce_chunked_workspace_size(n, v, chunk_size)
    ws = _workspace(nbytes, dev, workspace)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev) if return_lse else None
    _check("ce_chunked_fwd", lib.ce_chunked_fwd(
        _ptr(logits), n, v, ld, _ptr(labels), ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(loss), _ptr(lse), _ptr(status), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return loss, lse


def ce_chunked_bwd(logits, labels, *, out=None, ignore_index: int = -100, chunk_size: int = 1024,
                   num_label_tokens: int | None = None, grad_output=None, lse=None, status=None,
                   workspace=None):
    """Out-of-place backward: returns grad (bf16, shape of logits); logits are left intact."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    if out is None:
        out = torch.empty((n, v), dtype=torch.bfloat16, device=dev)
    _require(out, "out", torch.bfloat16, 2, dev)
    if tuple(out.shape) != (n, v) or (n > 0 and v > 1 and out.stride(1) != 1):
        raise ValueError("out must be [n, v] bf16 with contiguous rows")
    ldg = out.stride(0) if n > 1 else v
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    if lse is not None:
        _require_lse(lse, n, dev)
    ws = _workspace(ce_chunked_workspace_size(n, v, chunk_size), dev, workspace)
    _check("ce_chunked_bwd", lib.ce_chunked_bwd(
        _ptr(logits), n, v, ld, _ptr(out), ldg, _ptr(labels), ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(grad_output), _ptr(lse), _ptr(status), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return out


def ce_chunked_bwd_inplace(logits, labels, *, ignore_index: int = -100, chunk_size: int = 1024,
                           num_label_tokens: int | None = None, grad_output=None, lse=None,
                           status=None, workspace=None):
    """In-place backward: overwrites ``logits`` with the gradient and returns it."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    if lse is not None:
        _require_lse(lse, n, dev)
    ws = _workspace(ce_chunked_workspace_size(n, v, chunk_size), dev, workspace)
    _check("ce_chunked_bwd_inplace", lib.ce_chunked_bwd_inplace(
        _ptr(logits), n, v, ld, _ptr(labels), ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(grad_output), _ptr(lse), _ptr(status), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return logits


def ce_chunked_fwd_bwd_inplace(logits, labels, *, ignore_index: int = -100,
                               chunk_size: int = 1024, num_label_tokens: int | None = None,
                               grad_output=None, return_lse: bool = False, status=None,
                               workspace=None):
    """Forward and in-place backward in one call (the upstream gradient is known now).

    Overwrites ``logits`` with the gradient; returns (loss fp32 0-d tensor, lse fp32 [n] or
    None). Bitwise equal to ``ce_chunked_fwd`` followed by ``ce_chunked_bwd_inplace``."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    ws = _workspace(ce_chunked_workspace_size(n, v, chunk_size), dev, workspace)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev) if return_lse else None
    _check("ce_chunked_fwd_bwd_inplace", lib.ce_chunked_fwd_bwd_inplace(
        _ptr(logits), n, v, ld, _ptr(labels), ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(grad_output), _ptr(loss), _ptr(lse), _ptr(status),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return loss, lse


def ce_chunked_fwd_bwd_inplace_noalloc(logits, labels, *, ignore_index: int = -100,
                                       chunk_size: int = 1024,
                                       num_label_tokens: int | None = None, grad_output=None,
                                       loss=None, lse=None, status=None):
    """:func:`ce_chunked_fwd_bwd_inplace` without a workspace: the library keeps the step's
    O(n) scratch in a static per-GPU array (n <= LCE_NOALLOC_MAX_ROWS). Pass ``loss`` (fp32
    0-d) and optionally ``lse`` (fp32 [n]) to have nothing allocated here either; calls that
    may overlap on one GPU must be serialised by the caller. Returns (loss, lse)."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    if loss is None:
        loss = torch.empty((), dtype=torch.float32, device=dev)
    _require(loss, "loss", torch.float32, 0, dev)
    if lse is not None:
        _require_lse(lse, n, dev)
    _check("ce_chunked_fwd_bwd_inplace_noalloc", lib.ce_chunked_fwd_bwd_inplace_noalloc(
        _ptr(logits), n, v, ld, _ptr(labels), ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(grad_output), _ptr(loss), _ptr(lse), _ptr(status),
        _stream(dev)))
    return loss, lse


def ce_rows_fwd(logits, labels, *, ignore_index: int = -100, chunk_size: int = 1024,
                return_lse: bool = True, status=None, workspace=None):
    """Unreduced forward. Returns (row_loss fp32 [n], lse fp32 [n] or None); rows without a
    label get 0."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    ws = _workspace(ce_chunked_workspace_size(n, v, chunk_size), dev, workspace)
    rows = torch.empty(n, dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev) if return_lse else None
    _check("ce_rows_fwd", lib.ce_rows_fwd(
        _ptr(logits), n, v, ld, _ptr(labels), ignore_index, chunk_size, _ptr(rows), _ptr(lse),
        _ptr(status), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return rows, lse


def ce_rows_bwd(logits, labels, grad_rows, *, out=None, inplace: bool = False,
                ignore_index: int = -100, chunk_size: int = 1024, lse=None, status=None,
                workspace=None):
    """Unreduced backward: row i of the result is grad_rows[i] · (softmax − onehot). With
    ``inplace`` the gradient overwrites ``logits``; otherwise it goes to ``out`` (or a new
    tensor)."""
    import torch
    lib = load_library()
    n, v, ld = _logits_2d(logits)
    dev = logits.device
    labels = _labels_i32(labels, n, dev, ignore_index)
    _require(grad_rows, "grad_rows", torch.float32, 1, dev)
    if grad_rows.numel() != n or (n > 1 and grad_rows.stride(0) != 1):
        raise ValueError("grad_rows must be a contiguous fp32 [n] tensor")
    if lse is not None:
        _require_lse(lse, n, dev)
    if inplace:
        out, ldg = logits, ld
    else:
        if out is None:
            out = torch.empty((n, v), dtype=torch.bfloat16, device=dev)
        _require(out, "out", torch.bfloat16, 2, dev)
        if tuple(out.shape) != (n, v) or (n > 0 and v > 1 and out.stride(1) != 1):
            raise ValueError("out must be [n, v] bf16 with contiguous rows")
        ldg = out.stride(0) if n > 1 else v
    ws = _workspace(ce_chunked_workspace_size(n, v, chunk_size), dev, workspace)
    _check("ce_rows_bwd", lib.ce_rows_bwd(
        _ptr(logits), n, v, ld, _ptr(out), ldg, _ptr(labels), ignore_index, chunk_size,
        _ptr(grad_rows), _ptr(lse), _ptr(status), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(dev)))
    return out


def flce_fwd_bwd(hidden, weight, labels, bias=None, *, ignore_index: int = -100,
                 chunk_size: int = 1024, num_label_tokens: int | None = None,
                 recompute: bool = False, accumulate: bool = False, grad_output=None,
                 grad_hidden=True, grad_weight=True, grad_bias=None, return_lse=False,
                 status=None, workspace=None):
    """Fused linear CE forward+backward.

    ``grad_hidden`` / ``grad_weight`` / ``grad_bias``: True to allocate, False/None to skip, or
    a tensor to write into (required for ``accumulate``). grad_bias defaults to True when a
    bias is given. Returns (loss, grad_hidden, grad_weight, grad_bias, lse).
    """
    import torch
    lib = load_library()
    _require(hidden, "hidden", torch.bfloat16, 2)
    dev = hidden.device
    _require(weight, "weight", torch.bfloat16, 2, dev)
    n, h = hidden.shape
    v, h2 = weight.shape
    if h2 != h:
        raise ValueError(f"hidden has {h} columns but weight has {h2}")
    hidden = hidden.contiguous()
    weight = weight.contiguous()
    labels = _labels_i32(labels, n, dev, ignore_index)
    if bias is not None:
        _require(bias, "bias", torch.float32, 1, dev)
        if bias.shape[0] != v:
            raise ValueError("bias must have v entries")
        bias = bias.contiguous()
    if grad_bias is None:
        grad_bias = bias is not None
    flags = (FLCE_RECOMPUTE if recompute else 0) | (FLCE_ACCUMULATE if accumulate else 0)

    def out(spec, shape, dtype, name):
        if spec is True:
            if accumulate and name != "grad_hidden":
                raise ValueError(f"accumulate=True needs an existing {name} tensor")
            return torch.empty(shape, dtype=dtype, device=dev)
        if spec is False or spec is None:
            return None
        _require(spec, name, dtype, len(shape), dev)
        if tuple(spec.shape) != tuple(shape) or not spec.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor")
        return spec

    gh = out(grad_hidden, (n, h), torch.bfloat16, "grad_hidden")
    gw = out(grad_weight, (v, h), torch.float32, "grad_weight")
    gb = out(grad_bias, (v,), torch.float32, "grad_bias")
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev) if return_lse else None
    ws = _workspace(flce_workspace_size(n, h, v, chunk_size, flags), dev, workspace)
    _check("flce_fwd_bwd", lib.flce_fwd_bwd(
        _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(labels), n, h, v, ignore_index, chunk_size,
        _count_arg(num_label_tokens), flags, _ptr(grad_output), _ptr(loss), _ptr(lse), _ptr(gh),
        _ptr(gw), _ptr(gb), _ptr(status), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(dev)))
    return loss, gh, gw, gb, lse


def _flce_inputs(hidden, weight, labels, bias, ignore_index):
    import torch
    _require(hidden, "hidden", torch.bfloat16, 2)
    dev = hidden.device
    _require(weight, "weight", torch.bfloat16, 2, dev)
    n, h = hidden.shape
    v, h2 = weight.shape
    if h2 != h:
        raise ValueError(f"hidden has {h} columns but weight has {h2}")
    labels = _labels_i32(labels, n, dev, ignore_index)
    if bias is not None:
        _require(bias, "bias", torch.float32, 1, dev)
        if bias.shape[0] != v:
            raise ValueError("bias must have v entries")
        bias = bias.contiguous()
    return hidden.contiguous(), weight.contiguous(), labels, bias, dev, n, h, v


def flce_fwd(hidden, weight, labels, bias=None, *, ignore_index: int = -100,
             chunk_size: int = 1024, num_label_tokens: int | None = None, status=None,
             workspace=None):
    """Fused linear CE forward only. Returns (loss, lse); keep lse for :func:`flce_bwd`."""
    import torch
    lib = load_library()
    hidden, weight, labels, bias, dev, n, h, v = _flce_inputs(
        hidden, weight, labels, bias, ignore_index)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev)
    ws = _workspace(flce_workspace_size(n, h, v, chunk_size, 0), dev, workspace)
    _check("flce_fwd", lib.flce_fwd(
        _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(labels), n, h, v, ignore_index, chunk_size,
        _count_arg(num_label_tokens), _ptr(loss), _ptr(lse), _ptr(status), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(dev)))
    return loss, lse


def flce_bwd(hidden, weight, labels, lse, bias=None, *, ignore_index: int = -100,
             chunk_size: int = 1024, num_label_tokens: int | None = None,
             accumulate: bool = False, grad_output=None, grad_hidden=True, grad_weight=True,
             grad_bias=None, status=None, workspace=None):
    """Fused linear CE backward from :func:`flce_fwd`'s lse (the logits are recomputed).
    Output arguments as in :func:`flce_fwd_bwd`. Returns (grad_hidden, grad_weight, grad_bias)."""
    import torch
    lib = load_library()
    hidden, weight, labels, bias, dev, n, h, v = _flce_inputs(
        hidden, weight, labels, bias, ignore_index)
    _require(lse, "lse", torch.float32, 1, dev)
    if lse.shape[0] != n or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous [n] float32 tensor")
    if grad_bias is None:
        grad_bias = bias is not None
    flags = FLCE_ACCUMULATE if accumulate else 0

    def out(spec, shape, dtype, name):
        if spec is True:
            if accumulate and name != "grad_hidden":
                raise ValueError(f"accumulate=True needs an existing {name} tensor")
            return torch.empty(shape, dtype=dtype, device=dev)
        if spec is False or spec is None:
            return None
        _require(spec, name, dtype, len(shape), dev)
        if tuple(spec.shape) != tuple(shape) or not spec.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor")
        return spec

    gh = out(grad_hidden, (n, h), torch.bfloat16, "grad_hidden")
    gw = out(grad_weight, (v, h), torch.float32, "grad_weight")
    gb = out(grad_bias, (v,), torch.float32, "grad_bias")
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    ws = _workspace(flce_workspace_size(n, h, v, chunk_size, flags), dev, workspace)
    _check("flce_bwd", lib.flce_bwd(
        _ptr(hidden), _ptr(weight), _ptr(bias), _ptr(labels), _ptr(lse), n, h, v, ignore_index,
        chunk_size, _count_arg(num_label_tokens), flags, _ptr(grad_output), _ptr(gh), _ptr(gw),
        _ptr(gb), _ptr(status), _ptr(ws), ws.numel() * ws.element_size(), _stream(dev)))
    return gh, gw, gb


_FNS: dict = {}  # C entry points looked up so far


@functools.lru_cache(maxsize=512)
def _size(fn, *args):
    """A workspace size: a function of its arguments alone."""
    out = ctypes.c_size_t()
    _check(fn, getattr(load_library(), fn)(*args, ctypes.byref(out)))
    return out.value


def _call(fn, device, *args):
    """fn(*args) with ``device`` current (the library checks and launches on the current one);
    raises on a status code. The stream, the last argument, is the caller's current one there."""
    import torch
    f = _FNS.get(fn)
    if f is None:
        f = _FNS[fn] = getattr(load_library(), fn)
    index = device.index
    if index == torch.cuda.current_device():
        code = f(*args, _raw_stream(torch, index))
    else:
        with torch.cuda.device(device):
            code = f(*args, _raw_stream(torch, index))
    if code != 0:
        raise LceError(fn, code)


def _raw_stream(torch, index):
    """The current stream's handle; without building a Stream object where torch lets us, which
    takes 2 us, a sixth of a small call."""
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


def _adr(t):
    return None if t is None else t.data_ptr()


_DTYPE_CODES: dict = {}


def _dtype_code(dtype, name):
    code = _DTYPE_CODES.get(dtype)
    if code is None:
        import torch
        _DTYPE_CODES.update({torch.bfloat16: 0, torch.float16: 1, torch.float32: 2})
        code = _DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {dtype}")
    return code


def _rows_2d(t, name, dtype=None, shape=None, device=None):
    """The row stride of a 2-d tensor whose rows are contiguous."""
    _require(t, name, dtype, 2, device)
    n, h = t.shape
    if shape is not None and (n, h) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {(n, h)}")
    ld, step = t.stride()
    if step != 1 and h > 1 and n > 0:
        raise ValueError(f"{name} rows must be contiguous (stride(1) == 1)")
    return ld if n > 1 else h


def _status_ptr(status, device):
    if status is None:
        return None
    import torch
    _require(status, "status", torch.int32, status.dim(), device)
    if status.numel() < 1:
        raise ValueError("status must hold one int32")
    return status.data_ptr()


def _bytes_of(workspace):
    return workspace.numel() * workspace.element_size()


def embed_fwd(weight, tokens, *, scale: float = 1.0, ignore_index: int = -100, out=None,
              status=None):
    """Embedding lookup: row i of the result is scale · weight[tokens[i]], 0 where the token is
    ``ignore_index`` or outside the table (then LCE_STATUS_BAD_TOKEN is set in ``status``).
    weight bf16 / fp16 / fp32 [v, h], tokens int32 or int64 [n]; returns ``out`` [n, h]."""
    import torch
    code = _dtype_code(getattr(weight, "dtype", None), "weight")
    ldw = _rows_2d(weight, "weight")
    dev = weight.device
    v, h = weight.shape
    tokens = _tokens_i32(tokens, dev, ignore_index)
    n = tokens.shape[0]
    if out is None:
        out, ldo = weight.new_empty((n, h)), h
    else:
        ldo = _rows_2d(out, "out", weight.dtype, (n, h), dev)
    _call("embed_fwd", dev, weight.data_ptr(), code, v, h, ldw, tokens.data_ptr(), n,
          ignore_index, scale, out.data_ptr(), ldo, _status_ptr(status, dev))
    return out


def _ignore_arg(ignore_index):
    """ignore_index for the C ABI: one outside int32 would wrap onto a class."""
    if not -(2 ** 31) <= ignore_index < 2 ** 31:
        raise ValueError(f"ignore_index must fit in 32 bits, got {ignore_index}")
    return ignore_index


def _tokens_i32(tokens, device, ignore_index):
    import torch
    _ignore_arg(ignore_index)
    _require(tokens, "tokens", None, 1, device)
    if tokens.dtype == torch.int32:
        return tokens.contiguous()
    if tokens.dtype != torch.int64:
        raise TypeError("tokens must be int32 or int64")
    return _labels_i32(tokens, tokens.shape[0], device, ignore_index)


def embed_workspace_size(n: int, h: int, v: int) -> int:
    return _size("embed_workspace_size", n, h, v)


def embed_bwd(grad, tokens, num_embeddings: int, *, scale: float = 1.0, ignore_index: int = -100,
              grad_weight=None, dtype=None, accumulate: bool = False, status=None,
              workspace=None):
    """Gradient of :func:`embed_fwd` for its table: row v of the result is scale times the sum of
    the rows of ``grad`` [n, h] whose token is v, summed in fp32 in a fixed order. Written to
    ``grad_weight`` [num_embeddings, h] (added to it with ``accumulate``), or to a new tensor of
    ``dtype`` (default: grad's). Its type is grad's or float32."""
    import torch
    code = _dtype_code(getattr(grad, "dtype", None), "grad")
    ldg = _rows_2d(grad, "grad")
    dev = grad.device
    n, h = grad.shape
    v = int(num_embeddings)
    tokens = _tokens_i32(tokens, dev, ignore_index)
    if tokens.shape[0] != n:
        raise ValueError(f"tokens has {tokens.shape[0]} entries, expected {n}")
    if grad_weight is None:
        if accumulate:
            raise ValueError("accumulate=True needs an existing grad_weight tensor")
        grad_weight, ldw = torch.empty((v, h), dtype=dtype or grad.dtype, device=dev), h
    elif dtype is not None and grad_weight.dtype != dtype:
        raise TypeError(f"grad_weight must be {dtype}, got {grad_weight.dtype}")
    else:
        ldw = _rows_2d(grad_weight, "grad_weight", None, (v, h), dev)
    ws = _workspace(embed_workspace_size(n, h, v), dev, workspace)
    _call("embed_bwd", dev, grad.data_ptr(), code, ldg, tokens.data_ptr(), n, h, v, ignore_index,
          scale, EMBED_ACCUMULATE if accumulate else 0, grad_weight.data_ptr(),
          _dtype_code(grad_weight.dtype, "grad_weight"), ldw, _status_ptr(status, dev),
          ws.data_ptr(), _bytes_of(ws))
    return grad_weight


def _empty_rows(x):
    """A new contiguous tensor of x's shape and type (empty_like is the cheapest call that makes
    one, 1.2 us)."""
    import torch
    return torch.empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def _norm_param(t, name, h, device):
    _require(t, name, None, 1, device)
    if t.shape[0] != h:
        raise ValueError(f"{name} must have {h} entries, got {t.shape[0]}")
    return t.contiguous()


def layernorm_fwd(x, weight=None, bias=None, *, eps: float = 1e-5, out=None,
                  return_stats: bool = True):
    """Layer norm over the last dimension of x [n, h] (bf16 / fp16 / fp32). weight and bias: [h],
    of x's type or float32 (both the same type), or None. ``out`` may be x itself. Returns
    (y, mean, rstd), the fp32 [n] statistics None without ``return_stats``."""
    import torch
    code = _dtype_code(getattr(x, "dtype", None), "x")
    ldx = _rows_2d(x, "x")
    dev = x.device
    n, h = x.shape
    pdtype = x.dtype
    if weight is not None:
        weight = _norm_param(weight, "weight", h, dev)
        pdtype = weight.dtype
    if bias is not None:
        bias = _norm_param(bias, "bias", h, dev)
        if weight is not None and bias.dtype != pdtype:
            raise TypeError(f"bias is {bias.dtype}, weight {pdtype}: they must be of one type")
        pdtype = bias.dtype
    if out is None:
        out, ldy = _empty_rows(x), h
    else:
        ldy = _rows_2d(out, "out", x.dtype, (n, h), dev)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(n, dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
    _call("layernorm_fwd", dev, x.data_ptr(), code, n, h, ldx, _adr(weight), _adr(bias),
          _dtype_code(pdtype, "weight"), eps, out.data_ptr(), ldy, _adr(mean), _adr(rstd))
    return out, mean, rstd


def layernorm_workspace_size(n: int, h: int) -> int:
    return _size("layernorm_workspace_size", n, h)


def layernorm_bwd(grad, x, mean, rstd, weight=None, *, grad_x=True, grad_weight=None,
                  grad_bias=None, accumulate: bool = False, workspace=None):
    """Gradients of :func:`layernorm_fwd` from its x and statistics. ``grad_x`` /
    ``grad_weight`` / ``grad_bias``: True to allocate (the parameter gradients in the weight's
    type), False to skip, or a tensor to write into (grad_x may be ``grad`` itself; the
    parameter gradients may be float32, and are added to with ``accumulate``). grad_weight
    defaults to True when a weight is given, grad_bias to False. Returns (grad_x, grad_weight,
    grad_bias)."""
    import torch
    code = _dtype_code(getattr(x, "dtype", None), "x")
    ldx = _rows_2d(x, "x")
    dev = x.device
    n, h = x.shape
    ldg = _rows_2d(grad, "grad", x.dtype, (n, h), dev)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _require(t, name, torch.float32, 1, dev)
        if t.shape[0] != n or (n > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous float32 [{n}] tensor")
    pdtype = x.dtype
    if weight is not None:
        weight = _norm_param(weight, "weight", h, dev)
        pdtype = weight.dtype
    if grad_weight is None:
        grad_weight = weight is not None

    def param_out(spec, name):
        if spec is True:
            if accumulate:
                raise ValueError(f"accumulate=True needs an existing {name} tensor")
            return x.new_empty(h) if weight is None else torch.empty_like(weight)
        if spec is False or spec is None:
            return None
        _require(spec, name, None, 1, dev)
        if spec.shape[0] != h or (h > 1 and spec.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous [{h}] tensor")
        return spec

    lddx = h
    if grad_x is True:
        grad_x = _empty_rows(x)
    elif grad_x is False:
        grad_x = None
    elif grad_x is not None:
        lddx = _rows_2d(grad_x, "grad_x", x.dtype, (n, h), dev)
    gw, gb = param_out(grad_weight, "grad_weight"), param_out(grad_bias, "grad_bias")
    if gw is not None and gb is not None and gw.dtype != gb.dtype:
        raise TypeError("grad_weight and grad_bias must be of one type")
    gdtype = gw.dtype if gw is not None else gb.dtype if gb is not None else pdtype
    ws = None
    if gw is not None or gb is not None:
        ws = _workspace(layernorm_workspace_size(n, h), dev, workspace)
    _call("layernorm_bwd", dev, grad.data_ptr(), code, ldg, x.data_ptr(), ldx, mean.data_ptr(),
          rstd.data_ptr(), _adr(weight), _dtype_code(pdtype, "weight"), n, h,
          LAYERNORM_ACCUMULATE if accumulate else 0, _adr(grad_x), lddx, _adr(gw), _adr(gb),
          _dtype_code(gdtype, "grad_weight"), _adr(ws), 0 if ws is None else _bytes_of(ws))
    return grad_x, gw, gb


def flce_piece_fwd_workspace_size(n: int, h: int, v: int) -> int:
    return _size("flce_piece_fwd_workspace_size", n, h, v)


def flce_piece_loss_workspace_size(n: int) -> int:
    return _size("flce_piece_loss_workspace_size", n)


def flce_piece_bwd_workspace_size(n: int, h: int, v: int) -> int:
    return _size("flce_piece_bwd_workspace_size", n, h, v)


def _piece_weight(weight, bias, h, dev):
    import torch
    _require(weight, "weight", torch.bfloat16, 2, dev)
    v, h2 = weight.shape
    if h2 != h:
        raise ValueError(f"hidden has {h} columns but weight has {h2}")
    if bias is not None:
        _require(bias, "bias", torch.float32, 1, dev)
        if bias.shape[0] != v:
            raise ValueError("bias must have one entry per row of weight")
        bias = bias.contiguous()
    return weight.contiguous(), bias, v


def _contiguous_f32(t, name, shape, device):
    import torch
    _require(t, name, torch.float32, len(shape), device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)}")
    return t


def _piece_fwd(hidden, weight, bias, labels, state, n, h, v, v_start, vocab, first, ignore_index,
               ws, dev):
    _call("flce_piece_fwd", dev, hidden.data_ptr(), weight.data_ptr(), _adr(bias),
          labels.data_ptr(), n, h, v, v_start, vocab, ignore_index,
          FLCE_PIECE_FIRST if first else 0, state.data_ptr(), ws.data_ptr(), _bytes_of(ws))


def _piece_loss(state, labels, n, vocab, ignore_index, num_label_tokens, return_rows, status, ws,
                dev):
    import torch
    loss = torch.empty((), dtype=torch.float32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev)
    rows = torch.empty(n, dtype=torch.float32, device=dev) if return_rows else None
    _call("flce_piece_loss", dev, state.data_ptr(), labels.data_ptr(), n, vocab, ignore_index,
          _count_arg(num_label_tokens), loss.data_ptr(), lse.data_ptr(), _adr(rows),
          _status_ptr(status, dev), ws.data_ptr(), _bytes_of(ws))
    return loss, lse, rows


def flce_piece_fwd(hidden, weight, labels, state, bias=None, *, v_start: int, vocab: int,
                   first: bool, ignore_index: int = -100, workspace=None):
    """Takes the logits over one piece of the vocabulary, the classes v_start ... of ``vocab``,
    into ``state`` (fp32 [3, n]: maximum, sum of exponentials, label logit per row; overwritten
    with ``first``). Returns state."""
    import torch
    _require(hidden, "hidden", torch.bfloat16, 2)
    dev = hidden.device
    n, h = hidden.shape
    weight, bias, v = _piece_weight(weight, bias, h, dev)
    labels = _labels_i32(labels, n, dev, _ignore_arg(ignore_index))
    _contiguous_f32(state, "state", (3, n), dev)
    ws = _workspace(flce_piece_fwd_workspace_size(n, h, v), dev, workspace)
    _piece_fwd(hidden.contiguous(), weight, bias, labels, state, n, h, v, v_start, vocab, first,
               ignore_index, ws, dev)
    return state


def flce_piece_loss(state, labels, *, vocab: int, ignore_index: int = -100,
                    num_label_tokens: int | None = None, return_rows: bool = False, status=None,
                    workspace=None):
    """(loss, lse, rows) from the state over all pieces: the fp32 scalar divided by
    num_label_tokens (None: by the number of labelled rows), and fp32 [n] per-row logsumexp and
    terms (rows is None without ``return_rows``)."""
    import torch
    _require(state, "state", torch.float32, 2)
    dev = state.device
    n = state.shape[1]
    _contiguous_f32(state, "state", (3, n), dev)
    labels = _labels_i32(labels, n, dev, _ignore_arg(ignore_index))
    ws = _workspace(flce_piece_loss_workspace_size(n), dev, workspace)
    return _piece_loss(state, labels, n, vocab, ignore_index, num_label_tokens, return_rows, status,
                       ws, dev)


def _piece_bwd(hidden, weight, bias, labels, lse, n, h, v, v_start, vocab, ignore_index, count,
               flags, grad_output, grad_rows, hidden_acc, grad_hidden, grad_weight, grad_bias, ws,
               dev):
    wcode = 0 if grad_weight is None else _dtype_code(grad_weight.dtype, "grad_weight")
    _call("flce_piece_bwd", dev, hidden.data_ptr(), weight.data_ptr(), _adr(bias),
          labels.data_ptr(), lse.data_ptr(), n, h, v, v_start, vocab, ignore_index, count, flags,
          _adr(grad_output), _adr(grad_rows), _adr(hidden_acc), _adr(grad_hidden),
          _adr(grad_weight), wcode, _adr(grad_bias), ws.data_ptr(), _bytes_of(ws))


def _bwd_inputs(lse, grad_output, grad_rows, n, dev):
    import torch
    _contiguous_f32(lse, "lse", (n,), dev)
    if grad_output is not None:
        _require(grad_output, "grad_output", torch.float32, 0, dev)
    if grad_rows is not None:
        _contiguous_f32(grad_rows, "grad_rows", (n,), dev)


def _bwd_hidden(t, n, h, dev):
    import torch
    _require(t, "grad_hidden", torch.bfloat16, 2, dev)
    if tuple(t.shape) != (n, h) or not t.is_contiguous():
        raise ValueError(f"grad_hidden must be a contiguous {(n, h)} tensor")


def _bwd_params(grad_weight, grad_bias, v, h, dev):
    if grad_weight is not None:
        _require(grad_weight, "grad_weight", None, 2, dev)
        if tuple(grad_weight.shape) != (v, h) or not grad_weight.is_contiguous():
            raise ValueError(f"grad_weight must be a contiguous {(v, h)} tensor")
    if grad_bias is not None:
        _contiguous_f32(grad_bias, "grad_bias", (v,), dev)


def flce_piece_bwd(hidden, weight, labels, lse, bias=None, *, v_start: int, vocab: int,
                   first: bool, last: bool, ignore_index: int = -100,
                   num_label_tokens: int | None = None, accumulate: bool = False,
                   grad_output=None, grad_rows=None, hidden_acc=None, grad_hidden=None,
                   grad_weight=None, grad_bias=None, workspace=None):
    """Gradients of one piece from the lse over the whole vocabulary, written into the tensors
    given (None: not computed): ``hidden_acc`` fp32 [n, h], carried from the first piece to the
    last; ``grad_hidden`` bf16 [n, h], written with ``last`` from hidden_acc and that piece; ``grad_weight`` bf16 or fp32 and
    ``grad_bias`` fp32, of the piece's size. ``grad_rows`` fp32 [n]: the upstream gradient of
    each row's term, in place of grad_output / num_label_tokens."""
    import torch
    _require(hidden, "hidden", torch.bfloat16, 2)
    dev = hidden.device
    n, h = hidden.shape
    weight, bias, v = _piece_weight(weight, bias, h, dev)
    labels = _labels_i32(labels, n, dev, _ignore_arg(ignore_index))
    _bwd_inputs(lse, grad_output, grad_rows, n, dev)
    if hidden_acc is not None:
        _contiguous_f32(hidden_acc, "hidden_acc", (n, h), dev)
    if grad_hidden is not None:
        _bwd_hidden(grad_hidden, n, h, dev)
    _bwd_params(grad_weight, grad_bias, v, h, dev)
    flags = ((FLCE_PIECE_FIRST if first else 0) | (FLCE_PIECE_LAST if last else 0)
             | (FLCE_PIECE_ACCUMULATE if accumulate else 0))
    ws = _workspace(flce_piece_bwd_workspace_size(n, h, v), dev, workspace)
    _piece_bwd(hidden.contiguous(), weight, bias, labels, lse, n, h, v, v_start, vocab,
               ignore_index, _count_arg(num_label_tokens), flags, grad_output, grad_rows,
               hidden_acc, grad_hidden, grad_weight, grad_bias, ws, dev)


def _as_pieces(weight, bias):
    """([(weight, bias or None), ...], whether a sequence was given)."""
    many = isinstance(weight, (list, tuple))
    weights = list(weight) if many else [weight]
    if not weights:
        raise ValueError("weight holds no pieces")
    if bias is None:
        biases = [None] * len(weights)
    else:
        biases = list(bias) if isinstance(bias, (list, tuple)) else [bias]
        if len(biases) != len(weights):
            raise ValueError(f"{len(weights)} weight pieces but {len(biases)} biases")
    return list(zip(weights, biases)), many


def flce_pieces_fwd(hidden, weight, labels, bias=None, *, ignore_index: int = -100,
                    num_label_tokens: int | None = None, return_rows: bool = False, status=None):
    """Linear CE forward over a weight [v, h] or a sequence of weights that hold consecutive
    classes (with a sequence of biases, any of them None, or None). Returns (loss, lse, rows) as
    :func:`flce_piece_loss`; keep lse for :func:`flce_pieces_bwd`."""
    import torch
    pieces, _ = _as_pieces(weight, bias)
    _require(hidden, "hidden", torch.bfloat16, 2)
    hidden = hidden.contiguous()
    dev = hidden.device
    n, h = hidden.shape
    labels = _labels_i32(labels, n, dev, _ignore_arg(ignore_index))
    pieces = [_piece_weight(w, b, h, dev) for w, b in pieces]
    vocab = sum(v for _, _, v in pieces)
    state = torch.empty((3, n), dtype=torch.float32, device=dev)
    # one workspace for all of it: the calls follow one another on one stream
    ws = _workspace(max(flce_piece_loss_workspace_size(n),
                        *(flce_piece_fwd_workspace_size(n, h, v) for _, _, v in pieces)), dev)
    start = 0
    for w, b, v in pieces:
        _piece_fwd(hidden, w, b, labels, state, n, h, v, start, vocab, start == 0, ignore_index,
                   ws, dev)
        start += v
    return _piece_loss(state, labels, n, vocab, ignore_index, num_label_tokens, return_rows,
                       status, ws, dev)


# Bytes of the bf16 logit gradients that flce_pieces_bwd takes at a time by default, but at least
# _PIECE_LEAST classes: every piece reads and writes the fp32 hidden gradient and gathers the rows
# again, which shorter pieces would spend most of their time on (8192 x 4096 x 128256: 20.4 ms of
# backward in pieces of 16128 and more, 21.5 of 8192, 23.3 of 4096).
_PIECE_BYTES = 512 << 20
_PIECE_LEAST = 4096


def _piece_rows(n, v, piece_size):
    """Classes per piece: ``piece_size``, or as many as keep the logit gradients of a piece
    within _PIECE_BYTES (at least _PIECE_LEAST), in equal parts of whole 256-column tiles."""
    if piece_size is not None:
        if piece_size < 1:
            raise ValueError("piece_size must be at least 1")
        return piece_size
    rows = -(-max(n, 1) // 256) * 256
    most = max(_PIECE_LEAST, _PIECE_BYTES // (2 * rows) // 256 * 256)
    parts = -(-v // most)
    return -(-v // (256 * parts)) * 256


def flce_pieces_bwd(hidden, weight, labels, lse, bias=None, *, piece_size: int | None = None,
                    ignore_index: int = -100, num_label_tokens: int | None = None,
                    accumulate=False, grad_output=None, grad_rows=None, grad_hidden=True,
                    grad_weight=True, grad_bias=None):
    """Gradients of :func:`flce_pieces_fwd` from its lse. Each weight is taken ``piece_size``
    classes at a time (default: so that a piece's bf16 logit gradients stay within 512 MiB, but at
    least 4096, which past 65536 rows is 8 KiB a row).
    ``grad_rows`` fp32 [n]: the upstream gradient of each row's term, for per-row losses.

    ``grad_hidden`` / ``grad_weight`` / ``grad_bias``: True to allocate, False to skip, or what to
    write into; grad_weight (bf16, or fp32 where given so) and grad_bias are sequences where
    weight is one, and are added to with ``accumulate`` (True, or a sequence of one truth value per
    weight). grad_bias defaults to True when a bias is given (None for the pieces without one). Returns (grad_hidden, grad_weight, grad_bias)."""
    import torch
    pieces, many = _as_pieces(weight, bias)
    _require(hidden, "hidden", torch.bfloat16, 2)
    hidden = hidden.contiguous()
    dev = hidden.device
    n, h = hidden.shape
    labels = _labels_i32(labels, n, dev, _ignore_arg(ignore_index))
    _bwd_inputs(lse, grad_output, grad_rows, n, dev)
    if grad_bias is None:
        grad_bias = bias is not None
    if grad_bias is not False and bias is None:
        raise ValueError("grad_bias needs a bias")
    pieces = [_piece_weight(w, b, h, dev) for w, b in pieces]
    adds = [bool(accumulate)] * len(pieces)
    if isinstance(accumulate, (list, tuple)):
        adds = [bool(a) for a in accumulate]
        if len(adds) != len(pieces):
            raise ValueError(f"{len(pieces)} weight pieces but {len(adds)} of accumulate")

    def outs(spec, name, dtype, width):
        if spec is True:
            if any(adds):
                raise ValueError(f"accumulate=True needs an existing {name}")
            return [torch.empty((v, *width), dtype=dtype, device=dev) if width or b is not None
                    else None for _, b, v in pieces]
        if spec is False or spec is None:
            return [None] * len(pieces)
        spec = list(spec) if many else [spec]
        if len(spec) != len(pieces):
            raise ValueError(f"{len(pieces)} weight pieces but {len(spec)} of {name}")
        return spec

    gws = outs(grad_weight, "grad_weight", torch.bfloat16, (h,))
    gbs = outs(grad_bias, "grad_bias", torch.float32, ())
    gh = grad_hidden
    if gh is True:
        gh = torch.empty((n, h), dtype=torch.bfloat16, device=dev)
    elif gh is False:
        gh = None
    elif gh is not None:
        _bwd_hidden(gh, n, h, dev)
    vocab = sum(v for _, _, v in pieces)
    jobs = []  # (weight, bias, grad_weight, grad_bias, first class, classes, whether added to)
    start = 0
    for (w, b, v), gw, gb, add in zip(pieces, gws, gbs, adds):
        _bwd_params(gw, gb, v, h, dev)
        step = _piece_rows(n, v, piece_size)
        if step >= v:
            jobs.append((w, b, gw, gb, start, v, add))
        else:
            for lo in range(0, v, step):
                part = slice(lo, min(v, lo + step))
                jobs.append((*(None if t is None else t[part] for t in (w, b, gw, gb)),
                             start + lo, part.stop - lo, add))
        start += v
    acc = None
    if gh is not None and len(jobs) > 1:
        acc = torch.empty((n, h), dtype=torch.float32, device=dev)
    ws = _workspace(max(flce_piece_bwd_workspace_size(n, h, j[5]) for j in jobs), dev)
    count = _count_arg(num_label_tokens)
    for k, (w, b, gw, gb, at, v, add) in enumerate(jobs):
        flags = ((FLCE_PIECE_FIRST if k == 0 else 0)
                 | (FLCE_PIECE_LAST if k == len(jobs) - 1 else 0)
                 | (FLCE_PIECE_ACCUMULATE if add else 0))
        _piece_bwd(hidden, w, b, labels, lse, n, h, v, at, vocab, ignore_index, count, flags,
                   grad_output, grad_rows, acc, gh, gw, gb, ws, dev)
    return gh, gws if many else gws[0], gbs if many else gbs[0]


def lce_timing_enable(on: bool = True) -> None:
    """Bracket every library launch with hipEvents (measurement aid; off by default)."""
    _check("lce_timing_enable", load_library().lce_timing_enable(1 if on else 0))


def lce_timing_read() -> list[tuple[str, float, int]]:
    """(kernel name, total ms, launches) per kernel since the previous read; resets totals."""
    lib = load_library()
    cap = 64
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    cnt = (ctypes.c_longlong * cap)()
    k = ctypes.c_int()
    _check("lce_timing_read", lib.lce_timing_read(cap, names, ms, cnt, ctypes.byref(k)))
    return [(names[i].decode(), ms[i], cnt[i]) for i in range(min(k.value, cap))]
