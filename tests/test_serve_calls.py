"""CPU checks of calls of the norm, 8-bit product and beam search entry points beside those of
test_serve_boundary.py: what is refused and what passes the checks of arguments, with fake device
addresses."""
import ctypes

import torch

import linear_cross_entropy_masked_amd as lce
from test_serve_boundary import (A, ALIGN, AT_DEVICE_CHECK, BAD_DTYPE, BAD_SHAPE, BIG, NULL_ARG,
                                 OK, OVERLAP, WORKSPACE, caller, lib, no_gpu)  # noqa: F401


def test_fp8_matmul_precise_refusals(lib):  # noqa: F811
    """The same checks as fp8_matmul's, and the same workspace."""
    out = ctypes.c_size_t()
    call = caller(lib.fp8_matmul_precise,
                  dict(a=A[0], lda=1024, sa=A[1], ldas=200, b=A[2], ldb=1024, sb=A[3], ldbs=8,
                       sd=0, bias=A[4], m=200, n=300, k=1024, out=A[5], od=0, ldo=300, ws=A[6],
                       wsb=BIG, stream=None))
    assert lib.fp8_matmul_workspace_size(200, 300, 1024, ctypes.byref(out)) == OK and out.value > 0
    assert call(k=1000) == BAD_SHAPE and call(lda=1008) == BAD_SHAPE and call(ldo=299) == BAD_SHAPE
    assert call(sd=2) == BAD_DTYPE and call(od=3) == BAD_DTYPE
    assert call(a=None) == NULL_ARG and call(out=None) == NULL_ARG
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(b=A[2] + 8) == ALIGN and call(out=A[0] + 64) == OVERLAP
    if no_gpu():
        assert call(wsb=out.value) in AT_DEVICE_CHECK and call(od=2) in AT_DEVICE_CHECK


def test_precise_reaches_its_entry(monkeypatch):
    """The binding's choice of entry point, on host tensors that pass for device ones."""
    reached = []
    monkeypatch.setattr(lce, "_require", lambda *a, **k: None)
    monkeypatch.setattr(lce, "_call", lambda fn, *a: reached.append(fn))
    q, c = torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(2, 4)
    for kw in ({}, {"precise": False}, {"precise": True}, {"precise": True, "dtype": torch.float32}):
        lce.fp8_matmul(q, c, q, torch.ones(1, 2), **kw)
    assert reached == ["fp8_matmul", "fp8_matmul", "fp8_matmul_precise", "fp8_matmul_precise"]
