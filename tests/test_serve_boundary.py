"""CPU checks of the root-mean-square norm, 8-bit product and beam search entry points: bad
arguments are refused with the documented status codes before anything touches a GPU (fake device
addresses, as in test_ops_boundary.py), and the binding's own refusals."""
import ctypes
import os

import pytest
import torch

import linear_cross_entropy_masked_amd as lce

OK, NULL_ARG, BAD_SHAPE, _, WORKSPACE, HIP, DEVICE, BAD_FLAGS, ALIGN, OVERLAP = range(10)
BAD_DTYPE = 11
A = [0x10000000 * (k + 1) for k in range(14)]  # distinct 256-aligned fake buffers
AT_DEVICE_CHECK = (HIP, DEVICE)
BIG = 1 << 30


class BeamState(ctypes.Structure):
    """lce_beam_state of the C ABI."""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p)] + [
        (name, ctypes.c_int64) for name in
        ("in_entry", "in_beam", "in_segment", "out_entry", "out_beam", "out_segment", "segments",
         "segment_bytes")]


def no_gpu():
    return torch.cuda.device_count() == 0


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(lce.library_path()):
        pytest.skip("library not built")
    return lce.load_library()


def caller(f, base):
    def call(**kw):
        assert set(kw) <= set(base)
        return f(*dict(base, **kw).values())
    return call


def test_rmsnorm_fwd_refusals(lib):
    call = caller(lib.rmsnorm_fwd, dict(x=A[0], dtype=0, n=4, h=16, ldx=16, res=A[1], ldr=16,
                                        w=A[2], pd=0, eps=1e-6, y=A[3], ldy=16, so=A[4], ldso=16,
                                        rstd=A[5], stream=None))
    assert call(n=-1) == BAD_SHAPE and call(h=0) == BAD_SHAPE and call(n=1 << 31) == BAD_SHAPE
    assert call(h=lce.LAYERNORM_MAX_H + 1, ldx=BIG, ldr=BIG, ldy=BIG, ldso=BIG) == BAD_SHAPE
    assert call(ldx=15) == BAD_SHAPE and call(ldr=15) == BAD_SHAPE and call(ldy=15) == BAD_SHAPE
    assert call(ldso=15) == BAD_SHAPE and call(ldr=1 << 62) == BAD_SHAPE
    assert call(eps=-1.0) == BAD_SHAPE and call(eps=float("nan")) == BAD_SHAPE
    assert call(dtype=3) == BAD_DTYPE and call(pd=1) == BAD_DTYPE
    assert call(dtype=2) == BAD_DTYPE  # fp32 rows beside a bf16 weight
    assert call(x=None) == NULL_ARG and call(y=None) == NULL_ARG
    assert call(x=A[0] + 1) == ALIGN and call(res=A[1] + 1) == ALIGN
    assert call(so=A[4] + 1) == ALIGN and call(rstd=A[5] + 2) == ALIGN
    assert call(y=A[0] + 2) == OVERLAP and call(y=A[0], ldy=18) == OVERLAP
    assert call(so=A[1] + 32) == OVERLAP and call(so=A[1], ldso=20) == OVERLAP
    assert call(so=A[3]) == OVERLAP and call(so=A[0], y=A[0]) == OVERLAP
    assert call(rstd=A[0]) == OVERLAP and call(rstd=A[1] + 4) == OVERLAP
    assert call(y=A[2]) == OVERLAP and call(so=A[2]) == OVERLAP
    if no_gpu():
        for kw in ({}, dict(y=A[0]), dict(so=A[1]), dict(so=A[0]), dict(y=A[1], so=A[0]),
                   dict(res=None, ldr=0), dict(so=None, ldso=0), dict(w=None, rstd=None, pd=2),
                   dict(n=0, x=None, y=None)):
            assert call(**kw) in AT_DEVICE_CHECK, kw


def test_rmsnorm_fp8_fwd_refusals(lib):
    call = caller(lib.rmsnorm_fp8_fwd, dict(x=A[0], dtype=0, n=4, h=300, ldx=300, res=A[1],
                                            ldr=300, w=A[2], pd=0, eps=1e-6, q=A[3], ldq=300,
                                            scales=A[6], sd=0, lds=4, so=A[4], ldso=300,
                                            rstd=A[5], stream=None))
    assert call(lds=3) == BAD_SHAPE and call(ldq=299) == BAD_SHAPE
    assert call(sd=2) == BAD_DTYPE and call(sd=-1) == BAD_DTYPE
    assert call(scales=None) == NULL_ARG and call(q=None) == NULL_ARG
    assert call(scales=A[6] + 2) == ALIGN
    assert call(q=A[0]) == OVERLAP and call(q=A[1]) == OVERLAP  # 8-bit rows are no in-place form
    assert call(scales=A[3] + 4) == OVERLAP and call(scales=A[1]) == OVERLAP
    assert call(scales=A[4]) == OVERLAP
    if no_gpu():
        assert call() in AT_DEVICE_CHECK and call(so=A[1]) in AT_DEVICE_CHECK
        assert call(sd=1, scales=A[6] + 1) in AT_DEVICE_CHECK
        assert call(q=A[3] + 1, ldq=301) in AT_DEVICE_CHECK


def test_rmsnorm_bwd_refusals(lib):
    out = ctypes.c_size_t()
    assert lib.rmsnorm_workspace_size(4, 16, None) == NULL_ARG
    assert lib.rmsnorm_workspace_size(4, 0, ctypes.byref(out)) == BAD_SHAPE
    assert lib.rmsnorm_workspace_size(4, 16, ctypes.byref(out)) == OK and out.value >= 256
    call = caller(lib.rmsnorm_bwd, dict(g=A[0], dtype=0, ldg=16, x=A[1], ldx=16, rstd=A[2],
                                        w=A[3], pd=0, gr=A[4], ldgr=16, n=4, h=16, flags=0,
                                        gx=A[5], lddx=16, gw=A[6], gd=2, ws=A[7], wsb=BIG,
                                        stream=None))
    assert call(flags=2) == BAD_FLAGS
    assert call(h=0) == BAD_SHAPE and call(lddx=15) == BAD_SHAPE and call(ldgr=15) == BAD_SHAPE
    assert call(gd=1) == BAD_DTYPE and call(pd=2, gd=0) == BAD_DTYPE
    assert call(g=None) == NULL_ARG and call(x=None) == NULL_ARG and call(rstd=None) == NULL_ARG
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(gw=A[6] + 2) == ALIGN and call(ws=A[7] + 4) == ALIGN and call(gr=A[4] + 1) == ALIGN
    assert call(gx=A[1]) == OVERLAP and call(gx=A[0], ldg=20) == OVERLAP
    assert call(gx=A[4] + 32) == OVERLAP and call(gw=A[7]) == OVERLAP and call(ws=A[4]) == OVERLAP
    if no_gpu():
        for kw in ({}, dict(gx=A[0]), dict(gx=A[4]), dict(gx=None, lddx=0),
                   dict(gw=None, ws=None, wsb=0), dict(gr=None, ldgr=0),
                   dict(gr=A[0])):  # one gradient for both
            assert call(**kw) in AT_DEVICE_CHECK, kw


def test_fp8_quantize_refusals(lib):
    call = caller(lib.fp8_quantize, dict(x=A[0], dtype=0, n=300, h=200, ldx=200, rows=1, q=A[1],
                                         ldq=200, scales=A[2], sd=0, lds=300, stream=None))
    assert call(n=-1) == BAD_SHAPE and call(h=0) == BAD_SHAPE and call(rows=2) == BAD_SHAPE
    assert call(h=(1 << 20) + 1, ldx=BIG, ldq=BIG) == BAD_SHAPE
    assert call(n=1 << 20, h=(1 << 14) + 1, ldx=BIG, ldq=BIG, lds=BIG) == BAD_SHAPE
    assert call(ldx=199) == BAD_SHAPE and call(ldq=199) == BAD_SHAPE and call(lds=299) == BAD_SHAPE
    assert call(rows=128, lds=1) == BAD_SHAPE
    assert call(dtype=9) == BAD_DTYPE and call(sd=4) == BAD_DTYPE
    assert call(x=None) == NULL_ARG and call(q=None) == NULL_ARG and call(scales=None) == NULL_ARG
    assert call(x=A[0] + 1) == ALIGN and call(scales=A[2] + 1) == ALIGN
    assert call(q=A[0]) == OVERLAP and call(scales=A[1] + 4) == OVERLAP
    if no_gpu():
        assert call() in AT_DEVICE_CHECK and call(rows=128, lds=2, sd=1) in AT_DEVICE_CHECK
        assert call(n=0, x=None, q=None, scales=None) in AT_DEVICE_CHECK


def test_fp8_matmul_refusals(lib):
    out = ctypes.c_size_t()
    ref = ctypes.byref(out)
    size = lib.fp8_matmul_workspace_size
    assert size(4, 16, 16, None) == NULL_ARG
    for m, n, k in ((-1, 16, 16), (4, 0, 16), (4, 16, 0), (4, 16, 24), (4, 16, 8),
                    ((1 << 23) + 1, 16, 16), (4, (1 << 28) + 1, 16), (4, 16, (1 << 20) + 16),
                    (1 << 23, 1 << 16, 16)):
        assert size(m, n, k, ref) == BAD_SHAPE, (m, n, k)
    assert size(0, 16, 16, ref) == OK and out.value == 0
    call = caller(lib.fp8_matmul, dict(a=A[0], lda=1024, sa=A[1], ldas=200, b=A[2], ldb=1024,
                                       sb=A[3], ldbs=8, sd=0, bias=A[4], m=200, n=300, k=1024,
                                       out=A[5], od=0, ldo=300, ws=A[6], wsb=BIG, stream=None))
    assert size(200, 300, 1024, ref) == OK and out.value > 0
    assert call(k=1000) == BAD_SHAPE and call(lda=1008) == BAD_SHAPE and call(lda=1032) == BAD_SHAPE
    assert call(ldb=1020) == BAD_SHAPE and call(ldb=(1 << 22) + 16) == BAD_SHAPE
    assert call(ldo=299) == BAD_SHAPE and call(ldas=199) == BAD_SHAPE and call(ldbs=7) == BAD_SHAPE
    assert call(sd=2) == BAD_DTYPE and call(od=3) == BAD_DTYPE
    for name in ("a", "sa", "b", "sb", "out"):
        assert call(**{name: None}) == NULL_ARG, name
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(a=A[0] + 8) == ALIGN and call(b=A[2] + 8) == ALIGN and call(sa=A[1] + 2) == ALIGN
    assert call(out=A[5] + 1) == ALIGN and call(bias=A[4] + 2) == ALIGN
    assert call(out=A[0] + 64) == OVERLAP and call(out=A[4]) == OVERLAP
    assert call(ws=A[5]) == OVERLAP and call(ws=A[3]) == OVERLAP
    if no_gpu():
        assert call(wsb=out.value) in AT_DEVICE_CHECK
        assert call(m=0, a=None, sa=None, out=None) in AT_DEVICE_CHECK
        assert call(m=3, ws=None, wsb=0, bias=None) in AT_DEVICE_CHECK  # few rows need none


def test_beam_step_refusals(lib):
    out = ctypes.c_size_t()
    ref = ctypes.byref(out)
    size = lib.beam_step_workspace_size
    assert size(2, 4, 1000, 8, None) == NULL_ARG
    for args in ((-1, 4, 1000, 8), (2, 0, 1000, 8), (2, 65, 1000, 8), (2, 4, 0, 8),
                 (2, 4, 1000, 0), (2, 4, 1000, 65), (1 << 20, 64, 1 << 20, 8), (2, 4, 1 << 31, 8)):
        assert size(*args, ref) == BAD_SHAPE, args
    assert size(0, 4, 1000, 8, ref) == OK and out.value == 0
    assert size(2, 4, 1000, 8, ref) == OK and out.value >= 8 * 8 * 8
    call = caller(lib.beam_step, dict(z=A[0], dtype=0, batch=2, beams=4, v=1000, ldl=1000,
                                      scores=A[1], fin=A[2], eos=2, num=8, ign=-100, so=A[3],
                                      po=A[4], to=A[5], fo=A[6], status=A[7], ws=A[8], wsb=BIG,
                                      stream=None))
    assert call(ldl=999) == BAD_SHAPE and call(eos=1000) == BAD_SHAPE and call(eos=-1) == BAD_SHAPE
    assert call(dtype=5) == BAD_DTYPE
    for name in ("z", "scores", "so", "po", "to"):
        assert call(**{name: None}) == NULL_ARG, name
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(z=A[0] + 1) == ALIGN and call(scores=A[1] + 2) == ALIGN
    assert call(ws=A[8] + 8) == ALIGN and call(po=A[4] + 2) == ALIGN
    assert call(so=A[1]) == OVERLAP and call(fo=A[2]) == OVERLAP and call(po=A[5]) == OVERLAP
    assert call(ws=A[0]) == OVERLAP and call(status=A[3]) == OVERLAP
    if no_gpu():
        assert call(wsb=out.value) in AT_DEVICE_CHECK
        assert call(fin=None, fo=None, eos=-1, status=None) in AT_DEVICE_CHECK
        assert call(batch=0, z=None, scores=None, so=None, po=None, to=None, ws=None) \
            in AT_DEVICE_CHECK


def test_beam_reorder_refusals(lib):
    def call(states=({},), parents=A[0], batch=2, beams=4, slots=4, count=None):
        rows = (BeamState * max(1, len(states)))()
        for r, kw in zip(rows, states):
            kw = dict(dict(src=A[1], dst=A[2], in_entry=400, in_beam=100, in_segment=0,
                           out_entry=400, out_beam=100, out_segment=0, segments=1,
                           segment_bytes=100), **kw)
            for name, value in kw.items():
                setattr(r, name, value)
        return lib.beam_reorder(rows, len(states) if count is None else count, parents, batch,
                                beams, slots, None)
    assert call(batch=-1) == BAD_SHAPE and call(beams=0) == BAD_SHAPE and call(beams=65) == BAD_SHAPE
    assert call(slots=0) == BAD_SHAPE and call(slots=65) == BAD_SHAPE and call(count=-1) == BAD_SHAPE
    assert call(count=0) == OK and call(batch=0) == OK
    assert lib.beam_reorder(None, 1, A[0], 2, 4, 4, None) == NULL_ARG
    assert call(parents=None) == NULL_ARG and call(({"src": None},)) == NULL_ARG
    assert call(parents=A[0] + 2) == ALIGN
    assert call(({"segments": -1},)) == BAD_SHAPE and call(({"segment_bytes": -1},)) == BAD_SHAPE
    assert call(({"in_entry": -400},)) == BAD_SHAPE and call(({"in_entry": 1 << 62},)) == BAD_SHAPE
    # runs of the result that lie in one another
    assert call(({"out_beam": 99},)) == BAD_SHAPE and call(({"out_entry": 300},)) == BAD_SHAPE
    assert call(({"segments": 3, "out_segment": 50},)) == BAD_SHAPE
    assert call(({"dst": A[1] + 8},)) == OVERLAP and call(({"dst": A[0]},)) == OVERLAP
    assert call(({}, {"src": A[3]})) == OVERLAP  # two results in one place
    assert call(({}, {"src": A[2], "dst": A[3]})) == OVERLAP  # a state that another one overwrites
    assert call(({"dst": A[1]}, {"src": A[3]})) == OVERLAP  # one in place, the other not
    assert call(({"dst": A[1]},), slots=3) == OVERLAP
    assert call(({"dst": A[1], "out_beam": 50, "segment_bytes": 50},)) == OVERLAP
    if no_gpu():
        assert call() in AT_DEVICE_CHECK and call(({"dst": A[1]},)) in AT_DEVICE_CHECK
        assert call(({}, {"dst": A[3]})) in AT_DEVICE_CHECK  # one state read twice
        assert call(({"segment_bytes": 0, "src": None, "dst": None},)) in AT_DEVICE_CHECK
        # heads outside the beams: [heads, batch, beams, dim]
        assert call(({"segments": 5, "in_segment": 800, "out_segment": 800},)) in AT_DEVICE_CHECK


def test_launch_size_refusals(lib):
    """Sizes whose launches would pass 2^32 threads, and the largest below."""
    quant = caller(lib.fp8_quantize, dict(x=1 << 40, dtype=0, n=300, h=1, ldx=1, rows=1, q=1 << 50,
                                          ldq=1, scales=1 << 52, sd=0, lds=1 << 31, stream=None))
    at = dict(n=(1 << 28) - 16), dict(n=(1 << 31) - 256, rows=128)
    for kw in (dict(n=1 << 28), dict(n=(1 << 31) - 127, rows=128)):
        assert quant(**kw) == BAD_SHAPE, kw
    out = ctypes.c_size_t()
    size = lib.fp8_matmul_workspace_size
    assert size(1 << 15, 1 << 23, 16, ctypes.byref(out)) == BAD_SHAPE
    assert size((1 << 15) - 256, 1 << 23, 16, ctypes.byref(out)) == OK
    if no_gpu():
        for kw in at:
            assert quant(**kw) in AT_DEVICE_CHECK, kw


def test_beam_reorder_many_states(lib):
    """Overlaps among many states, a state without bytes ahead of one that has some, and strides
    whose products pass 64 bits."""
    def call(states, beams=4):
        rows = (BeamState * len(states))()
        for r, (src, dst, kw) in zip(rows, states):
            kw = dict(dict(src=src, dst=dst, in_entry=400, in_beam=100, out_entry=400,
                           out_beam=100, segments=1, segment_bytes=100), **kw)
            for name, value in kw.items():
                setattr(r, name, value)
        return lib.beam_reorder(rows, len(states), A[0], 2, beams, 4, None)
    many = [(A[1] + 800 * i, A[2] + 800 * ((i * 7919) % 20000), {}) for i in range(20000)]
    empty = (None, None, {"segment_bytes": 0})
    for i, dst in ((19999, A[2] + 800 * 5 + 799), (3, A[1] + 800 * 19999 + 799), (7, A[0] + 28)):
        bad = list(many)
        bad[i] = (bad[i][0], dst, {})
        assert call(bad) == OVERLAP, i
    huge = {"segments": (1 << 31) - 1, "in_segment": 1 << 50, "out_segment": 1 << 50}
    assert call([(A[1], A[2], huge)]) == BAD_SHAPE
    assert call([(A[1], A[2], {"in_entry": 1 << 50, "out_entry": 1 << 50})]) == BAD_SHAPE
    if no_gpu():
        assert call(many) in AT_DEVICE_CHECK
        assert call([empty, (A[1], A[2], {})]) in AT_DEVICE_CHECK
        assert call([empty, (A[1], A[1], {})]) in AT_DEVICE_CHECK


def test_binding_refusals():
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    x = torch.zeros(3, 32)
    for f in (lce.rmsnorm_fwd, lce.rmsnorm_fp8_fwd, lce.fp8_quantize):
        with pytest.raises(ValueError, match="HIP device"):
            f(x)
        with pytest.raises(TypeError, match="bfloat16"):
            f(x.double())
    with pytest.raises(ValueError, match="HIP device"):
        lce.rmsnorm_bwd(x, x, torch.zeros(3))
    with pytest.raises(ValueError, match="HIP device"):
        lce.fp8_matmul(x.to(f8), torch.zeros(1, 3).to(e8), x.to(f8), torch.zeros(1, 1).to(e8))
    with pytest.raises(ValueError, match="HIP device"):
        lce.beam_step(torch.zeros(1, 2, 9), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="HIP device"):
        lce.beam_reorder([x], torch.zeros(3, 2, dtype=torch.int32))


def test_binding_checks_shapes(monkeypatch):
    """The binding's own refusals, on host tensors that pass for device ones."""
    def require(t, name, dtype, dims, device=None):
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}")
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions")
    monkeypatch.setattr(lce, "_require", require)
    monkeypatch.setattr(lce, "_call", lambda *a: pytest.fail("reached the library"))
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="residual_out needs"):
        lce.rmsnorm_fwd(x, residual_out=x)
    with pytest.raises(ValueError, match="shape"):
        lce.rmsnorm_fwd(x, None, x[:2])
    with pytest.raises(TypeError, match="residual"):
        lce.rmsnorm_fwd(x, None, x.half())
    with pytest.raises(ValueError, match="entries"):
        lce.rmsnorm_fwd(x, torch.ones(255))
    with pytest.raises(TypeError, match="scale_dtype"):
        lce.rmsnorm_fp8_fwd(x, scale_dtype=torch.float16)
    with pytest.raises(ValueError, match="scales"):
        lce.rmsnorm_fp8_fwd(x, scales=torch.zeros(4, 2))  # rows by blocks, not blocks by rows
    with pytest.raises(ValueError, match="accumulate"):
        lce.rmsnorm_bwd(x, x, torch.ones(4), torch.ones(256), accumulate=True)
    with pytest.raises(ValueError, match="block_rows"):
        lce.fp8_quantize(x, block_rows=64)
    q, c = torch.zeros(4, 256).to(torch.float8_e4m3fn), torch.ones(2, 4)
    w = torch.ones(1, 2)
    with pytest.raises(ValueError, match="columns"):
        lce.fp8_matmul(q, c, q[:, :128], w)
    with pytest.raises(ValueError, match="b_scales"):
        lce.fp8_matmul(q, c, q, c)
    with pytest.raises(TypeError, match="one"):
        lce.fp8_matmul(q, c, q, w.to(torch.float8_e8m0fnu))
    with pytest.raises(ValueError, match="bias"):
        lce.fp8_matmul(q, c, q, w, torch.zeros(3))
    z, s = torch.zeros(2, 3, 9), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="finished needs eos"):
        lce.beam_step(z, s, finished=torch.zeros(2, 3, dtype=torch.bool))
    with pytest.raises(ValueError, match="eos"):
        lce.beam_step(z, s, eos=9)
    with pytest.raises(ValueError, match="scores"):
        lce.beam_step(z, s[:, :2])
    with pytest.raises(ValueError, match="contiguous"):
        lce.beam_step(torch.zeros(2, 9, 3).transpose(1, 2), s)


def test_runs_of_a_state():
    """What a beam holds as (runs, stride, bytes), and what is no such thing."""
    t = torch.zeros(2, 3, 4, 5, 6, dtype=torch.float16)
    assert lce._runs(t, "x") == (1, 0, 240)
    assert lce._runs(t[:, :, :, :2], "x") == (4, 60, 24)  # room behind a length
    assert lce._runs(t[:, :, :, :, :3], "x") == (20, 12, 6)
    assert lce._runs(t[:, :, :2], "x") == (1, 0, 120)
    assert lce._runs(t[:, :, :, 1], "x") == (4, 60, 12)
    assert lce._runs(t[:, :, 0, 0, 0], "x") == (1, 0, 2)
    assert lce._runs(t[:, :, :0], "x")[2] == 0
    with pytest.raises(ValueError, match="runs"):
        lce._runs(t[:, :, :, :2, :3], "x")
    with pytest.raises(ValueError, match="runs"):
        lce._runs(t.transpose(2, 4), "x")
