"""CPU checks of the embedding, layer norm and vocabulary-piece entry points: bad arguments are
refused with the documented status codes before anything touches a GPU (fake device addresses, as
in test_boundary.py), and the binding's own refusals."""
import ctypes
import os

import pytest
import torch

import linear_cross_entropy_masked_amd as lce

OK, NULL_ARG, BAD_SHAPE, _, WORKSPACE, HIP, DEVICE, BAD_FLAGS, ALIGN, OVERLAP = range(10)
BAD_DTYPE = 11
A = [0x10000000 * (k + 1) for k in range(12)]  # distinct 256-aligned fake buffers
AT_DEVICE_CHECK = (HIP, DEVICE)
BIG = 1 << 30


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


def test_status_string_of_the_new_code(lib):
    assert "type" in lce.lce_status_str(BAD_DTYPE)


def test_embed_fwd_refusals(lib):
    call = caller(lib.embed_fwd, dict(w=A[0], dtype=0, v=10, h=16, ldw=16, tok=A[1], n=4, ign=-100,
                                      scale=1.0, out=A[2], ldo=16, status=None, stream=None))
    assert call(n=-1) == BAD_SHAPE and call(v=0) == BAD_SHAPE and call(h=0) == BAD_SHAPE
    assert call(ldw=15) == BAD_SHAPE and call(ldo=15) == BAD_SHAPE
    assert call(v=1 << 31) == BAD_SHAPE and call(n=1 << 31) == BAD_SHAPE
    assert call(n=(1 << 31) - 1, h=1 << 20, ldw=1 << 20, ldo=1 << 20) == BAD_SHAPE
    assert call(ldw=1 << 62) == BAD_SHAPE
    assert call(dtype=3) == BAD_DTYPE and call(dtype=-1) == BAD_DTYPE
    assert call(w=None) == NULL_ARG and call(tok=None) == NULL_ARG and call(out=None) == NULL_ARG
    assert call(w=A[0] + 1) == ALIGN and call(out=A[2] + 2, dtype=2) == ALIGN
    assert call(tok=A[1] + 2) == ALIGN and call(status=A[3] + 1) == ALIGN
    assert call(out=A[0] + 32) == OVERLAP and call(out=A[1]) == OVERLAP
    assert call(status=A[2] + 4) == OVERLAP
    if no_gpu():
        assert call() in AT_DEVICE_CHECK
        assert call(n=0, tok=None, out=None) in AT_DEVICE_CHECK
        assert call(w=A[0] + 2, out=A[2] + 6, ldw=17, ldo=31) in AT_DEVICE_CHECK


def test_embed_bwd_refusals(lib):
    out = ctypes.c_size_t()
    assert lib.embed_workspace_size(4, 16, 10, None) == NULL_ARG
    assert lib.embed_workspace_size(-1, 16, 10, ctypes.byref(out)) == BAD_SHAPE
    assert lib.embed_workspace_size(4, 16, 10, ctypes.byref(out)) == OK and out.value >= 32
    call = caller(lib.embed_bwd, dict(g=A[0], dtype=0, ldg=16, tok=A[1], n=4, h=16, v=10, ign=-100,
                                      scale=1.0, flags=0, gw=A[2], gdtype=2, ldw=16, status=None,
                                      ws=A[3], wsb=BIG, stream=None))
    assert call(flags=2) == BAD_FLAGS
    assert call(h=0) == BAD_SHAPE and call(ldg=8) == BAD_SHAPE and call(ldw=8) == BAD_SHAPE
    assert call(h=(1 << 20) + 1, ldg=1 << 21, ldw=1 << 21) == BAD_SHAPE
    assert call(dtype=2, gdtype=0) == BAD_DTYPE and call(gdtype=1) == BAD_DTYPE
    assert call(dtype=7) == BAD_DTYPE
    assert call(g=None) == NULL_ARG and call(gw=None) == NULL_ARG and call(tok=None) == NULL_ARG
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(ws=A[3] + 64) == ALIGN and call(gw=A[2] + 2) == ALIGN
    assert call(gw=A[0]) == OVERLAP and call(ws=A[2]) == OVERLAP and call(status=A[3]) == OVERLAP
    if no_gpu():
        assert call(wsb=out.value, flags=1) in AT_DEVICE_CHECK
        assert call(n=0, g=None, tok=None) in AT_DEVICE_CHECK


def test_layernorm_refusals(lib):
    call = caller(lib.layernorm_fwd, dict(x=A[0], dtype=0, n=4, h=16, ldx=16, w=A[1], b=A[2],
                                          pd=0, eps=1e-5, y=A[3], ldy=16, mean=A[4], rstd=A[5],
                                          stream=None))
    assert call(n=-1) == BAD_SHAPE and call(h=0) == BAD_SHAPE and call(ldx=15) == BAD_SHAPE
    assert call(ldy=3) == BAD_SHAPE and call(eps=-1.0) == BAD_SHAPE
    assert call(eps=float("nan")) == BAD_SHAPE
    assert call(h=lce.LAYERNORM_MAX_H + 1, ldx=BIG, ldy=BIG) == BAD_SHAPE
    assert call(dtype=5) == BAD_DTYPE and call(pd=1) == BAD_DTYPE and call(dtype=2) == BAD_DTYPE
    assert call(x=None) == NULL_ARG and call(y=None) == NULL_ARG
    assert call(x=A[0] + 1) == ALIGN and call(mean=A[4] + 2) == ALIGN
    assert call(y=A[0] + 2) == OVERLAP and call(y=A[0], ldx=18) == OVERLAP
    assert call(mean=A[3]) == OVERLAP and call(rstd=A[4] + 4) == OVERLAP
    if no_gpu():
        assert call() in AT_DEVICE_CHECK and call(y=A[0]) in AT_DEVICE_CHECK
        assert call(w=None, b=None, mean=None, rstd=None, pd=2) in AT_DEVICE_CHECK
    out = ctypes.c_size_t()
    assert lib.layernorm_workspace_size(4, 16, None) == NULL_ARG
    assert lib.layernorm_workspace_size(4, 0, ctypes.byref(out)) == BAD_SHAPE
    assert lib.layernorm_workspace_size(4, 16, ctypes.byref(out)) == OK
    call = caller(lib.layernorm_bwd, dict(g=A[0], dtype=0, ldg=16, x=A[1], ldx=16, mean=A[2],
                                          rstd=A[3], w=A[4], pd=0, n=4, h=16, flags=0, gx=A[5],
                                          lddx=16, gw=A[6], gb=A[7], gd=2, ws=A[8], wsb=BIG,
                                          stream=None))
    assert call(flags=4) == BAD_FLAGS and call(lddx=15) == BAD_SHAPE and call(h=0) == BAD_SHAPE
    assert call(gd=1) == BAD_DTYPE and call(pd=2, gd=0) == BAD_DTYPE
    assert call(mean=None) == NULL_ARG and call(x=None) == NULL_ARG and call(g=None) == NULL_ARG
    assert call(ws=None) == WORKSPACE and call(wsb=out.value - 1) == WORKSPACE
    assert call(gw=A[6] + 2) == ALIGN and call(ws=A[8] + 4) == ALIGN
    assert call(gx=A[1]) == OVERLAP and call(gw=A[7]) == OVERLAP and call(gx=A[0], ldg=20) == OVERLAP
    if no_gpu():
        assert call(gx=A[0]) in AT_DEVICE_CHECK
        assert call(gx=None, gw=None, gb=None, ws=None, lddx=0) in AT_DEVICE_CHECK


def test_piece_refusals(lib):
    out = ctypes.c_size_t()
    ref = ctypes.byref(out)
    assert lib.flce_piece_fwd_workspace_size(4, 16, 10, None) == NULL_ARG
    assert lib.flce_piece_fwd_workspace_size(4, 12, 10, ref) == BAD_SHAPE
    assert lib.flce_piece_loss_workspace_size((1 << 23) + 1, ref) == BAD_SHAPE
    assert lib.flce_piece_bwd_workspace_size(4, 16, 0, ref) == BAD_SHAPE
    # the backward's workspace holds the piece's bf16 logit gradients, not the vocabulary's
    assert lib.flce_piece_bwd_workspace_size(8192, 4096, 16384, ref) == OK
    assert out.value >= 8192 * 16384 * 2 and out.value <= 8192 * 16384 * 2 + 8192 * 4096 * 3
    assert lib.flce_piece_bwd_workspace_size(4, 16, 10, ref) == OK
    need = out.value
    call = caller(lib.flce_piece_fwd, dict(hid=A[0], w=A[1], b=A[2], lab=A[3], n=4, h=16, v=10,
                                           start=0, vocab=10, ign=-100, flags=1, state=A[4],
                                           ws=A[5], wsb=BIG, stream=None))
    assert call(flags=2) == BAD_FLAGS and call(h=12) == BAD_SHAPE and call(n=-1) == BAD_SHAPE
    assert call(start=1) == BAD_SHAPE and call(start=-1) == BAD_SHAPE
    assert call(vocab=9) == BAD_SHAPE and call(vocab=1 << 31) == BAD_SHAPE
    assert call(n=(1 << 23) + 1) == BAD_SHAPE and call(h=(1 << 20) + 8) == BAD_SHAPE
    assert call(n=1 << 23, v=65536, vocab=65536) == BAD_SHAPE  # 2^23 tiles of 256 x 256
    assert call(hid=None) == NULL_ARG and call(w=None) == NULL_ARG and call(state=None) == NULL_ARG
    assert call(ws=None) == WORKSPACE and call(wsb=1) == WORKSPACE
    assert call(hid=A[0] + 8) == ALIGN and call(w=A[1] + 2) == ALIGN and call(ws=A[5] + 8) == ALIGN
    assert call(state=A[3]) == OVERLAP and call(ws=A[1]) == OVERLAP
    if no_gpu():
        assert call(start=90, vocab=100, flags=0, b=None) in AT_DEVICE_CHECK
        assert call(n=0, hid=None, lab=None, state=None) in AT_DEVICE_CHECK
    call = caller(lib.flce_piece_loss, dict(state=A[0], lab=A[1], n=4, vocab=10, ign=-100, t=-1,
                                            loss=A[2], lse=A[3], rows=A[4], status=A[5], ws=A[6],
                                            wsb=BIG, stream=None))
    assert call(vocab=0) == BAD_SHAPE and call(n=-1) == BAD_SHAPE
    assert call(state=None) == NULL_ARG and call(lab=None) == NULL_ARG
    assert call(wsb=8) == WORKSPACE and call(loss=A[2] + 2) == ALIGN
    assert call(lse=A[0]) == OVERLAP and call(rows=A[3] + 4) == OVERLAP
    if no_gpu():
        assert call(loss=None, lse=None, rows=None, status=None) in AT_DEVICE_CHECK
    call = caller(lib.flce_piece_bwd, dict(hid=A[0], w=A[1], b=A[2], lab=A[3], lse=A[4], n=4, h=16,
                                           v=10, start=0, vocab=10, ign=-100, t=-1, flags=3,
                                           gout=None, grows=None, acc=A[5], gh=A[6], gw=A[7], wd=0,
                                           gb=A[8], ws=A[9], wsb=BIG, stream=None))
    assert call(flags=8) == BAD_FLAGS and call(h=0) == BAD_SHAPE and call(vocab=5) == BAD_SHAPE
    assert call(wd=1) == BAD_DTYPE
    assert call(b=None) == NULL_ARG  # grad_bias needs one
    assert call(lse=None) == NULL_ARG and call(flags=2, acc=None) == NULL_ARG
    assert call(wsb=need - 1) == WORKSPACE
    assert call(gh=A[6] + 8) == ALIGN and call(gw=A[7] + 2) == ALIGN and call(acc=A[5] + 4) == ALIGN
    assert call(gh=A[0]) == OVERLAP and call(acc=A[6]) == OVERLAP and call(gb=A[4]) == OVERLAP
    assert call(grows=A[9]) == OVERLAP
    if no_gpu():
        assert call(wsb=need) in AT_DEVICE_CHECK and call(acc=None) in AT_DEVICE_CHECK
        assert call(gh=None, gw=None, gb=None, b=None, flags=0, acc=None) in AT_DEVICE_CHECK


def test_piece_size_rule():
    """Default pieces: whole 256-column tiles, equal parts, within the byte budget."""
    assert lce._piece_rows(8192, 128256, None) == 32256
    assert lce._piece_rows(64, 32777, None) == 33024
    assert lce._piece_rows(1 << 20, 128256, None) <= 4096
    assert lce._piece_rows(10, 100, 7) == 7
    with pytest.raises(ValueError, match="piece_size"):
        lce._piece_rows(10, 100, 0)


def test_binding_refuses_host_tensors_and_wrong_types():
    with pytest.raises(ValueError, match="HIP device"):
        lce.embed_fwd(torch.zeros(3, 4), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="bfloat16"):
        lce.embed_fwd(torch.zeros(3, 4, dtype=torch.float64), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="HIP device"):
        lce.embed_bwd(torch.zeros(3, 4), torch.zeros(3, dtype=torch.int32), 9)
    with pytest.raises(ValueError, match="HIP device"):
        lce.layernorm_fwd(torch.zeros(3, 4))
    with pytest.raises(TypeError, match="float32"):
        lce.layernorm_bwd(torch.zeros(3, 4), torch.zeros(3, 4, dtype=torch.int8), None, None)
    hid = torch.zeros(3, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        lce.flce_pieces_fwd(hid, hid, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="no pieces"):
        lce.flce_pieces_fwd(hid, [], torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="biases"):
        lce.flce_pieces_fwd(hid, [hid, hid], torch.zeros(3, dtype=torch.int32),
                            [torch.zeros(3)])


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A call for tensors of another device than the current one switches to it and takes that
    device's stream."""
    seen = []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("enter", self.device.index))

        def __exit__(self, *a):
            seen.append(("exit", self.device.index))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(lce, "_raw_stream", lambda t, index: 1000 + index)
    monkeypatch.setitem(lce._FNS, "embed_fwd", lambda *a: seen.append(("call", a)) or 0)
    lce._call("embed_fwd", torch.device("cuda", 0), "x")
    assert seen == [("call", ("x", 1000))]
    seen.clear()
    lce._call("embed_fwd", torch.device("cuda", 3), "x")
    assert seen == [("enter", 3), ("call", ("x", 1003)), ("exit", 3)]
    monkeypatch.setitem(lce._FNS, "embed_fwd", lambda *a: BAD_DTYPE)
    with pytest.raises(lce.LceError, match="type"):
        lce._call("embed_fwd", torch.device("cuda", 0))


def test_sizes_past_a_launch_are_refused(lib):
    """More threads than one launch holds (2^32 - 1) is a shape error, not the runtime's."""
    out = ctypes.c_size_t()
    ref = ctypes.byref(out)
    assert lib.embed_workspace_size(1 << 28, 16, 1 << 27, ref) == OK
    assert lib.embed_workspace_size((1 << 28) + 1, 16, 10, ref) == BAD_SHAPE
    assert lib.embed_workspace_size(4, 16, (1 << 27) + 1, ref) == BAD_SHAPE
    assert lib.embed_workspace_size(4, 1 << 20, (1 << 16) + 1, ref) == BAD_SHAPE
    assert lib.embed_workspace_size(1 << 28, 1 << 13, 10, ref) == BAD_SHAPE
    # weight, dtype, v, h, ldw, tokens, n, ignore_index, scale, out, ldo, status, stream
    far = 1 << 50

    def lookup(n, h, dtype=0):
        return lib.embed_fwd(A[0], dtype, 10, h, h, A[1] + far, n, -100, 1.0, A[2] + 2 * far, h,
                             None, None)
    assert lookup(1 << 24, 4096) == BAD_SHAPE and lookup(1 << 23, 4096, 2) == BAD_SHAPE
    assert lookup((1 << 31) - 1, 16) == BAD_SHAPE
    if no_gpu():
        assert lookup(15 << 20, 4096) in AT_DEVICE_CHECK
    assert lib.flce_piece_fwd_workspace_size(4, 8, 1 << 29, ref) == OK
    assert lib.flce_piece_fwd_workspace_size(4, 8, (1 << 29) + 1, ref) == BAD_SHAPE


def test_binding_refuses_a_wide_ignore_index(monkeypatch):
    monkeypatch.setattr(lce, "_require", lambda *a: None)
    hid = torch.zeros(3, 8, dtype=torch.bfloat16)
    idx = torch.zeros(3, dtype=torch.int64)
    f = torch.zeros(3)
    state = torch.zeros(3, 3)
    for ignore in (1 << 31, -(1 << 31) - 1, 1 << 40):
        kw = dict(ignore_index=ignore)
        for call in (lambda: lce.embed_fwd(hid, idx, **kw),
                     lambda: lce.embed_bwd(hid, idx, 5, **kw),
                     lambda: lce.flce_pieces_fwd(hid, hid, idx, **kw),
                     lambda: lce.flce_pieces_bwd(hid, hid, idx, f, **kw),
                     lambda: lce.flce_piece_fwd(hid, hid, idx, state, v_start=0, vocab=3,
                                                first=True, **kw),
                     lambda: lce.flce_piece_loss(state, idx, vocab=3, **kw),
                     lambda: lce.flce_piece_bwd(hid, hid, idx, f, v_start=0, vocab=3, first=True,
                                                last=True, **kw)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
    assert lce._ignore_arg(-(1 << 31)) == -(1 << 31)


def test_workspace_of_the_largest_piece_serves_the_others(lib):
    """At any batch the sizes grow with the piece, so that one workspace serves all pieces."""
    for n in (1, 32, 33, 128, 129, 700, 2048, 8192, 8193, 40000):
        for h in (64, 72, 1024):
            last = (0, 0)
            vs = sorted({1, 64, 100, 128, 2000, 65536} |
                        {k * 128 + d for k in (2, 4, 15, 16, 17, 64, 127, 128, 255, 256, 257)
                         for d in (0, 1)})
            for v in vs:
                size = (lce.flce_piece_fwd_workspace_size(n, h, v),
                        lce.flce_piece_bwd_workspace_size(n, h, v))
                assert size[0] >= last[0] and size[1] >= last[1], (n, h, v)
                last = size


def test_weights_without_a_buffer_get_their_gradient(monkeypatch):
    """None in a sequence of weight_grad_buffers: that weight's gradient is formed and returned
    (None where it needs none); the others' are added into their buffers."""
    from linear_cross_entropy_masked_amd import autograd as ag
    seen = {}

    def bwd(hidden, weights, labels, lse, bias, **kw):
        seen.update(kw)
        return "gh", None, None
    monkeypatch.setattr(ag, "flce_pieces_bwd", bwd)
    hid, lse = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(3)
    ws = [torch.ones(5, 8, dtype=torch.bfloat16), torch.ones(4, 8, dtype=torch.bfloat16)]
    buf = torch.full((4, 8), 2.0)
    cfg = (-100, 1, False, None, [None, buf])
    for need in (True, False):
        gh, gws, gbs = ag._piece_grads(hid, ws, [None, None], None, lse, lse.sum(), cfg, True,
                                       [need, True], [False, False])
        assert seen["accumulate"] == [False, True] and seen["grad_weight"][1] is buf
        assert gws[1] is None and gws[0] is seen["grad_weight"][0]
        assert (gws[0] is not None) == need
        assert not need or gws[0].dtype == torch.bfloat16 and gws[0].shape == (5, 8)


def test_a_hidden_gradient_without_a_place_is_refused(lib):
    """grad_hidden is written with the last piece: the pieces before need hidden_acc to carry it."""
    call = caller(lib.flce_piece_bwd, dict(hid=A[0], w=A[1], b=A[2], lab=A[3], lse=A[4], n=4, h=16,
                                           v=10, start=0, vocab=20, ign=-100, t=-1, flags=1,
                                           gout=None, grows=None, acc=None, gh=A[6], gw=A[7], wd=0,
                                           gb=A[8], ws=A[9], wsb=BIG, stream=None))
    assert call() == NULL_ARG and call(flags=0) == NULL_ARG and call(flags=2) == NULL_ARG
    if no_gpu():
        assert call(acc=A[5]) in AT_DEVICE_CHECK and call(flags=3) in AT_DEVICE_CHECK
        assert call(gh=None) in AT_DEVICE_CHECK


def test_default_pieces_stay_within_the_budget():
    """2 bytes a row (of whole tiles) and class, at least 4096 classes a piece."""
    for n in (1, 256, 257, 5000, 8192, 20000, 50000, 54321, 65536, 65537, 1 << 20, 1 << 23):
        up = -(-max(n, 1) // 256) * 256
        for v in (1, 700, 4097, 32777, 128256, 262144, 1 << 22):
            piece = lce._piece_rows(n, v, None)
            assert piece % 256 == 0 and 2 * up * piece <= max(lce._PIECE_BYTES, 2 * up * 4096)


def test_an_empty_batch_over_the_largest_table(lib):
    """Without positions one launch zeroes the table, a thread per 64 bytes: 2^32 of them at 2^36
    fp32 elements, one more than a launch holds."""
    out = ctypes.c_size_t()
    assert lib.embed_workspace_size(4, 1 << 20, 1 << 16, ctypes.byref(out)) == OK
    assert lib.embed_workspace_size(0, 1 << 20, 1 << 16, ctypes.byref(out)) == BAD_SHAPE
    call = caller(lib.embed_bwd, dict(g=None, dtype=2, ldg=1 << 20, tok=None, n=0, h=1 << 20,
                                      v=1 << 16, ign=-100, scale=1.0, flags=0, gw=A[2], gdtype=2,
                                      ldw=1 << 20, status=None, ws=1 << 45, wsb=BIG, stream=None))
    assert call() == BAD_SHAPE
    if no_gpu():
        assert call(v=64000) in AT_DEVICE_CHECK
