"""CPU checks of calls of the norm, 8-bit product and beam search entry points beside those of
test_serve_boundary.py: what is refused and what passes the checks of arguments, with fake device
addresses."""
import ctypes

import torch

import linear_cross_entropy_masked_amd as lce
from test_serve_boundary import (A, ALIGN, AT_DEVICE_CHECK, BAD_DTYPE, BAD_SHAPE, BIG,  # noqa: F401
                                 NULL_ARG, OK, OVERLAP, WORKSPACE, BeamState, caller, lib, no_gpu)


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


def states_call(lib):  # noqa: F811
    """beam_reorder over states (in, out, overrides) of 2 entries of 4 beams, runs of 100 bytes that
    lie 200 apart: two such states fit into one another."""
    def call(states, slots=4):
        rows = (BeamState * len(states))()
        for r, (src, dst, kw) in zip(rows, states):
            kw = dict(dict(src=src, dst=dst, in_entry=800, in_beam=200, out_entry=200 * slots,
                           out_beam=200, segments=1, segment_bytes=100), **kw)
            for name, value in kw.items():
                setattr(r, name, value)
        return lib.beam_reorder(rows, len(states), A[0], 2, 4, slots, None)
    return call


def test_states_that_interlace(lib):  # noqa: F811
    """States that share no byte although the ranges that they span do: accepted. One byte shared:
    refused."""
    call = states_call(lib)
    if no_gpu():
        passes = [
            [(A[1], A[1], {}), (A[1] + 100, A[1] + 100, {})],  # keys and values of one tensor
            [(A[1] + 100, A[1] + 100, {}), (A[1], A[1], {})],
            [(A[1], A[2], {}), (A[1] + 100, A[2] + 100, {})],
            [(A[1], A[1] + 100, {})],  # from one half of a tensor into the other
            # other strides: heads of 10 bytes, 20 apart, beside a run in each of their gaps' beams
            [(A[1], A[1], {"segments": 5, "in_segment": 20, "out_segment": 20,
                           "segment_bytes": 10}), (A[1] + 100, A[1] + 100, {})],
            [(A[1], A[1], {"segments": 5, "in_segment": 20, "out_segment": 20,
                           "segment_bytes": 10}),
             (A[1] + 10, A[1] + 10, {"segments": 5, "in_segment": 20, "out_segment": 20,
                                     "segment_bytes": 10})],
            # one within the other's first entry alone
            [(A[1], A[1], {}), (A[1] + 100, A[1] + 100, {"in_entry": 1 << 20, "out_entry": 1 << 20,
                                                         "in_beam": 200, "out_beam": 200})],
            [(A[1] + 10 * i, A[1] + 10 * i, {"segment_bytes": 10}) for i in range(20)],
        ]
        for states in passes:
            assert call(states) in AT_DEVICE_CHECK, states
    for states in (
            [(A[1], A[1], {}), (A[1] + 99, A[1] + 99, {})],
            [(A[1], A[1], {}), (A[1] + 101, A[1] + 101, {})],
            [(A[1], A[1] + 99, {})], [(A[1], A[1] + 101, {})],
            [(A[1], A[2], {}), (A[1] + 100, A[2] + 101, {})],
            [(A[1], A[2], {}), (A[2] + 99, A[3], {})],
            [(A[1], A[1], {"segments": 5, "in_segment": 20, "out_segment": 20,
                           "segment_bytes": 10}),
             (A[1] + 10, A[1] + 10, {"segments": 5, "in_segment": 20, "out_segment": 20,
                                     "segment_bytes": 11})],
            [(A[1], A[1], {}), (A[1] + 700 - 100, A[1] + 700 - 100, {})],
            # met in the second entry's third beam alone
            [(A[1], A[1], {}), (A[1] + 1300 - 99, A[1] + 1300 - 99, {"in_entry": 1 << 20,
                                                                     "out_entry": 1 << 20})],
            [(A[1], A[1], {}), (A[0] - 4096, A[0] - 4096, {"in_entry": 1 << 20, "in_beam": 1366,
                                                           "out_entry": 1 << 20, "out_beam": 1366,
                                                           "segment_bytes": 1366})],
            [(A[1] + 10 * i, A[1] + 10 * i, {"segment_bytes": 10}) for i in range(20)]
            + [(A[1] + 3, A[1] + 3, {"segment_bytes": 1})]):
        assert call(states) == OVERLAP, states


def test_interlaced_states_against_their_bytes(lib):  # noqa: F811
    """Two or three states of drawn strides, in place, judged byte by byte."""
    import random

    def bytes_of(st):
        return {st["at"] + b * st["entry"] + k * st["beam"] + s * st["seg"] + i
                for b in range(2) for k in range(4) for s in range(st["n"])
                for i in range(st["len"])}
    rng = random.Random(7)
    kinds = set()
    for _ in range(3000):
        states = []
        for _ in range(rng.choice([2, 2, 3])):
            n, size = rng.randint(1, 3), rng.randint(1, 6)
            seg = size + rng.randint(0, 12)
            beam = n * seg + rng.randint(0, 24)
            entry = 4 * beam + rng.randint(0, 40)
            if rng.random() < 0.5 and states:  # as another one's, a little further on
                st = dict(states[0], at=states[0]["at"] + rng.randint(1, 30))
            elif rng.random() < 0.3:  # entries inside beams
                st = dict(at=rng.randint(0, 60), n=n, len=size, seg=seg, entry=n * seg,
                          beam=2 * n * seg + rng.randint(0, 9))
            else:
                st = dict(at=rng.randint(0, 60), n=n, len=size, seg=seg, beam=beam, entry=entry)
            states.append(st)
        sets = [bytes_of(st) for st in states]
        meet = any(a & b for i, a in enumerate(sets) for b in sets[:i])
        rows = (BeamState * len(states))()
        for r, st in zip(rows, states):
            r.src = r.dst = A[1] + st["at"]
            r.in_entry = r.out_entry = st["entry"]
            r.in_beam = r.out_beam = st["beam"]
            r.in_segment = r.out_segment = st["seg"]
            r.segments, r.segment_bytes = st["n"], st["len"]
        got = lib.beam_reorder(rows, len(states), A[0], 2, 4, 4, None)
        if meet:
            assert got == OVERLAP, states
        elif no_gpu():
            assert got in AT_DEVICE_CHECK, states
        kinds.add(meet)
    assert kinds == {True, False}


def test_a_great_many_interlaced_states(lib):  # noqa: F811
    """They are told apart within a bounded time, or refused."""
    def call(count, step):
        rows = (BeamState * count)()
        for i, r in enumerate(rows):
            r.src = r.dst = A[1] + i * step
            r.in_entry = r.out_entry = 4 << 20
            r.in_beam = r.out_beam = 1 << 20
            r.segments, r.segment_bytes = 1, 16
        return lib.beam_reorder(rows, count, A[0], 2, 4, 4, None)
    if no_gpu():
        assert call(200, 16) in AT_DEVICE_CHECK
    assert call(200, 15) == OVERLAP and call(1 << 16, 15) == OVERLAP
    if no_gpu():
        assert call(1 << 16, 16) in (*AT_DEVICE_CHECK, OVERLAP)


def test_interlaced_pairs_of_many_layers(lib):  # noqa: F811
    """Keys and values of each of 5000 layers in a tensor of their own: pairs, not a crowd."""
    rows = (BeamState * 10000)()
    for i, r in enumerate(rows):
        r.src = r.dst = A[1] + i // 2 * 2048 + i % 2 * 100
        r.in_entry = r.out_entry = 800
        r.in_beam = r.out_beam = 200
        r.segments, r.segment_bytes = 1, 100
    if no_gpu():
        assert lib.beam_reorder(rows, 10000, A[0], 2, 4, 4, None) in AT_DEVICE_CHECK
    rows[7001].src = rows[7001].dst = A[1] + 3500 * 2048 + 99
    assert lib.beam_reorder(rows, 10000, A[0], 2, 4, 4, None) == OVERLAP
