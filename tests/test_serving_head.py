"""Fp8Head as a module, on the CPU: what a cast or a move of a model around it does to what it holds."""
import copy

import pytest
import torch

from linear_cross_entropy_masked_amd import serving

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture
def make(monkeypatch):
    def quantize(w, *, block_rows, scale_dtype=None):
        n, h = w.shape
        gen = torch.Generator().manual_seed(0)
        q = torch.randint(0, 127, (n, h), generator=gen, dtype=torch.uint8).view(F8)
        c = torch.randint(1, 254, (-(-n // 128), -(-h // 128)), generator=gen, dtype=torch.uint8)
        return q, c.float() / 7 if scale_dtype == torch.float32 else c.view(E8)
    monkeypatch.setattr(serving, "fp8_quantize", quantize)

    def make(scale=None):
        return serving.Fp8Head(torch.randn(300, 144), torch.randn(144).bfloat16(),
                               torch.randn(300), scale_dtype=scale)
    return make


def bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int32)


@pytest.mark.parametrize("scale", [None, torch.float32])
@pytest.mark.parametrize("cast", [lambda m: m.half(), lambda m: m.to(torch.bfloat16),
                                  lambda m: m.float(), lambda m: m.double(), lambda m: m.bfloat16(),
                                  lambda m: m.type(torch.bfloat16), lambda m: m.to("cpu"),
                                  copy.deepcopy, lambda m: m.half().bfloat16()])
def test_casts_keep_what_is_held(make, scale, cast):
    head = make(scale)
    model = torch.nn.ModuleDict({"body": torch.nn.Linear(3, 3), "head": head})
    was = {name: (t.dtype, bits(t).clone()) for name, t in head.named_buffers()
           if name != "norm_weight"}
    assert set(was) == {"weight", "scales", "bias"}
    model = cast(model)
    for name, (dtype, held) in was.items():
        now = getattr(model["head"], name)
        assert now.dtype == dtype and now.shape == held.shape, name
        assert torch.equal(bits(now), held), name
    # what follows the hidden states' type does
    assert model["head"].norm_weight.dtype == model["body"].weight.dtype \
        or cast(torch.zeros(1).bfloat16()).dtype == torch.bfloat16


def test_moves_and_states(make):
    head = make()
    meta = copy.deepcopy(head).to("meta")
    assert meta.weight.device.type == "meta" and meta.weight.dtype == F8
    assert meta.scales.dtype == E8 and meta.bias.dtype == torch.float32
    assert meta.to_empty(device="cpu").weight.shape == (300, 144)
    other = make()
    other.weight.view(torch.uint8).zero_()
    other.load_state_dict(head.bfloat16().state_dict())
    assert torch.equal(bits(other.weight), bits(head.weight))
    bare = serving.Fp8Head(torch.randn(10, 16)).half()
    assert bare.bias is None and bare.norm_weight is None and bare.weight.dtype == F8
