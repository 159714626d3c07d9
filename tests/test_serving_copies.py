"""Copies of the objects a model keeps for generation stand on their own: deep
copies and pickles of rotary maps work on their own frequencies (CPU only)."""
import copy
import ctypes
import pickle

import pytest
import torch

import exact_relative_position_b200 as rp
from exact_relative_position_b200 import serving


def _packed_steps(monkeypatch, rotary):
    """The steps that the call's argument block points to, read at the call."""
    seen = []

    def launch(name, dev, block):
        a = serving.relpos_rotary_args.from_buffer_copy(block)
        seen.extend((ctypes.c_uint64 * (a.rotary_dim // 2)).from_address(a.steps))
    monkeypatch.setattr(serving, "_launch", launch)

    class OnDevice(torch.Tensor):
        is_cuda = property(lambda self: True)
    rp.relpos_rotary(torch.zeros(1, 1, 1, 64).as_subclass(OnDevice), rotary=rotary)
    return seen


MAPS = [rp.RotaryMap(64), rp.RotaryMap(32, base=500000.0, interleaved=True, scaling="yarn", factor=8.0, original_length=8192),
        rp.RotaryMap(4, frequencies=(0.5, -2.0), magnitude=0.5)]


@pytest.mark.parametrize("how", [copy.deepcopy, copy.copy, lambda m: pickle.loads(pickle.dumps(m))], ids=["deepcopy", "copy", "pickle"])
@pytest.mark.parametrize("i", range(len(MAPS)))
def test_a_copied_map_has_its_own_steps(monkeypatch, how, i):
    make = lambda: type(MAPS[i])(**{f: getattr(MAPS[i], f) for f in MAPS[i].__dataclass_fields__})
    m = make()
    want = _packed_steps(monkeypatch, m)
    assert want == list(m._steps) and len(want) == m.rotary_dim // 2
    c = how(m)
    assert c == m and hash(c) == hash(m) and c._magnitude == m._magnitude
    del m
    junk = [make() for _ in range(50)]                   # whatever was freed is used again
    for j in junk:
        for n in range(len(j._steps)):
            j._steps[n] = 0x5555
    assert _packed_steps(monkeypatch, c) == want


def test_a_model_that_holds_a_map_is_copied_and_saved(monkeypatch):
    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.rotary = rp.RotaryMap(64)
    layer = Layer()
    other = copy.deepcopy(layer)
    layer.rotary._steps[0] = 1                           # the copy does not see it
    assert _packed_steps(monkeypatch, other.rotary) == _packed_steps(monkeypatch, rp.RotaryMap(64))
    assert pickle.loads(pickle.dumps(rp.RotaryMap(64))) == rp.RotaryMap(64)
