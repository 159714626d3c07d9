"""Copies of the objects a model keeps for generation stand on their own: deep
copies and pickles of rotary maps work on their own frequencies, copies of a
cache on their own pages (CPU only)."""
import copy
import ctypes
import pickle

import pytest
import torch

import exact_relative_position_b200 as rp
from exact_relative_position_b200 import serving


class _OnDevice(torch.Tensor):
    """A host tensor that passes for one on the device."""
    is_cuda = property(lambda self: True)

    def __deepcopy__(self, memo):
        return self.as_subclass(torch.Tensor).clone().as_subclass(_OnDevice)


def _packed_steps(monkeypatch, rotary):
    """The steps that the call's argument block points to, read at the call."""
    seen = []

    def launch(name, dev, block):
        a = serving.relpos_rotary_args.from_buffer_copy(block)
        seen.extend((ctypes.c_uint64 * (a.rotary_dim // 2)).from_address(a.steps))
    monkeypatch.setattr(serving, "_launch", launch)

    rp.relpos_rotary(torch.zeros(1, 1, 1, 64).as_subclass(_OnDevice), rotary=rotary)
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


def _cache(monkeypatch, coded=True):
    monkeypatch.setattr(serving, "_cuda", lambda *a: None)
    dt = torch.int8 if coded else torch.float16
    new = lambda *shape, dtype=dt: torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)
    scale = lambda: new(3, 2, 8, dtype=torch.float32) if coded else None
    return rp.KVCache(new(3, 2, 8, 64), new(3, 2, 8, 64), scale(), scale())


def _written_to(monkeypatch, cache):
    """The pointers of a write's argument block."""
    seen = []
    monkeypatch.setattr(serving, "_launch", lambda name, dev, block: seen.append(serving.relpos_cache_write_args.from_buffer_copy(block)))
    x = torch.zeros(1, 2, 64, dtype=torch.float16)
    rp.kv_cache_write(cache, x, x, torch.zeros(1, dtype=torch.int64))
    c = seen[0].cache
    return [c.k, c.v, c.k_scale, c.v_scale]


@pytest.mark.parametrize("coded", [True, False], ids=["int8", "f16"])
def test_a_copied_cache_has_its_own_pages(monkeypatch, coded):
    a = _cache(monkeypatch, coded)
    b = copy.deepcopy(a)
    for c in (a, b):
        assert _written_to(monkeypatch, c) == [None if t is None else t.data_ptr() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    assert a.k.data_ptr() != b.k.data_ptr() and _written_to(monkeypatch, a) != _written_to(monkeypatch, b)
    assert (b.num_pages, b.kv_heads, b.page_size, b.d, b.dtype) == (3, 2, 8, 64, a.dtype)
    for name in ("k", "v", "k_scale", "v_scale"):        # other pages are another cache
        with pytest.raises(AttributeError):
            setattr(a, name, getattr(b, name))
