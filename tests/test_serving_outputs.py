"""Outputs that a call cannot write while it reads: refused on the host (CPU
only; no kernel is launched)."""
import pytest
import torch

import exact_relative_position_b200 as rp
from exact_relative_position_b200 import serving
from test_serving_copies import _OnDevice, _cache


@pytest.fixture
def launches(monkeypatch):
    seen = []
    monkeypatch.setattr(serving, "_launch", lambda name, *a: seen.append(name))
    monkeypatch.setattr(serving, "_cuda", lambda *a: None)
    return seen


def _rows(*shape):
    return torch.zeros(shape, dtype=torch.float16).as_subclass(_OnDevice)


def test_rotary_outputs_that_overlap_are_refused(launches):
    m = rp.RotaryMap(64)
    q, k, y = _rows(2, 3, 5, 64), _rows(2, 3, 5, 64), _rows(2, 3, 5, 64)
    long = _rows(2 * 2 * 3 * 5 * 64)
    first, shifted = long[:1920].view(2, 3, 5, 64), long[64:1984].view(2, 3, 5, 64)
    for bad in (dict(q=q, k=k, out=(k, q)),              # exchanged: each would be read after it was written
                dict(q=q, k=k, out=(y, y)), dict(q=q, k=k, out=(k, y)), dict(q=q, k=k, out=(y, q)),
                dict(q=q, k=q, out=(q, q)),              # turned twice, or once, as the blocks come
                dict(q=first, out=(shifted,)), dict(q=first, k=y, out=(q, shifted)), dict(q=q, k=y, out=(first, shifted))):
        with pytest.raises(rp.RelPosError):
            rp.relpos_rotary(bad["q"], bad.get("k"), rotary=m, out=bad["out"])
    assert not launches


def test_rotary_outputs_in_place_and_side_by_side_are_taken(launches):
    m = rp.RotaryMap(64)
    q, k, y = _rows(2, 3, 5, 64), _rows(2, 3, 5, 64), _rows(2, 3, 5, 64)
    fused = _rows(2, 5, 9, 64).transpose(1, 2)           # queries, keys and values of a token next to each other
    empty = _rows(2, 3, 0, 64)
    for good in (dict(q=q, k=k, out=(q, k)), dict(q=q, k=k, out=(q, y)), dict(q=q, out=(q,)), dict(q=q, k=q, out=(y, k)),
                 dict(q=fused[:, :3], k=fused[:, 3:6], out=(fused[:, :3], fused[:, 3:6])),
                 dict(q=fused[:, :3], k=y, out=(fused[:, 6:], y)), dict(q=empty, k=empty, out=(empty, empty))):
        rp.relpos_rotary(good["q"], good.get("k"), rotary=m, out=good["out"])
    assert len(launches) == 7


def test_a_cache_is_not_read_into_one_tensor_twice(launches, monkeypatch):
    cache = _cache(monkeypatch)
    table, cu = torch.zeros(1, 1, dtype=torch.int32), torch.tensor([0, 8], dtype=torch.int32)
    both = _rows(20, 2, 64)
    for bad in ((both[:8], both[:8]), (both[:8], both[4:12])):
        with pytest.raises(rp.RelPosError):
            rp.kv_cache_read(cache, table, cu, out=bad)
    rp.kv_cache_read(cache, table, cu, out=(both[:8], both[8:16]))
    assert launches == ["relpos_cache_read"]
