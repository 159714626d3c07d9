"""Host-side checks of the generation entry points (CPU only; no CUDA call is
made): argument validation of the C ABI before any launch, workspace sizes,
frequencies and tree masks."""
import ctypes
import math

import pytest
import torch

import exact_relative_position_b200 as rp
from exact_relative_position_b200 import _binding as bd
from exact_relative_position_b200.build import build_library

FAKE = 1 << 20   # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bd.load_library()


def _cache(**kw):
    c = bd.relpos_kv_cache(4, 16, 2, 64, 0, 0, FAKE, FAKE, None, None)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHE = [dict(format=4), dict(format=-1), dict(num_pages=0), dict(page_size=0), dict(page_size=24), dict(page_size=1 << 17),
             dict(kv_heads=0), dict(d=8), dict(d=72), dict(d=512), dict(k=None), dict(v=FAKE + 8), dict(format=2),
             dict(format=3, k_scale=FAKE), dict(format=3, k_scale=FAKE, v_scale=FAKE + 2),
             dict(num_pages=1 << 30, page_size=1 << 10)]


def _tree(**kw):
    a = bd.relpos_tree_args()
    a.cache = _cache(**{k[6:]: kw.pop(k) for k in list(kw) if k.startswith("cache_")})
    a.B, a.T, a.H, a.tau, a.max_seqlen, a.pages_per_seq = 2, 3, 4, 0.125, 64, 4
    a.map = bd.RelPosMap("truncated", clip=4).desc()
    for n in ("page_table", "lengths", "q", "k", "v", "aq", "b", "o", "lse"):
        setattr(a, n, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_tree_refusals(lib):
    run = lambda a, ws=FAKE, n=1 << 40: lib.relpos_tree_attn(ctypes.byref(a), ws, n, None)
    for kw in BAD_CACHE:
        assert run(_tree(**{"cache_" + k: v for k, v in kw.items()})) < 0, kw
    bad = [dict(B=0), dict(B=4097), dict(T=0), dict(T=65), dict(H=3), dict(H=0), dict(tau=0.0), dict(tau=float("nan")),
           dict(tau=float("inf")), dict(pages_per_seq=0), dict(pages_per_seq=1 << 27), dict(max_seqlen=0), dict(dtype=1), dict(dtype=2),
           dict(out_dtype=1), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(page_table=None), dict(lengths=None),
           dict(q=FAKE + 8), dict(aq=FAKE + 2), dict(q_stride_n=4), dict(k_stride_h=1), dict(v_stride_b=12), dict(tree_mask=FAKE + 4),
           dict(map=bd.relpos_map_desc(9, 0, 0, 0, 0)), dict(map=bd.relpos_map_desc(0, -1, 0, 0, 0)), dict(cache_d=96)]
    for kw in bad:
        assert run(_tree(**kw)) in (-1, -2), kw
    assert run(_tree(), None) == -3 and run(_tree(), FAKE, 64) == -3 and run(_tree(), FAKE + 8) == -3
    assert lib.relpos_tree_attn(None, FAKE, 1 << 40, None) == -1
    n = ctypes.c_size_t()
    assert lib.relpos_tree_workspace_size(ctypes.byref(_tree()), None) == -1
    assert lib.relpos_tree_workspace_size(ctypes.byref(_tree(T=65)), ctypes.byref(n)) == -1


def test_tree_workspace_grows_with_the_relation_terms_only(lib):
    def size(**kw):
        n = ctypes.c_size_t()
        assert lib.relpos_tree_workspace_size(ctypes.byref(_tree(**kw)), ctypes.byref(n)) == 0
        return n.value
    plain = size(aq=None, b=None, pages_per_seq=1024, max_seqlen=16384)
    assert plain == size(aq=None, b=None, pages_per_seq=4096, max_seqlen=65536)      # partial results: one set a block
    trunc = size(pages_per_seq=1024, max_seqlen=16384)
    assert 0 < trunc - plain <= 2 * 4 * 3 * 16 * 4 + 512                             # 9 offsets, padded to 16
    ident = size(pages_per_seq=1024, max_seqlen=16400, map=bd.RelPosMap("identity").desc())
    cols = 16384 + 3 + 3 + 1
    assert cols * 24 * 4 <= ident - plain <= (cols + 8) * 24 * 4 + 512


def test_rotary_and_cache_refusals(lib):
    steps = (ctypes.c_uint64 * 32)()
    def rot(**kw):
        a = bd.relpos_rotary_args(1, 2, 3, 64, 64, 0, 0, 0, 1.0, 8, None, 0, ctypes.cast(steps, ctypes.c_void_p))
        a.t[0] = bd.relpos_rotary_tensor(FAKE, FAKE, 2, 0, *[64] * 6)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.relpos_rotary(ctypes.byref(a), None)
    for kw in [dict(n_tensors=0), dict(n_tensors=3), dict(steps=None), dict(B=-1), dict(d=0), dict(rotary_dim=0), dict(rotary_dim=3),
               dict(rotary_dim=66), dict(dtype=3), dict(position_bytes=2), dict(positions=FAKE + 4), dict(magnitude=float("nan")),
               dict(magnitude=float("inf"))]:
        assert rot(**kw) in (-1, -2), kw
    assert rot(B=0) == 0 and rot(N=0) == 0                # nothing to do, nothing launched
    assert lib.relpos_rotary(None, None) == -1
    def write(cache=None, **kw):
        a = bd.relpos_cache_write_args(cache or _cache(), 1, 3, 0, 0, FAKE, FAKE, *[64] * 6, FAKE)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.relpos_cache_write(ctypes.byref(a), None)
    def read(cache=None, **kw):
        a = bd.relpos_cache_read_args(cache or _cache(), 1, 1, 3, 0, FAKE, FAKE, FAKE, FAKE)
        for k, v in kw.items():
            setattr(a, k, v)
        return lib.relpos_cache_read(ctypes.byref(a), None)
    for kw in BAD_CACHE:
        assert write(_cache(**kw)) < 0 and read(_cache(**kw)) < 0, kw
    for kw in [dict(dtype=1), dict(dtype=2), dict(B=-1), dict(k=None), dict(v=None), dict(slots=None), dict(k=FAKE + 8), dict(slots=FAKE + 4),
               dict(k_stride_n=63), dict(v_stride_h=4), dict(N=1 << 31 - 1, B=1 << 10)]:
        assert write(**kw) in (-1, -2), kw
    for kw in [dict(dtype=2), dict(B=0), dict(pages_per_seq=-1), dict(total_tokens=-1), dict(page_table=None), dict(cu_seqlens=None), dict(k=None),
               dict(v=FAKE + 4)]:
        assert read(**kw) in (-1, -2), kw
    assert write(N=0) == 0 and read(total_tokens=0) == 0


def test_rotary_steps_are_the_frequencies():
    for m in (rp.RotaryMap(64), rp.RotaryMap(128, base=500000.0, scaling="yarn", factor=8.0, original_length=8192),
              rp.RotaryMap(4, frequencies=(-1.0, 100.0))):
        for w, s in zip(m.angular(), m._steps):
            turn = w / (2 * math.pi) % 1.0
            assert abs(s / 2.0 ** 64 - turn) <= 2.0 ** -50 or abs(abs(s / 2.0 ** 64 - turn) - 1) <= 2.0 ** -50
    for kw in [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(rotary_dim=64, scaling="other"), dict(rotary_dim=64, base=-1.0),
               dict(rotary_dim=64, factor=0.0), dict(rotary_dim=2, scaling="ntk", factor=2.0), dict(rotary_dim=64, scaling="yarn", factor=2.0),
               dict(rotary_dim=64, frequencies=(1.0,)), dict(rotary_dim=2, frequencies=(float("inf"),))]:
        with pytest.raises(rp.RelPosError):
            rp.RotaryMap(**kw)


def test_tree_masks():
    m = rp.tree_masks([-1, 0, 0, 1, None])
    assert m.tolist() == [1, 3, 5, 11, 0]
    chain = rp.tree_masks(list(range(-1, 63)))
    assert chain[63].item() == -1 and chain[62].item() == 2 ** 63 - 1
    assert torch.equal(rp.tree_masks([[-1, 0], [-1, -1]]), torch.tensor([[1, 3], [1, 2]]))
