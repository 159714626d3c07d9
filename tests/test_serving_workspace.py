"""Workspace sizes of the attention of drafted tokens (host only): the helper's
bytes are enough for the call whatever table an identity map brings, and the
saturated rows of a map are found wherever they begin."""
import ctypes

import pytest
import torch

import exact_relative_position_b200 as rp
from exact_relative_position_b200 import _binding as bd
from exact_relative_position_b200.build import build_library

FAKE = 1 << 20   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build_library()
    return bd.load_library()


def _bytes(lib, m, N, pages, page, B=1, T=4, H=2, aq=FAKE, b=FAKE):
    a = bd.relpos_tree_args()
    a.cache = bd.relpos_kv_cache(8, page, 2, 64, 0, 0, FAKE, FAKE, None, None)
    a.B, a.T, a.H, a.tau, a.max_seqlen, a.pages_per_seq = B, T, H, 0.125, N, pages
    a.map, a.aq, a.b = m.desc(), aq, b
    n = ctypes.c_size_t()
    assert lib.relpos_tree_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("pages,page", [(1, 64), (1, 16), (3, 16), (2, 1), (5, 32)])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 64])
def test_the_helper_covers_longer_identity_tables(lib, pages, page, T):
    # the helper does not know the table: it counts the offsets that the pages and nodes can reach
    m = rp.RelPosMap("identity")
    helper = _bytes(lib, m, pages * page + T, pages, page, T=T)
    for N in (1, pages * page, pages * page + T + 1, pages * page + 64, 10000):
        assert _bytes(lib, m, N, pages, page, T=T) <= helper


MAPS = [rp.RelPosMap("log", num_buckets=5, max_distance=64), rp.RelPosMap("log", num_buckets=16, max_distance=64),
        rp.RelPosMap("log_rev", num_buckets=5, max_distance=64), rp.RelPosMap("log_rev", num_buckets=33, max_distance=128),
        rp.RelPosMap("log", num_buckets=2, max_distance=8), rp.RelPosMap("log", num_buckets=3, max_distance=9),
        rp.RelPosMap("log", num_buckets=256, max_distance=512),
        rp.RelPosMap("t5", num_buckets=32, max_distance=128, bidirectional=0), rp.RelPosMap("t5", num_buckets=7, max_distance=50, bidirectional=0),
        rp.RelPosMap("t5", num_buckets=32, max_distance=128, bidirectional=1), rp.RelPosMap("t5", num_buckets=10, max_distance=1000, bidirectional=1),
        rp.RelPosMap("truncated", clip=0), rp.RelPosMap("truncated", clip=9), rp.RelPosMap("identity")]


@pytest.mark.parametrize("m", MAPS, ids=lambda m: f"{m.kind}-{m.num_buckets or m.clip}-{m.max_distance}-{m.bidirectional}")
def test_relation_rows_end_where_the_map_saturates(lib, m):
    # the layer's own bounds scan every offset; the stored offsets are those between them that can be reached
    for T in (1, 5):
        for pages in (1, 4, 150):                        # capacity 16, 64 and 2400
            for N in (1, 2, 17, 64 + T, 130, 2400 + T, 5000):
                lo, hi = ctypes.c_int32(), ctypes.c_int32()
                assert lib.relpos_expanded_bounds(ctypes.byref(m.desc()), N, ctypes.byref(lo), ctypes.byref(hi)) == 0
                lo, hi, back = lo.value, hi.value, -(16 * pages + T - 1)
                if lo > T:
                    hi = lo
                elif hi < back:
                    lo = hi
                else:
                    lo, hi = max(lo, back), min(hi, T)
                columns = (hi - lo + 1 + 7) // 8 * 8
                rows = _bytes(lib, m, N, pages, 16, T=T) - _bytes(lib, m, N, pages, 16, T=T, aq=None, b=None)
                assert rows == -(-4 * columns * T * 2 // 256) * 256, (T, pages, N)
