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
