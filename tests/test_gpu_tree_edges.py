"""Attention of drafted tokens where values, tables and queries take their
unusual sizes: results against the fp64 definition, and rows that must not
depend on their neighbours."""
import math

import pytest
import torch

import exact_relative_position_b200 as rp
from test_gpu_tree_attention import BF16, E4M3, F16, INT8, TYPE_IDS, TYPES, call, make
from tree_definition import check, definition

pytestmark = pytest.mark.gpu
SPLIT = [(1, 2, 1, 64, 64, 100), (1, 2, 1, 40, 128, 120), (2, 6, 2, 60, 64, 250)]     # B, H, Hkv, T, d, length


@pytest.mark.parametrize("val", [math.nan, math.inf], ids=["nan", "inf"])
@pytest.mark.parametrize("dt", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("B,H,Hkv,T,d,n", SPLIT)
def test_a_non_finite_value_of_a_node_reaches_its_rows_across_pieces(val, dt, B, H, Hkv, T, d, n):
    # the nodes lie in two tiles of keys, and so few tiles are pieces of one tile each
    s = make(B=B, H=H, Hkv=Hkv, T=T, d=d, lens=[n] * B, dt=dt)
    # node 0 is attended by its children of odd number only; the others descend from node 1
    s["mask"] = rp.tree_masks([-1, -1] + [0 if t % 2 else 1 for t in range(2, T)]).cuda()
    clean = call(s)
    for node in (0, T - 1):                              # in the first of the two tiles, and in the last
        bad = {**s, "v": s["v"].clone()}
        bad["v"][:, :, node, 5] = val
        o, lse = call(bad)
        sees = torch.tensor([(int(x) >> node) & 1 for x in s["mask"].tolist()]).bool().cuda()
        assert torch.equal(lse, clean[1])
        assert torch.equal(o[:, :, ~sees], clean[0][:, :, ~sees])
        assert bool((~torch.isfinite(o[:, :, sees, 5])).all())
        cols = [i for i in range(d) if i != 5]
        assert torch.equal(o[:, :, sees][..., cols], clean[0][:, :, sees][..., cols])


@pytest.mark.parametrize("dt,fmt", [(F16, F16), (BF16, INT8)], ids=["f16", "bf16-int8"])
@pytest.mark.parametrize("m", [rp.RelPosMap("log", num_buckets=5, max_distance=64), rp.RelPosMap("log_rev", num_buckets=7, max_distance=40),
                               rp.RelPosMap("t5", num_buckets=7, max_distance=64, bidirectional=0)], ids=lambda m: m.kind)
@pytest.mark.parametrize("H,Hkv,T", [(2, 1, 2), (4, 1, 20)])
def test_an_odd_number_of_buckets(dt, fmt, m, H, Hkv, T):
    # the rows of an odd number of log buckets end far beyond max_distance (here at 1985 and 270)
    s = make(B=2, H=H, Hkv=Hkv, T=T, lens=[2500, 400], page=64, dt=dt, fmt=fmt, map=m, aq="head", b=True)
    s["b"] *= 4
    check(call(s), definition(s), dt)
