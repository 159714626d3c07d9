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


@pytest.mark.parametrize("dt,fmt", [(F16, F16), (BF16, INT8)], ids=["f16", "bf16-int8"])
@pytest.mark.parametrize("m", [rp.RelPosMap("log", num_buckets=5, max_distance=64), rp.RelPosMap("log_rev", num_buckets=7, max_distance=40),
                               rp.RelPosMap("t5", num_buckets=7, max_distance=64, bidirectional=0)], ids=lambda m: m.kind)
@pytest.mark.parametrize("H,Hkv,T", [(2, 1, 2), (4, 1, 20)])
def test_an_odd_number_of_buckets(dt, fmt, m, H, Hkv, T):
    # the rows of an odd number of log buckets end far beyond max_distance (here at 1985 and 270)
    s = make(B=2, H=H, Hkv=Hkv, T=T, lens=[2500, 400], page=64, dt=dt, fmt=fmt, map=m, aq="head", b=True)
    s["b"] *= 4
    check(call(s), definition(s), dt)
