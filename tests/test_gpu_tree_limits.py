"""Attention of drafted tokens at the sizes where the kernels' limits lie."""
import pytest
import torch

import exact_relative_position_b200 as rp
from serving_harness import check_tree
from test_gpu_tree_attention import BF16, F16, call, make, want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dt", [(128, F16), (128, BF16), (64, F16)])
@pytest.mark.parametrize("B", [255, 256, 257])
def test_batches_around_the_list_of_sequences_of_a_block(B, d, dt):
    # 66 rows to a key head over a 16-bit cache: the many-row kernel as long as its list of sequences fits
    g = torch.Generator().manual_seed(B)
    s = make(B=B, H=2, Hkv=1, T=33, d=d, dt=dt, lens=torch.randint(0, 40, (B,), generator=g).tolist())
    check_tree(call(s), want(s), dt)
    y = rp.relpos_rotary(s["q"], rotary=rp.RotaryMap(d, magnitude=0.0))      # what follows is not disturbed
    assert bool((y == 0).all())


@pytest.mark.parametrize("T,n", [(4, 64), (7, 30), (40, 57)])
def test_a_workspace_by_the_helper_serves_a_longer_identity_table(T, n):
    s = make(B=1, H=4, Hkv=2, T=T, lens=[n], page=64, map=rp.RelPosMap("identity"), aq="head", b=True, N=500, tree="tree")
    ws = torch.empty(rp.tree_workspace_size(s["cache"], 1, T, 4, 1, aq=True, b=True, map=s["map"]), dtype=torch.uint8, device="cuda")
    check_tree(call(s, workspace=ws), want(s), F16)
    check_tree(call(s, workspace=ws, max_seqlen=None), want(s), F16)
