"""Rotary embedding of more heads than a grid has rows."""
import pytest
import torch

import exact_relative_position_b200 as rp
from serving_harness import check_rotary, rotary64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hk", [(40000, 40000), (65535, 65535), (65535, 1)])
def test_many_heads(H, Hk):
    g = torch.Generator().manual_seed(1)
    q, k = torch.randn(1, H, 1, 4, generator=g).cuda(), torch.randn(1, Hk, 1, 4, generator=g).cuda()
    m = rp.RotaryMap(4)
    pos = torch.tensor([3]).cuda()
    for x, y in zip((q, k), rp.relpos_rotary(q, k, pos, rotary=m)):
        want, size = rotary64(x, pos[None], m.angular(), 1.0, 4, False)
        check_rotary(y, want, size, torch.float32)
