"""A call that the CUDA runtime refuses leaves nothing behind for the next one."""
import ctypes

import pytest
import torch

import exact_relative_position_b200 as rp

pytestmark = pytest.mark.gpu


def test_a_refused_call_does_not_fail_the_next():
    x = torch.randn(1, 2, 3, 64, device="cuda")
    rot = rp.RotaryMap(64)
    want = rp.relpos_rotary(x, rotary=rot)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    runtime = ctypes.CDLL("libcudart.so.12")             # the one that torch has loaded
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    # reading a status waits for its stream, which a stream that is being captured refuses
    assert runtime.cudaStreamBeginCapture(ctypes.c_void_p(st.cuda_stream), 2) == 0
    with torch.cuda.stream(st), pytest.raises(rp.RelPosError):
        rp.check_workspace(ws)
    graph = ctypes.c_void_p()
    assert runtime.cudaStreamEndCapture(ctypes.c_void_p(st.cuda_stream), ctypes.byref(graph)) != 0
    runtime.cudaGetLastError()
    assert torch.equal(rp.relpos_rotary(x, rotary=rot), want)
    cache = rp.kv_cache(1, 8, 2, 64, torch.int8)
    rows = torch.randn(3, 2, 64, device="cuda").half()
    rp.kv_cache_write(cache, rows, rows, torch.arange(3).cuda())
    assert bool((cache.k_scale[0, :, :3] != 1).all())
