"""Rotary embedding against its fp64 definition: layouts, partial heads, far
positions, scalings, types, strides, in-place outputs, and gradients (against
the definition and against differences)."""
import math

import pytest
import torch

import exact_relative_position_b200 as rp
from serving_harness import check_rotary, rotary64

pytestmark = pytest.mark.gpu
gen = lambda s=0: torch.Generator().manual_seed(s)


def _pos(positions, B, N):
    if positions is None:
        return torch.arange(N)[None].expand(B, N)
    return positions.cpu()[None].expand(B, N) if positions.dim() == 1 else positions.cpu()


CASES = [
    dict(B=2, H=3, Hk=1, N=5, d=64, r=64, dtype=torch.float16),
    dict(B=1, H=4, Hk=2, N=129, d=128, r=96, dtype=torch.bfloat16, inter=True),
    dict(B=3, H=1, Hk=1, N=1, d=64, r=2, dtype=torch.float32),
    dict(B=1, H=2, Hk=2, N=7, d=66, r=22, dtype=torch.float16),              # no 16-byte rows
    dict(B=1, H=2, Hk=2, N=7, d=66, r=22, dtype=torch.float32, inter=True),
    dict(B=2, H=40, Hk=8, N=33, d=256, r=256, dtype=torch.bfloat16),
    dict(B=2, H=2, Hk=1, N=64, d=128, r=32, dtype=torch.float32),
    dict(B=1, H=12, Hk=12, N=3000, d=64, r=64, dtype=torch.float16, inter=True),   # several heads to a thread
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: f"{c['B']}x{c['H']}x{c['N']}x{c['d']}-r{c['r']}-{str(c['dtype'])[6:]}")
@pytest.mark.parametrize("pos", ["none", "far", "wide"])
def test_matches_definition(c, pos):
    g = gen(1)
    B, N, dt = c["B"], c["N"], c["dtype"]
    q = torch.randn(B, c["H"], N, c["d"], generator=g).to(dt).cuda()
    k = torch.randn(B, c["Hk"], N, c["d"], generator=g).to(dt).cuda()
    p = None
    if pos == "far":
        p = torch.randint(0, 1 << 20, (B, N), generator=g, dtype=torch.int32).cuda()
    if pos == "wide":
        p = (torch.arange(N) * 1001 - 500).cuda()       # int64, shared by the batch, negative ones among them
    m = rp.RotaryMap(c["r"], interleaved=c.get("inter", False))
    yq, yk = rp.rotary_embedding(q, k, p, rotary=m)
    for x, y in ((q, yq), (k, yk)):
        want, size = rotary64(x, _pos(p, B, N), m.angular(), 1.0, c["r"], m.interleaved)
        check_rotary(y, want, size, dt)
        assert torch.equal(y[..., c["r"]:], x[..., c["r"]:])
    assert torch.equal(rp.rotary_embedding(q, None, p, rotary=m), yq)


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=8.0, original_length=2048),
                                dict(scaling="yarn", factor=1.0, original_length=2048),
                                dict(base=500000.0, magnitude=0.5), dict(frequencies=tuple(7.0 / (i + 1) for i in range(32)))],
                         ids=["linear", "ntk", "yarn", "yarn1", "magnitude", "frequencies"])
def test_scalings(kw):
    g = gen(2)
    q = torch.randn(1, 2, 40, 64, generator=g).cuda()
    p = torch.randint(0, 200000, (40,), generator=g).cuda()
    m = rp.RotaryMap(64, **kw)
    i = torch.arange(32, dtype=torch.float64)
    base, f = kw.get("base", 10000.0), kw.get("factor", 1.0)
    w = base ** (-2 * i / 64)
    mag = kw.get("magnitude", 1.0)
    if kw.get("scaling") == "linear":
        w = w / f
    if kw.get("scaling") == "ntk":
        w = (base * f ** (64 / 62)) ** (-2 * i / 64)
    if kw.get("scaling") == "yarn":
        turns = 2048 * w / (2 * math.pi)
        share = ((turns - 1) / 31).clamp(0, 1)
        w, mag = share * w + (1 - share) * w / f, 1 + 0.1 * math.log(f)
    if "frequencies" in kw:
        w = torch.tensor(kw["frequencies"], dtype=torch.float64)
    want, size = rotary64(q, p[None], w.tolist(), mag, 64, False)
    check_rotary(rp.rotary_embedding(q, None, p, rotary=m), want, size, torch.float32)


@pytest.mark.parametrize("inter", [False, True])
def test_gradients(inter):
    g = gen(3)
    m = rp.RotaryMap(48, interleaved=inter, scaling="yarn", factor=4.0, original_length=512)
    q = torch.randn(2, 3, 17, 64, generator=g).cuda().requires_grad_()
    k = torch.randn(2, 1, 17, 64, generator=g).cuda().requires_grad_()
    p = torch.randint(0, 5000, (2, 17), generator=g).cuda()
    dq, dk = torch.randn(q.shape, generator=g).cuda(), torch.randn(k.shape, generator=g).cuda()
    yq, yk = rp.rotary_embedding(q, k, p, rotary=m)
    gq, gk = torch.autograd.grad((yq, yk), (q, k), (dq, dk))
    for x, y in ((dq, gq), (dk, gk)):
        want, size = rotary64(x, p, m.angular(), m._magnitude, 48, inter, inverse=True)
        check_rotary(y, want, size, torch.float32)
    # differences: the map is linear, so (f(x + e d) - f(x - e d)) / 2e equals f(d) up to rounding
    d = torch.randn(q.shape, generator=g).cuda()
    f = lambda x: (rp.rotary_embedding(x.detach(), None, p, rotary=m).double() * dq.double()).sum()
    num = (f(q + 0.5 * d) - f(q - 0.5 * d)).item()
    ana = (gq.double() * d.double()).sum().item()
    # about 6000 terms of size 1, each within 3 fp32 roundings of values up to 8: 6000^(1/2) x 8 x 2^-22 typical
    assert abs(num - ana) <= 6000 * 8 * 2.0 ** -22
    # one output unused, a broadcast upstream gradient, and the gradient's own gradient
    assert torch.autograd.grad(rp.rotary_embedding(q, k, p, rotary=m)[1].sum(), k)[0].shape == k.shape
    y = rp.rotary_embedding(q, None, p, rotary=m)
    first, = torch.autograd.grad(y, q, dq.requires_grad_(), create_graph=True)
    second, = torch.autograd.grad(first, dq, d)
    assert torch.equal(second, rp.relpos_rotary(d, None, p, rotary=m))
    assert torch.equal(torch.autograd.grad(rp.rotary_embedding(q, None, p, rotary=m).sum(), q)[0],
                       rp.relpos_rotary(torch.ones_like(d), None, p, rotary=m, inverse=True))


def test_layouts_agree():
    g = gen(4)
    m = rp.RotaryMap(64)
    x = torch.randn(2, 9, 5, 64, generator=g).half().cuda()                   # token-major storage
    p = torch.randint(0, 1000, (2, 9), generator=g).cuda()
    want = rp.relpos_rotary(x.transpose(1, 2).contiguous(), None, p, rotary=m)
    assert torch.equal(rp.relpos_rotary(x.transpose(1, 2), None, p, rotary=m), want)
    packed = rp.relpos_rotary(x.reshape(18, 5, 64), None, p.reshape(-1), rotary=m)
    assert torch.equal(packed.view(2, 9, 5, 64).transpose(1, 2), want)
    # rows that do not start on 16 bytes, a last dimension that is not contiguous, and in place
    odd = torch.randn(2, 5, 9, 67, generator=g).half().cuda()[..., 3:]
    assert torch.equal(rp.relpos_rotary(odd, None, p, rotary=m), rp.relpos_rotary(odd.contiguous(), None, p, rotary=m))
    cols = x.transpose(1, 2).contiguous().transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(rp.relpos_rotary(cols, None, p, rotary=m), want)
    y = x.transpose(1, 2).contiguous()
    assert rp.relpos_rotary(y, None, p, rotary=m, out=(y,)) is y and torch.equal(y, want)
    assert torch.equal(rp.relpos_rotary(want, None, p, rotary=rp.RotaryMap(64, magnitude=0.0)), torch.zeros_like(want))


def test_offsets_alone_matter():
    # q.k after the turn depends on the offset of the positions only
    g = gen(5)
    m = rp.RotaryMap(64, base=500000.0)
    q, k = (torch.randn(1, 1, 1, 64, generator=g).cuda() for _ in range(2))
    def dot(i, j):
        a = rp.relpos_rotary(q, None, torch.tensor([i]).cuda(), rotary=m)
        b = rp.relpos_rotary(k, None, torch.tensor([j]).cuda(), rotary=m)
        return (a.double() * b.double()).sum().item()
    assert abs(dot(5, 2) - dot(1000005, 1000002)) <= 64 * 4 * 1e-6   # 64 products of size ~1, each 2e-6 off


def test_empty_and_refusals():
    m = rp.RotaryMap(64)
    x = torch.randn(1, 2, 3, 64).cuda()
    assert rp.relpos_rotary(x[:, :, :0], rotary=m).shape == (1, 2, 0, 64)
    assert rp.relpos_rotary(x[:, :0], rotary=m).shape == (1, 0, 3, 64)
    bad = [lambda: rp.relpos_rotary(x.double(), rotary=m), lambda: rp.relpos_rotary(x[..., :32], rotary=m),
           lambda: rp.relpos_rotary(x.cpu(), rotary=m), lambda: rp.relpos_rotary(x, x.half(), rotary=m),
           lambda: rp.relpos_rotary(x, x[:, :, :2], rotary=m),
           lambda: rp.relpos_rotary(x, None, torch.arange(4).cuda(), rotary=m),
           lambda: rp.relpos_rotary(x, None, torch.arange(3.0).cuda(), rotary=m),
           lambda: rp.relpos_rotary(x, None, torch.arange(3), rotary=m),
           lambda: rp.relpos_rotary(x, rotary=m, out=(x[..., :32],)),
           lambda: rp.relpos_rotary(x, rotary=m, out=(x, x)),
           lambda: rp.relpos_rotary(x, rotary=m, out=(torch.empty(1, 1, 3, 64).cuda().expand(1, 2, 3, 64),))]
    for f in bad:
        with pytest.raises(rp.RelPosError):
            f()
