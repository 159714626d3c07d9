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
CODED = [(F16, E4M3), (BF16, E4M3), (F16, INT8), (BF16, INT8)]
CODED_IDS = ["f16-e4m3", "bf16-e4m3", "f16-int8", "bf16-int8"]
ROWS = [(1, 1, 1, 64), (4, 1, 4, 128), (4, 2, 13, 64), (2, 1, 30, 128), (8, 1, 20, 64)]   # H, Hkv, T, d: 1, 16, 26, 60, 160 rows
ROW_IDS = ["r1", "r16", "r26", "r60", "r160"]
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


def _values_of_one_size(s, size):
    """All value rows of about `size`, with a mean that does not cancel in a sum."""
    g = torch.Generator().manual_seed(11)
    c = s["cache"]
    rows = lambda *shape: (size * (1 + 0.3 * torch.randn(*shape, generator=g))).to(s["q"].dtype).cuda()
    n = c.num_pages * c.page_size
    k = torch.randn(n, c.kv_heads, c.d, generator=g).to(s["q"].dtype).cuda()
    rp.kv_cache_write(c, k, rows(n, c.kv_heads, c.d), torch.arange(n).cuda())
    s["v"] = rows(*s["v"].shape)


def _dominated(dt, fmt, H, Hkv, T, d, size, above, zero=False, node=True):
    """8000 keys and one, a node or a cached key, whose score lies about `above` over theirs for each row."""
    s = make(B=1, H=H, Hkv=Hkv, T=T, d=d, lens=[8000], page=64, dt=dt, fmt=fmt)
    _values_of_one_size(s, size)
    one = s["q"][:, :1, :1].float()
    s["q"] = (one + 0.05 * torch.randn(s["q"].shape, device="cuda")).to(dt)
    key = (one[:, 0, 0] * above / (s["tau"] * one.square().sum())).to(dt)                     # tau q.key = above
    if node:
        s["k"][:, :, 0] = key
        if zero:
            s["v"][:, :, 0] = 0
    else:
        slot = torch.tensor([int(s["table"][0, 70]) * 64 + 9]).cuda()
        row = key.expand(1, Hkv, d).contiguous()
        rp.kv_cache_write(s["cache"], row, row * 0 if zero else (row * 0 + size).to(dt), slot)
    return s


@pytest.mark.parametrize("dt,fmt", CODED, ids=CODED_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
@pytest.mark.parametrize("size", [0.02, 1e-4])
def test_small_values_beside_a_dominating_node(dt, fmt, H, Hkv, T, d, size):
    s = _dominated(dt, fmt, H, Hkv, T, d, size, 9.5)
    check(call(s), definition(s), dt)


@pytest.mark.parametrize("dt,fmt", CODED, ids=CODED_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
@pytest.mark.parametrize("node", [True, False], ids=["node", "cached"])
def test_small_values_beside_a_dominating_row_of_zeros(dt, fmt, H, Hkv, T, d, node):
    s = _dominated(dt, fmt, H, Hkv, T, d, 0.02, 9.5, zero=True, node=node)
    check(call(s), definition(s), dt)


def test_value_rows_of_zeros_only():
    for dt, fmt in CODED:
        s = make(B=2, H=2, Hkv=1, T=3, lens=[70, 9], dt=dt, fmt=fmt)
        c = s["cache"]
        z = torch.zeros(c.num_pages * c.page_size, 1, 64, dtype=dt, device="cuda")
        rp.kv_cache_write(c, z + 1, z, torch.arange(z.shape[0]).cuda())
        s["v"] *= 0
        o, lse = call(s)
        check((o, lse), definition(s), dt)
        assert bool((o == 0).all())


@pytest.mark.parametrize("dt,fmt", [(F16, F16), (BF16, INT8)], ids=["f16", "bf16-int8"])
@pytest.mark.parametrize("m", [rp.RelPosMap("log", num_buckets=5, max_distance=64), rp.RelPosMap("log_rev", num_buckets=7, max_distance=40),
                               rp.RelPosMap("t5", num_buckets=7, max_distance=64, bidirectional=0)], ids=lambda m: m.kind)
@pytest.mark.parametrize("H,Hkv,T", [(2, 1, 2), (4, 1, 20)])
def test_an_odd_number_of_buckets(dt, fmt, m, H, Hkv, T):
    # the rows of an odd number of log buckets end far beyond max_distance (here at 1985 and 270)
    s = make(B=2, H=H, Hkv=Hkv, T=T, lens=[2500, 400], page=64, dt=dt, fmt=fmt, map=m, aq="head", b=True)
    s["b"] *= 4
    check(call(s), definition(s), dt)


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
@pytest.mark.parametrize("tau", [None, 1.0])
def test_a_bias_of_minus_infinity_hides_far_keys(dt, fmt, H, Hkv, T, d, tau, low=-math.inf):
    # a window of 20: the saturated row of a truncated map hides all before it
    s = make(B=2, H=H, Hkv=Hkv, T=T, d=d, lens=[700, 15], dt=dt, fmt=fmt, map=rp.RelPosMap("truncated", clip=20), b=True, tree="tree")
    s["b"][:, 0] = low
    if tau is not None:
        s["tau"] = tau
    s["q"] *= 3
    for aq in (None, (0.5 * torch.randn(41, d, device="cuda")).to(dt)):
        s["aq"] = aq
        check(call(s), definition(s), dt)


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
@pytest.mark.parametrize("tau", [None, 1.0])
def test_the_lowest_bias_hides_far_keys(dt, fmt, H, Hkv, T, d, tau):
    test_a_bias_of_minus_infinity_hides_far_keys(dt, fmt, H, Hkv, T, d, tau, low=torch.finfo(torch.float32).min)


def test_a_bias_that_hides_everything():
    for dt, fmt in TYPES:
        for H, T in ((2, 3), (4, 30)):
            s = make(B=1, H=H, Hkv=1, T=T, lens=[300], dt=dt, fmt=fmt, map=rp.RelPosMap("truncated", clip=2), b=True)
            s["b"][:] = -math.inf
            o, lse = call(s)
            assert bool((o == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
def test_a_row_depends_on_its_own_query(dt, fmt, H, Hkv, T, d):
    # whatever one row holds (a padding node's anything, a head of another size), the others stay within their bounds
    s = make(B=2, H=H, Hkv=Hkv, T=T, d=d, lens=[90, 40], dt=dt, fmt=fmt, map=rp.RelPosMap("truncated", clip=8), aq="head", b=True)
    for big in ((3e38, 1e-30) if dt == BF16 else (6e4, 1e-6)):
        z = {**s, "q": s["q"].clone()}
        z["q"][0, H - 1, T - 1] = big
        got, want = call(z), definition(z)
        rest = [x.flatten(1, 2)[0, :H * T - 1] for x in want]
        if H * T > 1:
            check([x.flatten(1, 2)[0, :H * T - 1] for x in got], rest, dt, "the same sequence")
        check([x[1] for x in got], [x[1] for x in want], dt, "another sequence")


@pytest.mark.parametrize("fmt", [E4M3, INT8], ids=["e4m3", "int8"])
@pytest.mark.parametrize("q,k,v", [(1e-36, 1e36, 1.0), (1e30, 1e-30, 1e37), (1e-30, 3e29, 5e37)])
def test_bf16_numbers_near_the_ends_of_their_range(fmt, q, k, v):
    # the nodes alone: an 8-bit cache's own rows are coded with scales of their own
    s = make(B=1, H=2, Hkv=1, T=9, d=64, lens=[0], dt=BF16, fmt=fmt, tree="tree")
    s["q"] *= q
    s["k"] *= k
    s["v"] = (s["v"].clamp(-3, 3) * v).to(BF16)
    check(call(s), definition(s), BF16)


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("tau", [1e-39, 1e-30, 1e6])
def test_tau_far_from_its_usual_size(dt, fmt, T, tau):
    s = make(B=1, H=2, Hkv=1, T=T, d=64, lens=[200], dt=dt, fmt=fmt)
    s["tau"] = tau
    if tau > 1:
        s["q"] *= 1e-4
    check(call(s), definition(s), dt)


@pytest.mark.parametrize("dt,fmt", [(F16, F16), (BF16, INT8)], ids=["f16", "bf16-int8"])
def test_strides_of_dimensions_of_one_mean_nothing(dt, fmt):
    s = make(B=1, H=2, Hkv=1, T=1, d=64, lens=[40], dt=dt, fmt=fmt)
    want = call(s)
    z = dict(s)
    z["q"] = s["q"].as_strided((1, 2, 1, 64), (13, 64, 7, 1))
    z["k"], z["v"] = (s[x].as_strided((1, 1, 1, 64), (3, 5, 7, 1)) for x in "kv")
    got = call(z)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_cache_rows_and_rotary_with_strides_of_dimensions_of_one():
    x = torch.randn(1, 1, 1, 64, device="cuda").half()
    odd = x.as_strided((1, 1, 1, 64), (3, 5, 7, 1))
    a, b = (rp.kv_cache(1, 8, 1, 64, INT8) for _ in range(2))
    at = torch.tensor([[5]]).cuda()
    rp.kv_cache_write(a, x, x, at)
    rp.kv_cache_write(b, odd, odd, at)
    assert torch.equal(a.k, b.k) and torch.equal(a.v_scale, b.v_scale) and bool((a.k[0, 0, 5] != 0).any())
    rot = rp.RotaryMap(64)
    pos = torch.tensor([7]).cuda()
    want = rp.relpos_rotary(x, None, pos, rotary=rot)
    assert torch.equal(rp.relpos_rotary(odd, None, pos, rotary=rot), want)
    y = x.clone()                                        # in place through another view of the same rows
    rp.relpos_rotary(y, None, pos, rotary=rot, out=(y.as_strided((1, 1, 1, 64), (3, 5, 7, 1)),))
    assert torch.equal(y, want)


def test_the_lowest_bias_everywhere_stays_finite():
    for dt, fmt in TYPES:
        for H, T in ((2, 3), (4, 30)):
            s = make(B=2, H=H, Hkv=1, T=T, lens=[300, 0], dt=dt, fmt=fmt, map=rp.RelPosMap("truncated", clip=2), b=True)
            s["b"][:] = torch.finfo(torch.float32).min
            o, lse = call(s)
            assert bool(torch.isfinite(o).all()) and bool((lse < -1e7).all()) and bool(torch.isfinite(lse).all())


def test_a_tau_whose_base_2_form_is_infinite_is_refused():
    s = make(B=1, H=2, Hkv=1, T=2, lens=[20])
    for bad in (2.5e38, 1e39, math.inf):
        s["tau"] = bad
        with pytest.raises(rp.RelPosError):
            call(s)


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", ROWS, ids=ROW_IDS)
@pytest.mark.parametrize("low", [-1e6, -1e9])
@pytest.mark.parametrize("tau", [None, 1.0])
def test_a_large_bias_on_every_key_leaves_weights_and_lse(dt, fmt, H, Hkv, T, d, low, tau):
    # the same bias on all keys: the weights are those without it up to the rounding of the scores, the LSE is lower by it
    s = make(B=2, H=H, Hkv=Hkv, T=T, d=d, lens=[700, 15], dt=dt, fmt=fmt, map=rp.RelPosMap("truncated", clip=20), b=True, tree="tree")
    s["b"][:] = low
    if tau is not None:
        s["tau"] = tau
    o, lse = call(s)
    # scores carry rounding of 2^-24 of |bias| (64 at 1e9), so O is only an average of the values; the LSE is the bias, the
    # logarithm of at most 764 equal weights and the scores' own size away from it
    vmax = float(max(s["v"].abs().max(), (s["cache"].v.float().abs() * (1 if s["cache"].v_scale is None else s["cache"].v_scale[..., None])).max()))
    assert bool(torch.isfinite(o).all()) and float(o.abs().max()) <= vmax * (1 + 2.0 ** -7)
    # (the many-row kernel's terms end at 1.5 x 2^27 in base 2, 1.5 x 2^30 in bf16)
    end = math.log(2) * (1.5 * 2.0 ** (30 if dt == BF16 else 27) if fmt == dt and H // Hkv * T > 64 else math.inf)
    low = max(low, -end / s["tau"])
    own = s["tau"] * (8 * d ** 0.5 * 12 + 2.0 ** -22 * abs(low)) + 7
    assert float((lse.double() - s["tau"] * low).abs().max()) <= own + 2.0 ** -22 * abs(low) * s["tau"]


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("H,Hkv,T,d", [(1, 1, 33, 64), (2, 1, 11, 128), (4, 4, 3, 64), (8, 1, 31, 64), (8, 1, 8, 128)], ids=["r33", "r22", "r3", "r248", "r64"])
def test_nothing_depends_on_what_the_workspace_held(dt, fmt, H, Hkv, T, d):
    # rows of a tile that no query has must not vote on the maxima by relation terms that nobody wrote: sequence 0 is
    # empty, so most of its terms are left out
    s = make(B=3, H=H, Hkv=Hkv, T=T, d=d, lens=[0, 303, 1], dt=dt, fmt=fmt, map=rp.RelPosMap("identity"), aq="head", b=True)
    need = rp.tree_workspace_size(s["cache"], 3, T, H, s["table"].shape[1], aq=True, b=True, map=s["map"])
    want = None
    for fill in (0.0, 1e30, -1e30, 50.0, math.inf, -math.inf, math.nan):
        ws = torch.full((need // 4,), fill, device="cuda")
        got = call(s, workspace=ws)
        if want is None:
            want = got
            check(want, definition(s), dt)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), fill
