"""Attention of drafted tokens over the paged cache against its fp64
definition: formats, types, head sharing, tree shapes, maps, empty and odd
lengths, padding nodes, bad pages, non-finite values in masked places, split
work, streams and captured graphs."""
import pytest
import torch

import exact_relative_position_b200 as rp
from serving_harness import check_tree, make_pages, tree64

pytestmark = pytest.mark.gpu
F16, BF16, E4M3, INT8 = torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int8


def make(seed=0, B=1, H=2, Hkv=2, T=1, d=64, lens=(5,), page=16, dt=F16, fmt=None, map=None, aq=None, b=False, tree="chain",
         N=None, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    fmt = dt if fmt is None else fmt
    lens = list(lens)
    table, pages = make_pages(g, lens, page)
    cache = rp.kv_cache(pages, page, Hkv, d, fmt)
    total = pages * page
    rows = lambda n: (torch.randn(n, Hkv, d, generator=g) * torch.exp(0.5 * torch.randn(n, Hkv, 1, generator=g)) * scale).to(dt).cuda()
    rp.kv_cache_write(cache, rows(total), rows(total), torch.arange(total).cuda())
    s = dict(cache=cache, table=table.cuda(), lens=torch.tensor(lens, dtype=torch.int32).cuda(), tau=d ** -0.5, map=map)
    s["q"] = torch.randn(B, H, T, d, generator=g).to(dt).cuda()
    s["k"], s["v"] = (torch.randn(B, Hkv, T, d, generator=g).to(dt).cuda() for _ in range(2))
    if tree == "chain":
        s["mask"] = None
    elif tree == "tree":
        s["mask"] = rp.tree_masks([[-1] + [int(torch.randint(0, i, (1,), generator=g)) for i in range(1, T)] for _ in range(B)]).cuda()
    elif tree == "padded":
        s["mask"] = rp.tree_masks([-1] + [max(0, i - 2) if i < T - T // 3 else None for i in range(1, T)]).cuda()
    else:
        s["mask"] = torch.randint(-2 ** 62, 2 ** 62, (B, T), generator=g).cuda()   # any bits, no tree at all
    s["N"] = N if N is not None else table.shape[1] * page + T
    R = rp.table_rows(map, s["N"]) if map is not None else 0
    s["aq"] = None if aq is None else (0.5 * torch.randn(*((H,) if aq == "head" else ()), R, d, generator=g)).to(dt).cuda()
    s["b"] = torch.randn(H, R, generator=g).cuda() if b else None
    return s


def call(s, **kw):
    kw.setdefault("max_seqlen", s["N"] if s["map"] is not None else None)
    return rp.relpos_tree_attention(s["q"], s["k"], s["v"], s["cache"], s["table"], s["lens"], s["aq"], s["b"], tau=s["tau"],
                                    map=s["map"], tree_mask=s["mask"], **kw)


def want(s):
    return tree64(s["q"], s["k"], s["v"], s["cache"], s["table"], s["lens"], s["aq"], s["b"], s["tau"], s["map"], s["N"], s["mask"])


TYPES = [(F16, F16), (BF16, BF16), (F16, E4M3), (BF16, E4M3), (F16, INT8), (BF16, INT8)]
TYPE_IDS = ["f16", "bf16", "f16-e4m3", "bf16-e4m3", "f16-int8", "bf16-int8"]
SHAPES = [
    dict(B=1, H=1, Hkv=1, T=1, d=64, lens=[1], page=16),
    dict(B=3, H=4, Hkv=2, T=1, d=64, lens=[0, 63, 129], page=8),
    dict(B=2, H=8, Hkv=1, T=1, d=128, lens=[300, 17], page=32),
    dict(B=2, H=3, Hkv=3, T=7, d=64, lens=[64, 200], page=64, tree="tree"),
    dict(B=1, H=8, Hkv=2, T=6, d=64, lens=[257], page=1, tree="padded"),       # 24 rows a key head
    dict(B=2, H=4, Hkv=2, T=13, d=128, lens=[0, 131], page=16, tree="tree"),   # 26 rows
    dict(B=1, H=4, Hkv=1, T=64, d=64, lens=[95], page=16, tree="tree"),        # 256 rows
    dict(B=2, H=6, Hkv=2, T=33, d=128, lens=[70, 3], page=16, tree="bits"),    # 99 rows
    dict(B=1, H=1, Hkv=1, T=64, d=128, lens=[0], page=16, tree="bits"),
    dict(B=2, H=2, Hkv=1, T=33, d=64, lens=[500, 128], page=16, tree="tree"),  # 66 rows: one tile of 128
    dict(B=2, H=8, Hkv=2, T=61, d=128, lens=[700, 64], page=8, tree="tree"),   # 244 rows: two tiles
    dict(B=2, H=10, Hkv=2, T=64, d=64, lens=[1, 385], page=1, tree="bits"),    # 320 rows: a block of two, one of one
    dict(B=1, H=9, Hkv=1, T=60, d=128, lens=[0], page=64, tree="padded"),      # 540 rows, no cache
]


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"h{s['H']}-{s['Hkv']}-T{s['T']}-d{s['d']}-L{'-'.join(map(str, s['lens']))}")
def test_matches_definition(dt, fmt, shape):
    s = make(dt=dt, fmt=fmt, **shape)
    check_tree(call(s), want(s), dt)


MAPS = [
    (rp.RelPosMap("truncated", clip=16), "shared", True), (rp.RelPosMap("truncated", clip=0), "head", True),
    (rp.RelPosMap("truncated", clip=1000), None, True), (rp.RelPosMap("identity"), "head", True),
    (rp.RelPosMap("identity"), "shared", False),
    (rp.RelPosMap("t5", num_buckets=32, max_distance=128, bidirectional=0), None, True),
    (rp.RelPosMap("t5", num_buckets=32, max_distance=128, bidirectional=1), None, True),
    (rp.RelPosMap("log", num_buckets=16, max_distance=64), "shared", False),
    (rp.RelPosMap("log_rev", num_buckets=32, max_distance=128), "head", True),
]


@pytest.mark.parametrize("dt,fmt", [(F16, F16), (BF16, INT8)], ids=["f16", "bf16-int8"])
@pytest.mark.parametrize("m,aq,b", MAPS, ids=lambda x: x.kind + str(x.clip or "") if isinstance(x, rp.RelPosMap) else str(x))
@pytest.mark.parametrize("shape", [dict(B=2, H=4, Hkv=2, T=5, d=64, lens=[300, 0], page=16, tree="tree"),
                                   dict(B=1, H=2, Hkv=1, T=64, d=128, lens=[150], page=32, tree="tree"),
                                   dict(B=2, H=2, Hkv=2, T=1, d=64, lens=[700, 33], page=64)], ids=["T5", "T64", "T1"])
def test_relation_terms(dt, fmt, m, aq, b, shape):
    s = make(dt=dt, fmt=fmt, map=m, aq=aq, b=b, **shape)
    check_tree(call(s), want(s), dt)


def test_identity_table_longer_than_the_cache():
    s = make(B=1, H=2, Hkv=2, T=3, lens=[40], map=rp.RelPosMap("identity"), aq="shared", b=True, N=500)
    check_tree(call(s), want(s), F16)
    check_tree(call(s, max_seqlen=None), want(s), F16)


@pytest.mark.parametrize("T,H,dt", [(3, 4, BF16), (40, 8, F16)])            # 6 rows; 160, the many-row kernel
def test_identity_over_a_long_cache(T, H, dt):
    # more offsets than any bucketed map has, over several blocks of the projection
    s = make(B=2, H=H, Hkv=2, T=T, lens=[3001, 1290], page=16, dt=dt, map=rp.RelPosMap("identity"), aq="head", b=True, tree="tree")
    check_tree(call(s), want(s), dt)


def test_positions_past_the_table_are_clamped():
    s = make(B=1, H=2, Hkv=2, T=3, lens=[90], map=rp.RelPosMap("identity"), aq="shared", b=True, N=50)
    check_tree(call(s), want(s), F16)


@pytest.mark.parametrize("fmt", [F16, E4M3], ids=["f16", "e4m3"])
@pytest.mark.parametrize("T,H,Hkv,d", [(1, 4, 4, 64), (4, 8, 2, 128), (20, 8, 2, 64), (48, 8, 2, 128)])
def test_long_split_over_many_blocks(fmt, T, H, Hkv, d):
    s = make(B=3, H=H, Hkv=Hkv, T=T, d=d, lens=[9000, 1, 4097], page=64, fmt=fmt, tree="tree",
             map=rp.RelPosMap("truncated", clip=64), aq="shared", b=True)
    got = call(s)
    check_tree(got, want(s), F16)
    again = call(s)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_many_rows_many_items():
    # pieces of the line that hold several items and parts of others, one and two row tiles in turn
    g = torch.Generator().manual_seed(7)
    s = make(B=40, H=20, Hkv=4, T=64, d=64, lens=torch.randint(0, 700, (40,), generator=g).tolist(), tree="tree",
             map=rp.RelPosMap("log", num_buckets=16, max_distance=64), aq="head", b=True)
    got = call(s)
    check_tree(got, want(s), F16)
    for _ in range(3):
        again = call(s)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_bounded_waits_report():
    # a limit of one nanosecond lets the many-row kernel's waits run out: it stops, and the workspace says so
    s = make(B=4, H=16, Hkv=2, T=32, d=128, lens=[900, 700, 1000, 50], page=16)
    need = rp.tree_workspace_size(s["cache"], 4, 32, 16, s["table"].shape[1])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call(s, workspace=ws)
    assert rp.check_workspace(ws) == 0
    rp.set_wait_limit_ns(1)
    try:
        call(s, workspace=ws)
        with pytest.raises(rp.RelPosError, match="timed out"):
            rp.check_workspace(ws)
    finally:
        rp.set_wait_limit_ns(0)
    got = call(s, workspace=ws)
    assert rp.check_workspace(ws) == 0
    check_tree(got, want(s), F16)


def test_many_sequences():
    # more sequences than threads to a block, several items to a block
    B = 300
    g = torch.Generator().manual_seed(5)
    s = make(B=B, H=2, Hkv=1, T=2, lens=torch.randint(0, 90, (B,), generator=g).tolist(), fmt=INT8, tree="tree")
    check_tree(call(s), want(s), F16)


def test_large_scores_and_small_scales():
    # one key far above the others, and value rows 2^12 apart in size
    for fmt in (F16, E4M3, INT8):
        s = make(B=1, H=2, Hkv=2, T=2, lens=[200], fmt=fmt, scale=0.01)
        s["q"] *= 100
        c = s["cache"]
        if c.coded:
            c.v_scale[:, :, ::3] *= 2.0 ** -12
            c.k_scale[0] *= 64
        else:
            c.v[:, :, ::3] *= 2.0 ** -6
        check_tree(call(s), want(s), F16)


@pytest.mark.parametrize("fmt", [BF16, INT8], ids=["bf16", "int8"])
def test_bf16_range(fmt):
    # queries, drafted keys and values far outside fp16's range
    s = make(B=1, H=2, Hkv=1, T=4, d=64, lens=[50], dt=BF16, fmt=fmt, tree="tree")
    s["q"] *= 1e-30
    s["k"] *= 1e20
    s["v"] *= 1e25
    check_tree(call(s), want(s), BF16)


@pytest.mark.parametrize("dt,fmt", TYPES, ids=TYPE_IDS)
@pytest.mark.parametrize("val", [float("nan"), float("inf")])
@pytest.mark.parametrize("H", [2, 16])                  # 18 rows, 144 rows
def test_non_finite_in_masked_places(dt, fmt, val, H):
    s = make(B=2, H=H, Hkv=1, T=9, d=64, lens=[21, 130], dt=dt, fmt=fmt)
    # node 8 is padding; node 3 is a leaf that nobody else attends; the cache's unused rows are poisoned too
    s["mask"] = rp.tree_masks([-1, 0, 1, 1, 2, 4, 5, 6, None]).cuda()
    clean = call(s)
    s["k"][:, :, 8] = val
    s["v"][:, :, 8] = val
    s["v"][:, :, 3, 5] = val
    s["q"][:, :, 8] = val
    c = s["cache"]
    used = torch.zeros(c.num_pages * c.page_size, dtype=torch.bool)
    for b, n in enumerate(s["lens"].tolist()):
        for i in range(n):
            used[int(s["table"][b, i // c.page_size]) * c.page_size + i % c.page_size] = True
    dead = ~used.view(c.num_pages, c.page_size).cuda()
    if c.coded:
        c.v_scale.masked_fill_(dead[:, None, :], val)
        c.k_scale.masked_fill_(dead[:, None, :], val)
    else:
        c.k.masked_fill_(dead[:, None, :, None], val)
        c.v.masked_fill_(dead[:, None, :, None], val)
    o, lse = call(s)
    rows = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(o[:, :, rows], clean[0][:, :, rows]) and torch.equal(lse, clean[1])
    assert bool((o[:, :, 8] == 0).all()) and bool((lse[:, :, 8] == float("-inf")).all())
    cols = [i for i in range(64) if i != 5]
    assert torch.equal(o[:, :, 3][..., cols], clean[0][:, :, 3][..., cols])
    assert bool((~torch.isfinite(o[:, :, 3, 5])).all())


@pytest.mark.parametrize("H,T", [(2, 2), (4, 7), (4, 12), (8, 40)])
def test_bad_pages_far_from_the_queries(H, T):
    # a missing page among keys whose relation terms are saturated, and one among the others
    for fmt in (F16, INT8):
        s = make(B=2, H=H, Hkv=2, T=T, lens=[900, 700], fmt=fmt, page=16, map=rp.RelPosMap("truncated", clip=20), aq="head", b=True,
                 tree="tree")
        s["table"][0, 10] = -1
        s["table"][0, 55] = 10 ** 6
        s["table"][1, 0] = s["cache"].num_pages
        check_tree(call(s), want(s), F16)


def test_bad_pages_are_masked():
    for fmt in (F16, INT8):
        s = make(B=2, H=2, Hkv=2, T=2, lens=[100, 64], fmt=fmt, page=16)
        s["table"][0, 2] = -7
        s["table"][1, 0] = s["cache"].num_pages + 1000
        check_tree(call(s), want(s), F16)
        s["table"][:] = -1                               # nothing but the nodes
        check_tree(call(s), want(s), F16)


def test_lengths_are_clamped():
    s = make(B=2, H=2, Hkv=2, T=2, lens=[100, 64], page=16)
    s["lens"].copy_(torch.tensor([10 ** 9, -5], dtype=torch.int32))
    s["table"].clamp_(min=0)
    check_tree(call(s), want(s), F16)


def test_strides_outputs_and_streams():
    s = make(B=2, H=4, Hkv=2, T=5, lens=[77, 140], tree="tree", fmt=E4M3, map=rp.RelPosMap("identity"), aq="head", b=True)
    o, lse = call(s)
    token_major = {x: s[x].transpose(1, 2).contiguous().transpose(1, 2) for x in "qkv"}
    o2, lse2 = call({**s, **token_major})
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    o32, _ = call(s, out_f32=True)
    assert o32.dtype == torch.float32 and torch.equal(o32.half(), o)
    need = rp.tree_workspace_size(s["cache"], 2, 5, 4, s["table"].shape[1], aq=True, b=True, map=s["map"], max_seqlen=s["N"])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")          # NaN bits: nothing is read before it is written
    out, out_lse = torch.empty_like(o), torch.empty_like(lse)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(s, workspace=ws, o=out, lse=out_lse)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, o) and torch.equal(out_lse, lse)
    with pytest.raises(rp.RelPosError):
        call(s, workspace=ws[:need // 2])


@pytest.mark.parametrize("fmt,H,T", [(INT8, 4, 3), (F16, 8, 20)])        # 6 rows; 80, the many-row kernel
def test_captured_graph_follows_its_buffers(fmt, H, T):
    s = make(B=2, H=H, Hkv=2, T=T, lens=[200, 64], fmt=fmt, map=rp.RelPosMap("t5", num_buckets=32, max_distance=128, bidirectional=0), b=True)
    s["table"].clamp_(min=0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call(s)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = call(s)
    for lens in ([200, 64], [3, 208], [0, 1]):
        s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        s["q"].copy_(torch.randn(s["q"].shape).half())
        g.replay()
        eager = call(s)
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])


def test_calls_on_two_streams_at_once():
    a = make(seed=1, B=3, H=8, Hkv=2, T=20, lens=[900, 1500, 3], tree="tree", map=rp.RelPosMap("truncated", clip=16), aq="head", b=True)
    b = make(seed=2, B=5, H=4, Hkv=4, T=1, lens=[4000, 1, 77, 0, 900], fmt=E4M3, map=rp.RelPosMap("identity"), aq="shared")
    want_a, want_b = call(a), call(b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(10):
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                got.append((call(s), s is a))
    torch.cuda.synchronize()
    for (o, lse), first in got:
        w = want_a if first else want_b
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_refusals():
    s = make(B=2, H=4, Hkv=2, T=3, lens=[20, 6], map=rp.RelPosMap("truncated", clip=4), aq="shared", b=True)
    def f(**kw):
        z = dict(s)
        ck = {k: kw.pop(k) for k in list(kw) if k in ("o", "lse", "max_seqlen", "workspace")}
        z.update(kw)
        return lambda: call(z, **ck)
    bad = [f(q=s["q"].bfloat16()), f(q=s["q"].float()), f(q=s["q"].cpu()), f(q=s["q"][:, :3]), f(q=s["q"][..., :32]), f(k=s["k"][:, :, :2]),
           f(v=s["v"].bfloat16()), f(lens=s["lens"].long()), f(lens=s["lens"][:1]), f(table=s["table"].long()), f(table=s["table"][:1]),
           f(mask=torch.ones(3, dtype=torch.int32).cuda()), f(mask=torch.ones(4, dtype=torch.int64).cuda()), f(map=None),
           f(aq=s["aq"][:-1]), f(aq=s["aq"].bfloat16()), f(b=s["b"].half()), f(b=s["b"][:, :-1].contiguous()), f(max_seqlen=0),
           f(tau=0.0), f(tau=float("nan")), f(o=torch.empty(2, 4, 3, 64).cuda()), f(lse=torch.empty(2, 4, 3).half().cuda()),
           f(q=s["q"].repeat(1, 1, 22, 1)), f(q=torch.randn(2, 4, 3, 66).half().cuda()[..., 1:65]),
           f(q=torch.randn(2, 4, 3, 68).half().cuda()[..., :64])]
    for i, x in enumerate(bad):
        with pytest.raises(rp.RelPosError):
            x()
            pytest.fail(f"case {i}")
    with pytest.raises(rp.RelPosError):
        rp.tree_masks([0])
    with pytest.raises(rp.RelPosError):
        rp.tree_masks([-1] * 65)
