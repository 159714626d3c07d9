"""The paged K/V cache: codes and scales equal to the fp64 definition, values
read back within one rounding, rows that must stay as they were."""
import pytest
import torch

import exact_relative_position_b200 as rp
from serving_harness import half_step, make_pages, quantise64

pytestmark = pytest.mark.gpu
FORMATS = [torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int8]
IDS = ["f16", "bf16", "e4m3", "int8"]


def _rows(g, shape, dt):
    x = torch.randn(shape, generator=g) * torch.exp(3 * torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(dt).cuda()


def _values(cache):
    out = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        out.append((x.float().cpu().double(), None if s is None else s.cpu()))
    return out


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("Hkv,d,page,T", [(1, 64, 16, 1), (3, 128, 8, 57), (2, 16, 1, 5), (2, 48, 32, 70), (1, 256, 64, 130)])
def test_write_is_exact(fmt, Hkv, d, page, T):
    g = torch.Generator().manual_seed(T)
    dts = [fmt] if fmt in (torch.float16, torch.bfloat16) else [torch.float16, torch.bfloat16]
    pages = -(-T // page) + 2
    for dt in dts:
        cache = rp.kv_cache(pages, page, Hkv, d, fmt)
        k, v = _rows(g, (T, Hkv, d), dt), _rows(g, (T, Hkv, d), dt)
        if T > 4:
            k[1] = 0                                     # a row of zeros
            v[2, 0] = v[2, 0] * 0 + (2.0 ** -133 if dt == torch.bfloat16 else 2.0 ** -24)   # the smallest numbers
            k[3, :, 0] = 448.0                           # ties of e4m3 and of int8 around amax
            k[3, :, 1:] = torch.arange(1, d).to(dt).cuda() * 0.5
        slots = torch.randperm(pages * page, generator=g)[:T].cuda()
        skip = torch.rand(T, generator=g) < 0.2
        slots[skip.cuda()] = -1
        slots[T // 2] = pages * page + 5                 # past the pool: skipped
        before = _values(cache)
        rp.kv_cache_write(cache, k, v, slots)
        for (x, sc), (x0, sc0), src in zip(_values(cache), before, (k, v)):
            want, wsc = x0.clone(), None if sc0 is None else sc0.clone()
            codes, scale = (src.cpu().double(), None) if sc is None else quantise64(src, fmt)
            for t, s in enumerate(slots.tolist()):
                if 0 <= s < pages * page:
                    want[s // page, :, s % page] = codes[t]
                    if sc is not None:
                        wsc[s // page, :, s % page] = scale[t]
            assert torch.equal(x, want)
            if sc is not None:
                assert torch.equal(sc, wsc)


def test_write_every_16bit_value_is_coded_right():
    # every finite bf16 and fp16 number as an element of a row whose largest is fixed
    for dt in (torch.float16, torch.bfloat16):
        allbits = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dt)
        x = allbits[torch.isfinite(allbits) & (allbits.float().abs() <= 300)]
        x = torch.cat((x, x[: (-x.numel()) % 63])).view(-1, 1, 63)
        for top in (300.0, 301.0, 517.0):
            rows = torch.cat((torch.full((x.shape[0], 1, 1), top).to(dt), x), dim=2).cuda()
            for fmt in (torch.int8, torch.float8_e4m3fn):
                cache = rp.kv_cache(-(-rows.shape[0] // 64), 64, 1, 64, fmt)
                rp.kv_cache_write(cache, rows, rows, torch.arange(rows.shape[0]).cuda())
                codes, scale = quantise64(rows, fmt)
                n = rows.shape[0]
                assert torch.equal(cache.k.float().cpu().double().reshape(-1, 64)[:n], codes[:, 0])
                assert torch.equal(cache.v_scale.cpu().reshape(-1)[:n], scale[:, 0])


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_non_finite_rows_read_back_as_nan(fmt):
    cache = rp.kv_cache(1, 8, 2, 64, fmt)
    k = torch.randn(4, 2, 64, dtype=torch.float16, device="cuda")
    k[1, 0, 63] = float("inf")
    k[2, 1, 0] = float("nan")
    rp.kv_cache_write(cache, k, k, torch.arange(4).cuda())
    table, cu = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([0, 4], dtype=torch.int32).cuda()
    rk, rv = rp.kv_cache_read(cache, table, cu, total_tokens=4, dtype=torch.float16)
    bad = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    for r in (rk, rv):
        assert torch.equal(torch.isnan(r).all(-1), bad) and torch.equal(torch.isnan(r).any(-1), bad)


@pytest.mark.parametrize("fmt", FORMATS, ids=IDS)
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["to_f16", "to_bf16"])
@pytest.mark.parametrize("lens,Hkv,d,page", [([1], 1, 64, 16), ([33, 0, 1, 70], 3, 128, 16), ([40] * 3, 2, 48, 1),
                                             ([20000, 19], 1, 64, 128)])
def test_read_back(fmt, dt, lens, Hkv, d, page):
    g = torch.Generator().manual_seed(len(lens))
    table, pages = make_pages(g, lens, page)
    table = table.cuda()
    cache = rp.kv_cache(pages, page, Hkv, d, fmt)
    total = sum(lens)
    src = dt if fmt not in (torch.float16, torch.bfloat16) else fmt
    k, v = (torch.randn((total, Hkv, d), generator=g).to(src).cuda() for _ in range(2))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    at = [(b, i) for b, n in enumerate(lens) for i in range(n)]
    slots = torch.tensor([int(table[b, i // page]) * page + i % page for b, i in at] if total < 1000 else [], dtype=torch.int64)
    if total >= 1000:
        b = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)])
        i = torch.cat([torch.arange(n) for n in lens])
        slots = table.cpu().long()[b, i // page] * page + i % page
    rp.kv_cache_write(cache, k, v, slots.cuda())
    extra = 5
    out = tuple(torch.full((total + extra, Hkv, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
    rk, rv = rp.kv_cache_read(cache, table, cu, out=out)
    for r, x in ((rk, k), (rv, v)):
        codes, scale = (x.double().cpu(), None) if fmt in (torch.float16, torch.bfloat16) else quantise64(x, fmt)
        want = codes if scale is None else codes * scale.double()[..., None]
        # code x scale is rounded to fp32, then to dt
        tol = half_step(want, dt) + 2.0 ** -23 * want.abs()
        assert bool(((r[:total].double().cpu() - want).abs() <= tol).all())
        assert bool((r[total:] == 7.0).all())            # rows behind the last sequence
    # a table entry outside the pool, and a sequence longer than its table: zeros
    if len(lens) > 1 and lens[0] > page:
        table2 = table.clone()
        table2[0, 0] = pages + 3
        rk2, _ = rp.kv_cache_read(cache, table2, cu, total_tokens=total, dtype=dt)
        n0 = min(page, lens[0])
        assert bool((rk2[:n0] == 0).all()) and torch.equal(rk2[n0:], rk[n0:total])
        rk3, _ = rp.kv_cache_read(cache, table[:, :1].contiguous(), cu, total_tokens=total, dtype=dt)
        assert bool((rk3[n0:lens[0]] == 0).all()) and torch.equal(rk3[:n0], rk[:n0])


def test_layouts_and_refusals():
    g = torch.Generator().manual_seed(9)
    x = torch.randn(2, 3, 6, 64, generator=g).half().cuda()                  # [B, Hkv, N, d]
    slots = torch.randperm(16, generator=g)[:12].view(2, 6).cuda()
    a, b = rp.kv_cache(1, 16, 3, 64, torch.int8), rp.kv_cache(1, 16, 3, 64, torch.int8)
    rp.kv_cache_write(a, x, x, slots)
    packed = x.transpose(1, 2).reshape(12, 3, 64)
    rp.kv_cache_write(b, packed, packed, slots.reshape(-1))
    assert torch.equal(a.k, b.k) and torch.equal(a.v_scale, b.v_scale)
    rp.kv_cache_write(b, packed[:0], packed[:0], slots.reshape(-1)[:0])
    big = torch.randn(12, 3, 2, 64, generator=g).half().cuda()
    rp.kv_cache_write(b, big[:, :, 0], big[:, :, 1], slots.reshape(-1))       # strided rows
    rp.kv_cache_write(a, big[:, :, 0].contiguous(), big[:, :, 1].contiguous(), slots.reshape(-1))
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_scale, b.k_scale)
    table, cu = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([0, 4], dtype=torch.int32).cuda()
    c16 = rp.kv_cache(1, 16, 3, 64, torch.float16)
    bad = [lambda: rp.kv_cache_write(c16, x.bfloat16(), x.bfloat16(), slots),
           lambda: rp.kv_cache_write(a, x.float(), x.float(), slots),
           lambda: rp.kv_cache_write(a, x, x, slots.int()), lambda: rp.kv_cache_write(a, x, x, slots[:1]),
           lambda: rp.kv_cache_write(a, x[..., :32], x[..., :32], slots),
           lambda: rp.kv_cache_write(a, torch.randn(12, 3, 68).half().cuda()[..., 1:65], packed, slots.reshape(-1)),
           lambda: rp.kv_cache_write(a, x.cpu(), x, slots), lambda: rp.kv_cache_read(a, table, cu, total_tokens=4),
           lambda: rp.kv_cache_read(a, table, cu[:1], total_tokens=4, dtype=torch.float16),
           lambda: rp.kv_cache_read(a, table.long(), cu, total_tokens=4, dtype=torch.float16),
           lambda: rp.kv_cache_read(a, table, cu, dtype=torch.float16),
           lambda: rp.kv_cache_read(a, table, cu, total_tokens=4, dtype=torch.float32),
           lambda: rp.KVCache(a.k, a.v), lambda: rp.KVCache(a.k, a.v[:, :, :8], a.k_scale, a.v_scale),
           lambda: rp.KVCache(c16.k, c16.v, a.k_scale, a.v_scale), lambda: rp.kv_cache(1, 12, 1, 64, torch.int8),
           lambda: rp.kv_cache(1, 16, 1, 64, torch.float32)]
    for f in bad:
        with pytest.raises(rp.RelPosError):
            f()
