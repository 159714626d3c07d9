"""fp64 definitions of the generation operators and the error bounds their
results are held to (each derived from the roundings the operators make, see
the functions)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle as orc

EPS = {torch.float16: 2.0 ** -10, torch.bfloat16: 2.0 ** -7, torch.float32: 2.0 ** -23}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


def half_step(x, dtype):
    """Half a step of dtype at x (fp64): what one rounding to nearest may be off."""
    return EPS[dtype] / 2 * x.abs() + TINY[dtype] / 2


# ---------------------------------------------------------------- rotary
def rotary64(x, pos, w, mag, rotary_dim, interleaved, inverse=False):
    """x [B, H, N, d] turned at positions pos [B, N] (integers): fp64 result and the
    sum of the magnitudes it is made of."""
    x = x.detach().double().cpu()
    ang = pos.double().cpu()[:, None, :, None] * torch.tensor(w, dtype=torch.float64)
    c, s = mag * torch.cos(ang), mag * torch.sin(ang) * (-1 if inverse else 1)
    y, size = x.clone(), x.abs().clone()
    for i in range(rotary_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
        y[..., a] = x[..., a] * c[..., i] - x[..., b] * s[..., i]
        y[..., b] = x[..., b] * c[..., i] + x[..., a] * s[..., i]
        size[..., a] = size[..., b] = abs(mag) * (x[..., a].abs() + x[..., b].abs())
    return y, size


def check_rotary(got, want, size, dtype, ctx=""):
    # the sine's argument is rounded to 24 bits (2^-25 turns pi: 1e-7), the fp64 angle of
    # a far position is itself 2^-53 x 10^6 off, sincospif 1 to 2 units, three fp32
    # roundings: 1e-6 of the magnitudes covers them; then one rounding to the dtype
    tol = half_step(want, dtype) + 1e-6 * size
    err = (got.detach().double().cpu() - want).abs()
    assert torch.isfinite(got.detach().float()).all() and bool((err <= tol).all()), \
        f"{ctx}: worst {float((err / tol).max()):.3g} of the bound"


# ---------------------------------------------------------------- cache rows
def quantise64(x, fmt):
    """Codes' values (fp64) and fp32 scales of rows x [.., d], from the definition."""
    x = x.double().cpu()
    amax = x.abs().amax(-1)
    if fmt == torch.int8:
        scale = torch.from_numpy((amax.numpy().astype(np.float32) / np.float32(127))).double().clamp(min=2.0 ** -126)
    else:
        s = torch.tensor([[0.0 if a == 0 or not math.isfinite(a) else max(-126, _log2_up(a)) for a in r]
                          for r in amax.reshape(-1, 1).tolist()]).reshape(amax.shape)
        scale = torch.pow(2.0, s.double())
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    bad = ~torch.isfinite(x).all(-1)
    scale = torch.where(bad, torch.full_like(scale, math.nan), scale)
    u = torch.where(bad[..., None], torch.zeros_like(x), x / torch.where(bad, torch.ones_like(scale), scale)[..., None])
    if fmt == torch.int8:
        codes = torch.round(u).clamp(-127, 127)
    else:
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)
        codes = torch.round(u / step) * step
    return codes, scale.float()


def _log2_up(a):
    """Smallest integer s with a <= 448 2^s."""
    s = math.floor(math.log2(a / 448)) - 1
    while a > math.ldexp(448.0, s):
        s += 1
    return s


# ---------------------------------------------------------------- tree attention
def phi(m, delta, N):
    om = orc.MapDesc(m.kind, m.clip, m.num_buckets, m.max_distance, m.bidirectional)
    return torch.from_numpy(np.asarray(orc.phi_of_delta(om, delta.numpy(), N)).astype(np.int64))


def cache_rows(cache, table_row, n):
    """(k, v) values [Hkv, n, d] in fp64 of a sequence's first n tokens, the value
    scales [Hkv, n], and which tokens exist (their page lies in the pool)."""
    ps = cache.page_size
    pos = torch.arange(n)
    page = table_row.cpu().long()[pos // ps] if n else pos
    there = (page >= 0) & (page < cache.num_pages)
    page = torch.where(there, page, torch.zeros_like(page))
    out = []
    for x, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        y = x.float().cpu().double()[page, :, pos % ps]
        if sc is not None:
            y = y * sc.cpu().double()[page, :, pos % ps][..., None]
        out.append(y.transpose(0, 1))
    vs = torch.ones(out[1].shape[:2], dtype=torch.float64) if cache.v_scale is None else \
        cache.v_scale.cpu().double()[page, :, pos % ps].transpose(0, 1)
    return out[0], out[1], vs, there


def tree64(q, k, v, cache, table, lengths, aq, b, tau, m, N, mask):
    """fp64 (O, LSE) and their bounds (O's, LSE's), from the definition, sequence by
    sequence and head by head.

    Bounds, with u the half step of the 16-bit operand type of P V (fp16 for
    8-bit caches):
      scores: products of 16-bit numbers are exact in fp32; adding D of them (and the
        relation term's D) is off by at most 2^-23 a step relative to the sum of
        magnitudes, and a few more roundings apply tau: ds = (D + 8) 2^-23 tau (sum
        |q||k| + sum |q||aQ| + |b|) + 2^-20 (exponentials and logarithms of the scale)
      weights: relative 2 ds for the exponential and its sum, u for the 16-bit
        weight (or, for fp16, 2^-25 of the largest weight where it is subnormal)
      output: fp32 sums 2^-23 a key of the magnitudes, one rounding to q's type."""
    B, H, T, d = q.shape
    Hkv = cache.kv_heads
    G = H // Hkv
    qd, kd, vd = (x.double().cpu() for x in (q, k, v))
    O, E = torch.zeros(B, H, T, d, dtype=torch.float64), torch.full((B, H, T), -math.inf, dtype=torch.float64)
    tO, tE = torch.zeros_like(O), torch.zeros_like(E)
    u16 = EPS[q.dtype] / 2 if not cache.coded else 2.0 ** -11
    fp16 = cache.coded or q.dtype == torch.float16
    cap = table.shape[1] * cache.page_size
    for bi in range(B):
        n = min(max(int(lengths[bi]), 0), cap)
        ck, cv, vs, there = cache_rows(cache, table[bi], n)
        bits = [(1 << (t + 1)) - 1 for t in range(T)] if mask is None else \
            [int(x) & ((1 << T) - 1) for x in (mask if mask.dim() == 1 else mask[bi]).tolist()]
        depth = torch.tensor([max(bin(x).count("1") - 1, 0) for x in bits])
        node = torch.tensor([[(x >> c) & 1 for c in range(T)] for x in bits]).bool()
        live = torch.tensor([x != 0 for x in bits])
        keep = torch.cat((there[None, :].expand(T, n), node), 1) & live[:, None]
        pos = torch.cat((torch.arange(n), n + depth))
        row = None
        if m is not None and (aq is not None or b is not None):
            row = phi(m, (pos[None, :] - (n + depth)[:, None]).clamp(1 - N, N - 1), N)
        for h in range(H):
            g = h // G
            K, V = torch.cat((ck[g], kd[bi, g])), torch.cat((cv[g], vd[bi, g]))
            V = torch.where(keep.any(0)[:, None], V, torch.zeros_like(V))
            S, size = qd[bi, h] @ K.T, qd[bi, h].abs() @ K.abs().T
            if aq is not None:
                A = (aq[h] if aq.dim() == 3 else aq).double().cpu()
                S = S + (qd[bi, h] @ A.T).gather(1, row)
                size = size + (qd[bi, h].abs() @ A.abs().T).gather(1, row)
            if b is not None:
                S = S + b[h].double().cpu()[row]
                size = size + b[h].double().cpu().abs()[row]
            S = torch.where(keep, S * tau, torch.full_like(S, -math.inf))
            ds = (torch.where(keep, size, torch.zeros_like(size)).amax(1) * tau * (d + 8) * 2.0 ** -23 + 2.0 ** -20)
            E[bi, h] = torch.logsumexp(S, 1)
            tE[bi, h] = 2 * ds + 2.0 ** -22 * torch.where(live, E[bi, h].abs(), torch.zeros_like(ds)).nan_to_num(0, 0, 0)
            Pm = torch.where(keep.any(1)[:, None], torch.softmax(S, 1), torch.zeros_like(S))
            # each row sums over its own keys only: 0 weights times what is not attended are left out
            for t in range(T):
                kk = keep[t]
                O[bi, h, t] = Pm[t, kk] @ V[kk]
                mag = Pm[t, kk] @ V[kk].abs()
                scale = torch.cat((vs[g], torch.ones(T, dtype=torch.float64)))[kk]
                sub = 0.0
                if fp16 and kk.any():
                    top = (Pm[t, kk] * scale).max()
                    codes = (V[kk].abs() / scale[:, None]).sum(0)
                    sub = 2.0 ** -25 * top * codes
                tO[bi, h, t] = mag * (u16 + 2 * float(ds[t]) + 2.0 ** -20 + int(kk.sum()) * 2.0 ** -23) + sub
    return O, E, tO, tE


def check_tree(got, want, out_dtype, ctx=""):
    (o, lse), (O, E, tO, tE) = got, want
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isnan(o), torch.isnan(O)) and torch.equal(torch.isinf(lse), torch.isinf(E)), f"{ctx}: finiteness"
    fin = torch.isfinite(E)
    assert bool(((lse - E).abs()[fin] <= tE[fin]).all()), f"{ctx}: LSE off by {float(((lse - E).abs()[fin] / tE[fin]).max()):.3g} bounds"
    tol = tO + half_step(O, out_dtype) + EPS[out_dtype] / 2 * tO
    ok = torch.isfinite(O)
    err = (o - O).abs()
    bad = err[ok] > tol[ok]
    assert not bool(bad.any()), f"{ctx}: O off by {float((err[ok] / tol[ok]).max()):.3g} bounds"
    assert torch.equal(o[~ok & ~torch.isnan(O)], O[~ok & ~torch.isnan(O)])


def make_pages(gen, lens, page_size, extra=2):
    """A shuffled page table [B, P] int32 (unused entries -1) for these lengths, and the pool's size."""
    need = [-(-n // page_size) for n in lens]
    total = sum(need) + extra
    order = torch.randperm(total, generator=gen).tolist()
    P = max(1, max(need))
    rows = []
    for n in need:
        rows.append([order.pop() for _ in range(n)] + [-1] * (P - n))
    return torch.tensor(rows, dtype=torch.int32), total
