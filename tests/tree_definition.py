"""fp64 definition of the attention of drafted tokens with hidden keys, and the
error bounds that follow from what enters the 16-bit product P V: weights in
16 bits next to values, or to 8-bit codes whose scales are the values' own.

A weight is off by half a step of its type relative to itself, and in fp16, where
it is subnormal, by 2^-25 of the largest weight so far.  It multiplies the unit of its
key: over an 8-bit cache the value scale of a cached key (a value row of zeros sets
none), and of a node 1, or in bf16 the power of two that brings its row to 2^14 ..
2^15.  Cached keys come before the nodes, so their weights are measured by the
largest cached one."""
import math

import torch

from serving_harness import EPS, cache_rows, half_step, phi


def definition(s, hidden=None):
    """(O, LSE, bound of O, bound of LSE) for a call's tensors s (as test_gpu_tree_attention.make
    gives them).  hidden(b, h) -> bool [T, n + T]: keys that are left out (n cached, then T
    nodes); a bias below -1e30 hides its keys, too.  The bound of O is before the last rounding."""
    q, k, v, cache, table, lengths = (s[x] for x in ("q", "k", "v", "cache", "table", "lens"))
    aq, b, tau, m, N, mask = (s[x] for x in ("aq", "b", "tau", "map", "N", "mask"))
    B, H, T, d = q.shape
    G = H // cache.kv_heads
    qd, kd, vd = (x.double().cpu() for x in (q, k, v))
    O, E = torch.zeros(B, H, T, d, dtype=torch.float64), torch.full((B, H, T), -math.inf, dtype=torch.float64)
    tO, tE = torch.zeros_like(O), torch.zeros_like(E)
    fp16 = cache.coded or q.dtype == torch.float16
    u16 = 2.0 ** -11 if fp16 else EPS[q.dtype] / 2
    cap = table.shape[1] * cache.page_size
    for bi in range(B):
        n = min(max(int(lengths[bi]), 0), cap)
        ck, cv, vs, there = cache_rows(cache, table[bi], n)
        bits = [(1 << (t + 1)) - 1 for t in range(T)] if mask is None else \
            [int(x) & ((1 << T) - 1) for x in (mask if mask.dim() == 1 else mask[bi]).tolist()]
        depth = torch.tensor([max(bin(x).count("1") - 1, 0) for x in bits])
        node = torch.tensor([[(x >> c) & 1 for c in range(T)] for x in bits]).bool()
        pos = torch.cat((torch.arange(n), n + depth))
        row = None
        if m is not None and (aq is not None or b is not None):
            row = phi(m, (pos[None, :] - (n + depth)[:, None]).clamp(1 - N, N - 1), N)
        for h in range(H):
            g = h // G
            keep = torch.cat((there[None, :].expand(T, n), node), 1) & torch.tensor([x != 0 for x in bits])[:, None]
            if hidden is not None:
                keep = keep & ~hidden(bi, h)
            K, V = torch.cat((ck[g], kd[bi, g])), torch.cat((cv[g], vd[bi, g]))
            Q = torch.where(keep.any(1)[:, None], qd[bi, h], torch.zeros_like(qd[bi, h]))
            S, size = Q @ K.T, Q.abs() @ K.abs().T
            if aq is not None:
                A = (aq[h] if aq.dim() == 3 else aq).double().cpu()
                S, size = S + (Q @ A.T).gather(1, row), size + (Q.abs() @ A.abs().T).gather(1, row)
            if b is not None:
                x = b[h].double().cpu()[row]
                keep = keep & ~(x < -1e30)
                x = torch.where(keep, x, torch.zeros_like(x))
                S, size = S + x, size + x.abs()
            S = torch.where(keep, S * tau, torch.full_like(S, -math.inf))
            # scores: fp32 sums of exact products and a few roundings of tau's
            ds = torch.where(keep, size, torch.zeros_like(size)).amax(1) * tau * (d + 8) * 2.0 ** -23 + 2.0 ** -20
            E[bi, h] = torch.logsumexp(S, 1)
            tE[bi, h] = 2 * ds + 2.0 ** -22 * E[bi, h].abs().nan_to_num(0, 0, 0)
            P = torch.where(keep.any(1)[:, None], torch.softmax(S, 1), torch.zeros_like(S))
            unit = torch.ones(n + T, dtype=torch.float64)
            if cache.coded:
                unit[:n] = vs[g]
                if q.dtype == torch.bfloat16:
                    unit[n:] = torch.exp2(torch.floor(torch.log2(vd[bi, g].abs().nan_to_num(0, 0, 0).amax(-1))) - 14)
            sets = (V != 0).any(1) & (unit > 0)          # keys whose weight may be the largest
            if cache.coded and q.dtype == torch.float16:
                sets[n:] = True
            codes = torch.where(sets[:, None], V.abs() / torch.where(sets, unit, torch.ones_like(unit))[:, None], torch.zeros_like(V))
            cached = torch.arange(n + T) < n
            for t in range(T):
                kk = keep[t]
                if not kk.any():
                    continue
                O[bi, h, t] = P[t, kk] @ V[kk]
                tO[bi, h, t] = (P[t, kk] @ V[kk].abs()) * (u16 + 2 * float(ds[t]) + 2.0 ** -20 + int(kk.sum()) * 2.0 ** -23)
                if fp16:
                    weight = torch.where(kk & sets, P[t] * unit, torch.zeros_like(unit))
                    first = weight[:n].max() if n and cache.coded else weight.max()
                    tO[bi, h, t] += 2.0 ** -25 * (first * codes[kk & cached].sum(0) + weight.max() * codes[kk & ~cached].sum(0))
    return O, E, tO, tE


def check(got, want, dtype, ctx=""):
    """O within its bound and one rounding to dtype, LSE within its own, rows without a key 0 and -inf."""
    (o, lse), (O, E, tO, tE) = got, want
    o, lse = o.double().cpu(), lse.double().cpu()
    assert bool(torch.isfinite(o).all()) and torch.equal(torch.isinf(lse), torch.isinf(E)) and not bool(torch.isnan(lse).any()), f"{ctx}: finiteness"
    fin = torch.isfinite(E)
    worst_e = float(((lse - E).abs()[fin] / tE[fin]).max()) if bool(fin.any()) else 0.0
    tol = tO + half_step(O, dtype) + EPS[dtype] / 2 * tO
    worst_o = float(((o - O).abs() / tol).max())
    assert worst_o <= 1 and worst_e <= 1, f"{ctx}: O off by {worst_o:.3g} bounds, LSE by {worst_e:.3g}"
