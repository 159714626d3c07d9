"""Cases of the serving and rotary operators: rotary embedding (forward and
backward), the paged K/V cache written and read back in 16 or 8 bits, and
attention of a tree of drafted tokens over that cache with the library's
relative-position terms.  Each has its plain torch form here and the call of
the library that computes the same."""
import math

import torch

own = False

_DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_FMT = {"fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ---------------------------------------------------------------- cases
def _rotary(name, **kw):
    c = dict(name=name, op="rotary", train=True, B=1, H=12, Hkv=12, N=1, d=64, rotary_dim=64, interleaved=False,
             packed=False, dtype="fp16", scaling="none", factor=1.0, base=10000.0, start=0)
    c.update(kw)
    return c


def _cache(name, **kw):
    c = dict(name=name, op="cache", B=1, past=0, new=1, ragged=True, Hkv=12, d=64, page=16, dtype="fp16",
             format="int8")
    c.update(kw)
    return c


def _tree(name, **kw):
    c = dict(name=name, op="tree", B=1, T=1, L=512, ragged=True, H=12, Hkv=12, d=64, page=16, dtype="fp16",
             format="fp16", map="none", clip=64, aq=False, per_head=False, b=False, chain=False)
    c.update(kw)
    return c


def listed():
    return [
        # one decoding step of 32 sequences far into a stretched context
        _rotary("rotary_step", train=False, B=32, H=32, Hkv=8, N=1, d=128, rotary_dim=128, dtype="bf16",
                scaling="yarn", factor=8.0, start=100000),
        # a training step of the 8K layer with 12 heads of 64
        _rotary("rotary_train_8k", N=8192, interleaved=True),
        # a training batch of odd length, shared key heads, part of the head rotated
        _rotary("rotary_train_partial", B=4, H=32, Hkv=8, N=4097, d=128, rotary_dim=96, dtype="bf16",
                scaling="ntk", factor=4.0),
        # one token appended to each of 16 short sequences, which are then read back
        _cache("cache_step", B=16, past=60, new=1, format="int8"),
        # a long prompt of odd length quantised to e4m3 and read back
        _cache("cache_prompt_e4m3", B=4, past=0, new=8191, Hkv=8, d=128, page=64, dtype="bf16", format="e4m3"),
        # a chunk appended to long int8 sequences, the whole read back for the chunk's attention
        _cache("cache_chunk_int8", B=8, past=12000, new=512, page=32, format="int8"),
        # the same in 16 bits
        _cache("cache_chunk_16bit", B=4, past=3000, new=1024, Hkv=8, d=128, page=16, dtype="bf16", format="bf16"),
        # one sequence, one token: latency of a bucketed-bias decoder step
        _tree("decode_one", L=517, map="t5", b=True),
        # a serving batch of single tokens over an e4m3 cache, four query heads to a key head
        _tree("decode_batch_e4m3", B=64, L=8192, H=32, Hkv=8, d=128, page=64, dtype="bf16", format="e4m3"),
        # small trees over an int8 cache with truncated offsets
        _tree("tree_truncated_int8", B=16, T=13, L=4096, page=32, format="int8", map="truncated", aq=True, b=True),
        # one row per offset over long contexts: a chain of drafted tokens, tables per head
        _tree("tree_identity_16k", B=4, T=8, L=16384, H=8, Hkv=8, page=64, map="identity", aq=True, per_head=True,
              b=True, chain=True),
        # the widest trees with shared key heads, bucketed bias
        _tree("tree_wide", B=16, T=61, L=8192, H=32, Hkv=8, d=128, dtype="bf16", format="bf16", page=16, map="t5",
              b=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: the largest listed cases' work
_MOST_BYTES, _MOST_FLOPS = 6.0e8, 2.0e11


def _fits(c):
    w = work(c)
    return w["bytes"] <= _MOST_BYTES and w["flops"] <= _MOST_FLOPS


def draw(rng):
    op = rng.choice(["rotary", "cache", "tree", "tree"])
    while True:
        if op == "rotary":
            d = rng.choice([64, 128])
            Hkv = rng.choice([1, 2, 4, 8, 12])
            train = rng.random() < 0.6
            c = _rotary("", train=train, B=_log(rng, 1, 32), H=Hkv * rng.choice([1, 1, 2, 4]), Hkv=Hkv,
                        N=_log(rng, 1, 16384) if train or rng.random() < 0.3 else 1, d=d,
                        rotary_dim=rng.choice([d, d, d // 2, d // 4 * 3]), interleaved=rng.random() < 0.5,
                        packed=rng.random() < 0.3, dtype=rng.choice(["fp16", "bf16", "fp32"]),
                        scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=float(rng.choice([2, 4, 8])),
                        base=float(rng.choice([10000, 500000])), start=rng.choice([0, 0, _log(rng, 1, 500000)]))
        elif op == "cache":
            dtype = rng.choice(["fp16", "bf16"])
            c = _cache("", B=_log(rng, 1, 64), past=rng.choice([0, _log(rng, 1, 16384)]), new=_log(rng, 1, 8192),
                       ragged=rng.random() < 0.7, Hkv=rng.choice([1, 2, 4, 8, 12]), d=rng.choice([64, 128]),
                       page=rng.choice([16, 32, 64, 128]), dtype=dtype, format=rng.choice(["int8", "e4m3", dtype]))
        else:
            dtype = rng.choice(["fp16", "bf16"])
            Hkv = rng.choice([1, 2, 4, 8, 12])
            kind = rng.choice(["none", "t5", "truncated", "identity", "log"])
            aq = kind != "none" and kind != "t5" and rng.random() < 0.7
            c = _tree("", B=_log(rng, 1, 64), T=rng.choice([1, rng.randint(2, 16), rng.randint(2, 64)]),
                      L=_log(rng, 1, 32768), ragged=rng.random() < 0.7, H=Hkv * rng.choice([1, 1, 2, 4, 8]), Hkv=Hkv,
                      d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                      format=rng.choice(["int8", "e4m3", dtype, dtype]), map=kind, clip=rng.choice([16, 64, 100]),
                      aq=aq, per_head=rng.random() < 0.5, b=kind != "none" and (not aq or rng.random() < 0.6),
                      chain=rng.random() < 0.3)
        del c["name"]
        # a plain form of a small pass is host time only; a large one must not exceed the listed ones
        if _fits(c):
            return c


def _lengths(B, L, ragged):
    """Lengths of a batch: the longest first, the others spread over a quarter to the whole of it."""
    if not ragged:
        return [L] * B
    return [L if b == 0 else max(1, int(L * (0.25 + 0.75 * ((0.6180339887498949 * b) % 1.0)))) for b in range(B)]


def _rows(c):
    """Table rows and the longest position of a tree case."""
    N = c["L"] + c["T"] + 1
    R = {"none": 0, "t5": 32, "truncated": 2 * c["clip"] + 1, "identity": 2 * N - 1, "log": 128}[c["map"]]
    return R, N


def work(c):
    if c["op"] == "rotary":
        es = 4 if c["dtype"] == "fp32" else 2
        n = c["B"] * (c["H"] + c["Hkv"]) * c["N"] * c["d"]
        passes = 2 if c["train"] else 1
        return {"bytes": passes * 2 * n * es + 8 * c["B"] * c["N"], "flops": passes * 3 * n}
    es = 2 if c["format"] in ("fp16", "bf16") else 1
    scale = 0 if es == 2 else 4
    row = c["Hkv"] * (c["d"] * es + scale)              # one token's K (or V) in the cache
    if c["op"] == "cache":
        wide = c["Hkv"] * c["d"] * 2
        new = c["B"] * c["new"]
        total = sum(_lengths(c["B"], c["past"], c["ragged"])) + new if c["past"] else new
        return {"bytes": 2 * new * (wide + row) + 2 * total * (row + wide) + 8 * new, "flops": 4 * (new + total) * c["Hkv"] * c["d"]}
    keys = sum(_lengths(c["B"], c["L"], c["ragged"]))
    R, N = _rows(c)
    B, T, H, Hkv, d = c["B"], c["T"], c["H"], c["Hkv"], c["d"]
    tables = (2 * R * d * (H if c["per_head"] else 1) if c["aq"] else 0) + (4 * R * H if c["b"] else 0)
    if c["map"] == "identity":
        tables //= 2                                     # offsets ahead of every query are not read
    nbytes = 2 * keys * row + 4 * B * T * (H + Hkv) * d + 4 * B * H * T + tables
    flops = 4 * H * T * (keys + B * T) * d
    if c["aq"]:
        cols = (keys + B * T) if c["map"] == "identity" else B * min(R, c["L"] + T)
        flops += 2 * H * T * cols * d
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(dtype)


def _activations(g, shape, dtype):
    """Rows of uneven size with a few large columns, as keys and values have."""
    x = torch.randn(shape, device="cuda", generator=g)
    x *= torch.exp(0.3 * torch.randn(shape[:-1] + (1,), device="cuda", generator=g))
    x *= 1.0 + 2.0 * (torch.rand(shape[-1], device="cuda", generator=g) < 0.05)
    return x.to(dtype)


def _pages(g, lens, page):
    """A page table [B, P] of shuffled pages that holds `lens` tokens, and the number of pages."""
    need = [-(-n // page) for n in lens]
    P, total = max(1, max(need)), sum(need)
    order = torch.randperm(total + 3, device="cuda", generator=g).to(torch.int32)
    at, rows = 0, []
    for n in need:
        rows.append(torch.nn.functional.pad(order[at:at + n], (0, P - n)))
        at += n
    return torch.stack(rows).contiguous(), total + 3


def _map(c):
    R, N = _rows(c)
    if c["map"] == "t5":
        return dict(kind="t5", num_buckets=32, max_distance=128, bidirectional=0)
    if c["map"] == "log":
        return dict(kind="log", num_buckets=64, max_distance=256)
    if c["map"] == "truncated":
        return dict(kind="truncated", clip=c["clip"])
    return dict(kind=c["map"])


def _tree_masks(c, seed):
    """int64 [B, T]: bit u of row i is set where node i attends node u (its ancestors and itself)."""
    g = torch.Generator().manual_seed(seed + 1)
    T = c["T"]
    rows = []
    for _ in range(c["B"]):
        pick = torch.rand(T, generator=g).tolist()
        m = []
        for i in range(T):
            parent = i - 1 if c["chain"] else int(pick[i] * i) if i else -1
            m.append((m[parent] if i else 0) | (1 << i))
        rows.append([v - (1 << 64) if v >> 63 else v for v in m])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "rotary":
        dt = _DT[c["dtype"]]
        B, N, d = c["B"], c["N"], c["d"]
        shapes = [(B * N, h, d) if c["packed"] else (B, h, N, d) for h in (c["H"], c["Hkv"])]
        s["q"], s["k"] = (_randn(g, sh, dt) for sh in shapes)
        pos = c["start"] + torch.arange(N, device="cuda")[None, :] + torch.randint(0, 64, (B, 1), device="cuda", generator=g)
        s["pos"] = pos.reshape(-1) if c["packed"] else pos.contiguous()
        if c["train"]:
            s["dq"], s["dk"] = (_randn(g, sh, dt) for sh in shapes)
            s["q"].requires_grad_()
            s["k"].requires_grad_()
        if own:
            import exact_relative_position_b200 as rp
            s["rotary"] = rp.RotaryMap(c["rotary_dim"], base=c["base"], interleaved=c["interleaved"],
                                       scaling=c["scaling"], factor=c["factor"], original_length=8192)
        return s
    dt = _DT[c["dtype"]]
    Hkv, d, page = c["Hkv"], c["d"], c["page"]
    if c["op"] == "cache":
        past = _lengths(c["B"], c["past"], c["ragged"]) if c["past"] else [0] * c["B"]
        lens = [n + c["new"] for n in past]
    else:
        past = lens = _lengths(c["B"], c["L"], c["ragged"])
    s["table"], P = _pages(g, lens, page)
    for x in "kv":
        codes, scale = _quantise(_activations(g, (P, Hkv, page, d), dt), c["format"])
        s[x + "_pages"], s[x + "_scale"] = codes.contiguous(), scale
    if c["op"] == "cache":
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
        s["total"] = sum(lens)
        at = torch.tensor(past, device="cuda")[:, None] + torch.arange(c["new"], device="cuda")[None, :]
        s["slots"] = (torch.gather(s["table"].long(), 1, at // page) * page + at % page).reshape(-1)
        s["k"], s["v"] = (_activations(g, (c["B"] * c["new"], Hkv, d), dt) for _ in range(2))
    else:
        R, N = _rows(c)
        B, T, H = c["B"], c["T"], c["H"]
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        s["q"] = _randn(g, (B, H, T, d), dt)
        s["k"], s["v"] = (_activations(g, (B, Hkv, T, d), dt) for _ in range(2))
        s["mask"] = _tree_masks(c, seed)
        s["aq"] = _randn(g, (H, R, d) if c["per_head"] else (R, d), dt, 0.1) if c["aq"] else None
        s["b"] = torch.randn((H, R), device="cuda", generator=g) if c["b"] else None
        s["tau"], s["N"] = d ** -0.5, N
        if own and c["map"] != "none":
            import exact_relative_position_b200 as rp
            s["map"] = rp.RelPosMap(**_map(c))
    if own:
        import exact_relative_position_b200 as rp
        s["cache"] = rp.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------- plain forms
def _frequencies(c):
    """float64 [rotary_dim / 2] and the magnitude of the rotation."""
    r, f = c["rotary_dim"], c["factor"]
    base = c["base"] * (f ** (r / (r - 2)) if c["scaling"] == "ntk" else 1.0)
    w = torch.pow(torch.tensor(base, dtype=torch.float64, device="cuda"),
                  -torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "yarn":
        turns = 8192 * w / (2 * math.pi)
        keep = torch.clamp((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * keep + w / f * (1.0 - keep)
    return w, (0.1 * math.log(f) + 1.0 if c["scaling"] == "yarn" else 1.0)


def _rotate(x, cos, sin, c):
    """x [.., d] turned by the angles of cos / sin [.., rotary_dim / 2], in 32 bits."""
    r = c["rotary_dim"]
    y = x.detach().float()
    turned, rest = y[..., :r], y[..., r:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = turned[..., :r // 2], turned[..., r // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1).to(x.dtype)


def _quantise(x, fmt):
    """Codes and the float32 scale of each row of x; a 16-bit format keeps x."""
    if fmt not in ("int8", "e4m3"):
        return x.to(_FMT[fmt]), None
    x = x.float()
    amax = x.abs().amax(-1)
    if fmt == "e4m3":
        m, e = torch.frexp(amax)
        e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
        scale = torch.ldexp(torch.ones_like(amax), e)
    else:
        scale = (amax / 127.0).clamp(min=2.0 ** -126)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    fine = torch.isfinite(amax)
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    u = torch.where(fine[..., None], x.double() / scale.double()[..., None], torch.zeros((), dtype=torch.float64, device=x.device))
    codes = u.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else u.round().clamp(-127, 127).to(torch.int8)
    return codes, scale


def _gather(pages, scale, page_id, offset):
    """float32 rows [.., Hkv, d] of the cache at (page, offset) [..]."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = raw[page_id, :, offset]
    x = (x.view(torch.float8_e4m3fn) if pages.dtype == torch.float8_e4m3fn else x).float()
    return x if scale is None else x * scale[page_id, :, offset][..., None]


def _phi(m, delta, N):
    """Row of the relation tables for each offset."""
    if m["kind"] == "truncated":
        return delta.clamp(-m["clip"], m["clip"]) + m["clip"]
    if m["kind"] == "identity":
        return delta + N - 1
    if m["kind"] == "t5":
        n = (-delta).clamp(min=0)
        exact = m["num_buckets"] // 2
        far = torch.log(n.clamp(min=1).double() / exact) / math.log(m["max_distance"] / exact) * (m["num_buckets"] - exact)
        return torch.where(n < exact, n, (exact + torch.floor(far + 1e-9).long()).clamp(max=m["num_buckets"] - 1))
    mid, n = m["num_buckets"] // 2, delta.abs()
    far = torch.log(n.clamp(min=1).double() / mid) / math.log((m["max_distance"] - 1) / mid) * (mid - 1)
    far = torch.sign(delta) * (mid + torch.ceil(far - 1e-9).long())
    return (torch.where(n > mid, far, delta) + m["num_buckets"]).clamp(0, 2 * m["num_buckets"] - 1)


def _plain_rotary(s):
    c = s["case"]
    w, mag = _frequencies(c)
    angle = s["pos"].double()[..., None] * w
    cos, sin = (torch.cos(angle) * mag).float(), (torch.sin(angle) * mag).float()
    at = 1                                               # where the head dimension goes: [B, 1, N, r] or [T, 1, r]
    cos, sin = cos.unsqueeze(at), sin.unsqueeze(at)
    out = [_rotate(s["q"], cos, sin, c), _rotate(s["k"], cos, sin, c)]
    if c["train"]:
        out += [_rotate(s["dq"], cos, -sin, c), _rotate(s["dk"], cos, -sin, c)]
    return out


def _plain_cache(s):
    c = s["case"]
    page = c["page"]
    out = []
    at = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    pos = at - s["cu"].long()[seq]
    page_id = s["table"].long()[seq, pos // page]
    for x in "kv":
        pages, scale = s[x + "_pages"], s[x + "_scale"]
        codes, sc = _quantise(s[x], c["format"])
        slot = s["slots"]
        if c["format"] == "e4m3":
            pages.view(torch.uint8)[slot // page, :, slot % page] = codes.view(torch.uint8)
        else:
            pages[slot // page, :, slot % page] = codes
        if scale is not None:
            scale[slot // page, :, slot % page] = sc
        out.append(_gather(pages, scale, page_id, pos % page).to(_DT[c["dtype"]]))
    return out


def _plain_tree(s):
    c = s["case"]
    B, T, H, Hkv, d, page = c["B"], c["T"], c["H"], c["Hkv"], c["d"], c["page"]
    L, G = c["L"], H // Hkv
    j = torch.arange(L, device="cuda")
    page_id = s["table"].long()[:, j // page]
    keep_c = j[None, :] < s["lens"].long()[:, None]                              # [B, L]
    bit = torch.arange(T, device="cuda")
    keep_t = ((s["mask"][:, :, None] >> bit) & 1).bool()                         # [B, T, T]
    keep = torch.cat((keep_c[:, None, :].expand(B, T, L), keep_t), dim=2)
    lens = s["lens"].long()[:, None]
    here = lens + (keep_t.sum(-1) - 1)                                           # [B, T] positions of the nodes
    pos = torch.cat((j[None, :].expand(B, L), here), dim=1)                      # [B, L + T] positions of the keys
    k, v = (torch.cat((_gather(s[x + "_pages"], s[x + "_scale"], page_id, (j % page).expand(B, L)).permute(0, 2, 1, 3),
                       s[x].float()), dim=2) for x in "kv")                      # [B, Hkv, L + T, d]
    q = s["q"].float()
    S = torch.matmul(q.view(B, Hkv, G * T, d), k.transpose(2, 3)).view(B, H, T, L + T)
    if c["map"] != "none":
        row = _phi(_map(c), (pos[:, None, :] - here[:, :, None]).clamp(1 - s["N"], s["N"] - 1), s["N"])[:, None]     # [B, 1, T, L + T]
        if s["aq"] is not None:
            z = torch.matmul(q, s["aq"].float().transpose(-1, -2))               # [B, H, T, R]
            S = S + torch.gather(z, 3, row.expand(B, H, T, L + T))
        if s["b"] is not None:
            S = S + s["b"][:, row[:, 0]].transpose(0, 1)
    S = (S * s["tau"]).masked_fill(~keep[:, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - m)
    l = P.sum(-1, keepdim=True)
    o = torch.matmul(P.view(B, Hkv, G * T, L + T), v).view(B, H, T, d) / l
    return [o.to(s["q"].dtype), (m + torch.log(l))[..., 0]]


def run(s):
    c = s["case"]
    if not own:
        return {"rotary": _plain_rotary, "cache": _plain_cache, "tree": _plain_tree}[c["op"]](s)
    import exact_relative_position_b200 as rp
    if c["op"] == "rotary":
        q, k = rp.rotary_embedding(s["q"], s["k"], s["pos"], rotary=s["rotary"])
        if not c["train"]:
            return [q, k]
        return [q, k, *torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))]
    if c["op"] == "cache":
        rp.kv_cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return list(rp.kv_cache_read(s["cache"], s["table"], s["cu"], total_tokens=s["total"], dtype=_DT[c["dtype"]]))
    return list(rp.relpos_tree_attention(s["q"], s["k"], s["v"], s["cache"], s["table"], s["lens"], s["aq"], s["b"],
                                         tau=s["tau"], map=s.get("map"), max_seqlen=s["N"], tree_mask=s["mask"]))


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotary(s):
    c = s["case"]
    r, f, base = c["rotary_dim"], c["factor"], c["base"]
    pos = s["pos"].double()
    pos = pos[:, None] if c["packed"] else pos[:, None, :]                       # [T, 1] or [B, 1, N]
    out = [x.detach().double().clone() for x in (s["q"], s["k"])]
    if c["train"]:
        out += [s["dq"].double().clone(), s["dk"].double().clone()]
    for i in range(r // 2):
        w = base ** (-2.0 * i / r)
        mag = 1.0
        if c["scaling"] == "linear":
            w /= f
        elif c["scaling"] == "ntk":
            w = (base * f ** (r / (r - 2.0))) ** (-2.0 * i / r)
        elif c["scaling"] == "yarn":
            share = min(1.0, max(0.0, (8192 * w / (2 * math.pi) - 1.0) / 31.0))
            w = share * w + (1.0 - share) * w / f
            mag = 1.0 + 0.1 * math.log(f)
        turn = torch.polar(torch.full_like(pos, mag), pos * w)
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        for n, x in enumerate(out):
            z = torch.complex(x[..., a], x[..., b]) * (turn if n < 2 else turn.conj())
            x[..., a], x[..., b] = z.real, z.imag
    return out


def _exact_rows(x, fmt):
    """What a stored row stands for."""
    x = x.double()
    if fmt not in ("int8", "e4m3"):
        return x
    top = x.abs().max(-1, keepdim=True).values
    if fmt == "int8":
        step = torch.where(top > 0, (top / 127).float().double().clamp(min=2.0 ** -126), torch.ones_like(top))
        return torch.round(x / step) * step
    step = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448) - 1e-12).clamp(min=-126))
    u = x / step
    grid = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)  # spacing of e4m3 around u
    return torch.round(u / grid) * grid * step


def _exact_cache(s, past):
    c = s["case"]
    out = []
    for x in "kv":
        raw = s[x + "_pages"].double() if s[x + "_scale"] is None else s[x + "_pages"].double() * s[x + "_scale"].double()[..., None]
        rows = _exact_rows(s[x], c["format"])
        got = []
        for b, n in enumerate(past):
            ids = s["table"][b].long()
            whole = raw[ids].transpose(1, 2).reshape(-1, c["Hkv"], c["d"])[:n]   # page after page, token-major
            got += [whole, rows[b * c["new"]:(b + 1) * c["new"]]]
        out.append(torch.cat(got))
    return out


def _exact_phi(m, delta, N):
    if m["kind"] in ("truncated", "identity"):
        return _phi(m, delta, N)
    rows = {}
    for x in delta.unique().tolist():
        n = abs(x)
        if m["kind"] == "t5":
            n, e, nb = max(0, -x), m["num_buckets"] // 2, m["num_buckets"]
            rows[x] = n if n < e else min(nb - 1, e + math.floor(math.log(n / e) / math.log(m["max_distance"] / e) * (nb - e) + 1e-9))
        else:
            mid = m["num_buckets"] // 2
            p = x if n <= mid else int(math.copysign(mid + math.ceil(math.log(n / mid) / math.log((m["max_distance"] - 1) / mid) * (mid - 1) - 1e-9), x))
            rows[x] = min(2 * m["num_buckets"] - 1, max(0, p + m["num_buckets"]))
    keys = torch.tensor(sorted(rows), device=delta.device)
    vals = torch.tensor([rows[k] for k in sorted(rows)], device=delta.device)
    return vals[torch.searchsorted(keys, delta)]


def _exact_tree(s):
    c = s["case"]
    T, H, Hkv, d = c["T"], c["H"], c["Hkv"], c["d"]
    lens = s["lens"].tolist()
    masks = s["mask"].tolist()
    O = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    E = torch.empty(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        ids = s["table"][b, :-(-n // c["page"])].long()
        kv = []
        for x in "kv":
            raw = s[x + "_pages"][ids].double()
            if s[x + "_scale"] is not None:
                raw = raw * s[x + "_scale"][ids].double()[..., None]
            raw = raw.transpose(0, 1).reshape(Hkv, -1, d)[:, :n]
            kv.append(torch.cat((raw, s[x][b].double()), dim=1))
        depth = [bin(m & ((1 << 64) - 1)).count("1") - 1 for m in masks[b]]
        at = torch.tensor([n + u for u in depth], device="cuda")
        keys = torch.cat((torch.arange(n, device="cuda"), at))
        seen = torch.tensor([[(m >> u) & 1 for u in range(T)] for m in masks[b]], device="cuda", dtype=torch.bool)
        hide = torch.cat((torch.zeros((T, n), dtype=torch.bool, device="cuda"), ~seen), dim=1)
        row = None if c["map"] == "none" else _exact_phi(_map(c), keys[None, :] - at[:, None], s["N"])
        for h in range(H):
            q = s["q"][b, h].double()
            S = q @ kv[0][h * Hkv // H].T
            if s["aq"] is not None:
                S += (q @ (s["aq"][h] if c["per_head"] else s["aq"]).double().T).gather(1, row)
            if s["b"] is not None:
                S += s["b"][h].double()[row]
            S = (S * s["tau"]).masked_fill(hide, -math.inf)
            E[b, h] = torch.logsumexp(S, dim=1)
            O[b, h] = torch.softmax(S, dim=1) @ kv[1][h * Hkv // H]
    return [O, E]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(s)
    if case["op"] == "cache":
        return _exact_cache(s, _lengths(case["B"], case["past"], case["ragged"]) if case["past"] else [0] * case["B"])
    return _exact_tree(s)
