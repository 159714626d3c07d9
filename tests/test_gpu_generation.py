"""The operators as a decoder uses them: rotary or relation terms, a prompt
written to the cache, drafted trees attended and their accepted nodes written,
held against the library's own causal layer over the whole sequence."""
import pytest
import torch

import exact_relative_position_b200 as rp

pytestmark = pytest.mark.gpu


def _decode(q, k, v, prompt, fmt, m, aq, b, tau, draft=3, page=16):
    """Rows prompt .. N - 1 of the causal attention over q, k, v [1, H, N, d], by drafting
    `draft` tokens a step of which a wrong sibling is dropped: node 0 and its child chain
    are the true tokens, the last node a rejected one."""
    _, H, N, d = q.shape
    pages = -(-N // page)
    cache = rp.kv_cache(pages, page, H, d, fmt)
    table = torch.randperm(pages)[None].to(torch.int32).cuda()
    slot = lambda i: int(table[0, i // page]) * page + i % page
    write = lambda i0, n: rp.kv_cache_write(cache, k[:, :, i0:i0 + n], v[:, :, i0:i0 + n],
                                            torch.tensor([[slot(i) for i in range(i0, i0 + n)]]).cuda())
    write(0, prompt)
    out = []
    at = prompt
    while at < N:
        n = min(draft, N - at)
        wrong = torch.randn(1, H, 1, d, dtype=q.dtype, device="cuda")
        cat = lambda x: torch.cat((x[:, :, at:at + n], wrong), dim=2)
        mask = rp.tree_masks(list(range(-1, n - 1)) + [0]).cuda()
        o, _ = rp.relpos_tree_attention(cat(q), cat(k), cat(v), cache, table, torch.tensor([at], dtype=torch.int32).cuda(), aq, b,
                                        tau=tau, map=m, max_seqlen=N, tree_mask=mask)
        out.append(o[:, :, :n])
        slots = torch.tensor([[slot(i) for i in range(at, at + n)] + [-1]]).cuda()
        rp.kv_cache_write(cache, cat(k), cat(v), slots)
        at += n
    rk, rv = rp.kv_cache_read(cache, table, torch.tensor([0, N], dtype=torch.int32).cuda(), total_tokens=N, dtype=q.dtype)
    return torch.cat(out, dim=2), rk, rv


MAPS = [("truncated", dict(clip=16), True), ("identity", {}, True), ("t5", dict(num_buckets=32, max_distance=128, bidirectional=0), False)]


@pytest.mark.parametrize("kind,kw,has_aq", MAPS, ids=[m[0] for m in MAPS])
def test_decoding_equals_the_causal_layer(kind, kw, has_aq):
    g = torch.Generator().manual_seed(3)
    H, N, d, prompt = 2, 150, 64, 101
    m = rp.RelPosMap(kind, **kw)
    R = rp.table_rows(m, N)
    q, k, v = (torch.randn(1, H, N, d, generator=g).half().cuda() for _ in range(3))
    aq = (0.3 * torch.randn(H, R, d, generator=g)).half().cuda() if has_aq else None
    b = torch.randn(H, R, generator=g).cuda()
    full, _ = rp.relpos_attn_fwd(q, k, v, aq, None, b, tau=0.125, map=m, causal=True)
    got, rk, rv = _decode(q, k, v, prompt, torch.float16, m, aq, b, 0.125)
    # both hold the same definition within: P to fp16 (2^-11), the output to fp16 (2^-11), scores in
    # fp32: 2^-10 of the values averaged (|v| < 6) a side
    assert float((got - full[:, :, prompt:]).abs().max()) <= 2 * 6 * 2.0 ** -10
    assert torch.equal(rk.transpose(0, 1)[None], k) and torch.equal(rv.transpose(0, 1)[None], v)


@pytest.mark.parametrize("fmt", [torch.float8_e4m3fn, torch.int8], ids=["e4m3", "int8"])
def test_rotary_decoding_over_an_8bit_cache(fmt):
    g = torch.Generator().manual_seed(4)
    H, N, d, prompt = 3, 90, 64, 40
    q, k, v = (torch.randn(1, H, N, d, generator=g).half().cuda() for _ in range(3))
    q, k = rp.rotary_embedding(q, k, rotary=rp.RotaryMap(d))
    got, rk, rv = _decode(q, k, v, prompt, fmt, None, None, None, d ** -0.5)
    # what is attended: the values read back for cached tokens, the exact rows for the step's own
    for i in range(prompt, N):
        first = prompt + (i - prompt) // 3 * 3
        K = torch.cat((rk[:first].transpose(0, 1), k[0, :, first:i + 1]), dim=1).double()
        V = torch.cat((rv[:first].transpose(0, 1), v[0, :, first:i + 1]), dim=1).double()
        P = torch.softmax(q[0, :, i:i + 1].double() @ K.transpose(1, 2) * d ** -0.5, dim=-1)
        # read-back rounds the stored values to fp16 (2^-12 of |k| <= 6 in 64 products of |q| <= 6: 0.1 sqrt(64)
        # typical of 2^-12 36), P and O to fp16: 2^-8 of |v| < 6 covers them
        assert float((got[0, :, i - prompt] - (P @ V)[:, 0]).abs().max()) <= 6 * 2.0 ** -8


def test_rotary_trains_through_the_layer():
    # gradients reach q and k through rotary and the causal layer with a bias
    g = torch.Generator().manual_seed(6)
    H, N, d = 2, 70, 64
    m, rot = rp.RelPosMap("truncated", clip=8), rp.RotaryMap(32, interleaved=True)
    q, k, v, do = (torch.randn(1, H, N, d, generator=g).half().cuda() for _ in range(4))
    b = torch.randn(H, rp.table_rows(m, N), generator=g).cuda()
    q.requires_grad_(), k.requires_grad_()
    tq, tk = rp.rotary_embedding(q, k, rotary=rot)
    o = rp.relpos_attention(tq, tk, v, None, None, b, tau=0.125, map=m, causal=True)
    gq, gk = torch.autograd.grad(o, (q, k), do)
    dq, dk = torch.autograd.grad(rp.relpos_attention(*(x := [tq.detach().requires_grad_(), tk.detach().requires_grad_()]), v, None,
                                                     None, b, tau=0.125, map=m, causal=True), x, do)
    for got, up in ((gq, dq), (gk, dk)):
        assert torch.equal(got, rp.relpos_rotary(up, rotary=rot, inverse=True))


def test_transformer_xl_layer_decodes_its_own_rows():
    from exact_relative_position_b200.adapters import TransformerXLRelPos
    torch.manual_seed(8)
    H, N, d, prompt, page = 2, 75, 64, 60, 16
    layer = TransformerXLRelPos(H, d, init_std=0.3).cuda()
    q, k, v = (torch.randn(1, H, N, d, device="cuda").half() for _ in range(3))
    with torch.no_grad():
        full = layer(q, k, v)
    cache = rp.kv_cache(-(-N // page), page, H, d, torch.float16)
    table = torch.arange(cache.num_pages, dtype=torch.int32).flip(0)[None].contiguous().cuda()
    slots = torch.tensor([[int(table[0, i // page]) * page + i % page for i in range(prompt)]]).cuda()
    rp.kv_cache_write(cache, k[:, :, :prompt], v[:, :, :prompt], slots)
    o = layer.decode(q[:, :, prompt:], k[:, :, prompt:], v[:, :, prompt:], cache, table,
                     torch.tensor([prompt], dtype=torch.int32).cuda(), layer.decode_tables(N, torch.float16))
    # both round P and O to fp16 (2 x 2^-11 of |v| < 6 a side)
    assert float((o - full[:, :, prompt:]).abs().max()) <= 2 * 6 * 2.0 ** -10
