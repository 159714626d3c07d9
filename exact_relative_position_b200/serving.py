"""Generation next to the layer: rotary embedding, a paged K/V cache (16 or 8
bits), and attention of drafted tokens over it.

Argument marshalling and autograd only, like `_binding`: each call is one call
of the C ABI in include/relpos_attn.h, on the current stream of the tensors'
device.

    cache = rp.kv_cache(num_pages, page_size, kv_heads, d, torch.float8_e4m3fn)
    q, k = rp.rotary_embedding(q, k, positions, rotary=rp.RotaryMap(d))
    o, lse = rp.relpos_tree_attention(q, k, v, cache, page_table, lengths, tau=d ** -0.5, tree_mask=mask)
    rp.kv_cache_write(cache, k, v, slots)          # the accepted nodes' slots; -1 for the others
"""
from __future__ import annotations

import array
import ctypes
import math
import struct
from dataclasses import dataclass
from typing import Optional

import torch

from ._binding import (
    BF16, F16, F32, LIBPATH, MAP_KINDS, RelPosError, RelPosMap, _check, lib, relpos_cache_read_args, relpos_cache_write_args,
    relpos_rotary_args, relpos_tree_args, table_rows,
)

CACHE_FORMATS = {torch.float16: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2, torch.int8: 3}
_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
MAX_NODES = 64

# The argument blocks of the C ABI as struct formats (native alignment).  A decoding
# step makes these calls thousands of times a second and its kernels run for a few
# microseconds, so the blocks are packed in one go: 1 us, where setting the fields of a
# ctypes structure one by one takes 5.
_STRIDES = "3q3q"
_ROTARY = struct.Struct("@8ifiPqP" + 2 * ("PPii" + _STRIDES))
_CACHE = "6i4P"
_WRITE = struct.Struct("@" + _CACHE + "4iPP" + _STRIDES + "P")
_READ = struct.Struct("@" + _CACHE + "4iPPPP")
_TREE = struct.Struct("@" + _CACHE + "6ifiii5ii6P" + _STRIDES + "3q4P")
assert [s.size for s in (_ROTARY, _WRITE, _READ, _TREE)] == \
    [ctypes.sizeof(c) for c in (relpos_rotary_args, relpos_cache_write_args, relpos_cache_read_args, relpos_tree_args)]

_CALLS = None


def _calls():
    """The entry points, taking their packed blocks."""
    global _CALLS
    if _CALLS is None:
        lib()
        dll = ctypes.CDLL(LIBPATH)
        for name in ("relpos_rotary", "relpos_cache_write", "relpos_cache_read"):
            getattr(dll, name).argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        dll.relpos_tree_attn.argtypes = [ctypes.c_char_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        dll.relpos_tree_workspace_size.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_size_t)]
        _CALLS = dll
    return _CALLS


def _launch(name, dev, *args):
    """One call of the C ABI on the device's current stream, with the device current."""
    index = dev.index
    f = getattr(_CALLS or _calls(), name)
    if torch.cuda.current_device() == index:
        status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _check(status, name)


def _cuda(name, t, dtype, dev):
    if t.dtype is not dtype or t.get_device() != dev.index:
        raise RelPosError(f"{name} must be a CUDA tensor of {dtype} on {dev}")


def _view(name, t, packed_ok=True):
    """(B, H, N, d) and the (b, h, n) strides of [B, H, N, d] or packed [T, H, d]."""
    if t.dim() == 4:
        return t.shape, t.stride()[:3]
    if t.dim() == 3 and packed_ok:
        T, H, d = t.shape
        return (1, H, T, d), (0, t.stride(1), t.stride(0))
    raise RelPosError(f"{name} must be [B, H, N, d]" + (" or packed [T, H, d]" if packed_ok else ""))


def _overlap(a, b):
    """Whether two tensors share memory for sure: the same first element, or dense ones that
    meet.  (Views that lie side by side in one buffer do not, and are not looked into.)"""
    if a.numel() == 0 or b.numel() == 0:
        return False
    p, q = a.data_ptr(), b.data_ptr()
    return p == q or (a.is_contiguous() and b.is_contiguous() and p < q + b.numel() * b.element_size()
                      and q < p + a.numel() * a.element_size())


# ---------------------------------------------------------------- rotary embedding
@dataclass(frozen=True)
class RotaryMap:
    """The frequencies of a rotary embedding (host only).

    rotary_dim columns of each head are turned, pair i by position * w_i with
    w_i = base ** (-2 i / rotary_dim); interleaved pairs are (2i, 2i + 1), else
    (i, i + rotary_dim / 2).  For contexts `factor` times longer than the
    trained ones, scaling is
      "linear": w_i / factor (positions interpolated);
      "ntk":    base * factor ** (rotary_dim / (rotary_dim - 2)) as the base;
      "yarn":   w_i kept where a trained context of original_length turns it more than
                beta_fast times, divided by factor where fewer than beta_slow times, mixed
                linearly in the number of turns between (YaRN, Peng et al. 2023), and magnitude
                0.1 ln(factor) + 1.  A model that was run with a mix linear in the pair's index
                instead brings its own `frequencies`.
    magnitude, where given, multiplies the turned columns in place of the
    scaling's own; frequencies, where given, replace the w_i.
    """
    rotary_dim: int
    base: float = 10000.0
    interleaved: bool = False
    scaling: str = "none"
    factor: float = 1.0
    original_length: int = 0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    magnitude: Optional[float] = None
    frequencies: Optional[tuple] = None

    def __post_init__(self):
        r = self.rotary_dim
        if r < 2 or r % 2 or r > 256:
            raise RelPosError("rotary_dim must be even, 2 to 256")
        if self.scaling not in ("none", "linear", "ntk", "yarn"):
            raise RelPosError("scaling must be none, linear, ntk or yarn")
        if not (self.base > 0 and math.isfinite(self.base)) or not (self.factor > 0 and math.isfinite(self.factor)):
            raise RelPosError("base and factor must be positive")
        if self.scaling == "ntk" and r == 2:
            raise RelPosError("ntk scaling needs rotary_dim > 2")
        if self.scaling == "yarn" and (self.original_length < 1 or self.beta_fast <= self.beta_slow):
            raise RelPosError("yarn needs original_length and beta_fast > beta_slow")
        if self.frequencies is not None and len(self.frequencies) != r // 2:
            raise RelPosError("frequencies must hold rotary_dim / 2 values")
        w = self.angular()
        if not all(math.isfinite(x) for x in w):
            raise RelPosError("frequencies must be finite")
        # turns per position modulo 1, in units of 2^-64 (exact products: the kernel wraps them).  An
        # array, whose address is taken at each call: a copy of the map has, and uses, its own.
        steps = [int(math.fmod(x / (2 * math.pi), 1.0) * 2.0 ** 64) % (1 << 64) for x in w]
        object.__setattr__(self, "_steps", array.array("Q", steps))
        m = self.magnitude
        if m is None:
            m = 0.1 * math.log(self.factor) + 1.0 if self.scaling == "yarn" and self.factor > 1 else 1.0
        object.__setattr__(self, "_magnitude", float(m))

    def angular(self):
        """The angular frequencies w_i, as Python floats."""
        if self.frequencies is not None:
            return [float(x) for x in self.frequencies]
        r, f = self.rotary_dim, self.factor
        base = self.base * f ** (r / (r - 2)) if self.scaling == "ntk" else self.base
        w = [base ** (-2.0 * i / r) for i in range(r // 2)]
        if self.scaling == "linear":
            w = [x / f for x in w]
        elif self.scaling == "yarn":
            keep = [(self.original_length * x / (2 * math.pi) - self.beta_slow) / (self.beta_fast - self.beta_slow)
                    for x in w]
            keep = [min(1.0, max(0.0, g)) for g in keep]
            w = [x * g + x / f * (1.0 - g) for x, g in zip(w, keep)]
        return w


def relpos_rotary(q, k=None, positions=None, *, rotary: RotaryMap, inverse: bool = False, out=None):
    """Rotary embedding through the C ABI (one launch for q and k; no autograd).

    q, k: fp16, bf16 or fp32 CUDA tensors [B, H, N, d] of any strides with a
    contiguous last dimension, or packed [T, H, d]; they share all but the
    head count.  positions: int32 or int64 [N] or [B, N] (packed: [T]), None for
    0 .. N - 1.  out: (q_out, k_out), which may be q and k themselves, each its own
    input, but overlap nothing else.  Returns the turned q, or (q, k)."""
    dt, dev = q.dtype, q.device
    if dt not in _DTYPES or not q.is_cuda:
        raise RelPosError(f"q must be a float16, bfloat16 or float32 CUDA tensor, not {dt} on {dev}")
    (B, H, N, d), st = _view("q", q)
    if rotary.rotary_dim > d:
        raise RelPosError("rotary_dim exceeds the head dimension")
    pos_ptr, pos_bytes, pos_bs = 0, 8, 0
    if positions is not None:
        if positions.device != dev or positions.dtype not in (torch.int32, torch.int64):
            raise RelPosError(f"positions must be int32 or int64 on {dev}")
        if positions.shape != (N,) and (q.dim() != 4 or positions.shape != (B, N)):
            raise RelPosError("positions must be [N] or [B, N] (packed: [T])")
        if N > 1 and positions.stride(-1) != 1:
            positions = positions.contiguous()
        pos_ptr, pos_bytes = positions.data_ptr(), positions.element_size()
        pos_bs = positions.stride(0) if positions.dim() == 2 else 0
    if out is not None and (not isinstance(out, (tuple, list)) or len(out) != (1 if k is None else 2)):
        raise RelPosError("out must hold one tensor for each input")
    if out is not None:
        # q and k are turned in one launch, in no order
        if any(y.data_ptr() != x.data_ptr() and _overlap(y, x) for x, y in zip((q, k), out)):
            raise RelPosError("an output is its own input or does not overlap it")
        if k is not None and (_overlap(out[0], out[1]) or _overlap(out[0], k) or _overlap(out[1], q)):
            raise RelPosError("the outputs must not overlap one another, nor the other input")
    yq, blocks, x_q = _rotary_tensor(q, H, st, None if out is None else out[0])
    if k is not None:
        _cuda("k", k, dt, dev)
        (Bk, Hk, Nk, dk), st = _view("k", k)
        if (Bk, Nk, dk) != (B, N, d) or k.dim() != q.dim():
            raise RelPosError("k must match q in all but the head count")
        yk, more, x_k = _rotary_tensor(k, Hk, st, None if out is None else out[1])
        blocks += more
    else:
        blocks += _NO_TENSOR
    a = _ROTARY.pack(1 if k is None else 2, B, N, d, rotary.rotary_dim, rotary.interleaved, _DTYPES[dt], inverse,
                     rotary._magnitude, pos_bytes, pos_ptr, pos_bs, rotary._steps.buffer_info()[0], *blocks)
    _launch("relpos_rotary", dev, a)
    return yq if k is None else (yq, yk)


_NO_TENSOR = (0,) * 10


def _rotary_tensor(x, H, st, y):
    """The output for x, the block's fields, and what must live until the call."""
    d = x.shape[-1]
    if d > 1 and x.stride(-1) != 1:
        if y is x:
            raise RelPosError("the last dimension must be contiguous")
        x = x.contiguous()
        st = _view("x", x)[1]
    if y is None:
        y = torch.empty_like(x)
    else:
        _cuda("out", y, x.dtype, x.device)
        if y.shape != x.shape or (d > 1 and y.stride(-1) != 1):
            raise RelPosError("out must have its input's shape and a contiguous last dimension")
        if 0 in (s for s, n in zip(y.stride(), y.shape) if n > 1):
            raise RelPosError("out must not be an expanded tensor")
        if y.data_ptr() == x.data_ptr() and any(a != b for a, b, n in zip(y.stride(), x.stride(), x.shape) if n > 1):
            raise RelPosError("an output in place must have its input's strides")
    yst = st if y.stride() == x.stride() else _view("out", y)[1]
    return y, (x.data_ptr(), y.data_ptr(), H, 0, *st, *yst), x


class RotaryEmbedding(torch.autograd.Function):
    """Autograd wrapper: the gradient is the same turn backwards."""

    @staticmethod
    def forward(ctx, q, k, positions, rotary, inverse):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(positions)
        ctx.cfg = (rotary, inverse)
        return relpos_rotary(q, k, positions, rotary=rotary, inverse=inverse)

    @staticmethod
    def backward(ctx, dq, dk=None):
        rotary, inverse = ctx.cfg
        positions, = ctx.saved_tensors
        turn = lambda x, y=None: rotary_embedding(x, y, positions, rotary=rotary, inverse=not inverse)
        if dq is not None and dk is not None:
            dq, dk = turn(dq, dk)
        elif dq is not None:
            dq = turn(dq)
        elif dk is not None:
            dk = turn(dk)
        return dq, dk, None, None, None


def rotary_embedding(q, k=None, positions=None, *, rotary: RotaryMap, inverse: bool = False):
    """Differentiable rotary embedding of q (and k, in the same launch); arguments
    as relpos_rotary."""
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        return RotaryEmbedding.apply(q, k, positions, rotary, inverse)
    return relpos_rotary(q, k, positions, rotary=rotary, inverse=inverse)


# ---------------------------------------------------------------- paged K/V cache
class KVCache:
    """A pool of pages over the caller's tensors.

    k, v: contiguous [num_pages, kv_heads, page_size, d] of float16, bfloat16,
    float8_e4m3fn or int8 (the format); k_scale, v_scale: float32 [num_pages,
    kv_heads, page_size] for the 8-bit formats.  page_size is a power of two.  Token
    `offset` of page p has slot p * page_size + offset."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dtype not in CACHE_FORMATS:
            raise RelPosError(f"unsupported cache dtype {k.dtype}")
        if k.dim() != 4 or v.shape != k.shape:
            raise RelPosError("k and v must be [num_pages, kv_heads, page_size, d]")
        coded = CACHE_FORMATS[k.dtype] >= 2
        if coded != (k_scale is not None) or coded != (v_scale is not None):
            raise RelPosError("the 8-bit formats, and only they, take k_scale and v_scale")
        dev = k.device
        if not k.is_cuda:
            raise RelPosError("a cache lies in CUDA memory")
        for name, t, dt in (("k", k, k.dtype), ("v", v, k.dtype), ("k_scale", k_scale, torch.float32),
                            ("v_scale", v_scale, torch.float32)):
            if t is None:
                continue
            _cuda(name, t, dt, dev)
            if not t.is_contiguous() or (dt == torch.float32 and t.shape != k.shape[:3]):
                raise RelPosError(f"{name} must be contiguous" + (" [num_pages, kv_heads, page_size]" if dt == torch.float32 else ""))
        self._pages = (k, v, k_scale, v_scale)
        self.num_pages, self.kv_heads, self.page_size, self.d = k.shape
        self.dtype, self.device, self.coded = k.dtype, dev, coded
        if self.page_size < 1 or self.page_size & (self.page_size - 1):
            raise RelPosError("page_size must be a power of two")
        self._geometry = (self.num_pages, self.page_size, self.kv_heads, self.d, CACHE_FORMATS[k.dtype], 0)
        self._sizes = {}                                 # workspace bytes by call shape

    # the tensors the pool was made over; another set of tensors is another KVCache
    k = property(lambda self: self._pages[0])
    v = property(lambda self: self._pages[1])
    k_scale = property(lambda self: self._pages[2])
    v_scale = property(lambda self: self._pages[3])

    def _fields(self):
        """The argument block's cache: the pointers are the tensors' own at each call, so that a
        copy of the pool works on its own pages."""
        k, v, ks, vs = self._pages
        if ks is None:
            return (*self._geometry, k.data_ptr(), v.data_ptr(), 0, 0)
        return (*self._geometry, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())


def kv_cache(num_pages: int, page_size: int, kv_heads: int, d: int, dtype: torch.dtype, device="cuda") -> KVCache:
    """A zeroed pool (scales 1) in the format of `dtype`."""
    shape = (num_pages, kv_heads, page_size, d)
    if dtype not in CACHE_FORMATS:
        raise RelPosError(f"unsupported cache dtype {dtype}")
    coded = CACHE_FORMATS[dtype] >= 2
    new = lambda: (torch.zeros(shape, device=device, dtype=torch.uint8).view(dtype) if coded
                   else torch.zeros(shape, device=device, dtype=dtype))
    ones = lambda: torch.ones(shape[:3], device=device, dtype=torch.float32) if coded else None
    return KVCache(new(), new(), ones(), ones())


def kv_cache_write(cache: KVCache, k, v, slots) -> None:
    """Writes tokens' rows into their slots, quantised to the cache's format.

    k, v: packed [T, kv_heads, d] with slots [T], or [B, kv_heads, N, d] with slots
    [B, N]; fp16 or bf16, the cache's own type for a 16-bit cache.  slots: int64;
    a negative slot (or one past the pool) skips its token, and no two
    tokens of a call share one.  An 8-bit row stands for code x scale: e4m3 with the
    smallest power of two that keeps it within 448, int8 with amax / 127."""
    dev, dt = cache.device, k.dtype
    if dt not in (torch.float16, torch.bfloat16) or (not cache.coded and dt != cache.dtype):
        raise RelPosError(f"k and v of {dt} do not go into a cache of {cache.dtype}")
    _cuda("k", k, dt, dev)
    _cuda("v", v, dt, dev)
    _cuda("slots", slots, torch.int64, dev)
    (B, H, N, d), ks = _view("k", k)
    if v.shape != k.shape or H != cache.kv_heads or d != cache.d:
        raise RelPosError("k and v must have the cache's heads and head dimension")
    if slots.shape != ((N,) if k.dim() == 3 else (B, N)):
        raise RelPosError("slots must be [T] (packed) or [B, N]")
    if k.stride(-1) != 1 or v.stride(-1) != 1:
        raise RelPosError("the last dimension of k and v must be contiguous")
    if not slots.is_contiguous():
        slots = slots.contiguous()
    a = _WRITE.pack(*cache._fields(), B, N, _DTYPES[dt], 0, k.data_ptr(), v.data_ptr(), *ks, *_view("v", v)[1],
                    slots.data_ptr())
    _launch("relpos_cache_write", dev, a)


def kv_cache_read(cache: KVCache, page_table, cu_seqlens, *, total_tokens: Optional[int] = None, dtype=None,
                  out=None):
    """Sequences read back, packed: (k, v), each [total_tokens, kv_heads, d].

    Sequence b's tokens 0, 1, ... (pages page_table[b], int32 [B, P]) go to rows
    cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (int32 [B + 1]), as relpos_attention's packed
    batches take them.  total_tokens: rows of the outputs (the host knows it
    without asking the device); out: (k, v) to write into, whose rows past the
    last sequence are left alone (new ones are not initialised there).  dtype:
    fp16 or bf16; the default is a 16-bit cache's own."""
    dev = cache.device
    _cuda("page_table", page_table, torch.int32, dev)
    _cuda("cu_seqlens", cu_seqlens, torch.int32, dev)
    if page_table.dim() != 2 or cu_seqlens.shape != (page_table.shape[0] + 1,):
        raise RelPosError("page_table must be [B, P] and cu_seqlens [B + 1]")
    if not page_table.is_contiguous() or not cu_seqlens.is_contiguous():
        raise RelPosError("page_table and cu_seqlens must be contiguous")
    if out is not None:
        k, v = out
        dtype = dtype or k.dtype
        total_tokens = k.shape[0] if total_tokens is None else total_tokens
        for name, t in (("k", k), ("v", v)):
            _cuda(name, t, dtype, dev)
            if not t.is_contiguous() or t.dim() != 3 or t.shape[0] < total_tokens or t.shape[1:] != (cache.kv_heads, cache.d):
                raise RelPosError("out must be contiguous [total_tokens, kv_heads, d]")
        if _overlap(k, v):
            raise RelPosError("the outputs must not overlap")
    if dtype is None and not cache.coded:
        dtype = cache.dtype
    if dtype not in (torch.float16, torch.bfloat16):
        raise RelPosError("dtype must be float16 or bfloat16")
    if total_tokens is None:
        raise RelPosError("total_tokens is required without out")
    if out is None:
        shape = (total_tokens, cache.kv_heads, cache.d)
        k, v = torch.empty(shape, device=dev, dtype=dtype), torch.empty(shape, device=dev, dtype=dtype)
    a = _READ.pack(*cache._fields(), page_table.shape[0], page_table.shape[1], total_tokens, _DTYPES[dtype],
                   page_table.data_ptr(), cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr())
    _launch("relpos_cache_read", dev, a)
    return k, v


# ---------------------------------------------------------------- attention over the cache
_NO_MAP = (0, 0, 0, 0, 0)


def _rows(m, N):
    """table_rows without its call for the maps whose rows are plain."""
    return m.num_buckets if m.kind == "t5" else 2 * m.clip + 1 if m.kind == "truncated" else table_rows(m, N)


def _workspace_bytes(cache, B, T, H, P, code, aq, b, per_head, desc, N):
    key = (B, T, H, P, code, aq, b, desc, N)
    need = cache._sizes.get(key)
    if need is None:
        fake = 256                                       # only a table's not being NULL is read
        block = _TREE.pack(*cache._fields(), B, T, H, 0, code, code, 1.0, N, P, per_head, *desc, 0, *(0,) * 15,
                           fake if aq else 0, fake if b else 0, 0, 0)
        n = ctypes.c_size_t()
        _check(_calls().relpos_tree_workspace_size(block, ctypes.byref(n)), "relpos_tree_workspace_size")
        if len(cache._sizes) >= 256:                     # shapes of a serving loop; the pool's life is longer
            cache._sizes.clear()
        need = cache._sizes[key] = n.value
    return need


def relpos_tree_attention(q, k, v, cache: KVCache, page_table, lengths, aq=None, b=None, *, tau: float,
                          map: Optional[RelPosMap] = None, max_seqlen: Optional[int] = None, tree_mask=None,
                          out_f32: bool = False, workspace=None, o=None, lse=None):
    """Attention of drafted tokens over a cache and over one another: (O, LSE).

    q [B, H, T, d], k and v [B, kv_heads, T, d] are the T (1 to 64) new tokens of
    each sequence, d 64 or 128, fp16 or bf16, any strides with a contiguous last
    dimension; they are not in the cache yet.  lengths [B] int32: cached tokens;
    page_table [B, P] int32.  Query head h reads key head h // (H / kv_heads).

    tree_mask: int64 [T] or [B, T]; bit u of entry i is set where node i attends
    node u, its ancestors and itself; an entry 0 is padding (O = 0, LSE = -inf).
    None: a chain (T = 1: plain decoding).  Cached token j has position j, a
    node the position lengths[b] + its depth (set bits - 1).

    aq ([R, d] or [H, R, d], q's dtype) and b ([H, R] float32) with `map` add the
    relation terms of relpos_attention at those positions (a term of -inf hides its
    keys); tables of max_seqlen as
    there (by default a bucketed or truncated map needs no more than the pages
    hold, and an identity map's is (R + 1) / 2).  Inference only: no autograd.
    Calls that may overlap on the GPU need workspaces of their own; by default each
    call takes its own from PyTorch's allocator."""
    dev, dt = cache.device, q.dtype
    index = dev.index
    if dt not in (torch.float16, torch.bfloat16) or (not cache.coded and dt is not cache.dtype):
        raise RelPosError(f"q of {dt} does not go with a cache of {cache.dtype}")
    if q.get_device() != index or k.get_device() != index or v.get_device() != index or k.dtype is not dt or v.dtype is not dt:
        raise RelPosError(f"q, k and v must be CUDA tensors of one type on {dev}")
    if q.dim() != 4:
        raise RelPosError("q must be [B, H, T, d]")
    B, H, T, d = q.shape
    Hkv = cache.kv_heads
    if d != cache.d or d not in (64, 128) or H % Hkv:
        raise RelPosError("q must have the cache's head dimension (64 or 128) and a multiple of its heads")
    if not 0 < tau <= 2e38:
        raise RelPosError("tau must be positive, at most 2e38")
    if not 1 <= T <= MAX_NODES:
        raise RelPosError(f"1 to {MAX_NODES} drafted tokens")
    if k.shape != (B, Hkv, T, d) or v.shape != k.shape:
        raise RelPosError("k and v must be [B, kv_heads, T, d]")
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    if qs[3] != 1 or ks[3] != 1 or vs[3] != 1:
        raise RelPosError("the last dimension of q, k and v must be contiguous")
    if page_table.dtype is not torch.int32 or lengths.dtype is not torch.int32 or page_table.get_device() != index \
            or lengths.get_device() != index:
        raise RelPosError(f"page_table and lengths must be int32 on {dev}")
    if page_table.dim() != 2 or page_table.shape[0] != B or lengths.shape != (B,) \
            or not page_table.is_contiguous() or not lengths.is_contiguous():
        raise RelPosError("page_table must be contiguous [B, P] and lengths [B]")
    mask_ptr, per_seq = 0, 0
    if tree_mask is not None:
        _cuda("tree_mask", tree_mask, torch.int64, dev)
        if tree_mask.shape not in ((T,), (B, T)) or not tree_mask.is_contiguous():
            raise RelPosError("tree_mask must be contiguous int64 [T] or [B, T]")
        mask_ptr, per_seq = tree_mask.data_ptr(), int(tree_mask.dim() == 2)
    P = page_table.shape[1]
    desc, N, per_head = _NO_MAP, 1, 0
    if aq is not None or b is not None:
        if map is None:
            raise RelPosError("aq and b need a map")
        desc = (MAP_KINDS[map.kind], map.clip, map.num_buckets, map.max_distance, map.bidirectional)
        if max_seqlen is not None:
            N = max_seqlen
        elif map.kind == "identity":
            N = ((aq.shape[-2] if aq is not None else b.shape[-1]) + 1) // 2
        else:
            N = P * cache.page_size + T
        R = _rows(map, N)
        if aq is not None:
            _cuda("aq", aq, dt, dev)
            per_head = int(aq.dim() == 3)
            if aq.shape != ((H, R, d) if per_head else (R, d)) or not aq.is_contiguous():
                raise RelPosError(f"aq must be contiguous [{R}, {d}] or [{H}, {R}, {d}]")
        if b is not None:
            _cuda("b", b, torch.float32, dev)
            if b.shape != (H, R) or not b.is_contiguous():
                raise RelPosError(f"b must be contiguous float32 [{H}, {R}]")
    if o is None:
        o = torch.empty_like(q, dtype=torch.float32 if out_f32 else None, memory_format=torch.contiguous_format)
    elif o.shape != q.shape or not o.is_contiguous() or o.dtype != (torch.float32 if out_f32 else dt) or o.device != dev:
        raise RelPosError("o must be contiguous, shaped like q, of the output's dtype")
    if lse is None:
        lse = torch.empty((B, H, T), device=dev, dtype=torch.float32)
    elif lse.shape != (B, H, T) or not lse.is_contiguous() or lse.dtype != torch.float32 or lse.device != dev:
        raise RelPosError("lse must be contiguous float32 [B, H, T]")
    if B == 0:
        return o, lse
    code = _DTYPES[dt]
    need = _workspace_bytes(cache, B, T, H, P, code, aq is not None, b is not None, per_head, desc, N)
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise RelPosError(f"workspace must be contiguous on {dev}")
    a = _TREE.pack(*cache._fields(), B, T, H, 0, code, F32 if out_f32 else code, tau, N, P, per_head, *desc, per_seq,
                   page_table.data_ptr(), lengths.data_ptr(), mask_ptr, q.data_ptr(), k.data_ptr(), v.data_ptr(), qs[0],
                   qs[1], qs[2], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], 0 if aq is None else aq.data_ptr(),
                   0 if b is None else b.data_ptr(), o.data_ptr(), lse.data_ptr())
    _launch("relpos_tree_attn", dev, a, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return o, lse


def tree_workspace_size(cache: KVCache, B: int, T: int, H: int, pages_per_seq: int, aq: bool = False, b: bool = False,
                        map: Optional[RelPosMap] = None, max_seqlen: Optional[int] = None) -> int:
    """Bytes of workspace relpos_tree_attention needs for these sizes (host only)."""
    if map is None or not (aq or b):
        desc, N = _NO_MAP, 1
    else:
        desc = (MAP_KINDS[map.kind], map.clip, map.num_buckets, map.max_distance, map.bidirectional)
        N = max_seqlen if max_seqlen is not None else pages_per_seq * cache.page_size + T
    code = BF16 if cache.dtype == torch.bfloat16 else F16
    return _workspace_bytes(cache, B, T, H, pages_per_seq, code, aq, b, 0, desc, N)


def tree_masks(parents) -> torch.Tensor:
    """int64 masks of token trees from each node's parent (a list, or a list of
    lists for a batch; -1 for a root, parents before their children): bit u of
    entry i is set for i's ancestors and itself.  None marks a padding node."""
    if parents and isinstance(parents[0], (list, tuple)):
        return torch.stack([tree_masks(p) for p in parents])
    if len(parents) > MAX_NODES:
        raise RelPosError(f"at most {MAX_NODES} nodes")
    m = []
    for i, p in enumerate(parents):
        if p is None:
            m.append(0)
            continue
        if not -1 <= p < i or (p >= 0 and m[p] == 0):
            raise RelPosError(f"node {i}: its parent must be -1 or a node before it")
        m.append((m[p] if p >= 0 else 0) | (1 << i))
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in m], dtype=torch.int64)
