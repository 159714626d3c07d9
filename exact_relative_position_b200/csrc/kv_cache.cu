// kv_cache.cu -- the paged K/V cache: rows of new tokens written into their
// slots (as they are, or in 8 bits with a scale to each row) and whole
// sequences read back into the packed variable-length layout.
//
// int8:  scale = max(fl32(amax / 127), 2^-126), code = nearest (ties to even) of x / scale.
// e4m3:  scale = the smallest 2^s >= amax / 448 with s >= -126, code = nearest e4m3 of
//        x / scale.  A power of two costs a floating format no precision and makes the
//        division exact, so the code depends on x and amax alone.
// A row of zeros has scale 1.  A row with an infinity or a NaN has scale NaN and codes 0:
// it reads back as NaN.
//
// Both kernels move bytes only: each input is read once, each output written once,
// and both are bound by memory.  New rows are read, and values read back are
// written, past the caches (evict-first): 4 x 8191 tokens of 8 heads of 128 in bf16,
// written to e4m3 and read back, take 76 us that way (5.3 TB/s, 82% of a plain
// copy's rate) and 82 us without.
#include "serve.cuh"
#include "kernels.cuh"

#include <cuda_fp8.h>

namespace relpos {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, bool bf16, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}

// Nearest integer of x / s, ties to even, decided exactly: the products of
// x's 11 bits and s's 24 are compared through fused multiply-adds whose sign
// is exact.
__device__ __forceinline__ int quotient_int8(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float over = fmaf(-(q + 0.5f), s, x);    // sign of x / s - (q + 1/2)
  const float under = fmaf(-(q - 0.5f), s, x);   // sign of x / s - (q - 1/2)
  const bool odd = ((int)q) & 1;
  if (over > 0.f || (over == 0.f && odd)) q += 1.f;
  else if (under < 0.f || (under == 0.f && odd)) q -= 1.f;
  return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// LPR lanes to a row of d = 16 * (lanes in use) elements, 16 elements each.
template <int FMT, int LPR>
__global__ void __launch_bounds__(256) cache_write_kernel(const __grid_constant__ CacheWriteParams p) {
  // rows (token, head) of K, then of V; the host keeps their number below 2^31
  const uint32_t row = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int l = threadIdx.x % LPR;
  const int Hkv = p.c.Hkv, d = p.c.d;
  const bool is_v = blockIdx.y != 0;
  const uint32_t tok = row / (uint32_t)Hkv;
  const int h = (int)(row - tok * Hkv);
  long long slot = -1;
  if (tok < (uint32_t)p.B * (uint32_t)p.N) slot = p.slots[tok];
  const bool live = slot >= 0 && slot < ((long long)p.c.num_pages << p.c.page_shift) && l * 16 < d;
  uint4 u[2] = {};
  if (live) {
    const int b = p.B == 1 ? 0 : (int)(tok / (uint32_t)p.N), n = (int)(tok - (uint32_t)b * p.N);
    const Strides& st = is_v ? p.vst : p.kst;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_v ? p.v : p.k) + b * st.b +
                                                      h * st.h + n * st.n + l * 16);
    u[0] = __ldcs(src);
    u[1] = __ldcs(src + 1);
  }
  const long long page = slot >> p.c.page_shift, off = slot & ((1 << p.c.page_shift) - 1);
  const long long dst = ((page * Hkv + h) << p.c.page_shift) + off;   // row of the cache
  if (FMT == RELPOS_CACHE_F16 || FMT == RELPOS_CACHE_BF16) {
    if (live) {
      uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.c.v : p.c.k) + dst * d + l * 16);
      o[0] = u[0];
      o[1] = u[1];
    }
    return;
  }
  float f[16];
  unpack8(u[0], p.bf16, *reinterpret_cast<float (*)[8]>(f));
  unpack8(u[1], p.bf16, *reinterpret_cast<float (*)[8]>(f + 8));
  float amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    amax = fmaxf(amax, fabsf(f[i]));
    bad = bad || !(fabsf(f[i]) <= 3.4028235e38f);
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  // any lane's non-finite value spoils the row
  unsigned spoilt = __ballot_sync(0xffffffffu, bad);
  const int lane = threadIdx.x & 31;
  const unsigned mine = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << (lane / LPR * LPR);
  const bool nan_row = (spoilt & mine) != 0;
  float scale = 1.f;
  uint32_t code[4] = {};
  if (!nan_row && amax > 0.f) {
    if (FMT == RELPOS_CACHE_INT8) {
      scale = fmaxf(__fdiv_rn(amax, 127.f), 0x1p-126f);
      const float inv = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        code[i >> 2] |= (uint32_t)(quotient_int8(f[i], scale, inv) & 0xff) << (8 * (i & 3));
    } else {
      // amax = 1.m * 2^e: 448 = 1.75 * 2^8, so s = e - 8, or e - 7 past a mantissa of 1.75
      const uint32_t a = __float_as_uint(amax);
      int e = (int)(a >> 23) - 127;                                   // -127 for subnormal amax: clamped below
      e = (a & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7;
      e = max(e, -126);
      scale = __uint_as_float((uint32_t)(e + 127) << 23);
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);  // 2^-e: e <= 120
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 xy = make_float2(f[2 * i] * inv, f[2 * i + 1] * inv);
        const uint32_t c2 = __nv_cvt_float2_to_fp8x2(xy, __NV_SATFINITE, __NV_E4M3);
        code[i >> 1] |= c2 << (16 * (i & 1));
      }
    }
  }
  if (nan_row) scale = __uint_as_float(0x7fc00000u);
  if (live) {
    uint8_t* o = static_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + dst * d + l * 16;
    *reinterpret_cast<uint4*>(o) = make_uint4(code[0], code[1], code[2], code[3]);
    if (l == 0) (is_v ? p.c.vs : p.c.ks)[dst] = scale;
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  return bf16 ? DT<__nv_bfloat16>::pack(a, b) : DT<__half>::pack(a, b);
}

// A block takes TOK consecutive tokens: their sequence, page and row are found
// once, then all heads' K and V rows are copied, 16 elements to a thread.
template <int FMT>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ CacheReadParams p, int toks) {
  __shared__ long long base[32];       // page * Hkv << shift, plus the offset in the page; -1: zeros; -2: left alone
  const int t0 = blockIdx.x * toks;
  if (threadIdx.x < toks) {
    const int t = t0 + threadIdx.x;
    long long at = -2;
    if (t < p.total && t >= p.cu[0]) {
      int lo = 0, hi = p.B;            // the last sequence that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid; else hi = mid;
      }
      if (t < p.cu[lo + 1]) {
        const int pos = t - p.cu[lo];
        const int pg = pos >> p.c.page_shift;
        at = -1;
        if (pos >= 0 && pg < p.P) {
          const int id = p.page_table[(long long)lo * p.P + pg];
          if (id >= 0 && id < p.c.num_pages)
            at = (((long long)id * p.c.Hkv) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));
        }
      }
    }
    base[threadIdx.x] = at;
  }
  __syncthreads();
  const int cpr = p.c.d / 16;          // pieces of 16 elements to a row
  const int per_tok = 2 * p.c.Hkv * cpr;
  const int shift = __ffs(cpr) - 1, tshift = __ffs(toks) - 1;   // toks is a power of two
  const bool pow2 = (cpr & (cpr - 1)) == 0;
  const int Hkv = p.c.Hkv, d = p.c.d;
  // the block's tokens of one head after another: their rows follow each other in the cache
  const int group = toks * cpr;
#pragma unroll 4
  for (int i = threadIdx.x; i < toks * per_tok; i += 256) {
    const int kvh = pow2 ? i >> (shift + tshift) : i / group, rem = i - kvh * group;
    const int ti = pow2 ? rem >> shift : rem / cpr, ch = rem - ti * cpr;
    const long long at = base[ti];
    if (at == -2) continue;
    const bool is_v = kvh >= Hkv;
    const int h = is_v ? kvh - Hkv : kvh;
    uint4 o0 = make_uint4(0, 0, 0, 0), o1 = o0;
    if (at >= 0) {
      const long long row = at + ((long long)h << p.c.page_shift);
      const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.c.v : p.c.k);
      if (FMT == RELPOS_CACHE_F16 || FMT == RELPOS_CACHE_BF16) {
        const uint4* s4 = reinterpret_cast<const uint4*>(src + (row * d + ch * 16) * 2);
        o0 = __ldg(s4);
        o1 = __ldg(s4 + 1);
        if (p.bf16 != (FMT == RELPOS_CACHE_BF16)) {
          float f[8];
          unpack8(o0, FMT == RELPOS_CACHE_BF16, f);
          o0 = make_uint4(pack2(f[0], f[1], p.bf16), pack2(f[2], f[3], p.bf16), pack2(f[4], f[5], p.bf16), pack2(f[6], f[7], p.bf16));
          unpack8(o1, FMT == RELPOS_CACHE_BF16, f);
          o1 = make_uint4(pack2(f[0], f[1], p.bf16), pack2(f[2], f[3], p.bf16), pack2(f[4], f[5], p.bf16), pack2(f[6], f[7], p.bf16));
        }
      } else {
        const float sc = __ldg((is_v ? p.c.vs : p.c.ks) + row);
        const uint4 c4 = __ldg(reinterpret_cast<const uint4*>(src + row * d + ch * 16));
        const uint32_t w[4] = {c4.x, c4.y, c4.z, c4.w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[4];
          if (FMT == RELPOS_CACHE_INT8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = (float)(int)(int8_t)((w[j] >> (8 * e)) & 0xff);
          } else {
            const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j] & 0xffff), __NV_E4M3);
            const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j] >> 16), __NV_E4M3);
            const float2 fa = __half22float2(__half2(a)), fb = __half22float2(__half2(b));
            f[0] = fa.x; f[1] = fa.y; f[2] = fb.x; f[3] = fb.y;
          }
          o[2 * j] = pack2(f[0] * sc, f[1] * sc, p.bf16);
          o[2 * j + 1] = pack2(f[2] * sc, f[3] * sc, p.bf16);
        }
        o0 = make_uint4(o[0], o[1], o[2], o[3]);
        o1 = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? p.v : p.k) +
                                          ((long long)(t0 + ti) * Hkv + h) * d + ch * 16);
    __stcs(dst, o0);
    __stcs(dst + 1, o1);
  }
}

template <int FMT>
cudaError_t write_fmt(const CacheWriteParams& p, cudaStream_t s) {
  int lpr = 1;
  while (lpr * 16 < p.c.d) lpr <<= 1;
  const long long rows = (long long)p.B * p.N * p.c.Hkv;
  const dim3 grid((unsigned)((rows * lpr + 255) / 256), 2);
  switch (lpr) {
    case 1: cache_write_kernel<FMT, 1><<<grid, 256, 0, s>>>(p); break;
    case 2: cache_write_kernel<FMT, 2><<<grid, 256, 0, s>>>(p); break;
    case 4: cache_write_kernel<FMT, 4><<<grid, 256, 0, s>>>(p); break;
    case 8: cache_write_kernel<FMT, 8><<<grid, 256, 0, s>>>(p); break;
    default: cache_write_kernel<FMT, 16><<<grid, 256, 0, s>>>(p); break;
  }
  note_launch(1);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t read_fmt(const CacheReadParams& p, cudaStream_t s) {
  // tokens to a block: 8 once that gives each SM sixteen blocks (16 tokens: 2% slower), else
  // 2, so that short sequences still spread over the SMs
  const int toks = p.total >= 148 * 16 * 8 ? 8 : 2;
  cache_read_kernel<FMT><<<(unsigned)((p.total + toks - 1) / toks), 256, 0, s>>>(p, toks);
  note_launch(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s) {
  switch (p.c.format) {
    case RELPOS_CACHE_F16: return write_fmt<RELPOS_CACHE_F16>(p, s);
    case RELPOS_CACHE_BF16: return write_fmt<RELPOS_CACHE_BF16>(p, s);
    case RELPOS_CACHE_E4M3: return write_fmt<RELPOS_CACHE_E4M3>(p, s);
    default: return write_fmt<RELPOS_CACHE_INT8>(p, s);
  }
}

cudaError_t launch_cache_read(const CacheReadParams& p, cudaStream_t s) {
  switch (p.c.format) {
    case RELPOS_CACHE_F16: return read_fmt<RELPOS_CACHE_F16>(p, s);
    case RELPOS_CACHE_BF16: return read_fmt<RELPOS_CACHE_BF16>(p, s);
    case RELPOS_CACHE_E4M3: return read_fmt<RELPOS_CACHE_E4M3>(p, s);
    default: return read_fmt<RELPOS_CACHE_INT8>(p, s);
  }
}

}  // namespace relpos
