// tree_attn.cuh -- attention of a few drafted tokens (a tree of up to 64
// nodes; one node is plain decoding) over a paged cache and over one another,
// with the relation terms of the drafted queries.
//
//   S_ij = tau (q_i.k_j + q_i.aQ[phi(p_j - p_i)] + b[phi(p_j - p_i)]),  O = softmax(S) V
//
// over the cached keys j < length (position j) and the nodes u whose bit is
// set in the mask of node i (position length + depth(u)).
//
// Work: a block takes the G T rows (query heads of one key head, times nodes)
// against tiles of keys, so the cache is read once however many heads and
// nodes share it.  All tiles of all (sequence, key head, row block) items
// form one line that is cut into equal pieces, one to a block: ragged batches
// cost no more than even ones, and one long sequence fills the card.  An item
// cut by a piece's end leaves partial maxima, sums and outputs in the
// workspace, which a second kernel joins in the order of the pieces.
//
// Tensor work: mma.sync m16n8k16.  Up to 64 rows share each key, so the
// kernel does at most 2 x 64 multiply-adds for each element it loads and is
// bound by memory there; 128-row tcgen05 tiles would run mostly empty.
//
// Order of the operands.  An MMA sums over k in any order, and names its
// columns in any order, as long as both operands agree.  Each lane of a quad
// therefore takes 16 consecutive bytes of a key row for its k slots (one
// shared-memory load feeds 2 to 4 MMAs, 8-bit codes are expanded in
// registers), and column slot c of the two 8-key column tiles of 16 keys
// stands for key 4 (c / 2) + c % 2 (+ 2 in the second), which makes a lane's
// four score columns, and so its four rows of V, consecutive keys.
//
// 8-bit caches: codes are exact in fp16.  The scale of key j multiplies its
// score column; that of its value row is folded into the exponent, so that
// the fp16 weight is 2^(s_ij + log2 sv_j - m_i) <= 1 with m_i the row's
// running maximum of that sum, and the softmax sum divides it out in fp32:
//   P'_ij = 2^(s_ij + log2 sv_j - m_i),  l_i = sum_j P'_ij / sv_j,
//   O_i = sum_j P'_ij code_j / l_i,      LSE_i = m_i + log2 l_i (base 2).
// bf16 queries enter in fp16 after an exact power-of-two scaling of the
// warp's rows to a largest element in [2^14, 2^15).
#pragma once

#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "serve.cuh"
#include "warp_mma.cuh"

namespace relpos {
namespace tree {

constexpr float kMinLogScale = -100.f;   // value scales count as at least 2^-100: l stays finite

// Tiling of a row count: WM x WN warps, MT 16-row tiles to a warp, KW keys to
// a warp and step.
template <int D_, int WM_, int WN_, int MT_, int KW_, int STAGES_> struct Tiling {
  static constexpr int D = D_, WM = WM_, WN = WN_, MT = MT_, KW = KW_, STAGES = STAGES_;
  static constexpr int ROWS = WM * MT * 16, TK = WN * KW;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Sum-order-preserving join of (m, l): exponent base 2, -inf for nothing yet.
__device__ __forceinline__ float safe(float m) { return m == -INFINITY ? 0.f : m; }

// ---------------------------------------------------------------- the line of tiles
// pre[b]: tiles of one item summed over the sequences before b.
struct Line {
  const int* pre;
  int B, items;                      // items (key head, row block) of a sequence
  long long total, quantum;
  __device__ __forceinline__ int seq_of(long long at) const {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((long long)pre[mid] * items <= at) lo = mid; else hi = mid;
    }
    return lo;
  }
};

__device__ __forceinline__ int seq_len(const TreeParams& p, int b) {
  return iclamp(p.lengths[b], 0, p.P << p.c.page_shift);
}
// Tiles of an item: the cache's keys (and the nodes' behind them where the
// cache has their type); never none, for the nodes of an empty cache.
__device__ __forceinline__ int seq_tiles(const TreeParams& p, int b, int tk, bool wide) {
  const int n = seq_len(p, b) + (wide ? p.T : 0);
  return max(1, (n + tk - 1) / tk);
}

// Fills pre[0 .. B] (all threads of the block; ends with a barrier).
template <int NT>
__device__ __forceinline__ void build_line(const TreeParams& p, int tk, bool wide, int* pre, int* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int carry = 0;
  if (tid == 0) pre[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + tid;
    int x = b < p.B ? seq_tiles(p, b, tk, wide) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
      if (i < w) before += warp_sums[i];
      all += warp_sums[i];
    }
    if (b < p.B) pre[b + 1] = before + x;
    carry += all;
    __syncthreads();
  }
}

// Floats of one partial result: outputs, then maxima and sums of its rows.
RP_HD long long slot_floats(int rows, int d) { return (long long)rows * (d + 2); }

// ---------------------------------------------------------------- operand helpers
// Physical byte offset of 16-byte chunk ch of row r in a staged tile whose
// rows have CPR chunks.  Keys: odd rows are moved by four chunks, so that two
// adjacent rows' quads meet different banks.  Values: the four rows (of 16)
// that a quad reads at once, or the eight of an ldmatrix, go to different banks.
template <int CPR, bool WIDE, bool VAL>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  uint32_t li = (uint32_t)(r * CPR + ch);
  if (VAL) li ^= WIDE ? (uint32_t)((((r >> 2) & 3) << 1) | (r & 1)) : (uint32_t)(((r >> 2) & 3) << 1);
  else if (CPR >= 8) li ^= (uint32_t)((r & 1) << 2);
  return li << 4;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Four 8-bit codes as two pairs of fp16: (e0, e1), (e2, e3).
template <int FMT>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == RELPOS_CACHE_E4M3) {
    const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
    const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
  } else {
    // 1024 + (code + 128) is the fp16 number 0x6400 | (code ^ 0x80)
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&ra);
    hi = *reinterpret_cast<const uint32_t*>(&rb);
  }
}

// A pair of bf16 times a power of two, as a pair of fp16; fp16 stays.
template <typename QT>
__device__ __forceinline__ uint32_t to_half2(uint32_t w, float f);
template <>
__device__ __forceinline__ uint32_t to_half2<__half>(uint32_t w, float) { return w; }
template <>
__device__ __forceinline__ uint32_t to_half2<__nv_bfloat16>(uint32_t w, float f) {
  return DT<__half>::pack(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
}
// Largest |x| of bf16 pairs as fp32 bits (comparable as integers); an infinity
// or NaN does not count, so that it leaves its neighbours their precision.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  const uint32_t lo = (w << 16) & 0x7fffffffu, hi = w & 0x7fff0000u;
  m = lo < 0x7f800000u ? max(m, lo) : m;
  return hi < 0x7f800000u ? max(m, hi) : m;
}
// The power e with |x| 2^-e in [2^14, 2^15) for the largest |x| given by its bits.
__device__ __forceinline__ int exp_of(uint32_t bits) { return iclamp((int)(bits >> 23) - 127 - 14, -100, 100); }

// An infinity or NaN of a node's value row must not reach the rows that do not
// attend the node (0 times it is NaN): such elements enter the MMA as 0 and are
// added afterwards to the rows that do attend it.
template <typename T16>
__device__ __forceinline__ uint32_t clean2(uint32_t w, bool& seen) {
  constexpr uint32_t kExp = DT<T16>::kCoarse ? 0x7f80u : 0x7c00u;
  const bool lo = (w & kExp) == kExp, hi = ((w >> 16) & kExp) == kExp;
  seen = seen || lo || hi;
  return (lo ? 0u : w & 0xffffu) | (hi ? 0u : w & 0xffff0000u);
}

struct RowInfo {
  int t, h;                      // node and query head; t < 0: no such row
  int depth;
  unsigned long long mask;
  const float* z;                // its relation terms at offset 0 - e_lo ... (null: none)
};

__device__ __forceinline__ unsigned long long node_mask(const TreeParams& p, int b, int t) {
  const unsigned long long live = p.T == 64 ? ~0ull : (1ull << p.T) - 1;
  const unsigned long long m = p.mask ? (unsigned long long)p.mask[(long long)b * p.mask_bs + t]
                                      : (2ull << t) - 1;   // t = 63: 2 << 63 wraps to 0, minus 1 is all ones
  return m & live;
}

// Four finished columns of row gr (of a key head's G T rows): O = o / l, and the LSE.
__device__ __forceinline__ void store_row(const TreeParams& p, int b, int hkv, int gr, int c, float4 o, float m,
                                          float l) {
  const int t = gr / p.G, h = hkv * p.G + (gr - t * p.G);
  const long long row = ((long long)b * p.H + h) * p.T + t;
  // a row with no key has l = 0 and o = 0; a NaN goes on into the result
  const float inv = l == 0.f ? 0.f : 1.f / l;
  o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
  if (node_mask(p, b, t) == 0) {                       // a padding node attends nothing
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
  }
  if (p.o_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * p.c.d + 4 * c) = o;
  } else {
    uint2 w;
    if (p.bf16) w = make_uint2(DT<__nv_bfloat16>::pack(o.x, o.y), DT<__nv_bfloat16>::pack(o.z, o.w));
    else w = make_uint2(DT<__half>::pack(o.x, o.y), DT<__half>::pack(o.z, o.w));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * p.c.d + 4 * c) = w;
  }
  if (c == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// ---------------------------------------------------------------- the kernel
template <class TL, typename QT, int FMT>
__global__ void __launch_bounds__(128) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool WIDE = FMT == RELPOS_CACHE_F16;        // the cache has the queries' 16-bit type
  constexpr int D = TL::D, WM = TL::WM, WN = TL::WN, MT = TL::MT, KW = TL::KW, TK = TL::TK, ROWS = TL::ROWS;
  constexpr int ES = WIDE ? 2 : 1;
  constexpr int CPR = D * ES / 16;                      // chunks of a row
  constexpr int GT = WM * 32;                           // threads that share a group of KW keys
  constexpr int KS = D / 16;                            // k steps of q.k
  constexpr int NT = D / 8;                             // column tiles of the output
  constexpr int SG = KW / 16;                           // groups of 16 keys
  constexpr int HALF = KW * CPR * 16;                   // bytes of a group's keys (or values) in a stage
  constexpr int GSTAGE = 2 * HALF + (WIDE ? 0 : KW * 8);
  using MT16 = typename std::conditional<WIDE, QT, __half>::type;   // operand type of the MMAs

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sums[4];
  __shared__ uint32_t valid_bits[WN][TL::STAGES][(KW + 31) / 32];
  __shared__ float sm_m[WN][ROWS], sm_l[WN][ROWS];
  int* pre = reinterpret_cast<int*>(smem);              // [B + 1], rounded up to 128 bytes
  const uint32_t pre_bytes = (uint32_t)((p.B + 1) * 4 + 127) & ~127u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / WN, wn = warp % WN;             // WN == 4: wm = 0
  const int gtid = wm * 32 + lane;                      // place in the group of warps with this wn
  const int q4 = lane & 3, r8 = lane >> 2;
  const uint32_t stage0 = smem_u32(smem) + pre_bytes + (uint32_t)(wn * TL::STAGES * GSTAGE);
  float* merge = reinterpret_cast<float*>(smem + pre_bytes);   // [WN][ROWS][D], over the stages

  auto group_sync = [&]() {
    if (WM == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(wn + 1), "n"(GT) : "memory");
  };

  build_line<128>(p, TK, WIDE, pre, warp_sums);
  Line line;
  line.pre = pre;
  line.B = p.B;
  line.items = p.c.Hkv * p.row_blocks;
  line.total = (long long)pre[p.B] * line.items;
  line.quantum = (line.total + gridDim.x - 1) / gridDim.x;
  long long cur = line.quantum * blockIdx.x;
  const long long my_start = cur;
  const long long my_end = min(line.total, cur + line.quantum);
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int R = p.G * p.T;

  while (cur < my_end) {
    const int b = line.seq_of(cur);
    const int nt = pre[b + 1] - pre[b];
    const long long in_b = cur - (long long)pre[b] * line.items;
    const int item = (int)(in_b / nt), tile0 = (int)(in_b - (long long)item * nt);
    const int tile1 = (int)min((long long)nt, tile0 + (my_end - cur));
    const int hkv = item / p.row_blocks, rb = item - hkv * p.row_blocks;
    const int len = seq_len(p, b);

    // rows of this thread: MT tiles, rows r8 and r8 + 8 of each
    RowInfo row[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rb * ROWS + (wm * MT + mt) * 16 + r8 + 8 * e;
        RowInfo& x = row[mt][e];
        x.t = -1;
        x.h = 0;
        x.depth = 0;
        x.mask = 0;
        x.z = nullptr;
        if (r < R) {
          x.t = r / p.G;
          x.h = hkv * p.G + (r - x.t * p.G);
          x.mask = node_mask(p, b, x.t);
          x.depth = max(__popcll(x.mask) - 1, 0);
          if (p.z) x.z = p.z + b * p.z_b + x.h * p.z_h + x.t * p.z_t;
        }
      }

    // ---- queries: A fragments in the permuted k order
    uint32_t qa[MT][KS][4];
    uint32_t top = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const RowInfo& x = row[mt][e];
        const uint16_t* src = static_cast<const uint16_t*>(p.q) + b * p.qs.b + x.h * p.qs.h + (long long)x.t * p.qs.n;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          // 16-bit keys: 8 elements at 32 u + 8 q; 8-bit keys: 8 of the 16 elements at 64 (u / 2) + 16 q
          const int d0 = WIDE ? 32 * u + 8 * q4 : 64 * (u / 2) + 16 * q4 + 8 * (u % 2);
          uint4 w = make_uint4(0, 0, 0, 0);
          if (x.t >= 0) w = __ldg(reinterpret_cast<const uint4*>(src + d0));
          qa[mt][2 * u][e] = w.x;
          qa[mt][2 * u][2 + e] = w.y;
          qa[mt][2 * u + 1][e] = w.z;
          qa[mt][2 * u + 1][2 + e] = w.w;
          if (!WIDE && sizeof(QT) == 2 && DT<QT>::kCoarse)
            top = amax2(amax2(amax2(amax2(top, w.x), w.y), w.z), w.w);
        }
      }
    float qf = 1.f;                                     // the queries' power of two (8-bit caches)
    if (!WIDE && DT<QT>::kCoarse) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int e = exp_of(top);
      qf = pow2i(e);
      const float down = pow2i(-e);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 4; ++i) qa[mt][ks][i] = to_half2<QT>(qa[mt][ks][i], down);
    }
    const float kc = p.c2 * qf;                         // scores of 8-bit keys: acc * scale_j * kc (base 2)

    float oacc[MT][NT][4];
    float mrow[MT][2], lrow[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) oacc[mt][n][i] = 0.f;
      mrow[mt][0] = mrow[mt][1] = -INFINITY;
      lrow[mt][0] = lrow[mt][1] = 0.f;
    }

    // ---- loads: rows of the cache by page, nodes behind them (16-bit cache)
    const uint8_t* kc_base = static_cast<const uint8_t*>(p.c.k);
    const uint8_t* vc_base = static_cast<const uint8_t*>(p.c.v);
    const int* table = p.page_table + (long long)b * p.P;
    constexpr int LR = (KW + 31) / 32;                  // rows whose place a lane looks up
    auto lookup = [&](int tile, uint32_t (&at)[LR]) {
      // row of the cache of key `tile * TK + wn * KW + 32 i + lane`; all ones: none
#pragma unroll
      for (int i = 0; i < LR; ++i) {
        const int lr = 32 * i + lane, j = tile * TK + wn * KW + lr;
        at[i] = 0xffffffffu;
        if (lr < KW && tile < tile1 && j < len) {
          const int id = __ldg(table + (j >> p.c.page_shift));
          if (id >= 0 && id < p.c.num_pages)
            at[i] = (((uint32_t)id * (uint32_t)p.c.Hkv + (uint32_t)hkv) << p.c.page_shift) + (uint32_t)(j & page_mask);
        }
      }
    };
    auto issue = [&](int tile, int stage, const uint32_t (&at)[LR]) {
      const uint32_t sk = stage0 + (uint32_t)stage * GSTAGE, sv = sk + HALF;
      const int k0 = tile * TK + wn * KW;
      const bool nodes = WIDE && k0 + KW > len;         // some rows are nodes, or past the end
#pragma unroll
      for (int i = 0; i < KW * CPR / GT; ++i) {
        const int ci = i * GT + gtid, r = ci / CPR, ch = ci % CPR;
        const uint32_t at_r = __shfl_sync(0xffffffffu, at[(LR > 1) ? (i * GT / CPR) / 32 : 0], r & 31);
        const uint8_t *ksrc = kc_base, *vsrc = vc_base;
        int bytes = 0;
        if (at_r != 0xffffffffu) {
          const unsigned long long off = (unsigned long long)at_r * (D * ES) + ch * 16;
          ksrc += off;
          vsrc += off;
          bytes = 16;
        } else if (nodes) {
          const int u = k0 + r - len;
          if (u >= 0 && u < p.T) {
            ksrc = static_cast<const uint8_t*>(p.k) + 2 * (b * p.ks.b + hkv * p.ks.h + u * p.ks.n + ch * 8);
            vsrc = static_cast<const uint8_t*>(p.v) + 2 * (b * p.vs.b + hkv * p.vs.h + u * p.vs.n + ch * 8);
            bytes = 16;
          }
        }
        cp_async16(sk + chunk_at<CPR, WIDE, false>(r, ch), ksrc, bytes);
        cp_async16(sv + chunk_at<CPR, WIDE, true>(r, ch), vsrc, bytes);
      }
#pragma unroll
      for (int i = 0; i < LR; ++i) {
        const int lr = 32 * i + lane;
        bool ok = at[i] != 0xffffffffu;
        if (nodes) ok = ok || (lr < KW && k0 + lr >= len && k0 + lr < len + p.T);
        const uint32_t bits = __ballot_sync(0xffffffffu, ok);
        if (wm == 0 && lane == 0) valid_bits[wn][stage][i] = bits;
        if (!WIDE && wm == 0 && lr < KW) {
          const uint32_t ss = sk + 2 * HALF + lr * 4;
          const uint32_t src = ok ? at[i] : 0u;
          cp_async4(ss, p.c.ks + src, ok ? 4 : 0);
          cp_async4(ss + KW * 4, p.c.vs + src, ok ? 4 : 0);
        }
      }
    };

    // online softmax and P V of one group of scores: s[mt][2 g + j][..], base-2
    // exponents after `p.c2` (16-bit caches) or as they are (8-bit)
    auto new_max = [&](float (&s)[MT][2 * SG][4]) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = mrow[mt][e];
#pragma unroll
          for (int n = 0; n < 2 * SG; ++n) m = fmaxf(m, fmaxf(s[mt][n][2 * e], s[mt][n][2 * e + 1]));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
          if (m != mrow[mt][e]) {                       // the quad's lanes agree
            const float f = ex2((mrow[mt][e] - m) * (WIDE ? p.c2 : 1.f));   // 2^-inf = 0 at the first keys
            lrow[mt][e] *= f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              oacc[mt][n][2 * e] *= f;
              oacc[mt][n][2 * e + 1] *= f;
            }
            mrow[mt][e] = m;
          }
        }
    };

    // relation terms of four consecutive offsets from d0 on
    auto z4 = [&](const float* z, int d0, float (&out)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = z[iclamp(d0 + i, p.e_lo, p.e_hi) - p.e_lo];
    };

    // adds the non-finite value elements of nodes [ua, ub) to the rows that attend them
    auto add_non_finite = [&](int ua, int ub) {
      for (int u = max(ua, 0); u < min(ub, p.T); ++u) {
        const QT* src = static_cast<const QT*>(p.v) + b * p.vs.b + hkv * p.vs.h + u * p.vs.n;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = DT<QT>::to_f(src[WIDE ? n * 8 + 2 * q4 + c : (2 * q4 + c) * NT + n]);
            if (fabsf(x) <= 3.4028235e38f) continue;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if ((row[mt][e].mask >> u) & 1ull) oacc[mt][n][2 * e + c] += x;
          }
      }
    };

    uint32_t at_next[LR];
    {
      uint32_t at[LR];
#pragma unroll
      for (int s = 0; s < TL::STAGES - 1; ++s) {
        lookup(tile0 + s, at);
        if (tile0 + s < tile1) issue(tile0 + s, s, at);
        cp_async_commit();
      }
      lookup(tile0 + TL::STAGES - 1, at_next);
    }
    int stage = 0;
    for (int tile = tile0; tile < tile1; ++tile) {
      cp_async_wait<TL::STAGES - 2>();
      group_sync();
      {
        const int nx = tile + TL::STAGES - 1;
        int ns = stage + TL::STAGES - 1;
        if (ns >= TL::STAGES) ns -= TL::STAGES;
        if (nx < tile1) issue(nx, ns, at_next);
        cp_async_commit();
        lookup(nx + 1, at_next);
      }
      const uint32_t sk = stage0 + (uint32_t)stage * GSTAGE, sv = sk + HALF;
      const int k0 = tile * TK + wn * KW;
      bool full = true;
#pragma unroll
      for (int i = 0; i < LR; ++i)
        full = full && valid_bits[wn][stage][i] == (KW >= 32 ? 0xffffffffu : (1u << (KW & 31)) - 1u);
      const bool plain = full && k0 + KW <= len;        // every key is a valid cached one

      // ---- scores
      float s[MT][2 * SG][4];
      const bool low = k0 + KW <= len && k0 + KW - 1 - len <= p.e_lo;   // every offset is saturated: one value a row
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float z[4] = {0.f, 0.f, 0.f, 0.f};
            if (WIDE && p.z && row[mt][e].z) {
              if (low) {
                z[0] = z[1] = z[2] = z[3] = row[mt][e].z[0];
              } else {
                const int j = k0 + 16 * g + 4 * q4, here = len + row[mt][e].depth;
                z4(row[mt][e].z, j - here, z);
                if (j + 4 > len) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int u = j + i - len;
                    if (u >= 0 && u < p.T) {
                      const int du = max(__popcll(node_mask(p, b, u)) - 1, 0);
                      z[i] = row[mt][e].z[iclamp(du - row[mt][e].depth, p.e_lo, p.e_hi) - p.e_lo];
                    }
                  }
                }
              }
            }
            s[mt][2 * g][2 * e] = z[0];
            s[mt][2 * g][2 * e + 1] = z[1];
            s[mt][2 * g + 1][2 * e] = z[2];
            s[mt][2 * g + 1][2 * e + 1] = z[3];
          }
#pragma unroll
      for (int g = 0; g < SG; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int kr = 16 * g + 4 * (r8 >> 1) + (r8 & 1) + 2 * j;
#pragma unroll
          for (int u = 0; u < CPR / 4; ++u) {
            const uint4 w = lds128(sk + chunk_at<CPR, WIDE, false>(kr, 4 * u + q4));
            if (WIDE) {
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                MmaOp<MT16>::run(s[mt][2 * g + j], qa[mt][2 * u], w.x, w.y);
                MmaOp<MT16>::run(s[mt][2 * g + j], qa[mt][2 * u + 1], w.z, w.w);
              }
            } else {
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                expand4<FMT>(ww[i], b0, b1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) MmaOp<MT16>::run(s[mt][2 * g + j], qa[mt][(4 * u + i) % KS], b0, b1);
              }
            }
          }
        }
      float rsv[SG][4];                                 // 1 / value scale of the thread's keys
      if (!WIDE) {
#pragma unroll
        for (int g = 0; g < SG; ++g) {
          const uint4 a = lds128(sk + 2 * HALF + (16 * g + 4 * q4) * 4);
          const uint4 v4 = lds128(sk + 2 * HALF + KW * 4 + (16 * g + 4 * q4) * 4);
          const float kcol[4] = {__uint_as_float(a.x) * kc, __uint_as_float(a.y) * kc, __uint_as_float(a.z) * kc,
                                 __uint_as_float(a.w) * kc};
          const float vs4[4] = {__uint_as_float(v4.x), __uint_as_float(v4.y), __uint_as_float(v4.z),
                                __uint_as_float(v4.w)};
          float lg[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // not fmaxf, which would drop the NaN of a spoilt row
            const float v = vs4[i] < 0x1p-100f ? 0x1p-100f : vs4[i];
            lg[i] = lg2(v);
            rsv[g][i] = rcp(v);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float z[4] = {0.f, 0.f, 0.f, 0.f};
              if (p.z && row[mt][e].z) {
                if (low) z[0] = z[1] = z[2] = z[3] = row[mt][e].z[0];
                else z4(row[mt][e].z, k0 + 16 * g + 4 * q4 - len - row[mt][e].depth, z);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float& x = s[mt][2 * g + (i >> 1)][2 * e + (i & 1)];
                x = fmaf(x, kcol[i], lg[i] + z[i]);
              }
            }
        }
      }
      if (!plain) {
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kl = 16 * g + 4 * q4 + i;
            const bool there = (valid_bits[wn][stage][kl >> 5] >> (kl & 31)) & 1u;
            const int u = k0 + kl - len;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const bool keep = there && (u < 0 || ((row[mt][e].mask >> (u & 63)) & 1ull));
                if (!keep) s[mt][2 * g + (i >> 1)][2 * e + (i & 1)] = -INFINITY;
              }
          }
      }
      // ---- softmax
      new_max(s);
      uint32_t pa[MT][SG][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m0 = safe(mrow[mt][e]);
#pragma unroll
          for (int g = 0; g < SG; ++g) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = s[mt][2 * g + (i >> 1)][2 * e + (i & 1)];
              w[i] = WIDE ? ex2(fmaf(x, p.c2, -m0 * p.c2)) : ex2(x - m0);
              lrow[mt][e] = WIDE ? lrow[mt][e] + w[i] : fmaf(w[i], rsv[g][i], lrow[mt][e]);
            }
            pa[mt][g][e] = DT<MT16>::pack(w[0], w[1]);
            pa[mt][g][2 + e] = DT<MT16>::pack(w[2], w[3]);
          }
        }
      // ---- P V
      bool odd = false;                                 // a node's value element is not finite
#pragma unroll
      for (int g = 0; g < SG; ++g) {
        if (WIDE) {
          const int mi = lane >> 3, n = lane & 7;
          const int kr = 16 * g + 4 * (n >> 1) + (n & 1) + 2 * (mi & 1);
#pragma unroll
          for (int dp = 0; dp < NT / 2; ++dp) {
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(sv + chunk_at<CPR, WIDE, true>(kr, dp * 2 + (mi >> 1)), b0, b1, b2, b3);
            if (k0 + 16 * g + 16 > len) {               // some of these 16 keys are nodes
              const int kn = k0 + 16 * g + 4 * q4 - len;   // node of this lane's first key (b0: +0, +1; b1: +2, +3)
              bool x0 = false, x1 = false;
              const uint32_t n0 = clean2<QT>(b0, x0), n2 = clean2<QT>(b2, x0);
              const uint32_t n1 = clean2<QT>(b1, x1), n3 = clean2<QT>(b3, x1);
              // a pair that holds a cached key stays as it is where that key's element is the odd one
              if (x0 && kn + 1 >= 0) { b0 = kn >= 0 ? n0 : (n0 & 0xffff0000u) | (b0 & 0xffffu);
                                       b2 = kn >= 0 ? n2 : (n2 & 0xffff0000u) | (b2 & 0xffffu); odd = true; }
              if (x1 && kn + 3 >= 0) { b1 = kn + 2 >= 0 ? n1 : (n1 & 0xffff0000u) | (b1 & 0xffffu);
                                       b3 = kn + 2 >= 0 ? n3 : (n3 & 0xffff0000u) | (b3 & 0xffffu); odd = true; }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              MmaOp<MT16>::run(oacc[mt][2 * dp], pa[mt][g], b0, b1);
              MmaOp<MT16>::run(oacc[mt][2 * dp + 1], pa[mt][g], b2, b3);
            }
          }
        } else {
          // D / 8 consecutive columns of four consecutive keys
          uint32_t vw[4][D / 32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kr = 16 * g + 4 * q4 + i;
            if (D == 128) {
              const uint4 w = lds128(sv + chunk_at<CPR, WIDE, true>(kr, r8));
              vw[i][0] = w.x;
              vw[i][1] = w.y;
              vw[i][D / 32 - 2] = w.z;
              vw[i][D / 32 - 1] = w.w;
            } else {
              const uint2 w = lds64(sv + chunk_at<CPR, WIDE, true>(kr, r8 >> 1) + 8 * (r8 & 1));
              vw[i][0] = w.x;
              vw[i][1] = w.y;
            }
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {
            uint32_t b0[4], b1[4];
            expand4<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x5140), b0[0], b0[1]);
            expand4<FMT>(__byte_perm(vw[0][w], vw[1][w], 0x7362), b0[2], b0[3]);
            expand4<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x5140), b1[0], b1[1]);
            expand4<FMT>(__byte_perm(vw[2][w], vw[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) MmaOp<MT16>::run(oacc[mt][4 * w + c], pa[mt][g], b0[c], b1[c]);
          }
        }
      }
      if (WIDE && k0 + KW > len && __any_sync(0xffffffffu, odd)) add_non_finite(k0 - len, k0 + KW - len);
      if (++stage == TL::STAGES) stage = 0;
    }
    cp_async_wait<0>();

    // ---- 8-bit caches: the nodes' own keys, straight from their 16-bit tensors,
    // 16 nodes at a time; bf16 rows enter as fp16 times a power of two that
    // takes the place of the scale
    if (!WIDE && tile1 == nt) {
      for (int u0 = 16 * wn; u0 < p.T; u0 += 16 * WN) {
        float s[MT][2 * SG][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < 2 * SG; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][n][i] = n < 2 ? 0.f : -INFINITY;
        float kmul[2];
        bool odd = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int u = u0 + 4 * (r8 >> 1) + (r8 & 1) + 2 * j;
          uint32_t kw[D / 8];
          uint32_t kt = 0;
#pragma unroll
          for (int w = 0; w < D / 64; ++w)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              uint4 x = make_uint4(0, 0, 0, 0);
              if (u < p.T)
                x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + b * p.ks.b + hkv * p.ks.h +
                                                         u * p.ks.n + 64 * w + 16 * q4 + 8 * hh));
              kw[8 * w + 4 * hh] = x.x;
              kw[8 * w + 4 * hh + 1] = x.y;
              kw[8 * w + 4 * hh + 2] = x.z;
              kw[8 * w + 4 * hh + 3] = x.w;
              if (DT<QT>::kCoarse) kt = amax2(amax2(amax2(amax2(kt, x.x), x.y), x.z), x.w);
            }
          float down = 1.f;
          kmul[j] = 1.f;
          if (DT<QT>::kCoarse) {
            kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, 1));
            kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, 2));
            const int e = exp_of(kt);
            down = pow2i(-e);
            kmul[j] = pow2i(e);
          }
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint32_t b0 = to_half2<QT>(kw[2 * ks], down), b1 = to_half2<QT>(kw[2 * ks + 1], down);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) MmaOp<MT16>::run(s[mt][j], qa[mt][ks], b0, b1);
          }
        }
        // the power of key slot c lives in the lanes with r8 = c: columns 2 q and 2 q + 1 of this lane
        float kcol[4], lg[4], rv[4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) kcol[2 * j + c] = __shfl_sync(0xffffffffu, kmul[j], 4 * (2 * q4 + c)) * kc;
        uint32_t vh[4][D / 16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int u = u0 + 4 * q4 + i;
          uint32_t vt = 0;
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (u < p.T)
              x = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + b * p.vs.b + hkv * p.vs.h +
                                                       u * p.vs.n + r8 * (D / 8) + 8 * w));
            vh[i][4 * w] = x.x;
            vh[i][4 * w + 1] = x.y;
            vh[i][4 * w + 2] = x.z;
            vh[i][4 * w + 3] = x.w;
            if (DT<QT>::kCoarse) vt = amax2(amax2(amax2(amax2(vt, x.x), x.y), x.z), x.w);
          }
          lg[i] = 0.f;
          rv[i] = 1.f;
          if (DT<QT>::kCoarse) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) vt = max(vt, __shfl_xor_sync(0xffffffffu, vt, o));
            const int e = exp_of(vt);
            lg[i] = (float)e;
            rv[i] = pow2i(-e);
#pragma unroll
            for (int w = 0; w < D / 16; ++w) vh[i][w] = to_half2<QT>(vh[i][w], rv[i]);
          }
#pragma unroll
          for (int w = 0; w < D / 16; ++w) vh[i][w] = clean2<__half>(vh[i][w], odd);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int u = u0 + 4 * q4 + i;
          const int du = u < p.T ? max(__popcll(node_mask(p, b, u)) - 1, 0) : 0;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float z = 0.f;
              if (p.z && row[mt][e].z) z = row[mt][e].z[iclamp(du - row[mt][e].depth, p.e_lo, p.e_hi) - p.e_lo];
              float& x = s[mt][i >> 1][2 * e + (i & 1)];
              const bool keep = u < p.T && ((row[mt][e].mask >> (u & 63)) & 1ull);
              x = keep ? fmaf(x, kcol[i], lg[i] + z) : -INFINITY;
            }
        }
        new_max(s);
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m0 = safe(mrow[mt][e]);
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i] = ex2(s[mt][i >> 1][2 * e + (i & 1)] - m0);
              lrow[mt][e] = fmaf(w[i], rv[i], lrow[mt][e]);
            }
            pa[mt][e] = DT<MT16>::pack(w[0], w[1]);
            pa[mt][2 + e] = DT<MT16>::pack(w[2], w[3]);
          }
#pragma unroll
        for (int w = 0; w < D / 16; ++w)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t b0 = __byte_perm(vh[0][w], vh[1][w], c ? 0x7632 : 0x5410);
            const uint32_t b1 = __byte_perm(vh[2][w], vh[3][w], c ? 0x7632 : 0x5410);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) MmaOp<MT16>::run(oacc[mt][2 * w + c], pa[mt], b0, b1);
          }
        if (__any_sync(0xffffffffu, odd)) add_non_finite(u0, u0 + 16);
      }
    }

    // ---- join the key groups of the block
    const float cm = WIDE ? p.c2 : 1.f;                 // base-2 units of the maxima
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[mt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int r = (wm * MT + mt) * 16 + r8 + 8 * e;
        if (q4 == 0) {
          sm_m[wn][r] = mrow[mt][e] * cm;
          sm_l[wn][r] = l;
        }
      }
    __syncthreads();                                    // also: every stage has been read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = (wm * MT + mt) * 16 + r8 + 8 * e;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = fmaxf(m, sm_m[w][r]);
        const float f = ex2(mrow[mt][e] * cm - safe(m));
        float* dst = merge + (wn * ROWS + r) * D;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int slot = 2 * q4 + c;
            dst[WIDE ? n * 8 + slot : slot * NT + n] = oacc[mt][n][2 * e + c] * f;
          }
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == nt;
    float* slot = p.part + ((long long)blockIdx.x * 2 + (cur == my_start ? 0 : 1)) * slot_floats(ROWS, D);
    for (int i = tid; i < ROWS * (D / 4); i += 128) {
      const int r = i / (D / 4), c = i % (D / 4);
      const int gr = rb * ROWS + r;
      if (gr >= R) break;                               // rows ascend with i
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < WN; ++w) m = fmaxf(m, sm_m[w][r]);
#pragma unroll
      for (int w = 0; w < WN; ++w) l += sm_l[w][r] * ex2(sm_m[w][r] - safe(m));
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * ROWS + r) * D + 4 * c);
        o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
      }
      if (!whole) {
        *reinterpret_cast<float4*>(slot + (long long)r * D + 4 * c) = o;
        if (c == 0) {
          slot[ROWS * D + r] = m;
          slot[ROWS * D + ROWS + r] = l;
        }
      } else {
        store_row(p, b, hkv, gr, c, o, m, l);
      }
    }
    __syncthreads();                                    // the stages and sums are free again
    cur += tile1 - tile0;
  }
}

template <class TL, int FMT>
constexpr int stage_bytes() {
  constexpr bool wide = FMT == RELPOS_CACHE_F16;
  constexpr int st = TL::WN * TL::STAGES * (2 * TL::KW * TL::D * (wide ? 2 : 1) + (wide ? 0 : TL::KW * 8));
  constexpr int mg = TL::WN * TL::ROWS * TL::D * 4;
  return st > mg ? st : mg;
}

template <class TL, typename QT, int FMT>
cudaError_t run_tiling(const TreeParams& p, cudaStream_t s) {
  static std::atomic<unsigned long long> ready{0};      // devices whose limit has been raised
  const int smem = stage_bytes<TL, FMT>() + (((p.B + 1) * 4 + 127) & ~127);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(tree_kernel<TL, QT, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready |= 1ull << dev;
  }
  tree_kernel<TL, QT, FMT><<<p.grid, 128, smem, s>>>(p);
  note_launch(1);
  return cudaGetLastError();
}

// Tilings by head dimension and row count: up to 16 and 32 rows four (or two)
// groups of warps take different keys, beyond that the warps share the keys and
// take different rows.
using T64_16 = Tiling<64, 1, 4, 1, 32, 3>;
using T64_32 = Tiling<64, 1, 4, 2, 32, 3>;
using T64_64 = Tiling<64, 2, 2, 2, 32, 3>;
using T128_16 = Tiling<128, 1, 4, 1, 16, 3>;
using T128_32 = Tiling<128, 2, 2, 1, 32, 3>;
using T128_64 = Tiling<128, 4, 1, 1, 64, 3>;

template <typename QT, int FMT>
cudaError_t run_format(const TreeParams& p, cudaStream_t s) {
  if (p.c.d == 64) {
    if (p.rows_per_block == 16) return run_tiling<T64_16, QT, FMT>(p, s);
    if (p.rows_per_block == 32) return run_tiling<T64_32, QT, FMT>(p, s);
    return run_tiling<T64_64, QT, FMT>(p, s);
  }
  if (p.rows_per_block == 16) return run_tiling<T128_16, QT, FMT>(p, s);
  if (p.rows_per_block == 32) return run_tiling<T128_32, QT, FMT>(p, s);
  return run_tiling<T128_64, QT, FMT>(p, s);
}

cudaError_t run_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_bf16(const TreeParams& p, cudaStream_t s);
cudaError_t run_e4m3_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_e4m3_bf16(const TreeParams& p, cudaStream_t s);
cudaError_t run_int8_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_int8_bf16(const TreeParams& p, cudaStream_t s);

}  // namespace tree
}  // namespace relpos
