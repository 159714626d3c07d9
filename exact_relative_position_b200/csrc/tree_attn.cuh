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
// Tensor work: mma.sync m16n8k16 with the keys as the 16 rows and the query
// rows as the 8 columns, S^T = K Q^T and O^T = V^T P^T, so that decoding with
// up to eight query heads to a key head fills the tile.  With so few rows each
// loaded element feeds few multiply-adds and the kernel is bound by memory;
// 128-row tcgen05 tiles would run mostly empty.  64 single tokens over up to 8192
// keys, 32 / 8 heads of 128: e4m3 126 us (5.6 TB/s, 86% of a plain copy's rate); 32 of
// them over bf16 113 us (6.0 TB/s, 94% of it).  More rows over a 16-bit cache: tree_wide.cu.
// 61-node trees over 8 bits stay here, in blocks of 64 rows that each read and expand the
// cache: 16 of them over up to 8192 keys, 32 / 8 heads of 128, e4m3 with bf16 queries 531 us.
//
// Order of the operands.  An MMA sums over k in any order and names its rows in
// any order, as long as both operands agree.  Each lane of a quad therefore
// takes 16 consecutive bytes of a key row for its k slots (one shared-memory
// load feeds 2 to 4 MMAs, 8-bit codes are expanded in registers), and row slot
// c of 16 keys stands for key 4 (c / 2) + c % 2 (c < 8) or 2 more than slot c - 8,
// which makes the four rows of V that a lane pairs up consecutive keys.  P^T
// goes from the score layout to the operand layout by movmatrix.
//
// Weights enter P V in 16 bits, as in the layer's forward: the cache's own type, fp16 over 8
// bits; their sums stay fp32.  Split weights would double the MMAs of P V to take the error of
// O against 64 bits from 0.00023 to 0.00021 (fp16) and from 0.0021 to 0.0017 (bf16), where the
// rounding of O itself is the rest.
//
// The row maximum is moved only when a score exceeds it by 2^8: weights stay
// within 2^8, far from fp16's range, and most steps skip the rescaling of O and
// the reduction over lanes.
//
// 8-bit caches: codes are exact in fp16.  The scale of key j multiplies its
// score row; that of its value row is folded into the exponent, so that
// the fp16 weight is 2^(s_ij + log2 sv_j - m_i) with m_i the row's
// running maximum of that sum, and the softmax sum divides it out in fp32:
//   P'_ij = 2^(s_ij + log2 sv_j - m_i),  l_i = sum_j P'_ij / sv_j,
//   O_i = sum_j P'_ij code_j / l_i,      LSE_i = m_i + log2 l_i (base 2).
// A value row of zeros is stored with scale 1.  Taken at that, a key that is attended
// strongly and holds zeros (they are common where a model parks its attention) would set
// m_i far above what the other keys, with scales of 2^-10, add to O, and their 16-bit weights
// would be subnormal or 0.  Such a row enters at 2^-64, so that it sets the maximum only where
// it leaves the others less than 2^-50 of their values, and its share of l_i, kept in fp32, is
// exact for the others' scales up to 2^30.
// bf16 queries enter in fp16 after an exact power-of-two scaling of each row to a
// largest element in [2^14, 2^15): a power of the row's own, since what a padding node or
// another head holds must not cost this one its precision.
#pragma once

#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

#include "kernels.cuh"
#include "serve.cuh"
#include "warp_mma.cuh"

namespace relpos {
namespace tree {

using relpos::cp_async16;

// Tiling of a row count: WM x WN warps, NR tiles of 8 query rows to a warp, KW
// keys to a group of WM warps and stage, SK keys to a step, BPS blocks to an SM.
template <int D_, int WM_, int WN_, int NR_, int KW_, int SK_, int STAGES_, int BPS_> struct Tiling {
  static constexpr int D = D_, WM = WM_, WN = WN_, NR = NR_, KW = KW_, SK = SK_, STAGES = STAGES_, BPS = BPS_;
  static constexpr int ROWS = WM * NR * 8, TK = WN * KW;
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

// Sum-order-preserving join of (m, l): -inf for nothing yet.
__device__ __forceinline__ float safe(float m) { return m == -INFINITY ? 0.f : m; }

// ---------------------------------------------------------------- the line of tiles
// pre[b]: tiles of one item summed over the sequences before b.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src));
}

struct Line {
  const int* pre;
  int B, items;                      // items (key head, row block) of a sequence
  int total, quantum;                // tiles of the line and of a piece
  __device__ __forceinline__ int seq_of(int at) const {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] * items <= at) lo = mid; else hi = mid;
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
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
// The power e with |x| 2^-e in [2^14, 2^15) for the largest |x| given by its bits, not below
// `least`.  Keys and queries go down to -126 (bf16's smallest normal numbers), value rows to -100:
// they are divided out of the row sum again, which holds 2^-e times a weight.
__device__ __forceinline__ int exp_of(uint32_t bits, int least) { return max((int)(bits >> 23) - 127 - 14, least); }

// What a value row of zeros counts as (see above): as a scale, and as a node's power.
constexpr float kZeroRowScale = 0x1p-64f;
constexpr int kZeroRowPower = -64;

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
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <class TL, typename QT, int FMT>
__global__ void __launch_bounds__(128, TL::BPS) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool WIDE = FMT == RELPOS_CACHE_F16;        // the cache has the queries' 16-bit type
  constexpr int D = TL::D, WM = TL::WM, WN = TL::WN, NR = TL::NR, KW = TL::KW, TK = TL::TK, ROWS = TL::ROWS;
  constexpr int ES = WIDE ? 2 : 1;
  constexpr int CPR = D * ES / 16;                      // chunks of a row
  constexpr int GT = WM * 32;                           // threads that share a group of KW keys
  constexpr int KS = D / 16;                            // k steps of q.k
  constexpr int MTD = D / 16;                           // 16-row tiles of the output's d
  constexpr int SG = TL::SK / 16;                       // groups of 16 keys to a step
  constexpr int HALF = KW * CPR * 16;                   // bytes of a group's keys (or values) in a stage
  constexpr int GSTAGE = 2 * HALF + (WIDE ? 0 : KW * 8);
  using MT16 = typename std::conditional<WIDE, QT, __half>::type;   // operand type of the MMAs

  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sums[4];
  __shared__ uint32_t valid_bits[WN][TL::STAGES][(KW + 31) / 32];
  __shared__ float sm_m[WN][ROWS], sm_l[WN][ROWS];
  __shared__ const float* row_z[ROWS];                  // relation terms of a row at offset e_lo
  __shared__ unsigned long long row_mask[ROWS];         // nodes it attends (0: padding, or no row)
  __shared__ int row_depth[ROWS], node_depth[64];
  __shared__ __align__(8) float row_kc[ROWS];           // bf16, 8-bit caches: tau log2 e times the row's power of two
  int* pre = reinterpret_cast<int*>(smem);              // [B + 1], rounded up to 128 bytes
  const uint32_t pre_bytes = (uint32_t)((p.B + 1) * 4 + 127) & ~127u;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp / WN, wn = warp % WN;
  const int gtid = wm * 32 + lane;                      // place in the group of warps with this wn
  const int q4 = lane & 3, r8 = lane >> 2;
  const int key0 = 4 * (r8 >> 1) + (r8 & 1);            // key (of 16) of row slot r8; slot r8 + 8: two more
  const uint32_t stage0 = smem_u32(smem) + pre_bytes + (uint32_t)(wn * TL::STAGES * GSTAGE);
  static_assert(GSTAGE >= WM * 8 * D * 4, "a stage holds eight rows of outputs of each of its warps");

  auto group_sync = [&]() {
    if (WM == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(wn + 1), "n"(GT) : "memory");
  };

  build_line<128>(p, TK, WIDE, pre, warp_sums);
  Line line;
  line.pre = pre;
  line.B = p.B;
  line.items = p.c.Hkv * p.row_blocks;
  line.total = pre[p.B] * line.items;
  line.quantum = (line.total + gridDim.x - 1) / gridDim.x;
  const int my_start = line.quantum * blockIdx.x;
  const int my_end = min(line.total, my_start + line.quantum);
  if (my_start >= my_end) return;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const int R = p.G * p.T;

  // Two places on the line: the tile that is loaded next and the one that is
  // computed.  Loads run ahead across the borders of items.
  struct Place {
    int at, b, item, tile, nt, len, hkv;
  };
  auto seat = [&](Place& c) {
    c.b = line.seq_of(c.at);
    c.nt = pre[c.b + 1] - pre[c.b];
    const int in_b = c.at - pre[c.b] * line.items;
    c.item = in_b / c.nt;
    c.tile = in_b - c.item * c.nt;
    c.hkv = c.item / p.row_blocks;
    c.len = seq_len(p, c.b);
  };
  auto advance = [&](Place& c, int tiles) {             // to the next tile, or the next item's first
    c.at += tiles;
    c.tile += tiles;
    if (c.tile < c.nt) return;
    c.tile = 0;
    if (++c.item == line.items) {
      c.item = 0;
      if (++c.b >= p.B) return;
      c.nt = pre[c.b + 1] - pre[c.b];
      c.len = seq_len(p, c.b);
    }
    c.hkv = c.item / p.row_blocks;
  };

  // ---- loads: rows of the cache by page, nodes behind them (16-bit cache)
  const uint8_t* kc_base = static_cast<const uint8_t*>(p.c.k);
  const uint8_t* vc_base = static_cast<const uint8_t*>(p.c.v);
  // A group's KW keys lie in one page where pages are that large: one look-up, and
  // all addresses are constants away from the first row's.
  const bool one_page = KW <= page_mask + 1;
  // row of the cache of key j; all ones: none
  auto place_of = [&](const Place& c, int j) {
    uint32_t at = 0xffffffffu;
    if (j < c.len) {
      const int id = __ldg(p.page_table + (long long)c.b * p.P + (j >> p.c.page_shift));
      if (id >= 0 && id < p.c.num_pages)
        at = (((uint32_t)id * (uint32_t)p.c.Hkv + (uint32_t)c.hkv) << p.c.page_shift) + (uint32_t)(j & page_mask);
    }
    return at;
  };
  // ahead of the loads: the row of the group's first key
  auto lookup = [&](const Place& c) { return c.at < my_end && one_page ? place_of(c, c.tile * TK + wn * KW) : 0xffffffffu; };
  constexpr int LR = (KW + 31) / 32;                    // rows whose place a lane looks up otherwise
  // returns whether all KW keys are valid cached ones
  auto issue = [&](const Place& c, int stage, uint32_t first) {
    const uint32_t sk = stage0 + (uint32_t)stage * GSTAGE, sv = sk + HALF;
    const int k0 = c.tile * TK + wn * KW;
    const int ch = gtid % CPR, r0 = gtid / CPR;
    constexpr int RI = GT / CPR;                        // rows of an iteration
    if (first != 0xffffffffu && k0 + KW <= c.len) {
      const unsigned long long off = ((unsigned long long)first + r0) * (D * ES) + ch * 16;
      const uint8_t *ksrc = kc_base + off, *vsrc = vc_base + off;
#pragma unroll
      for (int i = 0; i < KW / RI; ++i) {
        cp_async16(sk + chunk_at<CPR, WIDE, false>(i * RI + r0, ch), ksrc + i * RI * D * ES);
        cp_async16(sv + chunk_at<CPR, WIDE, true>(i * RI + r0, ch), vsrc + i * RI * D * ES);
      }
      if (!WIDE && wm == 0) {
#pragma unroll
        for (int i = 0; i < LR; ++i) {
          const int lr = 32 * i + lane;
          if (KW % 32 == 0 || lr < KW) {
            cp_async4(sk + 2 * HALF + lr * 4, p.c.ks + first + lr, 4);
            cp_async4(sk + 2 * HALF + KW * 4 + lr * 4, p.c.vs + first + lr, 4);
          }
        }
      }
      return true;
    }
    // row by row: small or missing pages, the end of the cache, and (16-bit cache) the nodes behind it
    uint32_t at[LR];
    const bool nodes = WIDE && k0 + KW > c.len;
    bool all = !nodes;
#pragma unroll
    for (int i = 0; i < LR; ++i) {
      const int lr = 32 * i + lane;
      at[i] = lr < KW ? place_of(c, k0 + lr) : 0xffffffffu;
      all = all && (at[i] != 0xffffffffu || lr >= KW);
      const bool ok = at[i] != 0xffffffffu || (nodes && lr < KW && k0 + lr >= c.len && k0 + lr < c.len + p.T);
      const uint32_t bits = __ballot_sync(0xffffffffu, ok);
      if (wm == 0 && lane == 0) valid_bits[wn][stage][i] = bits;
      if (!WIDE && wm == 0 && lr < KW) {
        const uint32_t ss = sk + 2 * HALF + lr * 4;
        const uint32_t src = ok ? at[i] : 0u;
        cp_async4(ss, p.c.ks + src, ok ? 4 : 0);
        cp_async4(ss + KW * 4, p.c.vs + src, ok ? 4 : 0);
      }
    }
#pragma unroll 2
    for (int i = 0; i < KW / RI; ++i) {
      const int r = i * RI + r0;
      const uint32_t mine = LR > 1 && i * RI >= 32 ? at[LR - 1] : at[0];
      const uint32_t at_r = __shfl_sync(0xffffffffu, mine, r & 31);
      const uint8_t *ksrc = kc_base, *vsrc = vc_base;
      int bytes = 0;
      if (at_r != 0xffffffffu) {
        const unsigned long long off = (unsigned long long)at_r * (D * ES) + ch * 16;
        ksrc += off;
        vsrc += off;
        bytes = 16;
      } else if (nodes) {
        const int u = k0 + r - c.len;
        if (u >= 0 && u < p.T) {
          ksrc = static_cast<const uint8_t*>(p.k) + 2 * (c.b * p.ks.b + c.hkv * p.ks.h + u * p.ks.n + ch * 8);
          vsrc = static_cast<const uint8_t*>(p.v) + 2 * (c.b * p.vs.b + c.hkv * p.vs.h + u * p.vs.n + ch * 8);
          bytes = 16;
        }
      }
      cp_async16(sk + chunk_at<CPR, WIDE, false>(r, ch), ksrc, bytes);
      cp_async16(sv + chunk_at<CPR, WIDE, true>(r, ch), vsrc, bytes);
    }
    return (bool)__all_sync(0xffffffffu, all);
  };

  Place ld, cp;
  ld.at = my_start;
  seat(ld);
  cp = ld;
  uint32_t at_next, full_stages = 0;                    // bit s: stage s holds KW valid cached keys
  auto load = [&](int s, uint32_t first) {
    bool full = false;
    if (ld.at < my_end) full = issue(ld, s, first);
    cp_async_commit();
    full_stages = (full_stages & ~(1u << s)) | ((full ? 1u : 0u) << s);
    advance(ld, 1);
  };
  {
    uint32_t at[TL::STAGES - 1];
    Place c = ld;
#pragma unroll
    for (int s = 0; s < TL::STAGES - 1; ++s) {          // all look-ups first: their latencies overlap
      at[s] = lookup(c);
      advance(c, 1);
    }
    at_next = lookup(c);
#pragma unroll 1
    for (int s = 0; s < TL::STAGES - 1; ++s) load(s, s == 0 ? at[0] : at[TL::STAGES - 2]);
  }
  static_assert(TL::STAGES <= 3, "the first look-ups are picked from two");
  int stage = 0;
  // what ran before this kernel has been waited for by the relation kernel, where
  // there is one; its own results are read from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");

#pragma unroll 1
  while (cp.at < my_end) {
    const int b = cp.b, nt = cp.nt, hkv = cp.hkv, len = cp.len;
    const int rb = cp.item - hkv * p.row_blocks;
    const int tile0 = cp.tile, tile1 = min(nt, tile0 + (my_end - cp.at));
    const bool first_item = cp.at == my_start;

    // ---- the rows of the item
    if (tid < ROWS) {
      // a row that no query has attends nothing, and reads the last query's relation terms: it
      // votes on moving the maxima, which terms that nobody wrote must not decide
      const int r = min(rb * ROWS + tid, R - 1);
      const int t = r / p.G, h = hkv * p.G + (r - t * p.G);
      const unsigned long long mk = rb * ROWS + tid < R ? node_mask(p, b, t) : 0ull;
      const float* z = p.z + (b * p.z_b + h * p.z_h + t * p.z_t);
      row_mask[tid] = mk;
      row_depth[tid] = max(__popcll(mk) - 1, 0);
      row_z[tid] = z;
    } else if (tid - 64 >= 0 && tid - 64 < p.T) {
      node_depth[tid - 64] = max(__popcll(node_mask(p, b, tid - 64)) - 1, 0);
    }

    // ---- queries: B fragments in the permuted k order, row r8 of each tile
    uint32_t qb[NR][KS][2];
    constexpr bool POWERS = !WIDE && DT<QT>::kCoarse;   // rows of queries have powers of two
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = rb * ROWS + (wm * NR + n) * 8 + r8;
      const int t = r < R ? r / p.G : 0, h = hkv * p.G + (r < R ? r - t * p.G : 0);
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + b * p.qs.b + h * p.qs.h + (long long)t * p.qs.n;
      uint32_t top = 0;
#pragma unroll
      for (int u = 0; u < D / 32; ++u) {
        // 16-bit keys: 8 elements at 32 u + 8 q; 8-bit keys: 8 of the 16 elements at 64 (u / 2) + 16 q
        const int d0 = WIDE ? 32 * u + 8 * q4 : 64 * (u / 2) + 16 * q4 + 8 * (u % 2);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (r < R) w = __ldg(reinterpret_cast<const uint4*>(src + d0));
        qb[n][2 * u][0] = w.x;
        qb[n][2 * u][1] = w.y;
        qb[n][2 * u + 1][0] = w.z;
        qb[n][2 * u + 1][1] = w.w;
        if (POWERS) top = amax2(amax2(amax2(amax2(top, w.x), w.y), w.z), w.w);
      }
      if (POWERS) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int power = exp_of(top, -126);            // of row r8
        const float down = pow2i(-power);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) qb[n][ks][i] = to_half2<QT>(qb[n][ks][i], down);
        if (q4 == 0) row_kc[(wm * NR + n) * 8 + r8] = p.c2 * pow2i(power);
      }
    }

    // ---- rows 2 q and 2 q + 1 of each tile: their saturated relation terms
    __syncthreads();
    auto row_of = [&](int n, int e) { return (wm * NR + n) * 8 + 2 * q4 + e; };   // in the block
    // what turns the products of rows 2 q and 2 q + 1 with a key's codes into base-2 scores, but for the key's scale
    auto unit_of = [&](int n) {
      if (!POWERS) return make_float2(p.c2, p.c2);
      const uint2 w = lds64(smem_u32(&row_kc[row_of(n, 0)]));
      return make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    };
    float zlow[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) zlow[n][e] = p.z ? row_z[row_of(n, e)][0] : 0.f;

    float oacc[NR][MTD][4];
    float mrow[NR][2], lrow[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int i = 0; i < MTD; ++i) oacc[n][i][0] = oacc[n][i][1] = oacc[n][i][2] = oacc[n][i][3] = 0.f;
      mrow[n][0] = mrow[n][1] = -INFINITY;
      lrow[n][0] = lrow[n][1] = 0.f;
    }
    const float unit = WIDE ? p.c2 : 1.f;               // base-2 units of scores and maxima
    const float slack = WIDE ? fminf(8.f / p.c2, 3e38f) : 8.f;   // (finite for the smallest tau, too)

    // moves the maxima where a score exceeds its row's by more than the slack
    auto new_max = [&](const float (&lm)[NR][2]) {
      bool up = false;
#pragma unroll
      for (int n = 0; n < NR; ++n) up = up || lm[n][0] - mrow[n][0] > slack || lm[n][1] - mrow[n][1] > slack;
      if (!__any_sync(0xffffffffu, up)) return;
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = fmaxf(lm[n][e], mrow[n][e]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float f = m == mrow[n][e] ? 1.f : ex2((mrow[n][e] - m) * unit);   // 2^-inf = 0 at the first keys
          mrow[n][e] = m;
          lrow[n][e] *= f;
#pragma unroll
          for (int i = 0; i < MTD; ++i) {
            oacc[n][i][e] *= f;
            oacc[n][i][2 + e] *= f;
          }
        }
    };

    // adds the non-finite value elements of nodes [ua, ub) to the rows that attend them
    auto add_non_finite = [&](int ua, int ub) {
      for (int u = max(ua, 0); u < min(ub, p.T); ++u) {
        const QT* src = static_cast<const QT*>(p.v) + b * p.vs.b + hkv * p.vs.h + u * p.vs.n;
#pragma unroll
        for (int i = 0; i < MTD; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = DT<QT>::to_f(src[WIDE ? 16 * i + 8 * c + r8 : r8 * (D / 8) + 2 * i + c]);
            if (fabsf(x) <= 3.4028235e38f) continue;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if ((row_mask[row_of(n, e)] >> u) & 1ull) oacc[n][i][2 * c + e] += x;
              }
          }
      }
    };

    // Unsaturated relation terms of a step's scores: looked up a step ahead where the
    // registers for it are there (up to 16 rows to a warp; over 8-bit caches at d = 128 up to 8:
    // 16 trees of 61 over up to 8192 keys, 32 / 8 heads, int8, 534 us against 554 with them, and
    // with one relation row per offset, 4 trees over 4096 keys, 79 against 82)
    struct Terms {
      float v[NR][SG][4];
    };
    constexpr bool AHEAD = NR <= 2 && (WIDE || NR == 1 || D < 128);
    auto terms_of = [&](int kf, Terms& z) {             // kf: the step's first key
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* zr = row_z[row_of(n, e)] - p.e_lo;
          const int depth = row_depth[row_of(n, e)];
#pragma unroll
          for (int g = 0; g < SG; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              int at = kf + 16 * g + key0 + 2 * j - len;
              if (WIDE && at >= 0) at = at < p.T ? node_depth[at] : 0;
              z.v[n][g][2 * j + e] = zr[iclamp(at - depth, p.e_lo, p.e_hi)];
            }
        }
    };

    // One step of SK keys from key ko of the group's KW, staged at sk / sv.  EASY: every
    // key is a valid cached one, and its relation term saturated (or there is none).
    auto step = [&](auto easy, int k0, int ko, uint32_t sk, uint32_t sv, int stage, bool full, const Terms& z) {
      constexpr bool EASY = decltype(easy)::value;
      float s[NR][SG][4];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[n][g][i] = WIDE && EASY ? zlow[n][i & 1] : 0.f;
      // ---- scores: k steps outside, so that consecutive MMAs have their own sums
#pragma unroll
      for (int u = 0; u < CPR / 4; ++u) {
#pragma unroll
        for (int g = 0; g < SG; ++g) {
          const int kr = ko + 16 * g + key0;
          const uint4 w0 = lds128(sk + chunk_at<CPR, WIDE, false>(kr, 4 * u + q4));
          const uint4 w1 = lds128(sk + chunk_at<CPR, WIDE, false>(kr + 2, 4 * u + q4));
          if (WIDE) {
            const uint32_t a0[4] = {w0.x, w1.x, w0.y, w1.y}, a1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
            for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(s[n][g], a0, qb[n][2 * u][0], qb[n][2 * u][1]);
#pragma unroll
            for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(s[n][g], a1, qb[n][2 * u + 1][0], qb[n][2 * u + 1][1]);
          } else {
            const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a[4];
              expand4<FMT>(x0[i], a[0], a[2]);
              expand4<FMT>(x1[i], a[1], a[3]);
              const int ks = (4 * u + i) % KS;
#pragma unroll
              for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(s[n][g], a, qb[n][ks][0], qb[n][ks][1]);
            }
          }
        }
      }
      if (WIDE && !EASY && p.z) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int g = 0; g < SG; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[n][g][i] += z.v[n][g][i];
      }
      float rsv[SG][2];                                 // 1 / value scale of the thread's keys
      if (!WIDE) {
        float2 kc[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) kc[n] = unit_of(n);
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a = sk + 2 * HALF + (ko + 16 * g + key0 + 2 * j) * 4;
            const float ks = __uint_as_float(lds32(a));
            float v = __uint_as_float(lds32(a + KW * 4));
            v = v < 0x1p-100f ? 0x1p-100f : v;          // not fmaxf, which would drop the NaN of a spoilt row
            const float lg = lg2(v);
            rsv[g][j] = rcp(v);
            // two rows at a time, so that the rows' own factors cost few instructions
            const float2 ks2 = make_float2(ks, ks), lg2v = make_float2(lg, lg);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              const float2 f = __fmul2_rn(ks2, kc[n]);
              float2 a = lg2v;
              if (EASY) a = __fadd2_rn(a, make_float2(zlow[n][0], zlow[n][1]));
              else if (p.z) a = __fadd2_rn(a, make_float2(z.v[n][g][2 * j], z.v[n][g][2 * j + 1]));
              const float2 x = __ffma2_rn(make_float2(s[n][g][2 * j], s[n][g][2 * j + 1]), f, a);
              s[n][g][2 * j] = x.x;
              s[n][g][2 * j + 1] = x.y;
            }
          }
      }
      if (!EASY && !full) {
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int kl = ko + 16 * g + key0 + 2 * j;
            const bool there = (valid_bits[wn][stage][kl >> 5] >> (kl & 31)) & 1u;
            const int u = k0 + kl - len;
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                bool keep = there;
                if (WIDE && there && u >= 0) keep = (row_mask[row_of(n, e)] >> u) & 1ull;
                if (!keep) s[n][g][2 * j + e] = -INFINITY;
              }
          }
      }
      // ---- softmax
      float lm[NR][2];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          lm[n][e] = fmaxf(s[n][0][e], s[n][0][2 + e]);
#pragma unroll
          for (int g = 1; g < SG; ++g) lm[n][e] = fmaxf(lm[n][e], fmaxf(s[n][g][e], s[n][g][2 + e]));
        }
      new_max(lm);
      uint32_t pb[NR][SG][2];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        // the difference first: s c2 - m c2 would be off by half a unit of m c2's last place, which
        // beyond 2^27 (keys hidden by large negative biases) no 16-bit weight survives
        const float2 m2 = make_float2(-safe(mrow[n][0]), -safe(mrow[n][1])), unit2 = make_float2(unit, unit);
#pragma unroll
        for (int g = 0; g < SG; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float2 x = __fadd2_rn(make_float2(s[n][g][2 * j], s[n][g][2 * j + 1]), m2);
            if (WIDE) x = __fmul2_rn(x, unit2);
            const float w0 = ex2(x.x), w1 = ex2(x.y);
            lrow[n][0] = WIDE ? lrow[n][0] + w0 : fmaf(w0, rsv[g][j], lrow[n][0]);
            lrow[n][1] = WIDE ? lrow[n][1] + w1 : fmaf(w1, rsv[g][j], lrow[n][1]);
            pb[n][g][j] = transpose8(DT<MT16>::pack(w0, w1));
          }
      }
      // ---- O^T += V^T P^T
      bool odd = false;                                 // a node's value element is not finite
#pragma unroll
      for (int g = 0; g < SG; ++g) {
        if (WIDE) {
          const int mi = lane >> 3, c = lane & 7;       // this lane's row address: slot c of matrix mi
          const int kr = ko + 16 * g + 4 * (c >> 1) + (c & 1) + 2 * (mi >> 1);
#pragma unroll
          for (int i = 0; i < MTD; ++i) {
            uint32_t a[4];
            ldsm_x4_t(sv + chunk_at<CPR, WIDE, true>(kr, 2 * i + (mi & 1)), a[0], a[1], a[2], a[3]);
            if (!EASY && k0 + ko + 16 * g + 16 > len) { // some of these 16 keys are nodes
              const int kn = k0 + ko + 16 * g + 4 * q4 - len;   // node of this lane's first key (a0, a1: +0, +1; a2, a3: +2, +3)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int first = kn + (x >= 2 ? 2 : 0);
                bool seen = false;
                const uint32_t clean = clean2<QT>(a[x], seen);
                // a cached key's element stays as it is
                if (seen && first + 1 >= 0) {
                  a[x] = first >= 0 ? clean : (clean & 0xffff0000u) | (a[x] & 0xffffu);
                  odd = true;
                }
              }
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(oacc[n][i], a, pb[n][g][0], pb[n][g][1]);
          }
        } else {
          // D / 8 consecutive columns of four consecutive keys
          uint32_t vw[4][D / 32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kr = ko + 16 * g + 4 * q4 + i;
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
          for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t a[4];
              expand4<FMT>(__byte_perm(vw[0][w], vw[1][w], c ? 0x7362 : 0x5140), a[0], a[1]);
              expand4<FMT>(__byte_perm(vw[2][w], vw[3][w], c ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
              for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(oacc[n][2 * w + c], a, pb[n][g][0], pb[n][g][1]);
            }
        }
      }
      if (WIDE && !EASY && __any_sync(0xffffffffu, odd)) add_non_finite(k0 + ko - len, k0 + ko + TL::SK - len);
    };

    Terms z_next;
    auto unsaturated = [&](int kf) { return p.z && kf + TL::SK - 1 - len > p.e_lo; };
    if (AHEAD && unsaturated(tile0 * TK + wn * KW)) terms_of(tile0 * TK + wn * KW, z_next);
#pragma unroll 1
    for (int tile = tile0; tile < tile1; ++tile) {
      cp_async_wait<TL::STAGES - 2>();
      group_sync();
      {
        int ns = stage + TL::STAGES - 1;
        if (ns >= TL::STAGES) ns -= TL::STAGES;
        load(ns, at_next);
        at_next = lookup(ld);
      }
      const uint32_t sk = stage0 + (uint32_t)stage * GSTAGE, sv = sk + HALF;
      const int k0 = tile * TK + wn * KW;
      const bool full = (full_stages >> stage) & 1u;
      if (!WIDE) {
        // value rows of zeros (scale 1, all codes 0) get their scale in the stage, once a tile (looking
        // in every step cost 1 to 2%); warps that share the keys write the same
#pragma unroll
        for (int i = 0; i < LR; ++i) {
          const int kl = 32 * i + lane;
          const uint32_t at = sk + 2 * HALF + (KW + kl) * 4;
          const bool unit = (KW % 32 == 0 || kl < KW) && __uint_as_float(lds32(at)) == 1.f;
          if (__any_sync(0xffffffffu, unit)) {
            if (unit) {
              uint32_t any = 0;
#pragma unroll 1
              for (int ch = 0; ch < CPR; ++ch) {
                const uint4 w = lds128(sv + chunk_at<CPR, WIDE, true>(kl, ch));
                any |= w.x | w.y | w.z | w.w;
              }
              if (FMT == RELPOS_CACHE_E4M3) any &= 0x7f7f7f7fu;   // -0 is a zero
              if (any == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(kZeroRowScale) : "memory");
            }
            __syncwarp();
          }
        }
      }
#pragma unroll 1
      for (int ko = 0; ko < KW; ko += TL::SK) {
        if (full && !unsaturated(k0 + ko)) {
          step(std::true_type{}, k0, ko, sk, sv, stage, true, z_next);
        } else if (k0 + ko < len + (WIDE ? p.T : 0)) {
          Terms z = z_next;
          if (p.z && (!AHEAD || !unsaturated(k0 + ko))) terms_of(k0 + ko, z);   // (a missing page among saturated keys)
          if (AHEAD) {
            const int kn = ko + TL::SK < KW ? k0 + ko + TL::SK : k0 + TK;
            if (unsaturated(kn)) terms_of(kn, z_next);
          }
          step(std::false_type{}, k0, ko, sk, sv, stage, full, z);
          continue;
        }
        if (AHEAD) {
          const int kn = ko + TL::SK < KW ? k0 + ko + TL::SK : k0 + TK;
          if (unsaturated(kn)) terms_of(kn, z_next);
        }
      }
      if (++stage == TL::STAGES) stage = 0;
    }

    // ---- 8-bit caches: the nodes' own keys, straight from their 16-bit tensors,
    // 16 nodes at a time; bf16 rows enter as fp16 times a power of two that
    // takes the place of the scale
    if (!WIDE && tile1 == nt) {
#pragma unroll 1
      for (int u0 = 16 * wn; u0 < p.T; u0 += 16 * WN) {
        float s[NR][4];
#pragma unroll
        for (int n = 0; n < NR; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        const uint16_t* kn = static_cast<const uint16_t*>(p.k) + b * p.ks.b + hkv * p.ks.h;
        const uint16_t* vn = static_cast<const uint16_t*>(p.v) + b * p.vs.b + hkv * p.vs.h;
        auto part = [&](const uint16_t* base, long long stride, int u, int d0) {
          return u < p.T ? __ldg(reinterpret_cast<const uint4*>(base + u * stride + d0)) : make_uint4(0, 0, 0, 0);
        };
        float down[2] = {1.f, 1.f}, ks[2] = {1.f, 1.f};
        if (DT<QT>::kCoarse) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t kt = 0;
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              const uint4 x = part(kn, p.ks.n, u0 + key0 + 2 * j, 64 * (w / 2) + 16 * q4 + 8 * (w % 2));
              kt = amax2(amax2(amax2(amax2(kt, x.x), x.y), x.z), x.w);
            }
            kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, 1));
            kt = max(kt, __shfl_xor_sync(0xffffffffu, kt, 2));
            const int e = exp_of(kt, -126);
            down[j] = pow2i(-e);
            ks[j] = pow2i(e);
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const int d0 = 64 * (w / 2) + 16 * q4 + 8 * (w % 2);
          const uint4 x0 = part(kn, p.ks.n, u0 + key0, d0), x1 = part(kn, p.ks.n, u0 + key0 + 2, d0);
          const uint32_t a0[4] = {to_half2<QT>(x0.x, down[0]), to_half2<QT>(x1.x, down[1]), to_half2<QT>(x0.y, down[0]),
                                  to_half2<QT>(x1.y, down[1])};
          const uint32_t a1[4] = {to_half2<QT>(x0.z, down[0]), to_half2<QT>(x1.z, down[1]), to_half2<QT>(x0.w, down[0]),
                                  to_half2<QT>(x1.w, down[1])};
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            MmaOp<MT16>::run(s[n], a0, qb[n][2 * w][0], qb[n][2 * w][1]);
            MmaOp<MT16>::run(s[n], a1, qb[n][2 * w + 1][0], qb[n][2 * w + 1][1]);
          }
        }
        // the power of value row 4 q + i; the scores' rows (slots r8, r8 + 8) take theirs from the lanes that have it
        float vdown[4] = {1.f, 1.f, 1.f, 1.f};
        int ve[4] = {0, 0, 0, 0};
        if (DT<QT>::kCoarse) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t vt = 0;
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              const uint4 x = part(vn, p.vs.n, u0 + 4 * q4 + i, r8 * (D / 8) + 8 * w);
              vt = amax2(amax2(amax2(amax2(vt, x.x), x.y), x.z), x.w);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) vt = max(vt, __shfl_xor_sync(0xffffffffu, vt, o));
            ve[i] = vt == 0 ? kZeroRowPower : exp_of(vt, -100);
            vdown[i] = pow2i(-ve[i]);
          }
        }
        float rv[2];
        float lm[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) lm[n][0] = lm[n][1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e0 = __shfl_sync(0xffffffffu, ve[2 * j], r8 >> 1), e1 = __shfl_sync(0xffffffffu, ve[2 * j + 1], r8 >> 1);
          const int ev = r8 & 1 ? e1 : e0;
          rv[j] = pow2i(-ev);
          const int u = u0 + key0 + 2 * j;
          const int du = u < p.T ? node_depth[u] : 0;
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float2 kc = unit_of(n);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = row_of(n, e);
              const unsigned long long mk = row_mask[r];
              float x = (float)ev;
              if (p.z) x += row_z[r][iclamp(du - row_depth[r], p.e_lo, p.e_hi) - p.e_lo];
              const bool keep = u < p.T && ((mk >> (u & 63)) & 1ull);
              float& y = s[n][2 * j + e];
              y = keep ? fmaf(y, ks[j] * (e ? kc.y : kc.x), x) : -INFINITY;
              lm[n][e] = fmaxf(lm[n][e], y);
            }
          }
        }
        new_max(lm);
        uint32_t pb[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const float m0 = safe(mrow[n][0]), m1 = safe(mrow[n][1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float w0 = ex2(s[n][2 * j] - m0), w1 = ex2(s[n][2 * j + 1] - m1);
            lrow[n][0] = fmaf(w0, rv[j], lrow[n][0]);
            lrow[n][1] = fmaf(w1, rv[j], lrow[n][1]);
            pb[n][j] = transpose8(DT<MT16>::pack(w0, w1));
          }
        }
        bool odd = false;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t vh[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = part(vn, p.vs.n, u0 + 4 * q4 + i, r8 * (D / 8) + 8 * w);
            vh[i][0] = clean2<__half>(to_half2<QT>(x.x, vdown[i]), odd);
            vh[i][1] = clean2<__half>(to_half2<QT>(x.y, vdown[i]), odd);
            vh[i][2] = clean2<__half>(to_half2<QT>(x.z, vdown[i]), odd);
            vh[i][3] = clean2<__half>(to_half2<QT>(x.w, vdown[i]), odd);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t a[4] = {__byte_perm(vh[0][x], vh[1][x], 0x5410), __byte_perm(vh[0][x], vh[1][x], 0x7632),
                                   __byte_perm(vh[2][x], vh[3][x], 0x5410), __byte_perm(vh[2][x], vh[3][x], 0x7632)};
#pragma unroll
            for (int n = 0; n < NR; ++n) MmaOp<MT16>::run(oacc[n][4 * w + x], a, pb[n][0], pb[n][1]);
          }
        }
        if (__any_sync(0xffffffffu, odd)) add_non_finite(u0, u0 + 16);
      }
    }

    advance(cp, tile1 - tile0);
    // the join may be made ready while the last results are written
    if (cp.at >= my_end) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- join the key groups of the block
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = lrow[n][e];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        const int r = (wm * NR + n) * 8 + 2 * q4 + e;
        if (r8 == 0) {
          sm_m[wn][r] = mrow[n][e];
          sm_l[wn][r] = l;
        }
      }
    __syncthreads();                                    // also: the last tile's stage has been read
    // Eight rows of each warp at a time, through the stage that was read last: the
    // loads in flight go to the others.  Rows are turned against each other by
    // eight columns, which keeps the writes of a quad apart.
    const int freed = stage == 0 ? TL::STAGES - 1 : stage - 1;
    auto joined = [&](int w, int m) {                   // [8][D] of warp (m, w)
      return reinterpret_cast<float*>(smem + pre_bytes + (w * TL::STAGES + freed) * GSTAGE) + m * 8 * D;
    };
    const bool whole = tile0 == 0 && tile1 == nt;
    float* slot = p.part + ((long long)blockIdx.x * 2 + (first_item ? 0 : 1)) * slot_floats(ROWS, D);
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float* dst = joined(wn, wm);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row_of(n, e);
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = fmaxf(m, sm_m[w][r]);
        const float f = ex2((mrow[n][e] - safe(m)) * unit);
#pragma unroll
        for (int i = 0; i < MTD; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int d = WIDE ? 16 * i + 8 * c + r8 : r8 * (D / 8) + 2 * i + c;
            dst[(2 * q4 + e) * D + ((d + 8 * q4) & (D - 1))] = oacc[n][i][2 * c + e] * f;
          }
      }
      __syncthreads();
      for (int i = tid; i < WM * 8 * (D / 4); i += 128) {
        const int x = i / (D / 4), c = i % (D / 4), m8 = x >> 3;
        const int r = (m8 * NR + n) * 8 + (x & 7), gr = rb * ROWS + r;
        if (gr >= R) continue;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = fmaxf(m, sm_m[w][r]);
#pragma unroll
        for (int w = 0; w < WN; ++w) l += sm_l[w][r] * ex2((sm_m[w][r] - safe(m)) * unit);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WN; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(joined(w, m8) + (x & 7) * D +
                                                            ((4 * c + 8 * ((x & 7) >> 1)) & (D - 1)));
          o.x += y.x; o.y += y.y; o.z += y.z; o.w += y.w;
        }
        if (!whole) {
          *reinterpret_cast<float4*>(slot + (long long)r * D + 4 * c) = o;
          if (c == 0) {
            slot[ROWS * D + r] = m;
            slot[ROWS * D + ROWS + r] = l;
          }
        } else {
          store_row(p, b, hkv, gr, c, o, m * unit, l);
        }
      }
      __syncthreads();                                  // the stage (at the end: rows and sums, too) is free again
    }
  }
}

template <class TL, int FMT>
constexpr int stage_bytes() {
  constexpr bool wide = FMT == RELPOS_CACHE_F16;
  return TL::WN * TL::STAGES * (2 * TL::KW * TL::D * (wide ? 2 : 1) + (wide ? 0 : TL::KW * 8));
}

// Launches `threads` to a block; `early`: they may start while the kernel before
// them on the stream, which is this library's, still runs (they wait for it
// themselves before they use its results).
template <typename F, typename... A>
cudaError_t launch_after(F* f, int threads, dim3 grid, size_t smem, cudaStream_t s, bool early, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, f, args...);
}

template <class TL, typename QT, int FMT>
cudaError_t run_tiling(const TreeParams& p, cudaStream_t s) {
  // BPS blocks to an SM of 227 KB: the stages, 4 KB of rows, sums and reserve, and a short list of sequences
  static_assert(TL::BPS * (stage_bytes<TL, FMT>() + 4096 + 1024) <= 227 * 1024, "the blocks of a launch do not fit at once");
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
  note_launch(1);
  return launch_after(tree_kernel<TL, QT, FMT>, 128, dim3(p.grid), smem, s, p.z != nullptr, p);
}

// Tilings by head dimension and row count.  Up to 32 rows (16 at d = 128, where
// the outputs take twice the registers) four warps take different keys; beyond
// that warps share keys and take different rows.  Stages are sized for BPS blocks
// to an SM with some 100 KB of loads in flight.  A step of 32 keys in place of 16
// halves the votes and loop code of a step: int8, d = 64, 16 rows 41.7 to 35.1 us (at three
// blocks to an SM in place of four, for the registers), 32 rows 72 to 66; int8, d = 128, 8
// rows 115 to 106; 16-bit caches at d = 128 have no registers for it.  Two warps to 16 rows
// each beat one with 32 (72 to 66 us: the wider warp spills).  What still spills: 16 rows at d =
// 128 over 8 bits (132 bytes of stores, 220 to 248 with bf16 queries, whose look-ups of
// factors come on top), 64 rows there 80 to 84.
template <int D, bool WIDE> struct Tilings;
template <bool WIDE> struct Tilings<64, WIDE> {
  using R8 = Tiling<64, 1, 4, 1, 32, 32, WIDE ? 2 : 3, WIDE ? 3 : 4>;
  using R16 = Tiling<64, 1, 4, 2, WIDE ? 16 : 32, WIDE ? 16 : 32, 3, 3>;
  using R32 = Tiling<64, 2, 2, 2, 32, WIDE ? 16 : 32, 3, 3>;
  using R64 = Tiling<64, 4, 1, 2, 64, 32, 3, 3>;
};
template <bool WIDE> struct Tilings<128, WIDE> {
  using R8 = Tiling<128, 1, 4, 1, WIDE ? 16 : 32, WIDE ? 16 : 32, WIDE ? 3 : 2, WIDE ? 2 : 3>;
  using R16 = Tiling<128, 1, 4, 2, 16, 16, 3, WIDE ? 2 : 3>;
  using R32 = Tiling<128, 2, 2, 2, 32, 16, 3, 2>;
  using R64 = Tiling<128, 4, 1, 2, 64, 32, 3, 2>;
};

template <typename QT, int FMT, class T>
cudaError_t run_rows(const TreeParams& p, cudaStream_t s) {
  switch (p.rows_per_block) {
    case 8: return run_tiling<typename T::R8, QT, FMT>(p, s);
    case 16: return run_tiling<typename T::R16, QT, FMT>(p, s);
    case 32: return run_tiling<typename T::R32, QT, FMT>(p, s);
    default: return run_tiling<typename T::R64, QT, FMT>(p, s);
  }
}

template <typename QT, int FMT>
cudaError_t run_format(const TreeParams& p, cudaStream_t s) {
  constexpr bool wide = FMT == RELPOS_CACHE_F16;
  return p.c.d == 64 ? run_rows<QT, FMT, Tilings<64, wide>>(p, s) : run_rows<QT, FMT, Tilings<128, wide>>(p, s);
}

cudaError_t run_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_bf16(const TreeParams& p, cudaStream_t s);
cudaError_t run_e4m3_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_e4m3_bf16(const TreeParams& p, cudaStream_t s);
cudaError_t run_int8_f16(const TreeParams& p, cudaStream_t s);
cudaError_t run_int8_bf16(const TreeParams& p, cudaStream_t s);
bool takes_wide(const TreeParams& p);   // of a call with a 16-bit cache
cudaError_t launch_wide(const TreeParams& p, cudaStream_t s);

}  // namespace tree
}  // namespace relpos
