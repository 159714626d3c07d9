// tree_attn.cu -- the kernels around the tree attention (tree_attn.cuh): the
// relation terms of the drafted queries, and the join of split items.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
namespace {

// A finite term is bounded so that tau log2 e times it is finite, too: a table may hide keys
// with the lowest number of its type, and no maximum can be subtracted from -inf.  The
// many-row kernel's exponents are s c2 - m with m = s c2 rounded, off by half a unit of m's
// last place: its terms end at 1.5 x 2^27 in base 2, where fp16 weights are still within 2^8
// of their own (bf16: 1.5 x 2^30, 2^64).  An infinite term stays.
__device__ __forceinline__ float term(const TreeParams& p, float x) {
  if (fabsf(x) <= 3.4028235e38f) x = fminf(fmaxf(x, -p.z_limit), p.z_limit);
  return x * p.z_scale;
}

// z[b, h, t, e] = z_scale (q . aQ[phi(e_lo + e)] + b[phi(e_lo + e)]): one MMA
// product of a head's B T query rows with the table rows of the reachable
// offsets.  A warp keeps 16 table rows in registers and walks over the rows
// of queries, so the table is read once; z is written in fp32.  Offsets that no
// row of 16 can reach (they lie before position 0) are left out.
// BUCKETS: the map takes logarithms; the others' code is short, and at this length
// of kernel what the instruction caches must fetch shows.
template <bool BUCKETS>
__device__ __forceinline__ int row_at(const TreeParams& p, int delta) {
  const int r = BUCKETS ? phi_of(p.map, p.N, delta)
                        : p.map.kind == RELPOS_MAP_TRUNCATED ? iclamp(delta, -p.map.clip, p.map.clip) + p.map.clip : delta + p.N - 1;
  return iclamp(r, 0, p.R - 1);
}
template <int D, typename QT, bool BUCKETS>
__global__ void __launch_bounds__(128) relation_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, q4 = lane & 3, r8 = lane >> 2;
  const int c0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 16;
  const int W = p.e_hi - p.e_lo + 1;
  if (c0 >= W) return;
  const int h = blockIdx.y;
  uint4 bw[2][D / 32];
  int rows[2];                         // table rows of columns r8 and 8 + r8
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    rows[j] = row_at<BUCKETS>(p, p.e_lo + min(c0 + 8 * j + r8, W - 1));
    const uint16_t* src = static_cast<const uint16_t*>(p.aq) + h * p.aq_hs + (long long)rows[j] * D;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) bw[j][u] = __ldg(reinterpret_cast<const uint4*>(src + 32 * u + 8 * q4));
  }
  float bias[2][2] = {};
  if (p.bias) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = __shfl_sync(0xffffffffu, rows[j], 4 * (2 * q4 + c));   // the row of this lane's column
        bias[j][c] = p.bias[(long long)h * p.R + r];
      }
  }
  const int n = p.B * p.T;
  for (int r0 = blockIdx.z * 16; r0 < n; r0 += gridDim.z * 16) {
    int rr[2], bb[2], tt[2];
    bool need = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      rr[e] = r0 + r8 + 8 * e;
      const int r = min(rr[e], n - 1);
      bb[e] = r / p.T;
      tt[e] = r - bb[e] * p.T;
      need = need || p.e_lo + c0 + 15 >= -(seq_len(p, bb[e]) + p.T);
    }
    if (!__any_sync(0xffffffffu, need)) continue;
    float acc[2][4] = {};
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      uint4 w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + bb[e] * p.qs.b + h * p.qs.h +
                                                    tt[e] * p.qs.n + 32 * u + 8 * q4));
      const uint32_t a0[4] = {w[0].x, w[1].x, w[0].y, w[1].y}, a1[4] = {w[0].z, w[1].z, w[0].w, w[1].w};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        MmaOp<QT>::run(acc[j], a0, bw[j][u].x, bw[j][u].y);
        MmaOp<QT>::run(acc[j], a1, bw[j][u].z, bw[j][u].w);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (rr[e] >= n) continue;
      float* dst = p.z + bb[e] * p.z_b + h * p.z_h + tt[e] * p.z_t + c0 + 2 * q4;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (c0 + 8 * j + 2 * q4 < W)   // rows are padded to whole column tiles
          *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(term(p, acc[j][2 * e] + bias[j][0]), term(p, acc[j][2 * e + 1] + bias[j][1]));
    }
  }
}

// The bias alone: one row of offsets a head, shared by sequences and nodes.
__global__ void __launch_bounds__(128) bias_kernel(const __grid_constant__ TreeParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int e = blockIdx.x * 128 + threadIdx.x, h = blockIdx.y;
  if (e > p.e_hi - p.e_lo) return;
  const int r = iclamp(phi_of(p.map, p.N, p.e_lo + e), 0, p.R - 1);
  p.z[h * p.z_h + e] = term(p, p.bias[(long long)h * p.R + r]);
}

// Joins the partial results of an item that was cut: pieces c0 .. c1 of the
// line hold it, the first in the piece's last slot (unless the item begins the
// piece), the others in their first.  Summed in the order of the pieces.
// Block x looks at the border between pieces x and x + 1: it joins the item cut
// there, if that is the item's first cut.  A group of D / 4 lanes takes a row, each
// lane four columns; the weights of as many pieces are found at once, one to a lane.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const __grid_constant__ TreeParams p, int tk, int wide) {
  constexpr int GL = D / 4, RPB = 128 / GL;
  extern __shared__ int pre[];
  __shared__ int warp_sums[4];
  const int ROWS = p.rows_per_block, tid = threadIdx.x, c = tid % GL;
  build_line<128>(p, tk, wide != 0, pre, warp_sums);
  Line line;
  line.pre = pre;
  line.B = p.B;
  line.items = p.c.Hkv * p.row_blocks;
  line.total = pre[p.B] * line.items;
  line.quantum = (line.total + p.grid - 1) / p.grid;
  const int at = line.quantum * (int)(blockIdx.x + 1);
  const int b = line.seq_of(min(at, line.total - 1));
  const int nt = pre[b + 1] - pre[b];
  const int in_b = at - pre[b] * line.items, item = in_b / nt, tile = in_b - item * nt;
  const int start = at - tile, before = line.quantum * blockIdx.x;
  // base-2 units of the maxima: the narrow kernel's scores over a 16-bit cache are without tau log2 e
  const float unit = wide && ROWS != 256 ? p.c2 : 1.f;
  const bool mine = at < line.total && tile > 0 && start >= before;
  const int c0 = blockIdx.x, c1 = (start + nt - 1) / line.quantum;
  const int hkv = item / p.row_blocks, rb = item - hkv * p.row_blocks;
  const int n = min(ROWS, p.G * p.T - rb * ROWS);
  // every block waits, the idle ones too: what follows this kernel on the stream
  // must not start before the attention has ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the narrow kernel has no waits to run out; the wide one's word was cleared before it
  if (ROWS != 256 && blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.status = 0;
  if (!mine) return;
  const long long sf = slot_floats(ROWS, D);
  const float* first = p.part + (2LL * c0 + (start > before ? 1 : 0)) * sf;
  auto slot = [&](int k) { return k == c0 ? first : p.part + 2LL * k * sf; };
  for (int r0 = blockIdx.y * RPB; r0 < n; r0 += gridDim.y * RPB) {
    const int r = min(r0 + tid / GL, n - 1);             // lanes past the end repeat the last row
    // all loads of an item in up to four pieces are under way before the first is used
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c0 + i <= c1) x[i] = *reinterpret_cast<const float4*>(slot(c0 + i) + (long long)r * D + 4 * c);
    float mk = -INFINITY, lk = 0.f;
    if (c0 + c <= c1) {
      mk = slot(c0 + c)[ROWS * D + r];
      lk = slot(c0 + c)[ROWS * D + ROWS + r];
    }
    float m = mk;
    for (int k = c0 + c + GL; k <= c1; k += GL) m = fmaxf(m, slot(k)[ROWS * D + r]);
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float f, const float4& y) {
      o.x = fmaf(y.x, f, o.x); o.y = fmaf(y.y, f, o.y); o.z = fmaf(y.z, f, o.z); o.w = fmaf(y.w, f, o.w);
    };
    for (int k0 = c0; k0 <= c1; k0 += GL) {
      if (k0 > c0) {
        mk = -INFINITY;
        lk = 0.f;
        if (k0 + c <= c1) {
          mk = slot(k0 + c)[ROWS * D + r];
          lk = slot(k0 + c)[ROWS * D + ROWS + r];
        }
      }
      const float f = ex2((mk - safe(m)) * unit);
      float lf = lk * f;
#pragma unroll
      for (int q = 1; q < GL; q <<= 1) lf += __shfl_xor_sync(0xffffffffu, lf, q);
      l += lf;
      const int nk = min(GL, c1 - k0 + 1);
      int i = 0;
      if (k0 == c0) {
#pragma unroll
        for (; i < 4; ++i) {
          const float fi = __shfl_sync(0xffffffffu, f, i, GL);
          if (c0 + i <= c1) add(fi, x[i]);
        }
      }
#pragma unroll 4
      for (; i < nk; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i, GL);
        add(fi, *reinterpret_cast<const float4*>(slot(k0 + i) + (long long)r * D + 4 * c));
      }
    }
    if (r0 + tid / GL < n) store_row(p, b, hkv, rb * ROWS + r, c, o, m * unit, l);
  }
}

// Keys to a tile and blocks to an SM of the tiling a call takes.
struct Shape {
  int tk, bps;
};
template <class T>
Shape shape_rows(int rows_per_block) {
  switch (rows_per_block) {
    case 8: return {T::R8::TK, T::R8::BPS};
    case 16: return {T::R16::TK, T::R16::BPS};
    case 32: return {T::R32::TK, T::R32::BPS};
    default: return {T::R64::TK, T::R64::BPS};
  }
}
bool wide_cache(const TreeParams& p) {
  return p.c.format == RELPOS_CACHE_F16 || p.c.format == RELPOS_CACHE_BF16;
}
Shape shape_of(const TreeParams& p) {
  if (p.rows_per_block == 256) return {128, 1};
  if (p.c.d == 64)
    return wide_cache(p) ? shape_rows<Tilings<64, true>>(p.rows_per_block) : shape_rows<Tilings<64, false>>(p.rows_per_block);
  return wide_cache(p) ? shape_rows<Tilings<128, true>>(p.rows_per_block) : shape_rows<Tilings<128, false>>(p.rows_per_block);
}

}  // namespace
}  // namespace tree

using namespace tree;

int tree_rows_per_block(const TreeParams& p) {
  if (wide_cache(p) && takes_wide(p)) return 256;
  const int rows = p.G * p.T;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// One piece of the line of tiles to each block that can be resident; fewer
// where there are fewer tiles.
int tree_grid(const TreeParams& p) {
  const Shape sh = shape_of(p);
  const long long most = (((long long)p.P << p.c.page_shift) + p.T + sh.tk - 1) / sh.tk + 1;
  const long long tiles = most * p.B * p.c.Hkv * p.row_blocks;
  return (int)(tiles < 148LL * sh.bps ? tiles : 148LL * sh.bps);
}

cudaError_t launch_tree_relation(const TreeParams& p, cudaStream_t s) {
  const int W = p.e_hi - p.e_lo + 1;
  if (!p.aq) {
    bias_kernel<<<dim3((W + 127) / 128, p.H), 128, 0, s>>>(p);
  } else {
    const int row_tiles = (p.B * p.T + 15) / 16, cols = (W + 63) / 64;
    // walk the query rows in one block where the columns alone fill the card
    int gz = (int)(148LL * 32 / ((long long)cols * p.H)) + 1;
    gz = gz < row_tiles ? gz : row_tiles;
    const dim3 grid(cols, p.H, gz);
    const bool buckets = p.map.kind != RELPOS_MAP_TRUNCATED && p.map.kind != RELPOS_MAP_IDENTITY;
    void (*f)(TreeParams) =
        p.c.d == 64
            ? (p.bf16 ? (buckets ? relation_kernel<64, __nv_bfloat16, true> : relation_kernel<64, __nv_bfloat16, false>)
                      : (buckets ? relation_kernel<64, __half, true> : relation_kernel<64, __half, false>))
            : (p.bf16 ? (buckets ? relation_kernel<128, __nv_bfloat16, true> : relation_kernel<128, __nv_bfloat16, false>)
                      : (buckets ? relation_kernel<128, __half, true> : relation_kernel<128, __half, false>));
    f<<<grid, 128, 0, s>>>(p);
  }
  note_launch(1);
  return cudaGetLastError();
}

cudaError_t launch_tree_attention(const TreeParams& p, cudaStream_t s) {
  if (p.rows_per_block == 256) return launch_wide(p, s);
  switch (p.c.format) {
    case RELPOS_CACHE_F16: return run_f16(p, s);
    case RELPOS_CACHE_BF16: return run_bf16(p, s);
    case RELPOS_CACHE_E4M3: return p.bf16 ? run_e4m3_bf16(p, s) : run_e4m3_f16(p, s);
    default: return p.bf16 ? run_int8_bf16(p, s) : run_int8_f16(p, s);
  }
}

cudaError_t launch_tree_combine(const TreeParams& p, cudaStream_t s) {
  // a block to each border of pieces and (for the wide kernel's 256 rows, every
  // second) group of rows
  const int groups = p.rows_per_block * p.c.d / 512;
  const dim3 grid(p.grid > 1 ? p.grid - 1 : 1, groups > 32 ? groups / 2 : groups);
  note_launch(1);
  const int tk = shape_of(p).tk, wide = wide_cache(p);
  return launch_after(p.c.d == 64 ? combine_kernel<64> : combine_kernel<128>, 128, grid, (p.B + 1) * sizeof(int), s, true, p, tk, wide);
}

}  // namespace relpos
