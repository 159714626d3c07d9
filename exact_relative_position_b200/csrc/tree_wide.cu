// tree_wide.cu -- tree attention for many rows to a key head (more than 64) over
// a 16-bit cache, on tcgen05.
//
// The computation and the line of tiles are those of tree_attn.cuh; here an item
// is 256 query rows (two tiles of 128) of one key head, so that each K/V tile
// feeds four 128-row MMAs and the work per byte is that of a dense attention
// layer: the tensor and exponential units bound it, not memory.  16 trees of 61 nodes
// over up to 8192 keys, 32 / 8 heads of 128: 169 us, 495 TFLOP/s; a tile of keys takes 2.6 us
// where the tensor unit's share is 1.2: the softmax warpgroups and the MMAs wait for
// one another's hand-overs.  A softmax thread holds a row's 128 scores: 108 bytes spill at d =
// 128, 128 at d = 64.
//
// Warp roles of a block (one to an SM, walking its piece of the line):
//   warp 0        MMA issuer (one thread); allocates the tensor memory
//   warps 1..3    loaders: the item's queries, then K and V tiles in turn, a warp
//                 to a tile, into a ring of tiles.  A tile whose pages all exist
//                 comes by TMA, a box to a page (of at least 8 rows); one with
//                 smaller or missing pages, or with the nodes behind the cache, is
//                 gathered with cp.async into the same 128-byte-swizzled layout
//                 and handed over with a proxy fence, rows that do not exist as zeros.
//   warps 4..7    softmax of rows 0..127 (thread r owns row r = TMEM lane r)
//   warps 8..11   softmax of rows 128..255
// Tensor memory: S0 columns [0, 128), S1 [128, 256), O0 [256, 256 + D), O1 [384,
// 384 + D).  A row's 16-bit weights P replace the first half of its scores.  The
// tensor pipe runs in issue order, PV_g(t) then QK_g(t + 1), so the scores of a
// tile being there implies that the tile before has left O and P alone; the two
// row tiles alternate between the tensor and the exponential units.
#include <cudaTypedefs.h>

#include "sm100.cuh"
#include "tree_attn.cuh"

namespace relpos {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();   // attn_fwd.cu

namespace tree {
namespace {

using namespace sm100;

constexpr int kKeys = 128;              // keys of a tile
constexpr int kThreads = 384;
constexpr float kSlack = 8.f;           // log2 of the largest weight before O is rescaled
constexpr int kTileRing = 8;            // tiles whose row masks are kept

template <int D> struct Wide {
  static constexpr uint32_t kTile = 128 * D * 2;             // a K, V or Q tile
  static constexpr int kUnits = D == 128 ? 5 : 8;            // ring of K and V tiles
  static constexpr uint32_t kOffQ = 0, kOffKV = 2 * kTile, kOffEnd = kOffKV + kUnits * kTile;
};
// barriers
constexpr int kBarQFull = 0, kBarQFree = 1, kBarSFull = 2, kBarPReady = 4, kBarOFull = 6, kBarFull = 8, kBarEmpty = 16,
              kBarDrain = 24, kBars = 25;

struct WideShared {
  uint64_t bar[kBars];
  uint32_t valid[kTileRing][4];
  int odd[4];                           // number + 1 of the part whose nodes hold non-finite values, by its last two bits
  int depth[2][64];
  int abort;
  uint32_t tmem;
  int warp_sums[kThreads / 32];
};

// Dynamic shared memory of a block, and the most that one can have beside the static part
// (and 64 bytes of reserve): the ring of tiles, a kilobyte to align it, the list of sequences.
// 255 sequences fit at d = 128, thousands at d = 64.
constexpr int kDynamicMost = 227 * 1024 - (int)sizeof(WideShared) - 64;
template <int D> constexpr int dynamic_bytes(int B) { return (int)Wide<D>::kOffEnd + 1024 + (((B + 1) * 4 + 127) & ~127); }
static_assert(dynamic_bytes<128>(1) <= kDynamicMost && dynamic_bytes<64>(4096) <= kDynamicMost, "the tiles of a block do not fit");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tma_rows_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(col), "r"(row)
      : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// One 16-bit row chunk as the swizzled operand layout has it: 64-column halves of
// 128 rows x 128 bytes, chunk c of row r at (c ^ r % 8).
__device__ __forceinline__ uint32_t wide_at(int r, int ch) {
  return (uint32_t)((ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <int D, typename QT>
__global__ void __launch_bounds__(kThreads, 1) tree_wide_kernel(const __grid_constant__ TreeParams p,
                                                                const __grid_constant__ CUtensorMap tm_k,
                                                                const __grid_constant__ CUtensorMap tm_v, int box) {
  using W = Wide<D>;
  constexpr int CPR = D / 8;                           // 16-byte chunks of a row
  extern __shared__ uint8_t smem_raw[];
  __shared__ WideShared sh;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  int* pre = reinterpret_cast<int*>(smem_raw + (sb - raw) + W::kOffEnd);
  volatile int* abort_flag = &sh.abort;
  auto bar = [&](int i) { return smem_u32(&sh.bar[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(bar(kBarQFull), 3);
    mbar_init(bar(kBarQFree), 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(bar(kBarSFull + g), 1);
      mbar_init(bar(kBarPReady + g), 128);
      mbar_init(bar(kBarOFull + g), 1);
    }
    for (int u = 0; u < W::kUnits; ++u) {
      mbar_init(bar(kBarFull + u), 1);
      mbar_init(bar(kBarEmpty + u), 1);
    }
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < 4; ++i) sh.odd[i] = 0;
    sh.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  build_line<kThreads>(p, kKeys, true, pre, sh.warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  Line line;
  line.pre = pre;
  line.B = p.B;
  line.items = p.c.Hkv * p.row_blocks;
  line.total = pre[p.B] * line.items;
  line.quantum = (line.total + gridDim.x - 1) / gridDim.x;
  const int my_start = line.quantum * blockIdx.x;
  const int my_end = min(line.total, my_start + line.quantum);
  const int R = p.G * p.T;

  // the piece's part of one item: tiles [t0, t1) of nt
  struct Seg {
    int b, hkv, rb, nt, t0, t1, len, groups;
  };
  auto segment = [&](int at) {
    Seg s;
    s.b = line.seq_of(at);
    s.nt = pre[s.b + 1] - pre[s.b];
    const int in_b = at - pre[s.b] * line.items, item = in_b / s.nt;
    s.t0 = in_b - item * s.nt;
    s.t1 = min(s.nt, s.t0 + (my_end - at));
    s.hkv = item / p.row_blocks;
    s.rb = item - s.hkv * p.row_blocks;
    s.len = seq_len(p, s.b);
    s.groups = R - s.rb * 256 > 128 ? 2 : 1;
    return s;
  };
  const uint64_t limit = p.wait_ns;

  // Register split: the launch gives 168 to each of 384 threads (64512); the first
  // warpgroup drops to 88 and the softmax warpgroups take 208: 128 x 88 + 256 x 208 = 64512.
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------ MMA issuer
        constexpr bool bf = DT<QT>::kCoarse;
        const uint32_t id_qk = idesc_f16(bf, 128, 128, false, false), id_pv = idesc_f16(bf, 128, D, false, true);
        const uint64_t dq = sdesc_sw128(sb + W::kOffQ, 16, 1024);
        const uint64_t dk = sdesc_sw128(sb + W::kOffKV, 16, 1024);
        const uint64_t dv = sdesc_sw128(sb + W::kOffKV, 16384, 1024);   // 64-column halves 16 KB apart
        constexpr uint64_t kTile16 = W::kTile >> 4;
        auto issue_qk = [&](int g, int slot) {
          const uint64_t a = dq + g * kTile16, k = dk + slot * kTile16;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk >> 2) * 1024 + (kk & 3) * 2);   // 16 KB halves, 32-byte steps
            mma_ss(tmem + g * 128, a + off, k + off, id_qk, kk > 0);
          }
        };
        auto issue_pv = [&](int g, int slot, bool acc) {
          const uint64_t v = dv + slot * kTile16;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ts(tmem + 256 + g * 128, tmem + g * 128 + 8 * kk, v + 128 * kk, id_pv, (acc || kk > 0) ? 1u : 0u);
        };
        uint32_t unit = 0, seg_no = 0, np[2] = {0, 0};
        auto full = [&](uint32_t u) { return mbar_wait(bar(kBarFull + u % W::kUnits), (u / W::kUnits) & 1, abort_flag, limit); };
        bool ok = true;
        for (int at = my_start; at < my_end && ok; ++seg_no) {
          const Seg s = segment(at);
          const int n = s.t1 - s.t0;
          ok = mbar_wait(bar(kBarQFull), seg_no & 1, abort_flag, limit) && full(unit);
          if (!ok) break;
          tc_fence_after();
          for (int g = 0; g < s.groups; ++g) {
            issue_qk(g, unit % W::kUnits);
            mma_commit(bar(kBarSFull + g));
          }
          mma_commit(bar(kBarEmpty + unit % W::kUnits));
          if (n == 1) mma_commit(bar(kBarQFree));
#pragma unroll 1
          for (int t = 0; t < n && ok; ++t) {
            const uint32_t uv = unit + 1, uk = unit + 2;
            const bool more = t + 1 < n;
            ok = full(uv) && (!more || full(uk));
            for (int g = 0; g < s.groups && ok; ++g) {
              ok = mbar_wait(bar(kBarPReady + g), np[g]++ & 1, abort_flag, limit);
              if (!ok) break;
              tc_fence_after();
              issue_pv(g, uv % W::kUnits, t > 0);
              if (more) {
                issue_qk(g, uk % W::kUnits);
                mma_commit(bar(kBarSFull + g));
              } else {
                mma_commit(bar(kBarOFull + g));
              }
            }
            if (!ok) break;
            mma_commit(bar(kBarEmpty + uv % W::kUnits));
            if (more) mma_commit(bar(kBarEmpty + uk % W::kUnits));
            if (more && t + 2 == n) mma_commit(bar(kBarQFree));
            unit += 2;
          }
          at += n;
        }
        // every MMA issued is done before the tensor memory is freed, whoever gave up
        mma_commit(bar(kBarDrain));
        mbar_drain(bar(kBarDrain), 0);
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------- loaders
      const int lw = warp - 1;
      uint32_t unit = 0, tile_no = 0, seg_no = 0;
      const int nb = box ? kKeys / box : 0;              // boxes of a tile (0: pages too small)
      int last = -1;                                     // this warp's last tile by TMA
      int pending = -1;                                  // ring slot of the loads that have not been handed over
      auto publish = [&]() {
        if (pending < 0) return;
        asm volatile("cp.async.wait_all;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarFull + pending));
        pending = -1;
      };
      // warp-uniform wait; what is in flight is handed over before it may block
      auto wait = [&](int i, uint32_t parity) {
        bool got = mbar_test(bar(i), parity);           // try_wait may sleep on what is in flight here
        if (__all_sync(0xffffffffu, got)) return true;
        publish();
        got = mbar_wait(bar(i), parity, abort_flag, limit);
        return (bool)__all_sync(0xffffffffu, got);
      };
      bool ok = true;
      for (int at = my_start; at < my_end && ok; ++seg_no) {
        const Seg s = segment(at);
        // ---- queries, 32 rows to a warp in turn, once the first tiles are under way
        auto load_q = [&]() {
          if (seg_no > 0) ok = wait(kBarQFree, (seg_no - 1) & 1);
          if (!ok) return;
          publish();
          const uint16_t* q = static_cast<const uint16_t*>(p.q) + s.b * p.qs.b;
#pragma unroll 1
          for (int i = lw; i < s.groups * 4; i += 3) {
            const int gr = s.rb * 256 + i * 32 + lane, t = gr < R ? gr / p.G : 0;
            const int h = s.hkv * p.G + (gr < R ? gr - t * p.G : 0), ch = lane % CPR;
            const long long off = gr < R ? h * p.qs.h + (long long)t * p.qs.n : -1;
#pragma unroll 4
            for (int x = 0; x < 32; x += 32 / CPR) {
              const int rl = x + lane / CPR, r = i * 32 + rl;
              const long long at_r = __shfl_sync(0xffffffffu, off, rl);
              cp_async16(sb + W::kOffQ + (r >> 7) * W::kTile + wide_at(r & 127, ch), q + (at_r < 0 ? 0 : at_r) + ch * 8,
                         at_r < 0 ? 0 : 16);
            }
          }
          asm volatile("cp.async.wait_all;" ::: "memory");
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarQFull));
        };
        // ---- K and V tiles
        const int* table = p.page_table + (long long)s.b * p.P;
#pragma unroll 1
        for (int t = s.t0; t < s.t1 && ok; ++t, ++tile_no) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++unit) {
            if ((int)(unit % 3) != lw) continue;
            const int slot = (int)(unit % W::kUnits);
            const int k0 = t * kKeys;
            const uint32_t dst = sb + W::kOffKV + (uint32_t)slot * W::kTile;
            if (nb && k0 + kKeys <= s.len) {
              // lane i has box i, if its page exists
              int id = 0;
              if (lane < nb) id = __ldg(table + ((k0 + lane * box) >> p.c.page_shift));
              if (__all_sync(0xffffffffu, id >= 0 && id < p.c.num_pages)) {
                if (unit >= (uint32_t)W::kUnits) {
                  ok = wait(kBarEmpty + slot, (unit / W::kUnits - 1) & 1);
                  if (!ok) break;
                }
                publish();
                if (lane == 0) {
                  if (kv == 0)
                    for (int i = 0; i < 4; ++i) sh.valid[tile_no % kTileRing][i] = 0xffffffffu;
                  mbar_expect_tx(bar(kBarFull + slot), W::kTile);
                }
                __syncwarp();
                if (lane < nb) {
                  const int at = ((id * p.c.Hkv + s.hkv) << p.c.page_shift) +
                                 ((k0 + lane * box) & ((1 << p.c.page_shift) - 1));
                  const CUtensorMap* map = kv ? &tm_v : &tm_k;
#pragma unroll
                  for (int h = 0; h < D / 64; ++h)
                    tma_rows_load(dst + h * 16384 + lane * box * 128, map, bar(kBarFull + slot), h * 64, at);
                }
                last = (int)unit;
                continue;
              }
            }
            uint32_t row[4];                             // row of the cache of key 32 i + lane; all ones: none
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int j = k0 + 32 * i + lane;
              row[i] = 0xffffffffu;
              if (j < s.len) {
                const int id = __ldg(table + (j >> p.c.page_shift));
                if (id >= 0 && id < p.c.num_pages)
                  row[i] = (((uint32_t)id * (uint32_t)p.c.Hkv + (uint32_t)s.hkv) << p.c.page_shift) +
                           (uint32_t)(j & ((1 << p.c.page_shift) - 1));
              }
            }
            if (unit >= (uint32_t)W::kUnits) {
              ok = wait(kBarEmpty + slot, (unit / W::kUnits - 1) & 1);
              if (!ok) break;
            }
            if (kv == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = k0 + 32 * i + lane;
                const uint32_t bits = __ballot_sync(0xffffffffu, row[i] != 0xffffffffu || (j >= s.len && j < s.len + p.T));
                if (lane == 0) sh.valid[tile_no % kTileRing][i] = bits;
              }
              __threadfence_block();
            }
            publish();                                   // the tile before
            const uint8_t* base = static_cast<const uint8_t*>(kv ? p.c.v : p.c.k);
            const Strides& st = kv ? p.vs : p.ks;
            const uint16_t* nodes = static_cast<const uint16_t*>(kv ? p.v : p.k) + s.b * st.b + s.hkv * st.h;
            const int ch = lane % CPR;
            const bool all = __all_sync(0xffffffffu, row[0] != 0xffffffffu && row[1] != 0xffffffffu &&
                                                         row[2] != 0xffffffffu && row[3] != 0xffffffffu);
            // loops stay rolled: the block's warps run different code, and what does
            // not fit the instruction caches costs more than the loads
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const uint32_t mine = i == 0 ? row[0] : i == 1 ? row[1] : i == 2 ? row[2] : row[3];
              if (all) {
                const uint8_t* src = base + ch * 16;
#pragma unroll 8
                for (int x = 0; x < 32; x += 32 / CPR) {
                  const int rl = x + lane / CPR;
                  const uint32_t at_r = __shfl_sync(0xffffffffu, mine, rl);
                  cp_async16(dst + wide_at(32 * i + rl, ch), src + (unsigned long long)at_r * (D * 2));
                }
                continue;
              }
#pragma unroll 2
              for (int x = 0; x < 32; x += 32 / CPR) {
                // a cached row, a node, or zeros
                const int rl = x + lane / CPR, r = 32 * i + rl;
                const uint32_t at_r = __shfl_sync(0xffffffffu, mine, rl);
                const int u = k0 + r - s.len;
                const void* src = base;
                int bytes = 16;
                if (at_r != 0xffffffffu) src = base + (unsigned long long)at_r * (D * 2) + ch * 16;
                else if (u >= 0 && u < p.T) src = nodes + u * st.n + ch * 8;
                else bytes = 0;
                cp_async16(dst + wide_at(r, ch), src, bytes);
              }
            }
            if (kv && !all && k0 + kKeys > s.len) {
              // non-finite elements of the nodes' values are left out here and added by the rows that attend them
              asm volatile("cp.async.wait_all;" ::: "memory");
              __syncwarp();
              const int r0 = max(s.len - k0, 0), r1 = min(s.len + p.T - k0, kKeys);
#pragma unroll 1
              for (int r = r0 + lane / CPR; r < r1; r += 32 / CPR) {
                const uint32_t a = dst + wide_at(r, ch);
                const uint4 w = lds128(a);
                bool odd = false;
                const uint32_t c[4] = {clean2<QT>(w.x, odd), clean2<QT>(w.y, odd), clean2<QT>(w.z, odd), clean2<QT>(w.w, odd)};
                if (odd) {
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(c[0]), "r"(c[1]), "r"(c[2]), "r"(c[3])
                               : "memory");
                  *static_cast<volatile int*>(&sh.odd[seg_no & 3]) = (int)seg_no + 1;
                }
              }
            }
            pending = slot;
          }
          if (ok && t == s.t0) load_q();
        }
        at += s.t1 - s.t0;
      }
      publish();
      asm volatile("cp.async.wait_all;" ::: "memory");
      // after an abort nobody may have waited for the last tile; the tiles before
      // it in this warp's turn had been consumed or are waited for by theirs
      if (!ok && last >= 0) {
        mbar_drain(bar(kBarFull + last % W::kUnits), (last / W::kUnits) & 1);
        if (last >= 3) mbar_drain(bar(kBarFull + (last - 3) % W::kUnits), ((last - 3) / W::kUnits) & 1);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
    // ---------------------------------------------------------- softmax
    const int g = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t_lane + g * 128, tO = tmem + t_lane + 256 + g * 128;
    const float c2 = p.c2;
    uint32_t ns = 0, no = 0, tile_no = 0, seg_no = 0;
    bool ok = true;
    // the relation terms are read, and results written, from here on
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int at = my_start; at < my_end && ok; ++seg_no) {
      const Seg s = segment(at);
      const int n = s.t1 - s.t0;
      if (g >= s.groups) {
        tile_no += n;
        at += n;
        continue;
      }
      const int gr = s.rb * 256 + g * 128 + r;
      const bool row_ok = gr < R;
      const int t_row = row_ok ? gr / p.G : 0, h = s.hkv * p.G + (row_ok ? gr - t_row * p.G : 0);
      const unsigned long long mk = row_ok ? node_mask(p, s.b, t_row) : 0ull;
      const int depth = max(__popcll(mk) - 1, 0);
      const float* z = p.z ? p.z + s.b * p.z_b + h * p.z_h + t_row * p.z_t : nullptr;
      const float zlow = p.z ? z[0] * c2 : 0.f;
      // depths of the nodes, for this row tile's warps
      named_bar_sync(1 + g, 128);
      if (r < 64) sh.depth[g][r] = r < p.T ? max(__popcll(node_mask(p, s.b, r)) - 1, 0) : 0;
      named_bar_sync(1 + g, 128);
      float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
      for (int t = s.t0; t < s.t1; ++t, ++tile_no) {
        const int k0 = t * kKeys;
        const bool got = mbar_wait(bar(kBarSFull + g), ns++ & 1, abort_flag, limit);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        tc_fence_after();
        const volatile uint32_t* vw = sh.valid[tile_no % kTileRing];
        const bool easy = k0 + kKeys <= s.len && (vw[0] & vw[1] & vw[2] & vw[3]) == 0xffffffffu &&
                          (!p.z || k0 + kKeys - 1 - s.len <= p.e_lo);
        const float rowc = easy ? zlow : 0.f;           // base-2 score: x c2 + rowc
        if (!easy) {
          // masks and unsaturated relation terms, 32 keys at a time, back into tensor memory
          const float* zr = p.z ? z - p.e_lo : nullptr;
          const int* sh_depth = sh.depth[g];
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            float y[32];
            tmem_ld32(tS + 32 * i, reinterpret_cast<uint32_t*>(y));
            tmem_wait_ld();
            const uint32_t bits = vw[i];
            const int o0 = k0 + 32 * i - s.len, d0 = o0 - depth;   // from the end of the cache, and the offset, of column 0
            if (p.z && o0 + 32 <= 0 && d0 + 31 <= p.e_lo) {
              const float low = z[0];                   // saturated for this row
#pragma unroll
              for (int c = 0; c < 32; ++c) y[c] += low;
            } else if (p.z && o0 + 32 <= 0 && d0 >= p.e_lo && d0 + 31 <= p.e_hi) {
              // 32 consecutive terms: aligned groups of four (rows of z are padded to eight), turned by the rest.
              // A ninth group is needed, and then lies in the row, unless the first starts on a group.
              const int a = d0 - p.e_lo, sh = a & 3;
              const float4* src = reinterpret_cast<const float4*>(z + (a & ~3));
              float f[36];
#pragma unroll
              for (int c = 0; c < 9; ++c) {
                const float4 w = c < 8 || sh ? __ldg(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                f[4 * c] = w.x; f[4 * c + 1] = w.y; f[4 * c + 2] = w.z; f[4 * c + 3] = w.w;
              }
#pragma unroll
              for (int c = 0; c < 35; ++c) f[c] = sh & 1 ? f[c + 1] : f[c];
#pragma unroll
              for (int c = 0; c < 32; ++c) y[c] += sh & 2 ? f[c + 2] : f[c];
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                int o = o0 + c;                         // node, or the place from the end of the cache
                if (o >= 0) o = sh_depth[o & 63];
                if (p.z) y[c] += zr[iclamp(o - depth, p.e_lo, p.e_hi)];
              }
            }
            if (o0 + 32 > 0 || bits != 0xffffffffu) {
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const int o = o0 + c;
                if (!((bits >> c) & 1u) || (o >= 0 && !((mk >> (o & 63)) & 1ull))) y[c] = -INFINITY;
              }
            }
            __syncwarp();                               // the store is the whole warp's
            tmem_st32(tS + 32 * i, reinterpret_cast<uint32_t*>(y));
          }
          tmem_wait_st();
        }
        float x[128];
        tmem_ld32(tS, reinterpret_cast<uint32_t*>(x));
        tmem_ld32(tS + 32, reinterpret_cast<uint32_t*>(x) + 32);
        tmem_ld32(tS + 64, reinterpret_cast<uint32_t*>(x) + 64);
        tmem_ld32(tS + 96, reinterpret_cast<uint32_t*>(x) + 96);
        tmem_wait_ld();
        float pm[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) pm[u] = max3(x[u], x[u + 8], x[u + 16]);
#pragma unroll
        for (int c = 24; c < 120; c += 16)
#pragma unroll
          for (int u = 0; u < 8; ++u) pm[u] = max3(pm[u], x[c + u], x[c + 8 + u]);
#pragma unroll
        for (int u = 0; u < 8; ++u) pm[u] = fmaxf(pm[u], x[120 + u]);
        const float mx = max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
        const float m_new = fmaxf(m_run, mx * c2 + rowc);
        const bool grow = m_new - m_run > kSlack;      // (false for two infinities)
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2(m_run - m_new) : 1.f;
          if (t > s.t0) {                               // the tile before has left O: its P V came before these scores
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t ov[32];
              tmem_ld32(tO + c, ov);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st32(tO + c, ov);
            }
          }
          if (grow) {
            l_run *= alpha;
            m_run = m_new;
          }
        }
        // with nothing seen yet every score is -inf, if not by its mask then by rowc (a saturated bias
        // of -inf), which then has to stay in the exponent: 2^(x c2) alone could be infinite
        const float sub = m_run == -INFINITY ? rowc : rowc - m_run;
        const float2 cc = make_float2(c2, c2), ss = make_float2(sub, sub);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[32];
#pragma unroll
          for (int w = 0; w < 32; ++w) {
            const float2 y = ffma2(make_float2(x[64 * q + 2 * w], x[64 * q + 2 * w + 1]), cc, ss);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            sum[w & 1] = fadd2(sum[w & 1], e);
            pk[w] = DT<QT>::pack(e.x, e.y);
          }
          tmem_st32(tS + 32 * q, pk);
        }
        l_run += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(kBarPReady + g));
      }
      if (!ok) break;
      at += n;
      if (at >= my_end) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
      // ---- the item's (or its part's) result
      const bool got = mbar_wait(bar(kBarOFull + g), no++ & 1, abort_flag, limit);
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      const bool whole = s.t0 == 0 && s.t1 == s.nt;
      // nodes of this part's tiles, which may hold non-finite values: an item may be cut between its nodes
      const bool odd = *static_cast<volatile int*>(&sh.odd[seg_no & 3]) == (int)seg_no + 1;
      const int u0 = max(s.t0 * kKeys - s.len, 0), u1 = min(s.t1 * kKeys - s.len, p.T);
      // a padding node, or a row with no key, gives 0; a part is joined (and divided) later
      const bool empty = mk == 0 || l_run == 0.f;
      const float inv = !whole ? 1.f : empty ? 0.f : 1.f / l_run;
      const long long out_row = ((long long)s.b * p.H + h) * p.T + t_row;
      float* slot = p.part + ((long long)blockIdx.x * 2 + (at - n == my_start ? 0 : 1)) * slot_floats(256, D);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(tO + c, reinterpret_cast<uint32_t*>(o));
        tmem_wait_ld();
        if (odd && row_ok) {
          for (int u = u0; u < u1; ++u) {
            if (!((mk >> u) & 1ull)) continue;
            const QT* src = static_cast<const QT*>(p.v) + s.b * p.vs.b + s.hkv * p.vs.h + u * p.vs.n + c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float y = DT<QT>::to_f(src[i]);
              if (!(fabsf(y) <= 3.4028235e38f)) o[i] += y;
            }
          }
        }
        if (whole && empty) {                           // not 0 times it: a padding query may hold anything
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (row_ok) {
          float* dst = whole ? static_cast<float*>(p.o) + out_row * D + c : slot + (long long)(g * 128 + r) * D + c;
          if (whole && !p.o_f32) {
            uint16_t* d16 = static_cast<uint16_t*>(p.o) + out_row * D + c;
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(d16 + i) =
                  make_uint4(DT<QT>::pack(o[i] * inv, o[i + 1] * inv), DT<QT>::pack(o[i + 2] * inv, o[i + 3] * inv),
                             DT<QT>::pack(o[i + 4] * inv, o[i + 5] * inv), DT<QT>::pack(o[i + 6] * inv, o[i + 7] * inv));
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(dst + i) = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
          }
        }
        __syncwarp();                                   // the next load is the whole warp's
      }
      if (whole && row_ok) p.lse[out_row] = empty ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
      if (!whole && row_ok) {
        slot[256 * D + g * 128 + r] = m_run;
        slot[256 * D + 256 + g * 128 + r] = l_run;
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) *p.status = kStatusTimeout;
}

template <int D, typename QT>
cudaError_t run_wide(const TreeParams& p, cudaStream_t s) {
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int smem = dynamic_bytes<D>(p.B);
  if (dev > 63 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(tree_wide_kernel<D, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynamicMost);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready |= 1ull << dev;
  }
  // the cache's rows of a page as TMA boxes, where a page holds whole swizzle groups
  // of 8 rows and rows can be counted in an int
  const long long rows = ((long long)p.c.num_pages * p.c.Hkv) << p.c.page_shift;
  int box = p.c.page_shift >= 3 && rows < (1LL << 31) ? 1 << (p.c.page_shift < 7 ? p.c.page_shift : 7) : 0;
  CUtensorMap maps[2] = {};
  if (box) {
    auto fn = encode_fn();
    for (int i = 0; i < 2; ++i) {
      const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, pitch[1] = {D * 2};
      const cuuint32_t bx[2] = {64, (cuuint32_t)box}, one[2] = {1, 1};
      if (!fn || fn(&maps[i], DT<QT>::kCoarse ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                    i ? p.c.v : p.c.k, dims, pitch, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        box = 0;
    }
  }
  note_launch(1);
  return launch_after(tree_wide_kernel<D, QT>, kThreads, dim3(p.grid), smem, s, p.z != nullptr, p, maps[0], maps[1], box);
}

}  // namespace

// Whether this kernel takes a call: more rows than the narrow one's largest block,
// a cache of the queries' type, and a list of sequences that fits behind the ring of
// tiles.  16 sequences of up to 8192, 32 / 8 heads, bf16, against the narrow
// kernel: d = 128, 244 rows 176 us and 539, 68 rows 131 and 266; d = 64, 68 rows 108 and
// 162; with one relation row per offset (4 sequences of 4096) 244 rows 197 and 234, 68
// rows 104 and 117.
bool takes_wide(const TreeParams& p) {
  const int smem = p.c.d == 64 ? dynamic_bytes<64>(p.B) : dynamic_bytes<128>(p.B);
  return p.G * p.T > 64 && smem <= kDynamicMost;
}

cudaError_t launch_wide(const TreeParams& p, cudaStream_t s) {
  if (p.c.d == 64) return p.bf16 ? run_wide<64, __nv_bfloat16>(p, s) : run_wide<64, __half>(p, s);
  return p.bf16 ? run_wide<128, __nv_bfloat16>(p, s) : run_wide<128, __half>(p, s);
}

}  // namespace tree
}  // namespace relpos
