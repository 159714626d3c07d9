// serve.cuh -- parameter blocks and launch wrappers of the operators around
// generation: rotary embedding, the paged K/V cache and attention of drafted
// tokens over it.
#pragma once

#include "common.cuh"

namespace relpos {

// Element strides of a [B, H, N, d] view whose last dimension is contiguous.
struct Strides {
  long long b, h, n;
};

constexpr int kMaxPairs = 128;   // rotary pairs whose frequencies travel as kernel arguments

struct RotaryTensor {
  const void* x;
  void* y;
  int H;
  Strides xs, ys;
};

struct RotaryParams {
  RotaryTensor t[2];
  int n_tensors;
  int B, N, d, rotary_dim, interleaved;
  int pos_wide;                       // positions are int64 (else int32)
  const void* pos;                    // null: the token's index
  long long pos_bs;                   // elements between the positions of consecutive batch entries
  float cos_scale, sin_scale;         // magnitude, and magnitude times the direction of the turn
  unsigned long long step[kMaxPairs]; // turns per position as a fraction of 2^64
};
// es: bytes of an element (2 or 4); bf16 tells the two 16-bit types apart.
cudaError_t launch_rotary(const RotaryParams& p, int es, int bf16, cudaStream_t s);

// Geometry of the cache: rows of d elements at (page * Hkv + h) * page_size + offset.
struct CacheParams {
  void *k, *v;
  float *ks, *vs;
  int num_pages, page_shift, Hkv, d;
  int format;                         // relpos_cache_format
};

struct CacheWriteParams {
  CacheParams c;
  const void *k, *v;
  Strides kst, vst;
  int B, N;
  const long long* slots;             // [B * N]
  int bf16;                           // type of k and v
};
cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t s);

struct CacheReadParams {
  CacheParams c;
  const int* page_table;              // [B, P]
  int P, B;
  const int* cu;                      // [B + 1]
  int total;                          // rows of the outputs
  void *k, *v;                        // [total, Hkv, d]
  int bf16;                           // type of the outputs
};
cudaError_t launch_cache_read(const CacheReadParams& p, cudaStream_t s);

struct TreeParams {
  CacheParams c;
  int B, T, H, G;                     // G = H / Hkv query heads to a key head
  int bf16, o_f32;
  const int* page_table;              // [B, P]
  int P;
  const int* lengths;                 // [B]
  const long long* mask;              // bits of the attended nodes, [T] or [B, T]; null: a chain
  int mask_bs;                        // 0 or T
  const void *q, *k, *v;
  Strides qs, ks, vs;
  void* o;                            // [B, H, T, d]
  float* lse;                         // [B, H, T]
  float c2;                           // tau log2 e
  // relation terms over the offsets [e_lo, e_hi] (clamped there); z null: none
  float* z;
  long long z_b, z_h, z_t;            // element strides of z (0 where shared)
  int e_lo, e_hi;
  float z_scale;                      // what z is multiplied by when it is written
  float z_limit;                      // bound of a finite term before that
  const void* aq;                     // [R, d] or [H, R, d], or null
  long long aq_hs;
  const float* bias;                  // [H, R] or null
  int R, N;
  relpos_map_desc map;
  int* status;                        // device status word (a bounded wait expired)
  unsigned long long wait_ns;         // limit of the bounded waits
  // split work
  float* part;
  int grid, rows_per_block, row_blocks;
};
// Rows of query (heads times nodes) one block takes, and the blocks of a launch
// (256: the kernel for many rows).
int tree_rows_per_block(const TreeParams& p);
int tree_grid(const TreeParams& p);
cudaError_t launch_tree_relation(const TreeParams& p, cudaStream_t s);
cudaError_t launch_tree_attention(const TreeParams& p, cudaStream_t s);
cudaError_t launch_tree_combine(const TreeParams& p, cudaStream_t s);

}  // namespace relpos
