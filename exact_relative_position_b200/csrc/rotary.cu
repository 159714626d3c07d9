// rotary.cu -- rotary position embedding.
//
//   y_a = m (x_a cos t - x_b sin t),  y_b = m (x_b cos t + x_a sin t),
//   t = position * w_i,  (a, b) = (2i, 2i + 1) or (i, i + rotary_dim / 2);
//   columns from rotary_dim on are copied.
//
// The gradient is the same turn backwards (sin negated), so one kernel serves
// both.  The angle is kept as a fraction of a turn in 64-bit fixed point: the
// product position * step wraps modulo one turn by itself, so the angle of
// position 10^6 is as exact as that of position 1 (2^-33 of a turn before it
// is rounded to the 24 bits of the sine's argument), at the cost of one 64-bit
// multiply.
//
// Bound by memory: each element is read once and written once.  A thread turns one
// head at a time: blocks with more loads to a thread hold fewer threads and were
// slower (4 x 4097 tokens of 40 heads of 128, both directions: 140 us, 4.8 TB/s, at one
// head, 156 at four).
#include "serve.cuh"
#include "kernels.cuh"

namespace relpos {
namespace {

template <typename T> struct Elem;
template <> struct Elem<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// One thread: V frequencies of one token (two vectors of V elements), for up
// to `hpt` heads, so that the sines are taken once for all of them.
template <typename T, int V, bool SMALL>
__global__ void __launch_bounds__(256) rotary_kernel(const __grid_constant__ RotaryParams p, int pair_jobs,
                                                     int jobs, int hpt) {
  using VT = Vec<T, V>;
  // 32-bit division where the counts allow it: one in 64 bits costs as much as turning a row
  int job, b, n;
  if (SMALL) {
    const uint32_t idx = blockIdx.x * 256u + threadIdx.x, tok = idx / (uint32_t)jobs;
    if (tok >= (uint32_t)p.B * (uint32_t)p.N) return;
    job = (int)(idx - tok * jobs);
    b = (int)(tok / (uint32_t)p.N);
    n = (int)(tok - (uint32_t)b * p.N);
  } else {
    const long long idx = (long long)blockIdx.x * 256 + threadIdx.x, tok = idx / jobs;
    if (tok >= (long long)p.B * p.N) return;
    job = (int)(idx - tok * jobs);
    b = (int)(tok / p.N);
    n = (int)(tok - (long long)b * p.N);
  }

  const bool turn = job < pair_jobs;
  float cs[V], sn[V];
  int a0, b0;                          // columns of the two vectors
  int va = V, vb = V;                  // elements of them that exist
  if (turn) {
    long long pos = n;
    if (p.pos) {
      const long long at = (long long)b * p.pos_bs + n;
      pos = p.pos_wide ? static_cast<const long long*>(p.pos)[at] : (long long)static_cast<const int*>(p.pos)[at];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned long long f = (unsigned long long)pos * p.step[job * V + i];
      const float x = (float)(int)(f >> 32) * 0x1p-31f;   // half turns in [-1, 1)
      float s, c;
      sincospif(x, &s, &c);
      cs[i] = c * p.cos_scale;
      sn[i] = s * p.sin_scale;
    }
    a0 = p.interleaved ? job * 2 * V : job * V;
    b0 = p.interleaved ? a0 + V : a0 + p.rotary_dim / 2;
  } else {
    a0 = p.rotary_dim + (job - pair_jobs) * 2 * V;
    b0 = a0 + V;
    va = min(V, p.d - a0);
    vb = max(0, min(V, p.d - b0));
  }
  const int Ht = p.t[0].H + (p.n_tensors > 1 ? p.t[1].H : 0);
  const int h0 = blockIdx.y * hpt, h1 = min(h0 + hpt, Ht);
#pragma unroll 1
  for (int hh = h0; hh < h1; ++hh) {
    const RotaryTensor& t = hh < p.t[0].H ? p.t[0] : p.t[1];
    const int h = hh < p.t[0].H ? hh : hh - p.t[0].H;
    const T* x = static_cast<const T*>(t.x) + b * t.xs.b + h * t.xs.h + n * t.xs.n;
    T* y = static_cast<T*>(t.y) + b * t.ys.b + h * t.ys.h + n * t.ys.n;
    if (turn) {
      const VT u = *reinterpret_cast<const VT*>(x + a0), w = *reinterpret_cast<const VT*>(x + b0);
      VT yu, yw;
      if (p.interleaved) {
        // u and w together are V pairs (2i, 2i + 1)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e0 = 2 * i, e1 = 2 * i + 1;
          const float xa = Elem<T>::up(e0 < V ? u.e[e0 % V] : w.e[e0 % V]);
          const float xb = Elem<T>::up(e1 < V ? u.e[e1 % V] : w.e[e1 % V]);
          const T ya = Elem<T>::down(xa * cs[i] - xb * sn[i]), yb = Elem<T>::down(xb * cs[i] + xa * sn[i]);
          if (e0 < V) yu.e[e0 % V] = ya; else yw.e[e0 % V] = ya;
          if (e1 < V) yu.e[e1 % V] = yb; else yw.e[e1 % V] = yb;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xa = Elem<T>::up(u.e[i]), xb = Elem<T>::up(w.e[i]);
          yu.e[i] = Elem<T>::down(xa * cs[i] - xb * sn[i]);
          yw.e[i] = Elem<T>::down(xb * cs[i] + xa * sn[i]);
        }
      }
      *reinterpret_cast<VT*>(y + a0) = yu;
      *reinterpret_cast<VT*>(y + b0) = yw;
    } else if (x != y) {
      if (va == V) *reinterpret_cast<VT*>(y + a0) = *reinterpret_cast<const VT*>(x + a0);
      if (vb == V) *reinterpret_cast<VT*>(y + b0) = *reinterpret_cast<const VT*>(x + b0);
    }
  }
}

// Whether all rows start on whole vectors (the stride of a dimension of one means nothing).
bool fits(const RotaryParams& p, const RotaryTensor& t, int V, int es) {
  const long long m = V;
  auto ok = [&](const void* q, const Strides& s) {
    return reinterpret_cast<uintptr_t>(q) % (V * es) == 0 && (p.B == 1 || s.b % m == 0) && (t.H == 1 || s.h % m == 0) &&
           (p.N == 1 || s.n % m == 0);
  };
  return ok(t.x, t.xs) && ok(t.y, t.ys);
}

template <typename T, int V>
cudaError_t go(const RotaryParams& p, cudaStream_t s) {
  const int pair_jobs = p.rotary_dim / (2 * V);
  const int jobs = pair_jobs + (p.d - p.rotary_dim + 2 * V - 1) / (2 * V);
  const int Ht = p.t[0].H + (p.n_tensors > 1 ? p.t[1].H : 0);
  const long long threads = (long long)p.B * p.N * jobs;
  // heads a thread turns with one set of sines: as many as leave two blocks to an SM, up to
  // 8 (16 left too few threads: 151 us in place of 140)
  int hpt = (int)(threads * Ht / (148LL * 512));
  hpt = hpt < 1 ? 1 : hpt > 8 ? 8 : hpt;
  if (Ht > hpt * 65535) hpt = (Ht + 65534) / 65535;   // a grid's rows; two tensors have up to 131070 heads
  const int hy = (Ht + hpt - 1) / hpt;
  dim3 grid((unsigned)((threads + 255) / 256), (unsigned)hy);
  if (threads < (1LL << 31)) rotary_kernel<T, V, true><<<grid, 256, 0, s>>>(p, pair_jobs, jobs, hpt);
  else rotary_kernel<T, V, false><<<grid, 256, 0, s>>>(p, pair_jobs, jobs, hpt);
  note_launch(1);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t pick(const RotaryParams& p, cudaStream_t s) {
  bool wide = p.rotary_dim % (2 * V) == 0 && p.d % V == 0;
  for (int i = 0; i < p.n_tensors; ++i) wide = wide && fits(p, p.t[i], V, sizeof(T));
  return wide ? go<T, V>(p, s) : go<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, int es, int bf16, cudaStream_t s) {
  if (es == 4) return pick<float, 4>(p, s);
  return bf16 ? pick<__nv_bfloat16, 8>(p, s) : pick<__half, 8>(p, s);
}

}  // namespace relpos
