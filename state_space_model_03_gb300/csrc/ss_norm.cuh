// What the kernels of the root-mean-square norm share: a row's values by thread.
//
// A row is a warp's (a CTA's warps have rows of their own), or a CTA's; a thread has N accesses of V
// values of it, always the same columns, and goes from row to row with the weight in
// registers and the next row's values on their way while it works on this one's.
#pragma once
#include "ss_fwd_kernel.cuh"

#include <algorithm>

#include "ss_layer.h"

namespace ssk {

// V values as they are stored: 8 of 16 bits or 4 of 32 in a 16-byte access (8 of 32 in
// two), or one.
template <typename T, int V>
struct Piece {
  static constexpr int W = V * (int)sizeof(T) / 16;
  uint4 q[W];
  __device__ __forceinline__ void load(const T *src) {
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = reinterpret_cast<const uint4 *>(src)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + k] = __uint_as_float(w[k]);
        } else {
          const float2 f = unpack2<T>(w[k]);
          v[8 * i + 2 * k] = f.x;
          v[8 * i + 2 * k + 1] = f.y;
        }
      }
    }
  }
  // rounds v, which becomes what is stored
  __device__ __forceinline__ void round(float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(v[4 * i + k]);
        else w[k] = pack2<T>(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if constexpr (sizeof(T) != 4) widen(v);
  }
  __device__ __forceinline__ void store(T *dst) const {
#pragma unroll
    for (int i = 0; i < W; ++i) reinterpret_cast<uint4 *>(dst)[i] = q[i];
  }
};
template <typename T>
struct Piece<T, 1> {
  T x;
  __device__ __forceinline__ void load(const T *src) { x = *src; }
  __device__ __forceinline__ void zero() { x = from_f<T>(0.f); }
  __device__ __forceinline__ void widen(float (&v)[1]) const { v[0] = to_f<T>(x); }
  __device__ __forceinline__ void round(float (&v)[1]) {
    x = from_f<T>(v[0]);
    v[0] = to_f<T>(x);
  }
  __device__ __forceinline__ void store(T *dst) const { *dst = x; }
};
// The same pointer, of which the compiler does not know so: what is loaded through it in
// a loop is not kept in registers around the loop.
__device__ __forceinline__ const void *again(const void *p) {
  asm volatile("" : "+l"(p));
  return p;
}
template <typename T, int V>
__device__ __forceinline__ void load_weight(const void *w, bool f32, int c, float (&v)[V]) {
  if (sizeof(T) == 4 || f32) {
    Piece<float, V> p;
    p.load(static_cast<const float *>(w) + c);
    p.widen(v);
  } else {
    Piece<T, V> p;
    p.load(static_cast<const T *>(w) + c);
    p.widen(v);
  }
}

// The sum over a row's threads: a warp, or the CTA (sums: a place for each warp).
__device__ __forceinline__ float row_sum(float v, bool cta, float *sums) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if (!cta) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) sums[warp] = v;
  __syncthreads();
  v = lane < warps ? sums[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// How rows are laid out over threads: `values` of a row for each, as many as are
// instantiated (8, 16, 32 or 64).
struct RowPlan {
  int values, threads, ctas;
  bool cta;  // a CTA per row (else a warp)
};
constexpr int kNormSms = 152;
// Threads of a CTA at most: 640 with 102 registers where a thread has few enough values
// to keep the weight and the next row beside them, else 512 with 128.
constexpr int norm_threads(bool keeps) { return keeps ? 640 : 512; }
// by_warp: a warp has a row; least: values of a thread to begin with; kept: up to which
// the weight is kept; ctas: 0 for as many as 2048 threads an SM make.
inline RowPlan row_plan(int dim, long long rows, int v, bool by_warp, int least, int kept, int ctas) {
  RowPlan plan{least, 128, ctas, !by_warp};
  if (plan.cta) {
    while (plan.values < 64 && (long long)plan.values * norm_threads(plan.values <= kept) < dim) plan.values *= 2;
    const int n = plan.values / v, accesses = (dim + v - 1) / v;
    plan.threads = ((accesses + n - 1) / n + 31) / 32 * 32;
  }
  const long long at_once = plan.cta ? 1 : plan.threads / 32;
  if (!ctas) ctas = kNormSms * std::max(1, 2048 / plan.threads);
  plan.ctas = (int)std::max<long long>(1, std::min<long long>((rows + at_once - 1) / at_once, ctas));
  return plan;
}

}  // namespace ssk
