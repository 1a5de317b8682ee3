// What the kernels of the root-mean-square norm share: a row's values by thread.
#pragma once
#include "ss_fwd_kernel.cuh"
#include <algorithm>

#include "ss_layer.h"

namespace ssk {

// V values of a row as fp32: 8 (or 4) in 16-byte accesses, or one.
template <typename T, int V>
__device__ __forceinline__ void load_vals(const T *src, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f<T>(src[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4 *>(src + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  } else {
    static_assert(V == 8);
    const uint4 q = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<T>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_vals(T *dst, const float (&v)[V]) {
  if constexpr (V == 1) {
    dst[0] = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    static_assert(V == 8);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
}
template <typename T, int V>
__device__ __forceinline__ void load_weight(const void *w, bool f32, int c, float (&v)[V]) {
  if (sizeof(T) == 4 || f32) load_vals<float, V>(static_cast<const float *>(w) + c, v);
  else load_vals<T, V>(static_cast<const T *>(w) + c, v);
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

// How a row is laid out over threads: a warp's or a CTA's.
struct RowPlan {
  int pieces;   // accesses of a thread, rounded up to what is instantiated
  int threads;  // of the CTA
  bool cta;     // a CTA per row (else a warp)
};

}  // namespace ssk
