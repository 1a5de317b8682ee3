// What the kernels of the gated recurrence share: gates, loads of a lane's two
// channels, and the exchange within a cluster.
//
//   L = -rate softplus(decay) sigmoid(gate),  a = e^L
//   h = a h + sqrt(1 - a^2) sigmoid(input_gate) x
//
// A decay is held as n = a - 1, and the state moves by h + (n h + b). 1 - a is what a
// long memory depends on: a itself in fp32 is off by up to 2^-25, which adds up over
// the 1 / (1 - a) tokens that a state remembers (65536 tokens of one gate at a =
// 0.99993: 3e-4 off; by n 1e-6). sqrt(1 - a^2) = sqrt(-n (2 + n)) keeps its bits the
// same way. What is left is a state's own rounding, 2^-24 of the largest before it.
//
// Two channels at a time, in packed fp32 pairs.
#pragma once
#include "ss_fwd_kernel.cuh"
#include "ss_layer.h"

namespace ssk {

__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 both(float v) { return pk(v, v); }
__device__ __forceinline__ f2 pk(float2 v) { return pk(v.x, v.y); }

// e^L - 1 for L <= 0. In [-1/2, 0] as L (1 + L/2 + ...): a polynomial of degree 5
// interpolating (e^L - 1) / L at Chebyshev nodes (3e-9 off, coefficients in fp32).
// `near`: |L| <= 1/2 for every token of the warp's channels (|L| is at most rate
// softplus(decay)), so that the other form is not needed.
__device__ __forceinline__ f2 decay2(f2 L, bool near) {
  f2 q = both(1.1234042468e-03f);
  q = fma2(q, L, both(8.1896139309e-03f));
  q = fma2(q, L, both(4.1630074382e-02f));
  q = fma2(q, L, both(1.6666242480e-01f));
  q = fma2(q, L, both(4.9999982119e-01f));
  q = fma2(q, L, both(1.f));
  f2 n = mul2(q, L);
  if (!near) {
    const float2 l = upk(L);
    float2 v = upk(n);
    if (l.x < -0.5f) v.x = ex2(l.x * kLog2e) - 1.f;
    if (l.y < -0.5f) v.y = ex2(l.y * kLog2e) - 1.f;
    n = pk(v);
  }
  return n;
}

__device__ __forceinline__ f2 sigmoid2(f2 v) {
  float2 e = upk(mul2(v, both(-kLog2e)));
  e = upk(add2(pk(ex2(e.x), ex2(e.y)), both(1.f)));
  return pk(rcp(e.x), rcp(e.y));
}

__device__ __forceinline__ float rsqrt_ftz(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
// sqrt(1 - a^2) and its reciprocal. 1e-36 more under the root keeps both finite where
// a is 1; there the root is 1e-18.
__device__ __forceinline__ f2 root2(f2 n, f2 &inverse) {
  const f2 m = fma2(n, fma2(n, both(-1.f), both(-2.f)), both(1e-36f));
  const float2 v = upk(m);
  inverse = pk(rsqrt_ftz(v.x), rsqrt_ftz(v.y));
  return mul2(m, inverse);
}

// One token, and one token's map (n, b) after a run's (N, E).
__device__ __forceinline__ f2 step2(f2 n, f2 h, f2 b) { return add2(h, fma2(n, h, b)); }

// A lane's two channels as they are stored: neighbours in one access (PAIR), or one
// 32 channels after the other where rows do not start on such accesses.
template <typename T, bool PAIR>
struct Two {
  T a, b;
  __device__ __forceinline__ void load(const T *src, bool ok0, bool ok1) {
    a = ok0 ? src[0] : from_f<T>(0.f);
    b = ok1 ? src[32] : from_f<T>(0.f);
  }
  __device__ __forceinline__ f2 widen() const { return pk(to_f<T>(a), to_f<T>(b)); }
  static __device__ __forceinline__ void store(T *dst, float2 v, bool ok0, bool ok1) {
    if (ok0) dst[0] = from_f<T>(v.x);
    if (ok1) dst[32] = from_f<T>(v.y);
  }
};
template <typename T>
struct Two<T, true> {
  uint32_t w;
  __device__ __forceinline__ void load(const T *src, bool ok0, bool) { w = ok0 ? *reinterpret_cast<const uint32_t *>(src) : 0u; }
  __device__ __forceinline__ f2 widen() const { return pk(unpack2<T>(w)); }
  static __device__ __forceinline__ void store(T *dst, float2 v, bool ok0, bool) {
    if (ok0) *reinterpret_cast<uint32_t *>(dst) = pack2<T>(v.x, v.y);
  }
};
template <>
struct Two<float, true> {
  float2 v;
  __device__ __forceinline__ void load(const float *src, bool ok0, bool) {
    v = ok0 ? *reinterpret_cast<const float2 *>(src) : make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ f2 widen() const { return pk(v); }
  static __device__ __forceinline__ void store(float *dst, float2 x, bool ok0, bool) {
    if (ok0) *reinterpret_cast<float2 *>(dst) = x;
  }
};

// The exchange within a cluster.
__device__ __forceinline__ uint32_t remote_of(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_remote(void *p, int rank, ulonglong2 v) {
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(remote_of(p, rank)), "l"(v.x), "l"(v.y) : "memory");
}
__device__ __forceinline__ void store_remote(void *p, int rank, f2 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(remote_of(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace ssk
