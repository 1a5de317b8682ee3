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
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdlib>

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

// What follows takes N pairs at a time, step by step, so that the instructions of one
// step, which do not wait for one another, stand together.

// e^L - 1 for L <= 0. In [-1/2, 0] as L (1 + L/2 + ...): a polynomial of degree 5
// interpolating (e^L - 1) / L at Chebyshev nodes (3e-9 off, coefficients in fp32).
// `near`: |L| <= 1/2 for every token of the warp's channels (|L| is at most rate
// softplus(decay)), so that the other form is not needed.
template <int N>
__device__ __forceinline__ void decay2(const f2 (&L)[N], bool near, f2 (&n)[N]) {
  constexpr float c[5] = {8.1896139309e-03f, 4.1630074382e-02f, 1.6666242480e-01f, 4.9999982119e-01f, 1.f};
#pragma unroll
  for (int j = 0; j < N; ++j) n[j] = fma2(both(1.1234042468e-03f), L[j], both(c[0]));
#pragma unroll
  for (int k = 1; k < 5; ++k) {
#pragma unroll
    for (int j = 0; j < N; ++j) n[j] = fma2(n[j], L[j], both(c[k]));
  }
#pragma unroll
  for (int j = 0; j < N; ++j) n[j] = mul2(n[j], L[j]);
  if (!near) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float2 l = upk(L[j]);
      float2 v = upk(n[j]);
      if (l.x < -0.5f) v.x = ex2(l.x * kLog2e) - 1.f;
      if (l.y < -0.5f) v.y = ex2(l.y * kLog2e) - 1.f;
      n[j] = pk(v);
    }
  }
}

template <int N>
__device__ __forceinline__ void sigmoid2(f2 (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = mul2(v[j], both(-kLog2e));
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 e = upk(v[j]);
    v[j] = pk(ex2(e.x), ex2(e.y));
  }
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = add2(v[j], both(1.f));
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 e = upk(v[j]);
    v[j] = pk(rcp(e.x), rcp(e.y));
  }
}

__device__ __forceinline__ float rsqrt_ftz(float v) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
  return y;
}
// sqrt(1 - a^2) and its reciprocal. 1e-36 more under the root keeps both finite where
// a is 1; there the root is 1e-18.
template <int N>
__device__ __forceinline__ void root2(const f2 (&n)[N], f2 (&root)[N], f2 (&inverse)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) root[j] = fma2(n[j], both(-1.f), both(-2.f));
#pragma unroll
  for (int j = 0; j < N; ++j) root[j] = fma2(n[j], root[j], both(1e-36f));
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 v = upk(root[j]);
    inverse[j] = pk(rsqrt_ftz(v.x), rsqrt_ftz(v.y));
  }
#pragma unroll
  for (int j = 0; j < N; ++j) root[j] = mul2(root[j], inverse[j]);
}

// One token; as well one token's map (n, b) after a run's (N, E), part by part.
__device__ __forceinline__ f2 step2(f2 n, f2 h, f2 b) { return add2(h, fma2(n, h, b)); }

// A lane's two channels as they are stored: neighbours in one access (PAIR), or one
// 16 channels after the other where rows do not start on such accesses.
template <typename T, bool PAIR>
struct Two {
  T a, b;
  __device__ __forceinline__ void load(const T *src, bool ok0, bool ok1) {
    a = ok0 ? src[0] : from_f<T>(0.f);
    b = ok1 ? src[16] : from_f<T>(0.f);
  }
  __device__ __forceinline__ f2 widen() const { return pk(to_f<T>(a), to_f<T>(b)); }
  static __device__ __forceinline__ void store(T *dst, float2 v, bool ok0, bool ok1) {
    if (ok0) dst[0] = from_f<T>(v.x);
    if (ok1) dst[16] = from_f<T>(v.y);
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

// How rows come and go: single values, pairs, or tiles by TMA (pairs in shared memory).
// A tile is kGatedTile tokens by kGatedCh channels: runs of kRun tokens, two to a warp,
// whose halves have 16 lanes of two channels each.
constexpr int kRun = 8;
constexpr int kRuns = kGatedTile / kRun;
constexpr int kGatedWarps = kRuns / 2;
constexpr int kGatedThreads = kGatedWarps * 32;
enum RowAccess { kSingles, kPairs, kTma };

// SSFWD_TEST_STALL=<k>, SSFWD_TEST_STALL_MAPS=<k>: a round whose copies, or whose maps in a
// cluster, are lost, and short waits.
inline WaitHook wait_hook() {
  WaitHook w;
  const char *copy = std::getenv("SSFWD_TEST_STALL"), *maps = std::getenv("SSFWD_TEST_STALL_MAPS");
  w.limit = copy || maps ? 1u << 10 : kMaxWaitIters;
  if (copy) w.copy = std::atoi(copy);
  if (maps) w.maps = std::atoi(maps);
  return w;
}

// The exchange within a cluster.
__device__ __forceinline__ uint32_t remote_of(const void *p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
// 16 bytes to a place of CTA `rank`, counted by a barrier of that CTA: the data and its
// arrival in one, without a fence or a barrier of the whole cluster.
__device__ __forceinline__ void send(ulonglong2 *p, uint64_t *bar, int rank, ulonglong2 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];" ::"r"(remote_of(p, rank)),
               "l"(v.x), "l"(v.y), "r"(remote_of(bar, rank))
               : "memory");
}
// mbar_wait for what others have sent: it acquires at the scope that their stores'
// arrivals release at, which mbar_wait, of a CTA's own copies, does not.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, int32_t *err, int32_t code, uint32_t limit) {
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs) : "memory");
    if (ok) return true;
  }
  atomicCAS(err, 0, code);
  return false;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}

// Tiles by TMA: loads of a CTA's tile (thread 0), stores of a warp's rows.
__device__ __forceinline__ void store_rows(const CUtensorMap *tm, const void *src, int c, int t, int b) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(c), "r"(t), "r"(b), "r"(smem_u32(src))
               : "memory");
}
__device__ __forceinline__ void commit_stores() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// (dim, tokens, batch) in boxes of 32 channels by `rows` tokens. A dimension of one
// element may have any stride.
inline bool rows_map(TensorMapEncode enc, CUtensorMap *m, int esize, const void *base, int dim, int tokens, int batch, const long long *st, int rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)tokens, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {tokens > 1 ? (cuuint64_t)st[1] * esize : 16, batch > 1 ? (cuuint64_t)st[0] * esize : 16};
  const cuuint32_t box[3] = {kGatedCh, (cuuint32_t)rows, 1}, es[3] = {1, 1, 1};
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(enc)(
             m, esize == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of a unit's segments, one for each lane of a half warp.
__device__ __forceinline__ ulonglong2 *segment_maps(void *maps, long long unit, int segs, int seg) {
  return static_cast<ulonglong2 *>(maps) + (unit * segs + seg) * 16;
}

}  // namespace ssk
