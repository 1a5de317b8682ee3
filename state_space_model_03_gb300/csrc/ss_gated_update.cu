// One token of the gated recurrence, by state slot (include/ssfwd_layer.h):
//   h = h + (n h + b),  n = a - 1, b = sqrt(1 - a^2) sigmoid(input_gate) x,  out = h.
// Bound by the traffic of the fp32 states, read and written once, and of the rows
// beside them. A thread has V neighbouring channels, whose decay it takes once, of
// up to kRows rows. 512 x 5120 bf16: 8.3 us in a graph, 5.1 TB/s; 4 x 2560 3.2.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kCta = 128;
constexpr int kRows = 4;  // rows that a thread has in flight

template <typename T, int V>
struct Vals {
  float v[V];
  __device__ __forceinline__ void load(const T *src) {
    if constexpr (V == 1) {
      v[0] = to_f<T>(src[0]);
    } else if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4 *>(src);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2 *>(src);
      const float2 a = unpack2<T>(q.x), b = unpack2<T>(q.y);
      v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
  }
  __device__ __forceinline__ void store(T *dst) const {
    if constexpr (V == 1) dst[0] = from_f<T>(v[0]);
    else if constexpr (sizeof(T) == 4) *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
  }
};

template <typename T, int V, bool IG>
__global__ void __launch_bounds__(kCta) ss_gated_update_kernel(const __grid_constant__ GatedUpdateParams p) {
  const int c = (blockIdx.x * kCta + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int r0 = blockIdx.y * kRows;
  const T *x = static_cast<const T *>(p.x), *gate = static_cast<const T *>(p.gate), *igate = static_cast<const T *>(p.igate);
  Vals<T, V> xv[kRows], g[kRows], i[kRows];
  Vals<float, V> h[kRows];
  long long at[kRows];
  bool live[kRows];
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u;
    const int slot = r < p.rows ? (p.slot_map ? p.slot_map[r] : r) : -1;
    live[u] = slot >= 0 && slot < p.slots;
    at[u] = live[u] ? slot * p.ss + c : 0;
    if (!live[u]) continue;
    xv[u].load(x + r * p.sx + c);
    g[u].load(gate + r * p.sg + c);
    if constexpr (IG) i[u].load(igate + r * p.si + c);
    h[u].load(p.state + at[u]);
  }
  constexpr int W = V == 1 ? 1 : 2;  // channels at a time
  f2 open[V / W];                    // L of an open gate
  bool near = true;
  auto at2 = [](const float *v, int j) { return W == 2 ? pk(v[j], v[j + W - 1]) : both(v[j]); };
  {
    float k[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      k[j] = -p.rate * softplus_f(p.decay[c + j]);
      near = near && k[j] >= -0.5f;
    }
#pragma unroll
    for (int j = 0; j < V; j += W) open[j / W] = at2(k, j);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int r = r0 + u;
    if (r >= p.rows) return;
    Vals<T, V> o;
#pragma unroll
    for (int j = 0; j < V; j += W) {
      float2 v = make_float2(0.f, 0.f);
      if (live[u]) {
        f2 r[1] = {at2(g[u].v, j)}, n[1], root[1], inverse[1], w = at2(xv[u].v, j);
        sigmoid2(r);
        r[0] = mul2(open[j / W], r[0]);
        decay2(r, near, n);
        root2(n, root, inverse);
        if constexpr (IG) {
          f2 in[1] = {at2(i[u].v, j)};
          sigmoid2(in);
          w = mul2(w, in[0]);
        }
        v = upk(step2(n[0], at2(h[u].v, j), mul2(root[0], w)));
      }
      h[u].v[j] = o.v[j] = v.x;
      if constexpr (W == 2) h[u].v[j + 1] = o.v[j + 1] = v.y;
    }
    if (live[u]) h[u].store(p.state + at[u]);
    o.store(static_cast<T *>(p.out) + r * p.so + c);
  }
}

template <typename T>
cudaError_t pick(const GatedUpdateParams &p, cudaStream_t s) {
  const int per = kCta * (p.vec ? 4 : 1);
  const dim3 grid((p.dim + per - 1) / per, (p.rows + kRows - 1) / kRows);
  if (p.vec) {
    if (p.igate) ss_gated_update_kernel<T, 4, true><<<grid, kCta, 0, s>>>(p);
    else ss_gated_update_kernel<T, 4, false><<<grid, kCta, 0, s>>>(p);
  } else {
    if (p.igate) ss_gated_update_kernel<T, 1, true><<<grid, kCta, 0, s>>>(p);
    else ss_gated_update_kernel<T, 1, false><<<grid, kCta, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_update(int dtype, const GatedUpdateParams &p, cudaStream_t s) {
  return dtype == 0 ? pick<float>(p, s) : dtype == 1 ? pick<__half>(p, s) : pick<__nv_bfloat16>(p, s);
}

}  // namespace ssk
