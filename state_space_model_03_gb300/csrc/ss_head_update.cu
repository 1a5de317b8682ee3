// One token of the selective scan with one decay per head, by state slot
// (include/ssfwd_packed.h): for request r, head h, row p, state n
//   S = exp(dt A) S + dt x_p B_n;  out_p = (sum_n C_n S + D x_p) silu(z_p).
//
// Bound by the traffic of the fp32 states, read and written once (8 bytes per
// value). L lanes share a state row, NV 16-byte pieces each, and a warp has kPass
// rows in flight before it uses the first; dt, the decay and the B and C pieces
// are the same for all rows of a head and are taken once per warp. At 256 requests
// x 80 heads x 64 x 128: 249 us, 5.4 TB/s (80% of the copy bandwidth); 2 rows in
// flight 311, 8 258; CTAs of 8 warps 297, of 2 251; stores that leave the cache at
// once, as nothing reads them before the next step, against 253 without.
#include "ss_fwd_kernel.cuh"
#include "ss_packed.h"

namespace ssk {
namespace {

constexpr int kWarps = 4;
constexpr int kPass = 4;  // rows a lane group has in flight

template <typename T>
__device__ __forceinline__ void piece4(const T *src, bool vec, int valid, float (&v)[4]) {
  if (vec && valid == 4) {
    if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4 *>(src);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2 *>(src);
      const float2 a = unpack2<T>(q.x), b = unpack2<T>(q.y);
      v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = k < valid ? to_f<T>(src[k]) : 0.f;
}

template <typename T, int L, int NV>
__global__ void __launch_bounds__(kWarps * 32) ss_head_update_kernel(const __grid_constant__ HeadUpdateParams p) {
  constexpr int RW = 32 / L;  // rows of one warp access
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int j = lane % L, sub = lane / L;
  const int h = blockIdx.y, r = blockIdx.z;
  const int row0 = (blockIdx.x * kWarps + warp) * (kPass * RW) + sub;
  if (row0 - sub >= p.headdim) return;
  const int slot = p.slot_map ? p.slot_map[r] : r;
  const bool kept = slot >= 0 && slot < p.slots;
  float *st = p.state + (kept ? slot * p.ss[0] : 0) + h * p.ss[1];
  int valid[NV];
#pragma unroll
  for (int q = 0; q < NV; ++q) valid[q] = kept ? min(max(p.dstate - 4 * (j + q * L), 0), 4) : 0;
  float s[kPass][NV][4];
#pragma unroll
  for (int u = 0; u < kPass; ++u) {
    const int row = row0 + u * RW;
#pragma unroll
    for (int q = 0; q < NV; ++q)
      piece4<float>(st + (long long)row * p.dstate + 4 * (j + q * L), p.vec != 0, row < p.headdim ? valid[q] : 0, s[u][q]);
  }
  const int g = h / p.hpg;
  const T *B = static_cast<const T *>(p.B) + r * p.sB[0] + g * p.sB[1];
  const T *C = static_cast<const T *>(p.C) + r * p.sC[0] + g * p.sC[1];
  float b[NV][4], c[NV][4];
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    piece4<T>(B + 4 * (j + q * L), p.bcvec != 0, valid[q], b[q]);
    piece4<T>(C + 4 * (j + q * L), p.bcvec != 0, valid[q], c[q]);
  }
  const long long idt = r * p.sdt[0] + h * p.sdt[1];
  float dt = p.dt_f32 ? static_cast<const float *>(p.dt)[idt] : to_f<T>(static_cast<const T *>(p.dt)[idt]);
  if (p.bias) dt += p.bias[h];
  if (p.softplus) dt = softplus_f(dt);
  const float keep = ex2(dt * p.A[h] * kLog2e);
  const float skip = p.D ? p.D[h] : 0.f;
  const T *x = static_cast<const T *>(p.x) + r * p.sx[0] + h * p.sx[1];
  float y[kPass], xv[kPass];
#pragma unroll
  for (int u = 0; u < kPass; ++u) {
    const int row = row0 + u * RW;
    xv[u] = row < p.headdim ? to_f<T>(x[row]) : 0.f;
    const float in = dt * xv[u];
    y[u] = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[u][q][k] = fmaf(keep, s[u][q][k], in * b[q][k]);
        y[u] = fmaf(c[q][k], s[u][q][k], y[u]);
      }
      if (row < p.headdim && valid[q] > 0) {
        float *dst = st + (long long)row * p.dstate + 4 * (j + q * L);
        if (p.vec && valid[q] == 4) {
          __stcs(reinterpret_cast<float4 *>(dst), make_float4(s[u][q][0], s[u][q][1], s[u][q][2], s[u][q][3]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < valid[q]) dst[k] = s[u][q][k];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kPass; ++u)
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) y[u] += __shfl_xor_sync(0xffffffffu, y[u], o);
  // lane u of a row group writes its pass u
#pragma unroll
  for (int u = 0; u < kPass; ++u) {
    const int row = row0 + u * RW;
    if (j == u % L && row < p.headdim) {
      float v = fmaf(skip, xv[u], y[u]);
      if (p.z) v *= silu_f(to_f<T>(static_cast<const T *>(p.z)[r * p.sz[0] + h * p.sz[1] + row]));
      static_cast<T *>(p.out)[r * p.so[0] + h * p.so[1] + row] = from_f<T>(kept ? v : 0.f);
    }
  }
}

template <typename T, int L, int NV>
void go(const HeadUpdateParams &p, cudaStream_t s) {
  constexpr int rows = kWarps * kPass * (32 / L);
  const dim3 grid((p.headdim + rows - 1) / rows, p.heads, p.requests);
  ss_head_update_kernel<T, L, NV><<<grid, kWarps * 32, 0, s>>>(p);
}
template <typename T>
void by_states(const HeadUpdateParams &p, cudaStream_t s) {
  if (p.dstate > 128) go<T, 32, 2>(p, s);
  else if (p.dstate > 64) go<T, 32, 1>(p, s);
  else if (p.dstate > 32) go<T, 16, 1>(p, s);
  else if (p.dstate > 16) go<T, 8, 1>(p, s);
  else go<T, 4, 1>(p, s);
}

}  // namespace

cudaError_t launch_head_update(int dtype, const HeadUpdateParams &p, cudaStream_t s) {
  if (dtype == 0) by_states<float>(p, s);
  else if (dtype == 1) by_states<__half>(p, s);
  else by_states<__nv_bfloat16>(p, s);
  return cudaGetLastError();
}

}  // namespace ssk
