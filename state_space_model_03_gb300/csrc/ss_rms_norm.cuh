// (included by ss_rms_norm.cu and, with SS_NORM_QUANT, by ss_rms_norm_quant.cu)
#pragma once
// Root-mean-square norm with the residual's addition, output in the input's type or
// in e4m3 with scales (include/ssfwd_layer.h):
//   s = x + residual (rounded to the residual's type), out = s / rms(s) weight.
// Bound by the traffic of its rows. A row stays in its threads' registers from its
// one read to its writes: a warp's where it has up to 4 accesses a lane, else a
// CTA's. In the quantised form a group's largest value goes over the lanes that hold
// it, its bits as integers, so that a NaN is the largest of all.
#include <cuda_fp8.h>

#include "ss_norm.cuh"

namespace ssk {
namespace {

__device__ __forceinline__ float scale_of(float most, bool e8m0, uint8_t &byte) {
  float s = __fdiv_rn(most, 448.f);
  s = isnan(s) ? s : fmaxf(s, 1.17549435e-38f);
  if (e8m0) {  // the least power of two not below it
    uint32_t w = __float_as_uint(s);
    if (isnan(s)) {
      byte = 255;
    } else {
      w = (w + 0x7fffffu) & 0x7f800000u;
      byte = (uint8_t)(w >> 23);
      s = __uint_as_float(w);
    }
  }
  return s;
}

template <typename T, typename R, bool RES, int V, int N, bool QUANT>
__global__ void __launch_bounds__(1024) ss_rms_norm_kernel(const __grid_constant__ NormParams p, bool cta) {
  __shared__ float sums[32];
  extern __shared__ uint32_t most[];  // QUANT, where a group is not a part of a warp's access
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = cta ? blockIdx.x : (long long)blockIdx.x * (blockDim.x >> 5) + warp;
  const bool live = row < p.rows;  // a warp's last CTA may have fewer rows
  const int me = cta ? threadIdx.x : lane, width = cta ? blockDim.x : 32;
  const T *x = static_cast<const T *>(p.x) + row * p.sx;
  const R *res = RES ? static_cast<const R *>(p.residual) + row * p.sr : nullptr;
  float v[N][V];
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = (k * width + me) * V;
    if (live && c < p.dim) {
      load_vals<T, V>(x + c, v[k]);
      if constexpr (RES) {
        float r[V];
        load_vals<R, V>(res + c, r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] = to_f<R>(from_f<R>(v[k][i] + r[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
  }
  if (RES && p.sum && live) {
    R *sum = static_cast<R *>(p.sum) + row * p.ss;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c < p.dim) store_vals<R, V>(sum + c, v[k]);
    }
  }
  sq = row_sum(sq, cta, sums);
  const float rstd = rsqrtf(__fdiv_rn(sq, (float)p.dim) + p.eps);
  if (p.rstd && live && me == 0) p.rstd[row] = rstd;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = (k * width + me) * V;
    if (c < p.dim) {
      float w[V];
      load_weight<T, V>(p.weight, p.weight_f32, c, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rstd * w[i];
    }
  }
  if constexpr (!QUANT) {
    if (!live) return;
    T *out = static_cast<T *>(p.out) + row * p.so;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c < p.dim) store_vals<T, V>(out + c, v[k]);
    }
  } else {
    uint32_t m[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      m[k] = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) m[k] = max(m[k], __float_as_uint(v[k][i]) & 0x7fffffffu);
    }
    const int lanes = p.group / V;  // that share a group, where it is part of a warp's access
    if (p.group > 0 && lanes <= 32) {
#pragma unroll
      for (int k = 0; k < N; ++k)
        for (int o = lanes >> 1; o > 0; o >>= 1) m[k] = max(m[k], __shfl_xor_sync(~0u, m[k], o));
    } else if (p.group == 0) {
#pragma unroll
      for (int k = 1; k < N; ++k) m[0] = max(m[0], m[k]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(~0u, m[0], o));
      if (cta) {
        if (lane == 0) most[warp] = m[0];
        __syncthreads();
        m[0] = lane < (int)(blockDim.x >> 5) ? most[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(~0u, m[0], o));
      }
#pragma unroll
      for (int k = 1; k < N; ++k) m[k] = m[0];
    } else {  // single values, groups of two or four warps' accesses (V == 1, or lane groups above 32)
      uint32_t *mine = most + (cta ? 0 : warp * p.groups);
      for (int g = me; g < p.groups; g += width) mine[g] = 0;
      if (cta) __syncthreads();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        uint32_t q = m[k];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q = max(q, __shfl_xor_sync(~0u, q, o));
        const int c = k * width + (me & ~31);
        if (lane == 0 && c < p.dim) atomicMax(&mine[c / p.group], q);
      }
      if (cta) __syncthreads();
      __syncwarp();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = k * width + me;
        m[k] = c < p.dim ? mine[c / p.group] : 0;
      }
    }
    if (!live) return;
    uint8_t *out = static_cast<uint8_t *>(p.out) + row * p.so;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c >= p.dim) continue;
      uint8_t byte = 0;
      const float scale = scale_of(__uint_as_float(m[k]), p.e8m0, byte);
      if (p.group > 0 ? c % p.group == 0 : c == 0) {
        const long long at = row * p.groups + (p.group > 0 ? c / p.group : 0);
        if (p.e8m0) static_cast<uint8_t *>(p.scale)[at] = byte;
        else static_cast<float *>(p.scale)[at] = scale;
      }
      // a division, not a product with the reciprocal: where a value lies half way between two of e4m3's, the two differ
      if constexpr (V == 1) {
        out[c] = __nv_cvt_float_to_fp8(__fdiv_rn(v[k][0], scale), __NV_SATFINITE, __NV_E4M3);
      } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[k][i], scale), __fdiv_rn(v[k][i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[k][i + 2], scale), __fdiv_rn(v[k][i + 3], scale)), __NV_SATFINITE, __NV_E4M3);
          w[i / 4] = lo | hi << 16;
        }
        if constexpr (V == 8) *reinterpret_cast<uint2 *>(out + c) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(out + c) = w[0];
      }
    }
  }
}

template <typename T, typename R, bool RES, int V, int N, bool QUANT>
cudaError_t launch(const NormParams &p, const RowPlan &plan, cudaStream_t s) {
  const int warps = plan.threads / 32;
  const long long ctas = plan.cta ? p.rows : (p.rows + warps - 1) / warps;
  const int smem = QUANT ? 4 * std::max(32, p.groups * (plan.cta ? 1 : warps)) : 0;
  ss_rms_norm_kernel<T, R, RES, V, N, QUANT><<<(unsigned)ctas, plan.threads, smem, s>>>(p, plan.cta);
  return cudaGetLastError();
}
template <typename T, typename R, bool RES, bool QUANT>
cudaError_t pick(bool vec, const NormParams &p, int sms, cudaStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const int pieces = (p.dim + (vec ? V : 1) - 1) / (vec ? V : 1);
  RowPlan plan;
  auto spread = [&](int n) { plan.threads = ((pieces + n - 1) / n + 31) / 32 * 32; };
  if (vec) {
    // few rows: as many threads for each as it has accesses; else two accesses a thread
    plan.cta = pieces > 128 || (pieces > 32 && p.rows < 4 * sms);
    if (!plan.cta) {
      plan.threads = 128;
      plan.pieces = pieces <= 32 ? 1 : pieces <= 64 ? 2 : 4;
    } else {
      plan.pieces = pieces <= 1024 && p.rows < 4 * sms ? 1 : pieces <= 2048 ? 2 : pieces <= 4096 ? 4 : 8;
      spread(plan.pieces);
    }
    switch (plan.pieces) {
      case 1: return launch<T, R, RES, V, 1, QUANT>(p, plan, s);
      case 2: return launch<T, R, RES, V, 2, QUANT>(p, plan, s);
      case 4: return launch<T, R, RES, V, 4, QUANT>(p, plan, s);
    }
    if constexpr (V == 4) return launch<T, R, RES, V, 8, QUANT>(p, plan, s);
    return cudaErrorInvalidValue;
  }
  plan.cta = pieces > 256;
  if (!plan.cta) {
    plan.threads = 128;
    plan.pieces = 8;
  } else {
    plan.pieces = pieces <= 8192 ? 8 : 32;
    spread(plan.pieces);
  }
  return plan.pieces == 8 ? launch<T, R, RES, 1, 8, QUANT>(p, plan, s) : launch<T, R, RES, 1, 32, QUANT>(p, plan, s);
}
template <typename T, bool QUANT>
cudaError_t residual(int residual_dtype, bool vec, const NormParams &p, int sms, cudaStream_t s) {
  if (!p.residual) return pick<T, T, false, QUANT>(vec, p, sms, s);
  if constexpr (sizeof(T) == 2)
    if (residual_dtype == 0) return pick<T, float, true, QUANT>(vec, p, sms, s);
  return pick<T, T, true, QUANT>(vec, p, sms, s);
}
template <bool QUANT>
cudaError_t types(int dtype, int residual_dtype, bool vec, const NormParams &p, int sms, cudaStream_t s) {
  return dtype == 0   ? residual<float, QUANT>(residual_dtype, vec, p, sms, s)
         : dtype == 1 ? residual<__half, QUANT>(residual_dtype, vec, p, sms, s)
                      : residual<__nv_bfloat16, QUANT>(residual_dtype, vec, p, sms, s);
}

}  // namespace

#ifdef SS_NORM_QUANT
cudaError_t launch_rms_norm_quant(int dtype, int residual_dtype, bool vec, const NormParams &p, int sms, cudaStream_t s) {
  return types<true>(dtype, residual_dtype, vec, p, sms, s);
}
#else
cudaError_t launch_rms_norm(int dtype, int residual_dtype, bool vec, const NormParams &p, int sms, cudaStream_t s) {
  return types<false>(dtype, residual_dtype, vec, p, sms, s);
}
#endif

}  // namespace ssk
