// (included by ss_rms_norm.cu and, with SS_NORM_QUANT, by ss_rms_norm_quant.cu)
#pragma once
// Root-mean-square norm with the residual's addition, output in the input's type or
// in e4m3 with scales (include/ssfwd_layer.h):
//   s = x + residual (rounded to the residual's type), out = s / rms(s) weight.
// Bound by the traffic of its rows. A row stays in its threads' registers from its
// one read to its writes. In the quantised form a group's largest value goes over the
// lanes that hold it; a NaN is the largest of all.
//
// 16384 x 2560 bf16 with the residual in fp32: 78 us, 6.5 TB/s (95% of the copy); 16384 x
// 5120 bf16 in 8 bits, a scale of each 32 channels: 95 us, 6.2 TB/s (92%). A quotient by
// division took 139 instead (380 instructions for 8 values). CTAs that make 2048 threads
// an SM 181 us for norm and backward, 1024 187, 640 185.
#include <cuda_fp8.h>

#include "ss_norm.cuh"

namespace ssk {
namespace {

// The larger of two absolute values; a NaN where one is.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// The scale of a group with `most` as its largest (NaN: it has one), and its reciprocal.
// Both are NaN where most is infinite or NaN: no scale brings an infinity to 448.
// The least power of two not below most / 448 = most / (1.75 2^8): its exponent is most's
// less 8, and one more where most's fraction is above 1.75; at least 2^-126.
struct Scale {
  float scale, inverse;
  uint8_t byte;
};
__device__ __forceinline__ Scale scale_of(float most, bool e8m0) {
  Scale s;
  if (e8m0) {
    const uint32_t w = __float_as_uint(most);
    const uint32_t p = max((w + 0x1fffffu) >> 23, 9u) - 8;
    const bool fine = w < 0x7f800000u;
    s.byte = fine ? p : 255;
    s.scale = 0.f;
    s.inverse = __uint_as_float(fine ? (254 - p) << 23 : 0x7fffffffu);
  } else {
    s.scale = most / 448.f;
    if (s.scale < 1.17549435e-38f) s.scale = 1.17549435e-38f;
    if (!(most < __uint_as_float(0x7f800000u))) s.scale = __uint_as_float(0x7fffffffu);
    s.inverse = __frcp_rn(s.scale);
    s.byte = 0;
  }
  return s;
}

constexpr int kKept = 16;  // values of a thread up to which it keeps the weight and takes the next row early

template <typename T, typename R, bool RES, int V, int N, bool QUANT>
__global__ void __launch_bounds__(norm_threads(N * V <= kKept)) ss_rms_norm_kernel(const __grid_constant__ NormParams p, bool cta) {
  constexpr bool KEEP = N * V <= kKept;
  __shared__ float sums[2][32];
  extern __shared__ float most[];  // QUANT: largest values, by warp or by 32 channels
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = cta ? threadIdx.x : lane, width = cta ? blockDim.x : 32;
  const long long step = cta ? gridDim.x : (long long)gridDim.x * warps;
  long long row = cta ? blockIdx.x : (long long)blockIdx.x * warps + warp;
  if (row >= p.rows) return;  // the whole CTA, or a warp of one whose warps have rows of their own
  const float inv_dim = __frcp_rn((float)p.dim);
  int c[N], group[N];  // first channel, and QUANT its group
  bool in[N];
  float w[KEEP ? N : 1][V];
  Piece<T, V> nx[N];
  Piece<R, V> nr[N];
  auto load = [&](long long r) {
    const T *x = static_cast<const T *>(p.x) + r * p.sx;
    const R *res = RES ? static_cast<const R *>(p.residual) + r * p.sr : nullptr;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (in[k]) {
        nx[k].load(x + c[k]);
        if constexpr (RES) nr[k].load(res + c[k]);
      }
  };
#pragma unroll
  for (int k = 0; k < N; ++k) {
    c[k] = (k * width + me) * V;
    in[k] = c[k] < p.dim;
    group[k] = QUANT && p.group > 0 ? c[k] / p.group : 0;
    nx[k].zero();
    if constexpr (RES) nr[k].zero();
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[k][i] = 0.f;
      if (in[k]) load_weight<T, V>(p.weight, p.weight_f32, c[k], w[k]);
    }
  }
  if constexpr (KEEP) load(row);
  for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
    if constexpr (!KEEP) load(row);
    float v[N][V];
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      nx[k].widen(v[k]);
      if constexpr (RES) {
        float r[V];
        nr[k].widen(r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] += r[i];
      }
    }
    if constexpr (KEEP) {
      if (row + step < p.rows) load(row + step);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if constexpr (RES) {
        Piece<R, V> s;
        s.round(v[k]);
        if (p.sum && in[k]) s.store(static_cast<R *>(p.sum) + row * p.ss + c[k]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sq = fmaf(v[k][i], v[k][i], sq);
    }
    // two places in turn: a row's sums are read before the row after the next writes its own
    sq = row_sum(sq, cta, sums[turn]);
    const float rstd = rsqrtf(fmaf(sq, inv_dim, p.eps));
    if (p.rstd && me == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float u[V] = {};
      if constexpr (!KEEP) {
        if (in[k]) load_weight<T, V>(again(p.weight), p.weight_f32, c[k], u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * rstd * (KEEP ? w[KEEP ? k : 0][i] : u[i]);
    }
    if constexpr (!QUANT) {
      T *out = static_cast<T *>(p.out) + row * p.so;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (in[k]) {
          Piece<T, V> o;
          o.round(v[k]);
          o.store(out + c[k]);
        }
    } else {
      float m[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        m[k] = fabsf(v[k][0]);
#pragma unroll
        for (int i = 1; i < V; ++i) m[k] = larger(m[k], v[k][i]);
      }
      auto over = [&](int lanes) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          if (o >= lanes) break;
#pragma unroll
          for (int k = 0; k < N; ++k) m[k] = larger(m[k], __shfl_xor_sync(~0u, m[k], o));
        }
      };
      const int lanes = p.group / V;  // that share a group, where it is part of a warp's access
      if (p.group > 0 && lanes <= 32) {
        over(lanes);
      } else if (p.group == 0) {
#pragma unroll
        for (int k = 1; k < N; ++k) m[0] = larger(m[0], m[k]);
        over(32);
        if (cta) {
          if (lane == 0) most[32 * turn + warp] = m[0];
          __syncthreads();
          m[0] = lane < warps ? most[32 * turn + lane] : 0.f;
          over(32);
        }
#pragma unroll
        for (int k = 1; k < N; ++k) m[k] = m[0];
      } else {  // single values, groups of two or four warps' accesses: what the warps of a group have
        over(32);
        float *mine = most + (cta ? 0 : warp * 4 * p.groups);
        const int per = p.group / 32;
        if (cta) __syncthreads();  // the row before has read them
        __syncwarp();
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (lane == 0 && c[k] < p.dim) mine[c[k] / 32] = m[k];
        if (cta) __syncthreads();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < N; ++k) {
          m[k] = 0.f;
          if (in[k])
            for (int q = 0; q < per; ++q) {
              const int at = group[k] * per + q;
              if (at * 32 < p.dim) m[k] = larger(m[k], mine[at]);
            }
        }
      }
      uint8_t *out = static_cast<uint8_t *>(p.out) + row * p.so;
      Scale scale{};
#pragma unroll
      for (int k = 0; k < N; ++k) {
        if (k == 0 || p.group > 0) scale = scale_of(m[k], p.e8m0);
        if (!in[k]) continue;
        if ((c[k] & (p.group - 1)) == 0 && (p.group > 0 || c[k] == 0)) {
          const long long at = row * p.groups + group[k];
          if (p.e8m0) static_cast<uint8_t *>(p.scale)[at] = scale.byte;
          else static_cast<float *>(p.scale)[at] = scale.scale;
        }
        const float inverse = scale.inverse;
        // by the reciprocal, exact for a power of two; else within 2^-23 of the quotient
        if constexpr (V == 1) {
          out[c[k]] = __nv_cvt_float_to_fp8(v[k][0] * inverse, __NV_SATFINITE, __NV_E4M3);
        } else {
          uint32_t q[V / 4];
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[k][i] * inverse, v[k][i + 1] * inverse), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[k][i + 2] * inverse, v[k][i + 3] * inverse), __NV_SATFINITE, __NV_E4M3);
            q[i / 4] = lo | hi << 16;
          }
          if constexpr (V == 8) {
            *reinterpret_cast<uint2 *>(out + c[k]) = make_uint2(q[0], q[1]);
          } else {
            *reinterpret_cast<uint32_t *>(out + c[k]) = q[0];
          }
        }
      }
    }
  }
}

template <typename T, typename R, bool RES, int V, int N, bool QUANT>
cudaError_t launch(const NormParams &p, const RowPlan &plan, cudaStream_t s) {
  // largest values: two rows' by warp; or by 32 channels
  const int smem = QUANT ? 4 * std::max(64, 4 * p.groups * (plan.cta ? 1 : plan.threads / 32)) : 0;
  ss_rms_norm_kernel<T, R, RES, V, N, QUANT><<<plan.ctas, plan.threads, smem, s>>>(p, plan.cta);
  return cudaGetLastError();
}
template <typename T, typename R, bool RES, int V, bool QUANT>
cudaError_t by_values(const NormParams &p, const RowPlan &plan, cudaStream_t s) {
  switch (plan.values) {
    case 8: return launch<T, R, RES, V, 8 / V, QUANT>(p, plan, s);
    case 16: return launch<T, R, RES, V, 16 / V, QUANT>(p, plan, s);
    case 32: return launch<T, R, RES, V, 32 / V, QUANT>(p, plan, s);
    case 64: return launch<T, R, RES, V, 64 / V, QUANT>(p, plan, s);
  }
  return cudaErrorInvalidValue;
}
template <typename T, typename R, bool RES, bool QUANT>
cudaError_t pick(bool vec, const NormParams &p, cudaStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  // few rows, or single values: a CTA for each, 8 values a thread; else a warp for short
  // ones, and 16 values
  const bool fine = !vec || p.rows < 4 * kNormSms, by_warp = p.dim <= (fine ? 256 : 512);
  const RowPlan plan = row_plan(p.dim, p.rows, vec ? V : 1, by_warp, p.dim <= 256 || fine ? 8 : 16, kKept, 0);
  return vec ? by_values<T, R, RES, V, QUANT>(p, plan, s) : by_values<T, R, RES, 1, QUANT>(p, plan, s);
}
template <typename T, bool QUANT>
cudaError_t residual(int residual_dtype, bool vec, const NormParams &p, cudaStream_t s) {
  if (!p.residual) return pick<T, T, false, QUANT>(vec, p, s);
  if constexpr (sizeof(T) == 2) {
    if (residual_dtype == 0) return pick<T, float, true, QUANT>(vec, p, s);
  }
  return pick<T, T, true, QUANT>(vec, p, s);
}
template <bool QUANT>
cudaError_t types(int dtype, int residual_dtype, bool vec, const NormParams &p, cudaStream_t s) {
  return dtype == 0   ? residual<float, QUANT>(residual_dtype, vec, p, s)
         : dtype == 1 ? residual<__half, QUANT>(residual_dtype, vec, p, s)
                      : residual<__nv_bfloat16, QUANT>(residual_dtype, vec, p, s);
}

}  // namespace

#ifdef SS_NORM_QUANT
cudaError_t launch_rms_norm_quant(int dtype, int residual_dtype, bool vec, const NormParams &p, cudaStream_t s) {
  return types<true>(dtype, residual_dtype, vec, p, s);
}
#else
cudaError_t launch_rms_norm(int dtype, int residual_dtype, bool vec, const NormParams &p, cudaStream_t s) {
  return types<false>(dtype, residual_dtype, vec, p, s);
}
#endif

}  // namespace ssk
