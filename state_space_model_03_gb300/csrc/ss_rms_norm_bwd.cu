// Backward of the root-mean-square norm (include/ssfwd_layer.h): with n = s rstd,
//   ds = rstd (w dout - n mean(w dout n)) + dsum,  dw = sum over rows of dout n.
// Bound by the traffic of its rows. A CTA (or, for short rows, each warp of it) takes
// every so many-th row and keeps its columns' part of dw in registers; the parts go
// to the workspace by CTA and a second launch adds them up: no atomics.
#include "ss_norm.cuh"

namespace ssk {
namespace {

template <typename T, typename R, int V, int N>
__global__ void __launch_bounds__(1024) ss_rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p, bool cta) {
  __shared__ float sums[2][32];
  extern __shared__ float cols[];  // a warp per row: (warps, dim)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = cta ? threadIdx.x : lane, width = cta ? blockDim.x : 32;
  const long long first = cta ? blockIdx.x : (long long)blockIdx.x * warps + warp;
  const long long step = cta ? gridDim.x : (long long)gridDim.x * warps;
  float dw[N][V], w[N][V];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int c = (k * width + me) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = w[k][i] = 0.f;
    if (c < p.dim) load_weight<T, V>(p.weight, p.weight_f32, c, w[k]);
  }
  int turn = 0;
  for (long long row = first; row < p.rows; row += step, turn ^= 1) {
    const T *dout = static_cast<const T *>(p.dout) + row * p.sd;
    const R *sum = static_cast<const R *>(p.sum) + row * p.ss;
    const R *dsum = p.dsum ? static_cast<const R *>(p.dsum) + row * p.sds : nullptr;
    const float rstd = p.rstd[row];
    float d[N][V], n[N][V], e[N][V];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) d[k][i] = n[k][i] = e[k][i] = 0.f;
      if (c < p.dim) {
        load_vals<T, V>(dout + c, d[k]);
        load_vals<R, V>(sum + c, n[k]);
        if (dsum) load_vals<R, V>(dsum + c, e[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        n[k][i] *= rstd;
        dw[k][i] = fmaf(d[k][i], n[k][i], dw[k][i]);
        d[k][i] *= w[k][i];
        dot = fmaf(d[k][i], n[k][i], dot);
      }
    // two places in turn: a row's sums are read before the row after the next writes its own
    const float mean = __fdiv_rn(row_sum(dot, cta, sums[turn]), (float)p.dim);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c >= p.dim) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) d[k][i] = fmaf(rstd, fmaf(-n[k][i], mean, d[k][i]), e[k][i]);
      if (p.dx) store_vals<T, V>(static_cast<T *>(p.dx) + row * p.sdx + c, d[k]);
      if (p.dresidual) store_vals<R, V>(static_cast<R *>(p.dresidual) + row * p.sdr + c, d[k]);
    }
  }
  if (!p.parts) return;
  float *parts = p.parts + (long long)blockIdx.x * p.dim;
  if (cta) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c < p.dim)
#pragma unroll
        for (int i = 0; i < V; ++i) parts[c + i] = dw[k][i];
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int c = (k * width + me) * V;
      if (c < p.dim)
#pragma unroll
        for (int i = 0; i < V; ++i) cols[warp * p.dim + c + i] = dw[k][i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < p.dim; c += blockDim.x) {
      float s = 0.f;
      for (int k = 0; k < warps; ++k) s += cols[k * p.dim + c];
      parts[c] = s;
    }
  }
}

// dweight: the sum over the parts.
template <typename W>
__global__ void __launch_bounds__(512) ss_rms_norm_dweight_kernel(const float *parts, int n, int dim, W *dweight) {
  __shared__ float sums[16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < dim)
#pragma unroll 4
    for (int k = warp; k < n; k += 16) s += parts[(long long)k * dim + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < dim) {
    s = 0.f;
    for (int w = 0; w < 16; ++w) s += sums[w][lane];
    dweight[c] = from_f<W>(s);
  }
}

template <typename T, typename R, int V, int N>
cudaError_t launch(const NormBwdParams &p, const RowPlan &plan, cudaStream_t s) {
  const int smem = plan.cta ? 0 : 4 * (plan.threads / 32) * p.dim;
  ss_rms_norm_bwd_kernel<T, R, V, N><<<p.ctas, plan.threads, smem, s>>>(p, plan.cta);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dweight) return e;
  const int grid = (p.dim + 31) / 32;
  if (p.weight_f32) ss_rms_norm_dweight_kernel<float><<<grid, 512, 0, s>>>(p.parts, p.ctas, p.dim, static_cast<float *>(p.dweight));
  else ss_rms_norm_dweight_kernel<T><<<grid, 512, 0, s>>>(p.parts, p.ctas, p.dim, static_cast<T *>(p.dweight));
  return cudaGetLastError();
}
template <typename T, typename R>
cudaError_t pick(bool vec, const NormBwdParams &p, cudaStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const int pieces = (p.dim + (vec ? V : 1) - 1) / (vec ? V : 1);
  RowPlan plan;
  auto spread = [&](int n) { plan.threads = ((pieces + n - 1) / n + 31) / 32 * 32; };
  if (vec) {
    plan.cta = pieces > 64;
    plan.threads = 128;
    plan.pieces = plan.cta ? (pieces <= 1024 ? 1 : pieces <= 2048 ? 2 : pieces <= 4096 ? 4 : 8) : pieces <= 32 ? 1 : 2;
    if (plan.cta) spread(plan.pieces);
    switch (plan.pieces) {
      case 1: return launch<T, R, V, 1>(p, plan, s);
      case 2: return launch<T, R, V, 2>(p, plan, s);
      case 4: return launch<T, R, V, 4>(p, plan, s);
    }
    if constexpr (V == 4) return launch<T, R, V, 8>(p, plan, s);
    return cudaErrorInvalidValue;
  }
  plan.cta = pieces > 256;
  plan.threads = 128;
  plan.pieces = pieces <= 8192 ? 8 : 32;
  if (plan.cta) spread(plan.pieces);
  return plan.pieces == 8 ? launch<T, R, 1, 8>(p, plan, s) : launch<T, R, 1, 32>(p, plan, s);
}
template <typename T>
cudaError_t residual(int residual_dtype, bool vec, const NormBwdParams &p, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (residual_dtype == 0) return pick<T, float>(vec, p, s);
  return pick<T, T>(vec, p, s);
}

}  // namespace

// Each of 152 SMs four CTAs, as far as there are rows; a row's worth of dw per CTA is
// what the second launch has to read.
int norm_bwd_ctas(long long rows, int dim) {
  const long long rows_at_once = dim <= 256 ? 4 : 1;
  return (int)std::max<long long>(1, std::min<long long>((rows + rows_at_once - 1) / rows_at_once, 4 * 152));
}

cudaError_t launch_rms_norm_bwd(int dtype, int residual_dtype, bool vec, const NormBwdParams &p, cudaStream_t s) {
  return dtype == 0   ? residual<float>(residual_dtype, vec, p, s)
         : dtype == 1 ? residual<__half>(residual_dtype, vec, p, s)
                      : residual<__nv_bfloat16>(residual_dtype, vec, p, s);
}

}  // namespace ssk
