// Backward of the root-mean-square norm (include/ssfwd_layer.h): with n = s rstd,
//   ds = rstd (w dout - n mean(w dout n)) + dsum,  dw = sum over rows of dout n.
// Bound by the traffic of its rows. A CTA (or, for short rows, each warp of it) takes
// every so many-th row and keeps its columns' part of dw in registers; the parts go
// to the workspace by CTA and a second launch adds them up: no atomics. They are fp32: a
// thread adds rows / CTAs terms one after the other, 2^-24 sqrt(rows / 304) off. 16384 x 2560 bf16
// with the sum in fp32: 104 us, 6.4 TB/s (95% of the copy); three CTAs an SM 118, one 130.
#include "ss_norm.cuh"

namespace ssk {
namespace {

// Up to 256 channels a warp takes a row, 8 values a lane.
bool norm_bwd_cta_per_row(int dim) { return dim > 256; }

constexpr int kKept = 8;  // values of a thread up to which it keeps the weight and takes the next row early

template <typename T, typename R, int V, int N>
__global__ void __launch_bounds__(norm_threads(N * V <= kKept)) ss_rms_norm_bwd_kernel(const __grid_constant__ NormBwdParams p, bool cta) {
  constexpr bool KEEP = N * V <= kKept;
  __shared__ float sums[2][32];
  extern __shared__ float cols[];  // a warp per row: (warps, dim)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = cta ? threadIdx.x : lane, width = cta ? blockDim.x : 32;
  const long long first = cta ? blockIdx.x : (long long)blockIdx.x * warps + warp;
  const long long step = cta ? gridDim.x : (long long)gridDim.x * warps;
  const float inv_dim = __frcp_rn((float)p.dim);
  int c[N];
  bool in[N];
  float dw[N][V], w[KEEP ? N : 1][V], next_rstd = 0.f;
  Piece<T, V> nd[N];
  Piece<R, V> ns[N], ne[KEEP ? N : 1];
  auto load = [&](long long r) {
    const T *dout = static_cast<const T *>(p.dout) + r * p.sd;
    const R *sum = static_cast<const R *>(p.sum) + r * p.ss;
    const R *dsum = p.dsum ? static_cast<const R *>(p.dsum) + r * p.sds : nullptr;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (in[k]) {
        nd[k].load(dout + c[k]);
        ns[k].load(sum + c[k]);
        if constexpr (KEEP) {
          if (dsum) ne[k].load(dsum + c[k]);
        }
      }
    next_rstd = p.rstd[r];
  };
#pragma unroll
  for (int k = 0; k < N; ++k) {
    c[k] = (k * width + me) * V;
    in[k] = c[k] < p.dim;
    nd[k].zero();
    ns[k].zero();
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = 0.f;
    if constexpr (KEEP) {
      ne[k].zero();
#pragma unroll
      for (int i = 0; i < V; ++i) w[k][i] = 0.f;
      if (in[k]) load_weight<T, V>(p.weight, p.weight_f32, c[k], w[k]);
    }
  }
  if (KEEP && first < p.rows) load(first);
  int turn = 0;
  for (long long row = first; row < p.rows; row += step, turn ^= 1) {
    if constexpr (!KEEP) load(row);
    const float rstd = next_rstd;
    float d[N][V], n[N][V], e[KEEP ? N : 1][V];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      nd[k].widen(d[k]);
      ns[k].widen(n[k]);
      if constexpr (KEEP) ne[k].widen(e[k]);
    }
    if constexpr (KEEP) {
      if (row + step < p.rows) load(row + step);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      float u[V] = {};
      if constexpr (!KEEP) {
        if (in[k]) load_weight<T, V>(again(p.weight), p.weight_f32, c[k], u);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        n[k][i] *= rstd;
        dw[k][i] = fmaf(d[k][i], n[k][i], dw[k][i]);
        d[k][i] *= KEEP ? w[KEEP ? k : 0][i] : u[i];
        dot = fmaf(d[k][i], n[k][i], dot);
      }
    }
    // two places in turn: a row's sums are read before the row after the next writes its own
    const float mean = row_sum(dot, cta, sums[turn]) * inv_dim;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (!in[k]) continue;
      float v[V], f[V] = {};
      if constexpr (!KEEP) {
        if (p.dsum) {
          Piece<R, V> q;
          q.load(static_cast<const R *>(p.dsum) + row * p.sds + c[k]);
          q.widen(f);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = d[k][i] = fmaf(rstd, fmaf(-n[k][i], mean, d[k][i]), KEEP ? e[KEEP ? k : 0][i] : f[i]);
      if (p.dx) {
        Piece<T, V> o;
        o.round(v);
        o.store(static_cast<T *>(p.dx) + row * p.sdx + c[k]);
      }
      if (p.dresidual) {
        Piece<R, V> o;
        o.round(d[k]);
        o.store(static_cast<R *>(p.dresidual) + row * p.sdr + c[k]);
      }
    }
  }
  if (!p.parts) return;
  float *parts = p.parts + (long long)blockIdx.x * p.dim;
  if (cta) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (in[k])
#pragma unroll
        for (int i = 0; i < V; ++i) parts[c[k] + i] = dw[k][i];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (in[k])
#pragma unroll
        for (int i = 0; i < V; ++i) cols[warp * p.dim + c[k] + i] = dw[k][i];
    __syncthreads();
    for (int k = threadIdx.x; k < p.dim; k += blockDim.x) {
      float s = 0.f;
      for (int u = 0; u < warps; ++u) s += cols[u * p.dim + k];
      parts[k] = s;
    }
  }
}

// dweight: the sum over the parts.
template <typename W>
__global__ void __launch_bounds__(1024) ss_rms_norm_dweight_kernel(const float *parts, int n, int dim, W *dweight) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < dim) {
#pragma unroll 10
    for (int k = warp; k < n; k += 32) s += parts[(long long)k * dim + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  // column `warp`: its 32 sums, one a lane
  s = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
  if (lane == 0 && blockIdx.x * 32 + warp < dim) dweight[blockIdx.x * 32 + warp] = from_f<W>(s);
}

template <typename T, typename R, int V, int N>
cudaError_t launch(const NormBwdParams &p, const RowPlan &plan, cudaStream_t s) {
  const int smem = plan.cta ? 0 : 4 * (plan.threads / 32) * p.dim;
  ss_rms_norm_bwd_kernel<T, R, V, N><<<p.ctas, plan.threads, smem, s>>>(p, plan.cta);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.dweight) return e;
  const int grid = (p.dim + 31) / 32;
  if (p.weight_f32) ss_rms_norm_dweight_kernel<float><<<grid, 1024, 0, s>>>(p.parts, p.ctas, p.dim, static_cast<float *>(p.dweight));
  else ss_rms_norm_dweight_kernel<T><<<grid, 1024, 0, s>>>(p.parts, p.ctas, p.dim, static_cast<T *>(p.dweight));
  return cudaGetLastError();
}
template <typename T, typename R, int V>
cudaError_t by_values(const NormBwdParams &p, const RowPlan &plan, cudaStream_t s) {
  switch (plan.values) {
    case 8: return launch<T, R, V, 8 / V>(p, plan, s);
    case 16: return launch<T, R, V, 16 / V>(p, plan, s);
    case 32: return launch<T, R, V, 32 / V>(p, plan, s);
    case 64: return launch<T, R, V, 64 / V>(p, plan, s);
  }
  return cudaErrorInvalidValue;
}
template <typename T, typename R>
cudaError_t pick(bool vec, const NormBwdParams &p, cudaStream_t s) {
  constexpr int V = sizeof(T) == 4 ? 4 : 8;
  const RowPlan plan = row_plan(p.dim, p.rows, vec ? V : 1, !norm_bwd_cta_per_row(p.dim), 8, kKept, p.ctas);
  return vec ? by_values<T, R, V>(p, plan, s) : by_values<T, R, 1>(p, plan, s);
}
template <typename T>
cudaError_t residual(int residual_dtype, bool vec, const NormBwdParams &p, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (residual_dtype == 0) return pick<T, float>(vec, p, s);
  }
  return pick<T, T>(vec, p, s);
}

}  // namespace

// Each SM two CTAs (of 320 threads at 2560 channels), four of them where a warp has a
// row, as far as there are rows; a row's worth of dw per CTA is what the second launch has
// to read.
int norm_bwd_ctas(long long rows, int dim) {
  const bool cta = norm_bwd_cta_per_row(dim);
  return (int)std::max<long long>(1, std::min<long long>(cta ? rows : (rows + 3) / 4, (cta ? 2 : 4) * kNormSms));
}

cudaError_t launch_rms_norm_bwd(int dtype, int residual_dtype, bool vec, const NormBwdParams &p, cudaStream_t s) {
  return dtype == 0   ? residual<float>(residual_dtype, vec, p, s)
         : dtype == 1 ? residual<__half>(residual_dtype, vec, p, s)
                      : residual<__nv_bfloat16>(residual_dtype, vec, p, s);
}

}  // namespace ssk
