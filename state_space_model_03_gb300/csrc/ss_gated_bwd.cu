// Backward of the gated linear recurrence (include/ssfwd_layer.h). With e_t what
// token t hands back to the state before it,
//   g_t = dout_t + e_{t+1},  e_t = a_t g_t = g_t + n_t g_t,
// the same kind of recurrence as the forward's, backwards, with a token's own a. The
// states h_{t-1} that the decays' gradients need are taken up again in fp32 from the
// one that the forward kept before each tile of 64 tokens (1/32 of an operand in 16
// bits), so that both recurrences are local to a tile but for e.
//
// Tiles, warps and clusters are the forward's, the tiles in falling order. A warp's
// map has three parts: the product of its a (both directions'), the forward's end
// and the backward's. The sum over tokens for the decay's gradient stays in
// registers, then goes by CTA to the workspace and is added up by a second launch:
// no atomics, the same result in every call.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kSteps = 4;  // tokens of a warp: all that a token needs stays in registers
constexpr int kWarps = kGatedTile / kSteps;
constexpr int kThreads = kWarps * 32;

template <typename T, bool PAIR, bool IG>
__global__ void __launch_bounds__(kThreads, 1) ss_gated_bwd_kernel(const __grid_constant__ GatedBwdParams p) {
  __shared__ f2 prod[2][kWarps][32], fwd[2][kWarps][32], rev[2][kWarps][32];
  __shared__ ulonglong2 tiles[2][kGatedMostCluster][32];  // (N, R) of whole tiles
  __shared__ f2 carry[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int K = p.cluster, rank = blockIdx.x % K, unit = blockIdx.x / K;
  const int ct = unit % p.channel_tiles, b = unit / p.channel_tiles;
  const int c0 = ct * kGatedCh + (PAIR ? 2 * lane : lane), c1 = c0 + (PAIR ? 1 : 32);
  const bool ok0 = c0 < p.dim, ok1 = c1 < p.dim;
  const float2 most = make_float2(ok0 ? -p.rate * softplus_f(p.decay[c0]) : 0.f, ok1 ? -p.rate * softplus_f(p.decay[c1]) : 0.f);
  const bool near = __all_sync(~0u, most.x >= -0.5f && most.y >= -0.5f);
  const f2 open = pk(most);  // L of an open gate
  const T *const x = static_cast<const T *>(p.x) + b * p.sx[0] + c0;
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + c0;
  const T *const igate = IG ? static_cast<const T *>(p.igate) + b * p.si[0] + c0 : nullptr;
  const T *const dout = static_cast<const T *>(p.dout) + b * p.sd[0] + c0;
  T *const dx = p.dx ? static_cast<T *>(p.dx) + b * p.sdx[0] + c0 : nullptr;
  T *const dgate = p.dgate ? static_cast<T *>(p.dgate) + b * p.sdg[0] + c0 : nullptr;
  T *const digate = IG && p.digate ? static_cast<T *>(p.digate) + b * p.sdi[0] + c0 : nullptr;
  auto pair_at = [&](const float *q) { return pk(ok0 ? q[c0] : 0.f, ok1 ? q[c1] : 0.f); };

  Two<T, PAIR> rx[kSteps], rg[kSteps], ri[IG ? kSteps : 1], rd[kSteps];
  f2 next = 0;  // the state before the tile that comes next
  auto load = [&](int tile) {
    const int t0 = tile * kGatedTile + warp * kSteps;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const bool in = t0 + j < p.tokens;
      const long long t = t0 + j;
      rx[j].load(x + t * p.sx[1], ok0 && in, ok1 && in);
      rg[j].load(gate + t * p.sg[1], ok0 && in, ok1 && in);
      if constexpr (IG) ri[j].load(igate + t * p.si[1], ok0 && in, ok1 && in);
      rd[j].load(dout + t * p.sd[1], ok0 && in, ok1 && in);
    }
    next = tile < p.tiles ? pair_at(p.kept + ((long long)b * p.tiles + tile) * p.dim) : 0;
  };
  const int rounds = (p.tiles + K - 1) / K;
  load((rounds - 1) * K + rank);
  f2 e = 0, sum = 0;
  if (p.dlast) e = pair_at(p.dlast + (long long)b * p.dim);
  if (K > 1) cluster_sync();
  const f2 one = both(1.f), minus = both(-1.f);
  for (int it = rounds - 1; it >= 0; --it) {
    const int buf = it & 1, tile = it * K + rank, t0 = tile * kGatedTile + warp * kSteps;
    f2 xv[kSteps], d[kSteps], r[kSteps], i[kSteps], n[kSteps], root[kSteps], inv[kSteps], h[kSteps];
    f2 N = 0, E = 0, R = 0, start = next;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      xv[j] = rx[j].widen();
      d[j] = rd[j].widen();
      r[j] = sigmoid2(rg[j].widen());
      i[j] = one;
      if constexpr (IG) i[j] = sigmoid2(ri[j].widen());
      if (t0 + j >= p.tokens) r[j] = 0;  // past the end: L = 0, a = 1, and x = dout = 0
      n[j] = decay2(mul2(open, r[j]), near);
      root[j] = root2(n[j], inv[j]);
      h[j] = mul2(root[j], mul2(i[j], xv[j]));  // b; the state before later
      N = step2(n[j], N, n[j]);
      E = step2(n[j], E, h[j]);
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      const f2 g = add2(d[j], R);
      R = fma2(n[j], g, g);
    }
    if (it > 0) load(tile - K);
    prod[buf][warp][lane] = N;
    fwd[buf][warp][lane] = E;
    rev[buf][warp][lane] = R;
    __syncthreads();
    if (K > 1) {
      if (warp == 0) {
        ulonglong2 all = make_ulonglong2(0, 0);
#pragma unroll
        for (int w = kWarps - 1; w >= 0; --w) {
          const f2 q = prod[buf][w][lane];
          all.y = step2(q, all.y, rev[buf][w][lane]);
          all.x = step2(q, all.x, q);
        }
        for (int c = 0; c < K; ++c) store_remote(&tiles[buf][rank][lane], c, all);
      }
      cluster_sync();
    }
    if (it + 1 < rounds) e = carry[buf ^ 1][lane];
    for (int c = K - 1; c > rank; --c) {
      const ulonglong2 q = tiles[buf][c][lane];
      e = step2(q.x, e, q.y);
    }
#pragma unroll
    for (int w = kWarps - 1; w > 0; --w)
      if (w > warp) e = step2(prod[buf][w][lane], e, rev[buf][w][lane]);
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) start = step2(prod[buf][w][lane], start, fwd[buf][w][lane]);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const f2 v = h[j];
      h[j] = start;
      start = step2(n[j], start, v);
    }
#pragma unroll
    for (int j = kSteps - 1; j >= 0; --j) {
      const f2 g = add2(d[j], e), a = add2(n[j], one), L = mul2(open, r[j]), u = mul2(i[j], xv[j]);
      e = fma2(n[j], g, g);
      // G = g L a (h - u a / sqrt(1 - a^2))
      const f2 G = mul2(mul2(g, mul2(L, a)), fma2(mul2(mul2(u, a), inv[j]), minus, h[j]));
      sum = add2(sum, G);
      if (t0 + j < p.tokens) {
        const long long t = t0 + j;
        const f2 gr = mul2(g, root[j]);
        if (dx) Two<T, PAIR>::store(dx + t * p.sdx[1], upk(mul2(gr, i[j])), ok0, ok1);
        if (dgate) Two<T, PAIR>::store(dgate + t * p.sdg[1], upk(mul2(G, fma2(r[j], minus, one))), ok0, ok1);
        if (IG && digate) Two<T, PAIR>::store(digate + t * p.sdi[1], upk(mul2(mul2(gr, u), fma2(i[j], minus, one))), ok0, ok1);
      }
    }
    if (warp == 0) {
      if (K == 1) {
        carry[buf][lane] = e;
      } else if (rank == 0) {
        for (int c = 0; c < K; ++c) store_remote(&carry[buf][lane], c, e);
      }
    }
  }
  auto put_pair = [&](float *q, f2 v) {
    const float2 w = upk(v);
    if (ok0) q[c0] = w.x;
    if (ok1) q[c1] = w.y;
  };
  if (p.dinit && rank == 0 && warp == 0) put_pair(p.dinit + (long long)b * p.dim, e);
  __syncthreads();
  prod[0][warp][lane] = sum;
  __syncthreads();
  if (p.parts && warp == 0) {
    f2 s = prod[0][0][lane];
    for (int w = 1; w < kWarps; ++w) s = add2(s, prod[0][w][lane]);
    put_pair(p.parts + ((long long)b * K + rank) * p.dim, s);
  }
  if (K > 1) cluster_sync();
}

// ddecay = sigmoid(decay) / softplus(decay) times the sum over the parts.
__global__ void __launch_bounds__(256) ss_gated_ddecay_kernel(const float *parts, int n, int dim, const float *decay, float *ddecay) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < dim)
    for (int k = warp; k < n; k += 8) s += parts[(long long)k * dim + c];
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < dim) {
    s = 0.f;
    for (int w = 0; w < 8; ++w) s += sums[w][lane];
    const float v = decay[c];
    // far below 0 both are e^decay
    const float ratio = v < -20.f ? 1.f : __fdividef(rcp(1.f + ex2(-v * kLog2e)), softplus_f(v));
    ddecay[c] = s * ratio;
  }
}

template <typename T, bool PAIR, bool IG>
cudaError_t launch(const GatedBwdParams &p, cudaStream_t s) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)p.batch * p.channel_tiles * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster > 1;
  return cudaLaunchKernelEx(&cfg, ss_gated_bwd_kernel<T, PAIR, IG>, p);
}
template <typename T>
cudaError_t pick(bool pair, const GatedBwdParams &p, cudaStream_t s) {
  if (pair) return p.igate ? launch<T, true, true>(p, s) : launch<T, true, false>(p, s);
  return p.igate ? launch<T, false, true>(p, s) : launch<T, false, false>(p, s);
}

}  // namespace

cudaError_t launch_gated_bwd(int dtype, bool pair, const GatedBwdParams &p, cudaStream_t s) {
  cudaError_t e = dtype == 0 ? pick<float>(pair, p, s) : dtype == 1 ? pick<__half>(pair, p, s) : pick<__nv_bfloat16>(pair, p, s);
  if (e != cudaSuccess || !p.ddecay) return e;
  ss_gated_ddecay_kernel<<<(p.dim + 31) / 32, 256, 0, s>>>(p.parts, p.batch * p.cluster, p.dim, p.decay, p.ddecay);
  return cudaGetLastError();
}

}  // namespace ssk
