// Selective scan with one decay per head over packed requests
// (include/ssfwd_packed.h): the form that takes every type and size, token by
// token in fp32. Per request and head, with S (headdim x dstate):
//   S = exp(dt A) S + dt x B^T;  y = S C + D x;  out = y silu(z).
//
// One CTA carries 64 (or 32) rows of one head's state in registers through one
// block of a request (16 lanes a row), and stages 16 tokens at a time in shared
// memory. It is bound by the fp32 operations, three for every state value
// and token. When requests may have several blocks, a first launch brings every
// block but the last from zero (the first one from the request's start) to its
// end, a second one carries these ends on from block to block, and the third
// starts every block where the one before it ends. 4096 ragged tokens x 24 heads of
// 64 with 128 states in fp32: 304 us.
#include "ss_fwd_kernel.cuh"
#include "ss_packed.h"

namespace ssk {
namespace {

constexpr int kLanes = 16, kScanThreads = 256, kTokens = 16;

// NPL states and RPL rows per lane.
template <typename T, int NPL, int RPL, bool SUMMARY>
__global__ void __launch_bounds__(kScanThreads) ss_head_scan_kernel(const __grid_constant__ HeadScanParams p) {
  constexpr int V = NPL < 4 ? NPL : 4, Q = NPL / V, NP = kLanes * NPL, NF = (NPL + 1) / 2;
  constexpr int kRows = kScanThreads / kLanes * RPL;
  __shared__ __align__(16) float xs[kTokens][kRows];
  __shared__ __align__(16) float bs[kTokens][NP];
  __shared__ __align__(16) float cs[SUMMARY ? 1 : kTokens][NP];
  __shared__ float ys[SUMMARY ? 1 : kTokens][kRows];
  __shared__ float dts[kTokens], keeps[kTokens];
  const int tid = threadIdx.x, j = tid % kLanes, rg = tid / kLanes;
  const int ptiles = (p.headdim + kRows - 1) / kRows;
  const int h = blockIdx.y / ptiles, p0 = (blockIdx.y % ptiles) * kRows;
  const int prow = min(kRows, p.headdim - p0);
  const int g = h / p.hpg;
  T *out = static_cast<T *>(p.out) + h * p.so[1] + p0;
  if (!SUMMARY && (int)blockIdx.x == p.t.max_blocks) {  // past the last token: zeros
    for (int t = p.t.counts[0]; t < p.t.tokens; ++t)
      for (int i = tid; i < prow; i += kScanThreads) out[t * p.so[0] + i] = from_f<T>(0.f);
    return;
  }
  if (SUMMARY) let_next_start(); else wait_for_previous();
  const int blk = SUMMARY ? p.t.carried[blockIdx.x] : blockIdx.x;
  if (blk < 0) return;
  const int4 row = reinterpret_cast<const int4 *>(p.t.blocks)[blk];
  const int r = row.x, first = row.y, size = row.z, index = row.w;
  if (r < 0) return;
  const int len = p.t.offsets[r + 1] - p.t.offsets[r];
  const int last = (len - 1) / p.t.block;  // index of the request's last block
  const int slot0 = p.state ? p.t.slot_map[r] : -1;
  const bool kept = slot0 >= 0 && slot0 < p.slots;
  const bool goes_on = kept && p.t.context && p.t.context[r] > 0;
  float *cache = kept ? p.state + slot0 * p.ss[0] + h * p.ss[1] + (long long)p0 * p.dstate : nullptr;
  const long long pn = (long long)p.headdim * p.dstate;
  auto entry = [&](int i) {  // summary of the request's block i
    return p.ws_state + ((long long)(blk - index + i) * p.heads + h) * pn + (long long)p0 * p.dstate;
  };
  auto decay_of = [&](int i) { return p.ws_decay + (long long)(blk - index + i) * p.heads + h; };

  f2 s[RPL][NF];  // pairs of states; a lone one is paired with 0
  auto each = [&](auto f) {  // f(is one, offset of row and state, value)
#pragma unroll
    for (int u = 0; u < RPL; ++u)
#pragma unroll
      for (int k = 0; k < NF; ++k) {
        float2 v = upk(s[u][k]);
        const int pr = rg * RPL + u, n = V * (j + kLanes * (2 * k / V)) + 2 * k % V;
        f(pr < prow && n < p.dstate, (long long)pr * p.dstate + n, v.x);
        if (NPL > 1) f(pr < prow && n + 1 < p.dstate, (long long)pr * p.dstate + n + 1, v.y);
        s[u][k] = pk(v.x, v.y);
      }
  };
#pragma unroll
  for (int u = 0; u < RPL; ++u)
#pragma unroll
    for (int k = 0; k < NF; ++k) s[u][k] = pk(0.f, 0.f);
  auto load = [&](const float *src) {
    each([&](bool in, long long at, float &v) { v = src && in ? src[at] : 0.f; });
  };
  auto store = [&](float *dst) {
    each([&](bool in, long long at, float &v) { if (in) dst[at] = v; });
  };
  if (SUMMARY) {
    load(index == 0 && goes_on ? cache : nullptr);
    // the last block's entry keeps the start, which the cache loses when that block ends
    if (index == 0 && goes_on) store(entry(last));
  } else if (index == 0) {
    load(goes_on ? (last > 0 ? entry(last) : cache) : nullptr);
  } else {
    load(entry(index - 1));
  }

  const float A = p.A[h], bias = p.bias ? p.bias[h] : 0.f, skip = p.D ? p.D[h] : 0.f;
  const T *x = static_cast<const T *>(p.x) + h * p.sx[1] + p0;
  const T *z = p.z ? static_cast<const T *>(p.z) + h * p.sz[1] + p0 : nullptr;
  const T *B = static_cast<const T *>(p.B) + g * p.sB[1], *C = static_cast<const T *>(p.C) + g * p.sC[1];
  float decay = 0.f;
  for (int base = 0; base < size; base += kTokens) {
    const int n_tok = min(kTokens, size - base);
    const long long t0 = first + base;
    __syncthreads();
    for (int i = tid; i < kTokens * kRows; i += kScanThreads) {
      const int t = i / kRows, k = i % kRows;
      xs[t][k] = t < n_tok && k < prow ? to_f<T>(x[(t0 + t) * p.sx[0] + k]) : 0.f;
    }
    for (int i = tid; i < kTokens * NP; i += kScanThreads) {
      const int t = i / NP, k = i % NP;
      const bool in = t < n_tok && k < p.dstate;
      bs[t][k] = in ? to_f<T>(B[(t0 + t) * p.sB[0] + k]) : 0.f;
      if (!SUMMARY) cs[t][k] = in ? to_f<T>(C[(t0 + t) * p.sC[0] + k]) : 0.f;
    }
    if (tid < n_tok) {
      const long long at = (t0 + tid) * p.sdt[0] + h * p.sdt[1];
      float dt = bias + (p.dt_f32 ? static_cast<const float *>(p.dt)[at] : to_f<T>(static_cast<const T *>(p.dt)[at]));
      if (p.softplus) dt = softplus_f(dt);
      dts[tid] = dt;
      keeps[tid] = dt * A * kLog2e;
    }
    __syncthreads();
    for (int t = 0; t < n_tok; ++t) {
      const float dt = dts[t], keep = ex2(keeps[t]);
      decay += keeps[t];
      const f2 keep2 = pk(keep, keep);
      f2 b[NF], c[NF];
      auto pairs = [&](const float *src, f2 (&v)[NF]) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const float *at = src + V * (j + kLanes * q);
          if constexpr (V == 4) {
            const float4 f = *reinterpret_cast<const float4 *>(at);
            v[2 * q] = pk(f.x, f.y);
            v[2 * q + 1] = pk(f.z, f.w);
          } else if constexpr (V == 2) {
            const float2 f = *reinterpret_cast<const float2 *>(at);
            v[q] = pk(f.x, f.y);
          } else {
            v[q] = pk(*at, 0.f);
          }
        }
      };
      pairs(bs[t], b);
      if (!SUMMARY) pairs(cs[t], c);
      float y[RPL];
#pragma unroll
      for (int u = 0; u < RPL; ++u) {
        const float in = dt * xs[t][rg * RPL + u];
        const f2 in2 = pk(in, in);
        f2 acc = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NF; ++k) {
          s[u][k] = fma2(keep2, s[u][k], mul2(in2, b[k]));
          if (!SUMMARY) acc = fma2(c[k], s[u][k], acc);
        }
        const float2 a = upk(acc);
        y[u] = a.x + a.y;
      }
      if (!SUMMARY) {
        // sums over the 16 lanes: with several rows a lane hands half of them over at
        // each exchange, until it has one
        int row = rg * RPL;
        if constexpr (RPL == 4) {
          const bool up = j & 8;
          const float a0 = up ? y[0] : y[2], a1 = up ? y[1] : y[3];
          const float k0 = up ? y[2] : y[0], k1 = up ? y[3] : y[1];
          y[0] = k0 + __shfl_xor_sync(0xffffffffu, a0, 8);
          y[1] = k1 + __shfl_xor_sync(0xffffffffu, a1, 8);
          row += up ? 2 : 0;
        }
        constexpr int kPair = RPL == 4 ? 4 : 8;  // the exchange that leaves one row of two
        if constexpr (RPL >= 2) {
          const bool up = j & kPair;
          const float a = up ? y[0] : y[1], k = up ? y[1] : y[0];
          y[0] = k + __shfl_xor_sync(0xffffffffu, a, kPair);
          row += up ? 1 : 0;
        }
#pragma unroll
        for (int o = RPL >= 2 ? kPair / 2 : 8; o > 0; o >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
        if (j % (kLanes / RPL) == 0) ys[t][row] = y[0];
      }
    }
    if (!SUMMARY) {
      __syncthreads();
      for (int i = tid; i < n_tok * kRows; i += kScanThreads) {
        const int t = i / kRows, k = i % kRows;
        if (k < prow) {
          float v = fmaf(skip, xs[t][k], ys[t][k]);
          if (z) v *= silu_f(to_f<T>(z[(t0 + t) * p.sz[0] + k]));
          out[(t0 + t) * p.so[0] + k] = from_f<T>(v);
        }
      }
    }
  }
  if (SUMMARY) {
    store(entry(index));
    if (tid == 0 && p0 == 0) *decay_of(index) = decay;
  } else if (index == last && kept) {
    store(cache);
  }
}

// One thread: 4 values of one head's state, along a request's blocks. The loads
// do not wait for one another, only the sums do.
__global__ void __launch_bounds__(256) ss_head_scan_carry_kernel(const __grid_constant__ HeadScanParams p, int pieces) {
  let_next_start();
  wait_for_previous();
  const int blk = p.t.carried[blockIdx.x / (p.heads * pieces)], rest = blockIdx.x % (p.heads * pieces), h = rest / pieces;
  if (blk < 0) return;
  const int4 row = reinterpret_cast<const int4 *>(p.t.blocks)[blk];
  if (row.w != 0) return;
  const int last = (p.t.offsets[row.x + 1] - p.t.offsets[row.x] - 1) / p.t.block;
  const int pn = p.headdim * p.dstate, n = ((rest % pieces) * 256 + threadIdx.x) * 4;
  if (last < 2 || n >= pn) return;
  const long long step = (long long)p.heads * pn;
  float *e = p.ws_state + ((long long)blk * p.heads + h) * pn + n;
  const float *decay = p.ws_decay + (long long)blk * p.heads + h;
  const bool vec = pn % 4 == 0;
  float v[4] = {};
  auto get = [&](const float *src, float (&f)[4]) {
    if (vec) {
      const float4 q = *reinterpret_cast<const float4 *>(src);
      f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
    } else {
      for (int k = 0; k < 4; ++k) f[k] = n + k < pn ? src[k] : 0.f;
    }
  };
  get(e, v);
#pragma unroll 4
  for (int i = 1; i < last; ++i) {
    e += step;
    float f[4];
    get(e, f);
    const float keep = ex2(decay[(long long)i * p.heads]);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = fmaf(keep, v[k], f[k]);
    if (vec) {
      *reinterpret_cast<float4 *>(e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      for (int k = 0; k < 4; ++k)
        if (n + k < pn) e[k] = v[k];
    }
  }
}

template <typename T, int NPL, int RPL>
cudaError_t go(const HeadScanParams &p, cudaStream_t s) {
  constexpr int rows = kScanThreads / kLanes * RPL;
  const dim3 grid(p.t.max_blocks + 1, p.heads * ((p.headdim + rows - 1) / rows));
  if (p.split) {
    ss_head_scan_kernel<T, NPL, RPL, true><<<dim3(p.t.tokens / p.t.block, grid.y), kScanThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_head_scan_carry(p, s);
    if (e != cudaSuccess) return e;  // the scan would start from what no one has written
  }
  return launch_after(ss_head_scan_kernel<T, NPL, RPL, false>, grid, kScanThreads, 0, s, p.split, p);
}
template <typename T, int RPL>
cudaError_t by_states(const HeadScanParams &p, cudaStream_t s) {
  if (p.dstate > 128) return go<T, 16, RPL>(p, s);
  if (p.dstate > 64) return go<T, 8, RPL>(p, s);
  if (p.dstate > 32) return go<T, 4, RPL>(p, s);
  if (p.dstate > 16) return go<T, 2, RPL>(p, s);
  return go<T, 1, RPL>(p, s);
}
// 64 rows of a head's state per CTA, or 32 where that leaves fewer rows empty
template <typename T>
cudaError_t by_rows(const HeadScanParams &p, cudaStream_t s) {
  return (p.headdim + 31) / 32 % 2 ? by_states<T, 2>(p, s) : by_states<T, 4>(p, s);
}

}  // namespace

cudaError_t launch_head_scan_carry(const HeadScanParams &p, cudaStream_t s) {
  return launch_after(ss_head_scan_carry_kernel, dim3((unsigned)head_scan_carry_ctas(p)), 256, 0, s, true, p,
                      head_scan_carry_pieces(p));
}

cudaError_t launch_head_scan(int dtype, const HeadScanParams &p, cudaStream_t s) {
  if (dtype == 0) return by_rows<float>(p, s);
  return dtype == 1 ? by_rows<__half>(p, s) : by_rows<__nv_bfloat16>(p, s);
}

}  // namespace ssk
