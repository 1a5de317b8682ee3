// Short causal depthwise convolution of packed requests, in the (tokens,
// channels) layout that a projection leaves, and its one-token step by slot
// (include/ssfwd_packed.h). For token t of a request, channel c, width W:
//   out[t,c] = act(bias[c] + sum_{k<W} weight[c,k] * x[t-(W-1)+k, c])
// with the request's kept window (or zeros) before its first token.
//
// Both are bound by memory traffic: x in, out out. A thread owns V adjacent
// channels (one 16-byte access) and walks a run of tokens with the last W-1
// inputs in registers, so an input is read from memory once, but for the W-1
// rows before each run. The thread that has a request's first token also takes
// its first W-1 ones past the end of its run, so that it alone reads the kept
// window and can replace it at once: the exchange needs no second pass.
// 16384 x 1792 bf16, width 4: 26.9 us, 4.4 TB/s (65% of the copy bandwidth); the
// step at 512 x 5376: 14.3 us, 3.1 TB/s.
#include "ss_fwd_kernel.cuh"
#include "ss_packed.h"

namespace ssk {
namespace {

constexpr int kConvCta = 128;

// V values as they are stored: one 16-byte access, or one value.
template <typename T, int V>
struct Raw {
  uint4 q;
  __device__ __forceinline__ void load(const T *src) { q = *reinterpret_cast<const uint4 *>(src); }
  __device__ __forceinline__ void widen(float (&v)[V]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = unpack2<T>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T x;
  __device__ __forceinline__ void load(const T *src) { x = *src; }
  __device__ __forceinline__ void widen(float (&v)[1]) const { v[0] = to_f<T>(x); }
};
template <typename T, int V>
__device__ __forceinline__ void load_v(const T *src, float (&v)[V]) {
  Raw<T, V> r;
  r.load(src);
  r.widen(v);
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T *dst, const float (&v)[V]) {
  if constexpr (V == 1) {
    *dst = from_f<T>(v[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
      else w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
    }
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// V channels' windows (V x H values, contiguous) as V values per tap.
template <typename T, int V, int H>
__device__ __forceinline__ void load_window(const T *src, float (&win)[H][V]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int k = 0; k < H; ++k) win[k][0] = to_f<T>(src[k]);
  } else {
    float flat[V * H];
#pragma unroll
    for (int q = 0; q < H; ++q) {
      float part[V];
      load_v<T, V>(src + q * V, part);
#pragma unroll
      for (int i = 0; i < V; ++i) flat[q * V + i] = part[i];
    }
#pragma unroll
    for (int k = 0; k < H; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) win[k][i] = flat[i * H + k];
  }
}

template <typename T, int V, int H>
__device__ __forceinline__ void store_window(T *dst, const float (&win)[H][V]) {
  float flat[V * H];
#pragma unroll
  for (int k = 0; k < H; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) flat[i * H + k] = win[k][i];
  if constexpr (V == 1) {
#pragma unroll
    for (int k = 0; k < H; ++k) dst[k] = from_f<T>(flat[k]);
  } else {
#pragma unroll
    for (int q = 0; q < H; ++q) {
      float part[V];
#pragma unroll
      for (int i = 0; i < V; ++i) part[i] = flat[q * V + i];
      store_v<T, V>(dst + q * V, part);
    }
  }
}

// Taps and bias of V channels (V x W contiguous values).
template <int V, int W>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int c, float (&w)[W][V], float (&b)[V]) {
  const float *src = weight + (long long)c * W;
  if (V > 1 && reinterpret_cast<uintptr_t>(weight) % 16 == 0) {
    float flat[V * W];
#pragma unroll
    for (int q = 0; q < V * W / 4; ++q) {
      const float4 f = reinterpret_cast<const float4 *>(src)[q];
      flat[4 * q] = f.x;
      flat[4 * q + 1] = f.y;
      flat[4 * q + 2] = f.z;
      flat[4 * q + 3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = flat[i * W + k];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = src[i * W + k];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = bias ? bias[c + i] : 0.f;
}

// One output of V channels from their window and the new input, which the window takes in.
template <int V, int W>
__device__ __forceinline__ void advance(const float (&w)[W][V], const float (&b)[V], float (&win)[W - 1][V], const float (&v)[V],
                                        int act, float (&y)[V]) {
  constexpr int H = W - 1;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float acc = b[i];
#pragma unroll
    for (int k = 0; k < H; ++k) acc = fmaf(w[k][i], win[k][i], acc);
    acc = fmaf(w[H][i], v[i], acc);
    y[i] = act ? silu_f(acc) : acc;
#pragma unroll
    for (int k = 0; k + 1 < H; ++k) win[k][i] = win[k + 1][i];
    win[H - 1][i] = v[i];
  }
}

// `run` tokens per thread, loaded STEP at a time. What is particular about a
// request's start stands once, outside the loop over its tokens: inside it, it
// is repeated for every unrolled token and the loop no longer fits the
// instruction cache (125 us instead of 31 at 16384 x 1792 bf16).
template <typename T, int V, int W, int STEP>
__global__ void __launch_bounds__(kConvCta, V == 1 ? 4 : 3) ss_packed_conv1d_kernel(const __grid_constant__ PackedConvParams p, const int run) {
  constexpr int H = W - 1;
  // a warp is 32 channel pieces wide, so that few lanes pass the last channel
  const int c = (blockIdx.y * 32 + (threadIdx.x & 31)) * V;
  const int t0 = (blockIdx.x * (kConvCta / 32) + (threadIdx.x >> 5)) * run;
  if (c >= p.dim || t0 >= p.t.tokens) return;
  int t1 = min(t0 + run, p.t.tokens);
  const T *x = static_cast<const T *>(p.x) + c;
  T *out = static_cast<T *>(p.out) + c;
  float w[W][V], b[V], win[H][V];
  const int live = p.t.offsets[p.t.requests];
  int r = p.t.token_request[t0];
  const int rl = p.t.token_request[t1 - 1];
  load_taps<V, W>(p.weight, p.bias, c, w, b);
  int t = t0, first = 0, end = t0;  // the request's tokens are [first, end)
  if (r >= 0) {
    first = p.t.offsets[r];
    end = p.t.offsets[r + 1];
    // a request's first H tokens belong to the thread that has its first one
    if (first < t0 && t0 - first < H) t = min(first + H, end);
  }
  if (rl >= 0) {
    const int f = p.t.offsets[rl], e = p.t.offsets[rl + 1];
    if (t1 - f < H) t1 = max(t1, min(f + H, e));
  }
  if (r >= 0 && t < end && t != first) {
#pragma unroll
    for (int j = 0; j < H; ++j) load_v<T, V>(x + (long long)(t - H + j) * p.sx, win[j]);
  }
  const int stop = min(t1, live);
#pragma unroll 1
  while (t < stop) {
    if (t >= end) {  // on to the next request that has tokens
      do ++r; while (p.t.offsets[r + 1] <= t);
      first = t;
      end = p.t.offsets[r + 1];
    }
    if (t == first) {
      const int slot = p.state ? p.t.slot_map[r] : -1;
      T *kept = slot < 0 || slot >= p.slots ? nullptr : static_cast<T *>(p.state) + slot * p.ss + (long long)c * H;
      if (kept && p.t.context && p.t.context[r] > 0) {
        load_window<T, V, H>(kept, win);
      } else {
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) win[j][i] = 0.f;
      }
      if (kept) {  // and the window that the request leaves behind
        float nw[H][V];
#pragma unroll
        for (int j = 0; j < H; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) nw[j][i] = win[j][i];
        const int from = max(first, end - H), count = end - from;  // the last inputs, at most H
#pragma unroll
        for (int k = 0; k < H; ++k)
          if (k < count) {
#pragma unroll
            for (int j = 0; j + 1 < H; ++j)
#pragma unroll
              for (int i = 0; i < V; ++i) nw[j][i] = nw[j + 1][i];
            load_v<T, V>(x + (long long)(from + k) * p.sx, nw[H - 1]);
          }
        store_window<T, V, H>(kept, nw);
      }
    }
    const int to = min(end, stop);
    const T *xp = x + (long long)t * p.sx;
    T *op = out + (long long)t * p.so;
#pragma unroll 1
    for (; t + STEP <= to; t += STEP) {
      Raw<T, V> in[STEP];
#pragma unroll
      for (int s = 0; s < STEP; ++s) in[s].load(xp + s * p.sx);
#pragma unroll
      for (int s = 0; s < STEP; ++s) {
        float v[V], y[V];
        in[s].widen(v);
        advance<V, W>(w, b, win, v, p.act, y);
        store_v<T, V>(op + s * p.so, y);
      }
      xp += STEP * p.sx;
      op += STEP * p.so;
    }
#pragma unroll 1
    for (; t < to; ++t) {
      float v[V], y[V];
      load_v<T, V>(xp, v);
      advance<V, W>(w, b, win, v, p.act, y);
      store_v<T, V>(op, y);
      xp += p.sx;
      op += p.so;
    }
  }
  const float zero[V] = {};
#pragma unroll 1
  for (t = max(t0, live); t < min(t0 + run, p.t.tokens); ++t) store_v<T, V>(out + (long long)t * p.so, zero);
}

// ROWS requests per thread, one after another on the same taps; the loads of all
// of them are under way before the first is used.
template <typename T, int V, int W, int ROWS>
__global__ void __launch_bounds__(kConvCta) ss_packed_conv1d_update_kernel(const __grid_constant__ PackedConvUpdateParams p) {
  constexpr int H = W - 1;
  const int c = (blockIdx.y * kConvCta + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int r0 = blockIdx.x * ROWS;
  int slot[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = r0 + i;
    slot[i] = r >= p.requests ? -1 : p.slot_map ? p.slot_map[r] : r;
  }
  float w[W][V], b[V], win[ROWS][H][V];
  Raw<T, V> in[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (r0 + i < p.requests) in[i].load(static_cast<const T *>(p.x) + (r0 + i) * p.sx + c);
    if (slot[i] >= 0 && slot[i] < p.slots)
      load_window<T, V, H>(static_cast<const T *>(p.state) + slot[i] * p.ss + (long long)c * H, win[i]);
  }
  load_taps<V, W>(p.weight, p.bias, c, w, b);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (r0 + i >= p.requests) break;
    T *out = static_cast<T *>(p.out) + (r0 + i) * p.so + c;
    float y[V] = {};
    if (slot[i] >= 0 && slot[i] < p.slots) {
      float v[V];
      in[i].widen(v);
      advance<V, W>(w, b, win[i], v, p.act, y);
      store_window<T, V, H>(static_cast<T *>(p.state) + slot[i] * p.ss + (long long)c * H, win[i]);
    }
    store_v<T, V>(out, y);
  }
}

template <typename T, int V, int W>
void go(const PackedConvParams &p, cudaStream_t s) {
  // Runs that fill the SMs once: 3 CTAs of the 16-byte form fit one SM (168
  // registers a thread, for 16 loads under way; with 8 and 4 CTAs 25.3 us against
  // 24.4 at 16384 x 1792 bf16), 9 or 10 of the other (56 to 48 registers). Longer ones
  // leave SMs idle, shorter ones a part of a second wave (31.5 us against 28.8 at
  // 16384 x 1792 bf16, runs of 32 against 56).
  constexpr int STEP = V == 1 ? 8 : 16, resident = V == 1 ? 10 : 3;
  const int cols = (p.dim + 32 * V - 1) / (32 * V), warps = 152 * resident * (kConvCta / 32);
  const long long want = ((long long)p.t.tokens * cols + warps - 1) / warps;
  const int run = (int)(want < STEP ? STEP : want > 128 ? 128 : (want + STEP - 1) / STEP * STEP);
  const int per = run * (kConvCta / 32);
  ss_packed_conv1d_kernel<T, V, W, STEP><<<dim3((p.t.tokens + per - 1) / per, cols), kConvCta, 0, s>>>(p, run);
}
template <typename T, int V, int W>
void go(const PackedConvUpdateParams &p, cudaStream_t s) {
  const int cols = (p.dim + kConvCta * V - 1) / (kConvCta * V);
  // two requests per thread once that leaves each SM some CTAs: the taps are as many
  // bytes as a window (512 x 5376 bf16: 14.3 us, with one request 19.3, with four 14.8)
  if ((long long)p.requests * cols >= 8 * 152)
    ss_packed_conv1d_update_kernel<T, V, W, 2><<<dim3((p.requests + 1) / 2, cols), kConvCta, 0, s>>>(p);
  else
    ss_packed_conv1d_update_kernel<T, V, W, 1><<<dim3(p.requests, cols), kConvCta, 0, s>>>(p);
}
template <typename T, int V, typename P>
void by_width(const P &p, cudaStream_t s) {
  if (p.width == 2) go<T, V, 2>(p, s);
  else if (p.width == 3) go<T, V, 3>(p, s);
  else go<T, V, 4>(p, s);
}
template <typename P>
cudaError_t by_type(int dtype, const P &p, cudaStream_t s) {
  if (dtype == 0) {
    if (p.vec) by_width<float, 4>(p, s); else by_width<float, 1>(p, s);
  } else if (dtype == 1) {
    if (p.vec) by_width<__half, 8>(p, s); else by_width<__half, 1>(p, s);
  } else {
    if (p.vec) by_width<__nv_bfloat16, 8>(p, s); else by_width<__nv_bfloat16, 1>(p, s);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_conv(int dtype, const PackedConvParams &p, cudaStream_t s) { return by_type(dtype, p, s); }
cudaError_t launch_packed_conv_update(int dtype, const PackedConvUpdateParams &p, cudaStream_t s) {
  return by_type(dtype, p, s);
}

}  // namespace ssk
