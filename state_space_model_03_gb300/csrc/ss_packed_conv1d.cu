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
#include "ss_fwd_kernel.cuh"
#include "ss_packed.h"

namespace ssk {
namespace {

constexpr int kConvCta = 128;

template <typename T, int V>
__device__ __forceinline__ void load_v(const T *src, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f<T>(*src);
  } else {
    const uint4 q = *reinterpret_cast<const uint4 *>(src);
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

template <int V, int W>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int c, float (&w)[W][V], float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = weight[(long long)(c + i) * W + k];
    b[i] = bias ? bias[c + i] : 0.f;
  }
}

// TOK tokens per thread, loaded STEP at a time.
template <typename T, int V, int W, int TOK, int STEP>
__global__ void __launch_bounds__(kConvCta) ss_packed_conv1d_kernel(const __grid_constant__ PackedConvParams p) {
  constexpr int H = W - 1;
  const int c = (blockIdx.y * kConvCta + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int t0 = blockIdx.x * TOK;
  int t1 = min(t0 + TOK, p.t.tokens);
  const T *x = static_cast<const T *>(p.x) + c;
  T *out = static_cast<T *>(p.out) + c;
  float w[W][V], b[V], win[H][V];
  load_taps<V, W>(p.weight, p.bias, c, w, b);
  const int live = p.t.offsets[p.t.requests];
  int r = p.t.token_request[t0];
  const int rl = p.t.token_request[t1 - 1];
  int tb = t0, first = 0, end = t0;  // the request's tokens are [first, end)
  if (r >= 0) {
    first = p.t.offsets[r];
    end = p.t.offsets[r + 1];
    // a request's first H tokens belong to the thread that has its first one
    if (first < t0 && t0 - first < H) tb = min(first + H, end);
  }
  if (rl >= 0) {
    const int f = p.t.offsets[rl], e = p.t.offsets[rl + 1];
    if (t1 - f < H) t1 = max(t1, min(f + H, e));
  }
  auto kept = [&](int rr) -> T * {
    if (!p.state) return nullptr;
    const int slot = p.t.slot_map[rr];
    return slot < 0 || slot >= p.slots ? nullptr : static_cast<T *>(p.state) + slot * p.ss + (long long)c * H;
  };
  auto start_window = [&](int rr, float (&v)[H][V]) {
    T *k = kept(rr);
    if (k && p.t.context && p.t.context[rr] > 0) {
      load_window<T, V, H>(k, v);
    } else {
#pragma unroll
      for (int j = 0; j < H; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] = 0.f;
    }
  };
  // at the request's first token: the window that it leaves behind
  auto replace_window = [&](int rr, int f, int e, const float (&old)[H][V]) {
    T *k = kept(rr);
    if (!k) return;
    float nw[H][V];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      const int t = e - H + j;
      if (t >= f) {
        load_v<T, V>(x + (long long)t * p.sx, nw[j]);
      } else {  // shorter than the window: its tail moves up
#pragma unroll
        for (int o = 0; o < H; ++o)
          if (o == t - f + H) {
#pragma unroll
            for (int i = 0; i < V; ++i) nw[j][i] = old[o][i];
          }
      }
    }
    store_window<T, V, H>(k, nw);
  };
  if (r >= 0 && tb < end) {
    if (tb == first) {
      start_window(r, win);
      replace_window(r, first, end, win);
    } else {
#pragma unroll
      for (int j = 0; j < H; ++j) load_v<T, V>(x + (long long)(tb - H + j) * p.sx, win[j]);
    }
  }
  for (int t = tb; t < t1; t += STEP) {
    float v[STEP][V];
#pragma unroll
    for (int s = 0; s < STEP; ++s) {
      if (t + s < t1) {
        load_v<T, V>(x + (long long)(t + s) * p.sx, v[s]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[s][i] = 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < STEP; ++s) {
      if (t + s >= t1) break;
      if (t + s >= live) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[s][i] = 0.f;
        store_v<T, V>(out + (long long)(t + s) * p.so, v[s]);
        continue;
      }
      if (t + s == end) {
        do ++r; while (p.t.offsets[r + 1] <= t + s);
        first = end;
        end = p.t.offsets[r + 1];
        start_window(r, win);
        replace_window(r, first, end, win);
      }
      float y[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float acc = b[i];
#pragma unroll
        for (int k = 0; k < H; ++k) acc = fmaf(w[k][i], win[k][i], acc);
        acc = fmaf(w[H][i], v[s][i], acc);
        y[i] = p.act ? silu_f(acc) : acc;
      }
      store_v<T, V>(out + (long long)(t + s) * p.so, y);
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k + 1 < H; ++k) win[k][i] = win[k + 1][i];
        win[H - 1][i] = v[s][i];
      }
    }
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kConvCta) ss_packed_conv1d_update_kernel(const __grid_constant__ PackedConvUpdateParams p) {
  constexpr int H = W - 1;
  const int c = (blockIdx.y * kConvCta + threadIdx.x) * V;
  if (c >= p.dim) return;
  const int r = blockIdx.x;
  const int slot = p.slot_map ? p.slot_map[r] : r;
  float w[W][V], y[V], v[V];
  load_taps<V, W>(p.weight, p.bias, c, w, y);
  load_v<T, V>(static_cast<const T *>(p.x) + r * p.sx + c, v);
  T *out = static_cast<T *>(p.out) + r * p.so + c;
  if (slot < 0 || slot >= p.slots) {
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = 0.f;
    store_v<T, V>(out, y);
    return;
  }
  T *st = static_cast<T *>(p.state) + slot * p.ss + (long long)c * H;
  float win[H][V];
  load_window<T, V, H>(st, win);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float acc = y[i];
#pragma unroll
    for (int k = 0; k < H; ++k) acc = fmaf(w[k][i], win[k][i], acc);
    acc = fmaf(w[H][i], v[i], acc);
    y[i] = p.act ? silu_f(acc) : acc;
#pragma unroll
    for (int k = 0; k + 1 < H; ++k) win[k][i] = win[k + 1][i];
    win[H - 1][i] = v[i];
  }
  store_v<T, V>(out, y);
  store_window<T, V, H>(st, win);
}

template <typename T, int V, int W>
void go(const PackedConvParams &p, cudaStream_t s) {
  constexpr int TOK = 32, STEP = V == 1 ? 16 : 8;
  const dim3 grid((p.t.tokens + TOK - 1) / TOK, (p.dim + kConvCta * V - 1) / (kConvCta * V));
  ss_packed_conv1d_kernel<T, V, W, TOK, STEP><<<grid, kConvCta, 0, s>>>(p);
}
template <typename T, int V, int W>
void go(const PackedConvUpdateParams &p, cudaStream_t s) {
  const dim3 grid(p.requests, (p.dim + kConvCta * V - 1) / (kConvCta * V));
  ss_packed_conv1d_update_kernel<T, V, W><<<grid, kConvCta, 0, s>>>(p);
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
