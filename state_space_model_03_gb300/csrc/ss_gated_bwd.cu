// Backward of the gated linear recurrence (include/ssfwd_layer.h). With e_t what
// token t hands back to the state before it,
//   g_t = dout_t + e_{t+1},  e_t = a_t g_t = g_t + n_t g_t,
// the same kind of recurrence as the forward's, backwards, with a token's own a. The
// states h_{t-1} that the decays' gradients need are taken up again in fp32 from the
// one that the forward kept before each tile of 64 tokens (1/32 of an operand in 16
// bits), so that both recurrences are local to a tile but for e.
//
// Tiles, runs, clusters and segments are the forward's, the tiles in falling order. A run's map
// has three parts: N (both directions'), the forward's end and the backward's. Of a
// token, n, the state before it and 1 / sqrt(1 - a^2) stay in registers; its gates are
// taken again from the tile in shared memory for the gradients, which costs less than
// registers that would halve the CTAs of an SM. The sum over tokens for the decay's
// gradient stays in registers (fp32: a lane adds an eighth of its CTA's tokens one after
// the other, 2^-24 of the root of their number off), then goes by CTA to the workspace and
// is added up by a second launch: no atomics, the same result in every call.
//
// 8 x 2048 x 2560 bf16: 120 us, 4.9 TB/s (72% of the copy), five CTAs an SM, so that 640
// run at once; with places of their own for the gradients (four an SM, two rounds) 142.
// Bound by latency at 17 warps an SM and by their uneven share, as the forward: 132
// instructions a token and pair of channels, 18 of them on the special-function unit, at
// 0.65 of the issue rate, DRAM at 0.54.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kStages = 2;
constexpr int G = 4;  // tokens whose gates are taken side by side

struct BwdMaps {
  CUtensorMap x, gate, igate, dout, dx, dgate, digate;
};
template <typename T>
struct BwdSmem {
  // x, gate, input gate and dout of a tile; where a token's have been used, its gradients
  // dx, dgate and dinput_gate take their place and leave from there
  T rows[kStages][4][kGatedTile][kGatedCh];
  uint64_t full[kStages];
};

// The maps (N, R) of all segments but the first: each half warp takes a part of the
// segment's tokens that no other comes between.
template <typename T, bool PAIR>
__global__ void __launch_bounds__(kGatedThreads, 4) ss_gated_bwd_maps_kernel(const __grid_constant__ GatedBwdParams p) {
  __shared__ ulonglong2 maps[kRuns][16];
  let_next_start();
  const int segs = p.plan.segs - 1, seg = blockIdx.x % segs + 1, unit = blockIdx.x / segs;
  const int ct = unit % p.channel_tiles, b = unit / p.channel_tiles, l = threadIdx.x & 15, run = threadIdx.x >> 4;
  const int c0 = ct * kGatedCh + (PAIR ? 2 * l : l), c1 = c0 + (PAIR ? 1 : 16);
  const bool ok0 = c0 < p.dim, ok1 = c1 < p.dim;
  const float2 most = make_float2(ok0 ? -p.rate * softplus_f(p.decay[c0]) : 0.f, ok1 ? -p.rate * softplus_f(p.decay[c1]) : 0.f);
  const bool near = __all_sync(~0u, most.x >= -0.5f && most.y >= -0.5f);
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + c0;
  const T *const dout = static_cast<const T *>(p.dout) + b * p.sd[0] + c0;
  const int tokens = p.plan.seg_tiles * kGatedTile, end = min(p.tokens, (seg + 1) * tokens);
  const int steps = (tokens + kGatedTile - 1) / kGatedTile, first = seg * tokens + run * steps * kRun;
  Two<T, PAIR> rg[kRun], rd[kRun];
  auto load = [&](int k) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const long long t = first + k * kRun + j;
      const bool in = t < end;
      rg[j].load(gate + t * p.sg[1], ok0 && in, ok1 && in);
      rd[j].load(dout + t * p.sd[1], ok0 && in, ok1 && in);
    }
  };
  load(steps - 1);
  f2 N = 0, R = 0;
#pragma unroll 1
  for (int k = steps - 1; k >= 0; --k) {
    f2 L[kRun], n[kRun], d[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      L[j] = rg[j].widen();
      d[j] = rd[j].widen();
    }
    if (k > 0) load(k - 1);
    sigmoid2(L);
#pragma unroll
    for (int j = 0; j < kRun; ++j) L[j] = first + k * kRun + j < end ? mul2(pk(most), L[j]) : 0;
    decay2(L, near, n);
#pragma unroll
    for (int j = kRun - 1; j >= 0; --j) {
      const f2 g = add2(d[j], R);
      R = fma2(n[j], g, g);
      N = step2(n[j], N, n[j]);
    }
  }
  maps[run][l] = make_ulonglong2(N, R);
  __syncthreads();
  if (threadIdx.x < 16) {
    N = R = 0;
#pragma unroll
    for (int r = kRuns - 1; r >= 0; --r) {
      const ulonglong2 q = maps[r][l];
      R = step2(q.x, R, q.y);
      N = step2(q.x, N, q.x);
    }
    *(segment_maps(p.maps, unit, p.plan.segs, seg) + l) = make_ulonglong2(N, R);
  }
}

template <typename T, int ROWS, bool IG, bool CL>
__global__ void __launch_bounds__(kGatedThreads, ROWS != kTma ? 3 : sizeof(T) == 4 ? 3 : 5)
    ss_gated_bwd_kernel(const __grid_constant__ GatedBwdParams p, const __grid_constant__ BwdMaps tm) {
  constexpr int S = kRun;
  constexpr bool TMA = ROWS == kTma, PAIR = ROWS != kSingles;
  extern __shared__ __align__(128) unsigned char dyn[];
  BwdSmem<T> &sm = *reinterpret_cast<BwdSmem<T> *>(dyn);
  __shared__ ulonglong2 maps[2][kRuns][16];  // (N, E) of the lane's channels, by run
  __shared__ f2 backs[2][kRuns][16];         // R
  __shared__ ulonglong2 tiles[CL ? 2 : 1][kGatedMostCluster][16];  // CL: (N, R) of whole tiles
  __shared__ uint64_t here[2];                                     // CL: they have come
  __shared__ int asked;  // thread 0's: turns whose copies it has asked for
  __shared__ f2 carry[2][16];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), l = lane & 15, half = lane >> 4;
  // CL: a unit's CTAs are a cluster; else they have a segment each
  const int K = CL ? p.plan.cluster : 1, share = CL ? K : p.plan.segs, rank = blockIdx.x % share, unit = blockIdx.x / share;
  const int ct = unit % p.channel_tiles, b = unit / p.channel_tiles;
  const int run = 2 * warp + half;
  const int c0 = ct * kGatedCh + (PAIR ? 2 * l : l), c1 = c0 + (PAIR ? 1 : 16);
  const bool ok0 = c0 < p.dim, ok1 = c1 < p.dim;
  const float2 most = make_float2(ok0 ? -p.rate * softplus_f(p.decay[c0]) : 0.f, ok1 ? -p.rate * softplus_f(p.decay[c1]) : 0.f);
  const bool near = __all_sync(~0u, most.x >= -0.5f && most.y >= -0.5f);
  const f2 open = pk(most);  // L of an open gate
  auto pair_at = [&](const float *q) { return pk(ok0 ? q[c0] : 0.f, ok1 ? q[c1] : 0.f); };
  auto put_pair = [&](float *q, f2 v) {
    const float2 w = upk(v);
    if (ok0) q[c0] = w.x;
    if (ok1) q[c1] = w.y;
  };
  const int rounds = CL ? (p.tiles + K - 1) / K : min(p.plan.seg_tiles, p.tiles - rank * p.plan.seg_tiles);

  constexpr int H = TMA ? 1 : S;
  Two<T, PAIR> rx[H] = {}, rg[H] = {}, ri[H] = {}, rd[H] = {};
  const T *const x = static_cast<const T *>(p.x) + b * p.sx[0] + c0;
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + c0;
  const T *const igate = IG ? static_cast<const T *>(p.igate) + b * p.si[0] + c0 : nullptr;
  const T *const dout = static_cast<const T *>(p.dout) + b * p.sd[0] + c0;
  T *const dx = p.dx ? static_cast<T *>(p.dx) + b * p.sdx[0] + c0 : nullptr;
  T *const dgate = p.dgate ? static_cast<T *>(p.dgate) + b * p.sdg[0] + c0 : nullptr;
  T *const digate = IG && p.digate ? static_cast<T *>(p.digate) + b * p.sdi[0] + c0 : nullptr;
  bool fine = true;  // no wait has given up; after one has, nothing more is asked of a barrier
  // turns count up while the tiles go down
  auto tile_of = [&](int turn) { return CL ? (rounds - 1 - turn) * K + rank : rank * p.plan.seg_tiles + rounds - 1 - turn; };
  auto load = [&](int turn) {
    const int first = tile_of(turn) * kGatedTile;
    if constexpr (TMA) {
      if (threadIdx.x == 0 && fine) {
        const int s = turn % kStages;
        asked = turn + 1;
        mbar_arrive_expect_tx(&sm.full[s], (IG ? 4 : 3) * sizeof(sm.rows[0][0]));
        if (turn == p.wait.copy) return;
        tma_load_3d(sm.rows[s][0], &tm.x, &sm.full[s], ct * kGatedCh, first, b);
        tma_load_3d(sm.rows[s][1], &tm.gate, &sm.full[s], ct * kGatedCh, first, b);
        if constexpr (IG) tma_load_3d(sm.rows[s][2], &tm.igate, &sm.full[s], ct * kGatedCh, first, b);
        tma_load_3d(sm.rows[s][3], &tm.dout, &sm.full[s], ct * kGatedCh, first, b);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int t = first + run * S + j;
        const bool in = t < p.tokens;
        rx[j].load(x + t * p.sx[1], ok0 && in, ok1 && in);
        rg[j].load(gate + t * p.sg[1], ok0 && in, ok1 && in);
        if constexpr (IG) ri[j].load(igate + t * p.si[1], ok0 && in, ok1 && in);
        rd[j].load(dout + t * p.sd[1], ok0 && in, ok1 && in);
      }
    }
  };
  auto kept_of = [&](int turn) {
    const int tile = tile_of(turn);
    return tile < p.tiles ? pair_at(p.kept + ((long long)b * p.tiles + tile) * p.dim) : 0;
  };
  auto expect_maps = [&](int turn) { mbar_arrive_expect_tx(&here[turn & 1], K * sizeof(tiles[0][0])); };
  if constexpr (CL) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < 2; ++s) mbar_init(&here[s], 1);
      fence_barrier_init();
      for (int s = 0; s < 2 && s < rounds; ++s) expect_maps(s);
    }
  }
  if constexpr (TMA) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
      fence_barrier_init();
      for (int s = 0; s < kStages && s < rounds; ++s) load(s);
    }
  }
  f2 next = kept_of(0);  // the state before the tile that comes next
  // what comes back from past the last token; !CL: as if from a turn before the first
  f2 back = p.dlast ? pair_at(p.dlast + (long long)b * p.dim) : 0, e = 0, sum = 0;
  if constexpr (CL) {
    cluster_sync();
  } else {
    const int after = share - 1 - rank;  // segments after this one: a part of them for each half warp
    if (after > 0) {
      wait_for_previous();
      const int per = (after + kRuns - 1) / kRuns, from = rank + 1 + run * per, to = min(share, from + per);
      const ulonglong2 *seg = segment_maps(p.maps, unit, share, 0) + l;
      f2 N = 0, R = 0;
#pragma unroll 4
      for (int k = to - 1; k >= from; --k) {
        const ulonglong2 q = seg[k * 16];
        R = step2(q.x, R, q.y);
        N = step2(q.x, N, q.x);
      }
      maps[0][run][l] = make_ulonglong2(N, R);
      __syncthreads();
#pragma unroll
      for (int r = kRuns - 1; r >= 0; --r) back = step2(maps[0][r][l].x, back, maps[0][r][l].y);
    }
    if (threadIdx.x < 16) carry[1][l] = back;
    __syncthreads();
  }
  const f2 one = both(1.f), minus = both(-1.f);
  for (int turn = 0; turn < rounds; ++turn) {
    const int buf = turn & 1, stage = turn % kStages, t0 = tile_of(turn) * kGatedTile + run * S;
    const bool whole = (tile_of(turn) + 1) * kGatedTile <= p.tokens;
    f2 n[S], inv[S], h[S];
    f2 N = 0, E = 0, R = 0, start = next;
    if constexpr (TMA) {
      fine = mbar_wait(&sm.full[stage], (turn / kStages) & 1, p.err, kErrWaitFull, fine ? p.wait.limit : 1) && fine;
    } else {
      load(turn);
    }
    // a token's rows, from shared memory or from the registers that they were loaded to
    auto get = [&](int which, int j) {
      Two<T, PAIR> v;
      if constexpr (TMA) {
        v.load(&sm.rows[stage][which][run * S + j][2 * l], true, true);
      } else {
        v = which == 0 ? rx[j] : which == 1 ? rg[j] : which == 2 ? ri[IG ? j : 0] : rd[j];
      }
      return v.widen();
    };
#pragma unroll
    for (int k = 0; k < S; k += G) {
      f2 L[G], u[G], part[G], root[G], inverse[G];
#pragma unroll
      for (int j = 0; j < G; ++j) L[j] = get(1, k + j);
      sigmoid2(L);
#pragma unroll
      for (int j = 0; j < G; ++j) L[j] = mul2(open, L[j]);
      decay2(L, near, part);
      root2(part, root, inverse);
#pragma unroll
      for (int j = 0; j < G; ++j) {
        n[k + j] = part[j];
        inv[k + j] = inverse[j];
        root[j] = mul2(root[j], get(0, k + j));
      }
      if constexpr (IG) {
#pragma unroll
        for (int j = 0; j < G; ++j) u[j] = get(2, k + j);
        sigmoid2(u);
#pragma unroll
        for (int j = 0; j < G; ++j) root[j] = mul2(root[j], u[j]);
      }
#pragma unroll
      for (int j = 0; j < G; ++j) h[k + j] = root[j];  // b; the state before later
    }
    if (!whole) {  // past the end the state and what comes back stay (x and dout are 0 there)
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (t0 + j >= p.tokens) n[j] = 0;
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      N = step2(n[j], N, n[j]);
      E = step2(n[j], E, h[j]);
    }
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
      const f2 g = add2(get(3, j), R);
      R = fma2(n[j], g, g);
    }
    maps[buf][run][l] = make_ulonglong2(N, E);
    backs[buf][run][l] = R;
    if (turn + 1 < rounds) next = kept_of(turn + 1);
    if (TMA && lane == 0) stores_read();
    __syncthreads();
    // every warp is done with the tile before this one, whose place the next one takes, and
    // its gradients have left
    if (TMA && turn > 0 && turn + 1 < rounds) load(turn + 1);
    if constexpr (CL) {
      if (warp == 0) {
        ulonglong2 all = make_ulonglong2(0, 0);
#pragma unroll
        for (int r = kRuns - 1; r >= 0; --r) {
          const f2 q = maps[buf][r][l].x;
          all.y = step2(q, all.y, backs[buf][r][l]);
          all.x = step2(q, all.x, q);
        }
        // its place there was read in the turn before the last, and every CTA has begun the last one
        for (int r = turn == p.wait.maps ? K : half; r < K; r += 2) send(&tiles[buf][rank][l], &here[buf], r, all);
      }
      fine = mbar_wait_cluster(&here[buf], (turn >> 1) & 1, p.err, kErrWaitReady, fine ? p.wait.limit : 1) && fine;
      if (threadIdx.x == 0 && fine && turn + 2 < rounds) expect_maps(turn + 2);
      for (int c = K - 1; c >= 0; --c) {
        if (c == rank) e = back;
        const ulonglong2 q = tiles[buf][c][l];
        back = step2(q.x, back, q.y);
      }
    } else {
      e = carry[buf ^ 1][l];
    }
#pragma unroll
    for (int w = kGatedWarps - 1; w >= 0; --w) {
      if (w > warp) {
        e = step2(maps[buf][2 * w + 1][l].x, e, backs[buf][2 * w + 1][l]);
        e = step2(maps[buf][2 * w][l].x, e, backs[buf][2 * w][l]);
      }
    }
#pragma unroll
    for (int w = 0; w < kGatedWarps; ++w) {
      if (w < warp) {
        const ulonglong2 q = maps[buf][2 * w][l], r = maps[buf][2 * w + 1][l];
        start = step2(r.x, step2(q.x, start, q.y), r.y);
      }
    }
    if (half) {
      const ulonglong2 q = maps[buf][2 * warp][l];
      start = step2(q.x, start, q.y);
    } else {
      e = step2(maps[buf][2 * warp + 1][l].x, e, backs[buf][2 * warp + 1][l]);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      const f2 v = h[j];
      h[j] = start;
      start = step2(n[j], start, v);
    }
    if (!whole) {  // nothing for the decay's gradient: G = 0
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (t0 + j >= p.tokens) h[j] = 0;
    }
#pragma unroll
    for (int k = S - G; k >= 0; k -= G) {
      f2 r[G], i[G], g[G];
#pragma unroll
      for (int j = 0; j < G; ++j) r[j] = get(1, k + j);
      sigmoid2(r);
#pragma unroll
      for (int j = 0; j < G; ++j) i[j] = one;
      if constexpr (IG) {
#pragma unroll
        for (int j = 0; j < G; ++j) i[j] = get(2, k + j);
        sigmoid2(i);
      }
#pragma unroll
      for (int j = G - 1; j >= 0; --j) {
        g[j] = add2(get(3, k + j), e);
        e = fma2(n[k + j], g[j], g[j]);
      }
#pragma unroll
      for (int j = G - 1; j >= 0; --j) {
        const f2 m = n[k + j], a = add2(m, one), u = mul2(i[j], get(0, k + j));
        // G = g L a (h - u a / sqrt(1 - a^2))
        const f2 Gr = mul2(mul2(g[j], mul2(mul2(open, r[j]), a)), fma2(mul2(mul2(u, a), inv[k + j]), minus, h[k + j]));
        sum = add2(sum, Gr);
        // sqrt(1 - a^2) = (1 - a^2) / sqrt(1 - a^2)
        const f2 gr = mul2(g[j], mul2(fma2(m, fma2(m, minus, both(-2.f)), both(1e-36f)), inv[k + j]));
        const f2 vx = mul2(gr, i[j]), vg = mul2(Gr, fma2(r[j], minus, one)), vi = mul2(mul2(gr, u), fma2(i[j], minus, one));
        if constexpr (TMA) {
          const int row = run * S + k + j;
          Two<T, PAIR>::store(&sm.rows[stage][0][row][2 * l], upk(vx), true, true);
          Two<T, PAIR>::store(&sm.rows[stage][1][row][2 * l], upk(vg), true, true);
          if constexpr (IG) Two<T, PAIR>::store(&sm.rows[stage][2][row][2 * l], upk(vi), true, true);
        } else if (t0 + k + j < p.tokens) {
          const long long t = t0 + k + j;
          if (dx) Two<T, PAIR>::store(dx + t * p.sdx[1], upk(vx), ok0, ok1);
          if (dgate) Two<T, PAIR>::store(dgate + t * p.sdg[1], upk(vg), ok0, ok1);
          if (IG && digate) Two<T, PAIR>::store(digate + t * p.sdi[1], upk(vi), ok0, ok1);
        }
      }
    }
    if constexpr (TMA) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && t0 < p.tokens) {
        const int row = 2 * warp * S;
        if (dx) store_rows(&tm.dx, sm.rows[stage][0][row], ct * kGatedCh, t0, b);
        if (dgate) store_rows(&tm.dgate, sm.rows[stage][1][row], ct * kGatedCh, t0, b);
        if (IG && digate) store_rows(&tm.digate, sm.rows[stage][2][row], ct * kGatedCh, t0, b);
        commit_stores();
      }
    }
    if (!CL && threadIdx.x < 16) carry[buf][l] = e;
  }
  if (p.dinit && rank == 0 && threadIdx.x < 16) put_pair(p.dinit + (long long)b * p.dim, e);
  __syncthreads();
  backs[0][run][l] = sum;
  __syncthreads();
  if (p.parts && threadIdx.x < 16) {
    f2 s = backs[0][0][l];
    for (int r = 1; r < kRuns; ++r) s = add2(s, backs[0][r][l]);
    put_pair(p.parts + ((long long)b * share + rank) * p.dim, s);
  }
  if constexpr (TMA) {
    if (lane == 0) stores_done();
    if (!fine && threadIdx.x == 0) {  // a wait gave up: the copies under way land before the CTA leaves
      for (int turn = max(asked - kStages, 0); turn < asked; ++turn)
        mbar_wait(&sm.full[turn % kStages], (turn / kStages) & 1, p.err, kErrWaitFull, p.wait.limit);
    }
  }
  if constexpr (CL) cluster_sync();  // nobody leaves while its shared memory is written to
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

template <typename T, int ROWS, bool IG, bool CL>
cudaError_t launch(const GatedBwdParams &p, const BwdMaps &tm, cudaStream_t s) {
  const auto kernel = ss_gated_bwd_kernel<T, ROWS, IG, CL>;
  const int smem = ROWS == kTma ? sizeof(BwdSmem<T>) : 0;
  if (smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const long long units = (long long)p.batch * p.channel_tiles;
  if (!CL) {
    if (p.plan.segs > 1) {
      ss_gated_bwd_maps_kernel<T, ROWS != kSingles><<<(unsigned)(units * (p.plan.segs - 1)), kGatedThreads, 0, s>>>(p);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    return launch_after(kernel, dim3((unsigned)(units * p.plan.segs)), kGatedThreads, smem, s, p.plan.segs > 1, p, tm);
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.plan.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(units * p.plan.cluster));
  cfg.blockDim = dim3(kGatedThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, tm);
}
template <typename T, int ROWS>
cudaError_t form(const GatedBwdParams &p, const BwdMaps &tm, cudaStream_t s) {
  const bool cl = p.plan.cluster > 1;
  if (p.igate) return cl ? launch<T, ROWS, true, true>(p, tm, s) : launch<T, ROWS, true, false>(p, tm, s);
  return cl ? launch<T, ROWS, false, true>(p, tm, s) : launch<T, ROWS, false, false>(p, tm, s);
}
template <typename T>
cudaError_t pick(int rows, TensorMapEncode enc, const GatedBwdParams &p, cudaStream_t s) {
  BwdMaps tm;
  if (rows == kTma) {
    // what is not there has the map of what is
    auto map = [&](CUtensorMap *m, const void *base, const long long *st, int box) {
      return base ? rows_map(enc, m, sizeof(T), base, p.dim, p.tokens, p.batch, st, box) : rows_map(enc, m, sizeof(T), p.x, p.dim, p.tokens, p.batch, p.sx, box);
    };
    if (!map(&tm.x, p.x, p.sx, kGatedTile) || !map(&tm.gate, p.gate, p.sg, kGatedTile) || !map(&tm.igate, p.igate, p.si, kGatedTile) ||
        !map(&tm.dout, p.dout, p.sd, kGatedTile) || !map(&tm.dx, p.dx, p.sdx, 2 * kRun) || !map(&tm.dgate, p.dgate, p.sdg, 2 * kRun) ||
        !map(&tm.digate, p.digate, p.sdi, 2 * kRun))
      return cudaErrorInvalidValue;
    return form<T, kTma>(p, tm, s);
  }
  return rows == kPairs ? form<T, kPairs>(p, tm, s) : form<T, kSingles>(p, tm, s);
}

}  // namespace

cudaError_t launch_gated_bwd(int dtype, int rows, TensorMapEncode enc, const GatedBwdParams &given, cudaStream_t s) {
  GatedBwdParams p = given;
  p.wait = wait_hook();
  cudaError_t e = dtype == 0   ? pick<float>(rows, enc, p, s)
                  : dtype == 1 ? pick<__half>(rows, enc, p, s)
                               : pick<__nv_bfloat16>(rows, enc, p, s);
  if (e != cudaSuccess || !p.ddecay) return e;
  ss_gated_ddecay_kernel<<<(p.dim + 31) / 32, 256, 0, s>>>(p.parts, p.batch * p.plan.cluster * p.plan.segs, p.dim, p.decay, p.ddecay);
  return cudaGetLastError();
}

}  // namespace ssk
