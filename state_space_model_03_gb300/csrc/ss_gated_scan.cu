// Gated linear recurrence, forward, on dense batches and on packed requests
// (include/ssfwd_layer.h):
//   h_t = h_{t-1} + (n_t h_{t-1} + b_t),  n = a - 1 and b from the gates (ss_gated.cuh).
//
// A step is a linear map of h, and maps compose: (N, E) of a run of tokens and then
// (n, b) is (N + n + n N, E + n E + b). Half a warp takes a run of 8 tokens of 32
// channels, two channels a lane, and keeps their n and b in registers; its map goes to
// shared memory; every run then starts from the tile's first state taken through the
// maps before its own and goes over its 8 tokens once more. So inputs are read once and
// the gates' arithmetic, which is most of the work, is spread over all warps, whatever
// the chain. Where sequences and channels alone leave SMs idle, the CTAs of a cluster
// take consecutive tiles and hand on their tiles' maps through distributed shared
// memory: nothing is read twice, no workspace, and no wait on memory.
//
// A packed request's first token takes the request's start state in its b, and cuts:
// what comes out of it does not depend on what came before, NaN or not. A map with a
// cut in it has N = kCut.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kStages = 2;
constexpr int kResident = 4;  // CTAs of a cluster that an SM holds
constexpr int kBuffers = 3;   // of maps: one is written while the one before is read, up to a barrier later
constexpr float kCut = 1.f;   // no decay's n, which lies in [-1, 0]

struct ScanMaps {
  CUtensorMap x, gate, igate, out;
};

template <typename T>
struct ScanSmem {
  // (stage, tensor) tiles of [tokens][channels], and a warp's rows on their way out
  T rows[kStages][3][kGatedTile][kGatedCh];
  T out[kGatedWarps][2 * kRun][kGatedCh];
  uint64_t full[kStages];
};

// The map q = (N, E) applied to h; a cut leaves nothing of it (PACKED).
template <bool PACKED>
__device__ __forceinline__ f2 through(ulonglong2 q, f2 h) {
  f2 r = step2(q.x, h, q.y);
  if constexpr (PACKED) {
    if (upk(q.x).x == kCut) r = q.y;
  }
  return r;
}

// PACKED, of a lane's run: bit j of last (first) says that token j ends (starts) a
// request; of cut, that it starts one or is past the last. request: lane j + 1 of the
// half has token j's; any: the bits of last of both halves.
struct Marks {
  uint32_t cut, first, last, any;
  int request;
};
__device__ __forceinline__ Marks marks_of(int request, int lane) {
  const int l = lane & 15, half = lane & 16;
  const int before = __shfl_up_sync(~0u, request, 1), after = __shfl_down_sync(~0u, request, 1);
  const bool mine = l >= 1 && l <= kRun;
  const uint32_t first = __ballot_sync(~0u, mine && request >= 0 && before != request);
  const uint32_t last = __ballot_sync(~0u, mine && request >= 0 && after != request);
  const uint32_t none = __ballot_sync(~0u, mine && request < 0);
  Marks m;
  m.first = first >> (half + 1) & 0xffu;
  m.last = last >> (half + 1) & 0xffu;
  m.cut = m.first | (none >> (half + 1) & 0xffu);
  m.any = (last >> 1 | last >> 17) & 0xffu;
  m.request = request;
  return m;
}

// CL: a cluster's CTAs take consecutive tiles; a tile's output then waits until the next
// tile's gates are done, so that the exchange is under way meanwhile.
template <typename T, int ROWS, bool IG, bool PACKED, bool CL>
__global__ void __launch_bounds__(kGatedThreads, ROWS != kTma ? 4 : CL ? 4 : sizeof(T) == 4 ? 4 : 6)
    ss_gated_scan_kernel(const __grid_constant__ GatedScanParams p, const __grid_constant__ ScanMaps tm) {
  constexpr int S = kRun;
  constexpr bool TMA = ROWS == kTma, PAIR = ROWS != kSingles;
  extern __shared__ __align__(128) unsigned char dyn[];
  ScanSmem<T> &sm = *reinterpret_cast<ScanSmem<T> *>(dyn);
  __shared__ ulonglong2 maps[kBuffers][kRuns][16];                         // (N, E) of the lane's channels, by run
  __shared__ ulonglong2 tiles[CL ? kBuffers : 1][kGatedMostCluster][16];   // CL: the same by CTA
  __shared__ f2 carry[2][16];                                              // !CL: the state after a tile
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), l = lane & 15, half = lane >> 4;
  const int K = CL ? p.cluster : 1, rank = CL ? blockIdx.x % K : 0, unit = CL ? blockIdx.x / K : blockIdx.x;
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
  const int rounds = (p.tiles + K - 1) / K;

  // rows: by TMA two tiles ahead, or into registers one tile ahead
  constexpr int H = TMA ? 1 : S;
  Two<T, PAIR> rx[H], rg[H], ri[H];
  const T *const x = static_cast<const T *>(p.x) + b * p.sx[0] + c0;
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + c0;
  const T *const igate = IG ? static_cast<const T *>(p.igate) + b * p.si[0] + c0 : nullptr;
  T *const out = static_cast<T *>(p.out) + b * p.so[0] + c0;
  bool fine = true;  // no wait has given up
  auto load = [&](int it) {
    const int first = (it * K + rank) * kGatedTile;
    if constexpr (TMA) {
      if (threadIdx.x == 0) {
        const int s = it % kStages;
        mbar_arrive_expect_tx(&sm.full[s], (IG ? 3 : 2) * sizeof(sm.rows[0][0]));
        tma_load_3d(sm.rows[s][0], &tm.x, &sm.full[s], ct * kGatedCh, first, b);
        tma_load_3d(sm.rows[s][1], &tm.gate, &sm.full[s], ct * kGatedCh, first, b);
        if constexpr (IG) tma_load_3d(sm.rows[s][2], &tm.igate, &sm.full[s], ct * kGatedCh, first, b);
      }
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int t = first + run * S + j;
        const bool in = t < p.tokens;
        rx[j].load(x + t * p.sx[1], ok0 && in, ok1 && in);
        rg[j].load(gate + t * p.sg[1], ok0 && in, ok1 && in);
        if constexpr (IG) ri[j].load(igate + t * p.si[1], ok0 && in, ok1 && in);
      }
    }
  };
  int request = -1;
  auto load_requests = [&](int it) {
    const int t = (it * K + rank) * kGatedTile + run * S + l - 1;
    request = l < S + 2 && t >= 0 && t < p.tokens ? p.token_request[t] : -1;
  };
  if constexpr (TMA) {
    if (threadIdx.x == 0) {
      for (int s = 0; s < kStages; ++s) mbar_init(&sm.full[s], 1);
      fence_barrier_init();
      for (int s = 0; s < kStages && s < rounds; ++s) load(s);
    }
  } else {
    load(0);
  }
  if constexpr (PACKED) load_requests(0);

  f2 h = p.init ? pair_at(p.init + (long long)b * p.dim) : 0;  // CL: the state before the cluster's tiles; else what a run ends in
  if (!CL && threadIdx.x < 16) carry[1][l] = h;
  if constexpr (CL) cluster_sync();  // every CTA's shared memory is there
  else __syncthreads();

  f2 n[S], e[S], pn[CL ? S : 1], pe[CL ? S : 1];
  Marks now{}, past{};
  // n, e and the map of a run's tokens in tile `it`
  auto gates = [&](int it) {
    const int t0 = (it * K + rank) * kGatedTile + run * S;
    if constexpr (TMA) {
      fine = mbar_wait(&sm.full[it % kStages], (it / kStages) & 1, p.err, kErrWaitFull, fine ? kMaxWaitIters : 1) && fine;
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      Two<T, PAIR> vx, vg, vi;
      if constexpr (TMA) {
        vx.load(&sm.rows[it % kStages][0][run * S + j][2 * l], true, true);
        vg.load(&sm.rows[it % kStages][1][run * S + j][2 * l], true, true);
        if constexpr (IG) vi.load(&sm.rows[it % kStages][2][run * S + j][2 * l], true, true);
      } else {
        vx = rx[j];
        vg = rg[j];
        if constexpr (IG) vi = ri[j];
      }
      n[j] = decay2(mul2(open, sigmoid2(vg.widen())), near);
      f2 inverse, u = vx.widen();
      if constexpr (IG) u = mul2(u, sigmoid2(vi.widen()));
      e[j] = mul2(root2(n[j], inverse), u);
    }
    if ((it * K + rank + 1) * kGatedTile > p.tokens) {  // past the end the state stays
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (t0 + j >= p.tokens) n[j] = e[j] = 0;
    }
    if constexpr (PACKED) {
      now = marks_of(request, lane);
      if (__any_sync(~0u, now.cut != 0)) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          const int r = __shfl_sync(~0u, request, (lane & 16) + j + 1);
          if (now.first >> j & 1) {
            const int slot = p.slot_map[r];
            if (p.state && p.context && p.context[r] > 0 && slot >= 0 && slot < p.slots)
              e[j] = step2(n[j], pair_at(p.state + slot * p.state_stride), e[j]);
          } else if (now.cut >> j & 1) {
            e[j] = 0;
          }
        }
      }
      if (it + 1 < rounds) load_requests(it + 1);
    }
    if constexpr (!TMA) {
      if (it + 1 < rounds) load(it + 1);
    }
    ulonglong2 m = make_ulonglong2(n[0], e[0]);
#pragma unroll
    for (int j = 1; j < S; ++j) {
      m.x = step2(n[j], m.x, n[j]);
      m.y = PACKED && (now.cut >> j & 1) ? e[j] : step2(n[j], m.y, e[j]);
    }
    if (PACKED && now.cut) m.x = both(kCut);
    maps[it % kBuffers][run][l] = m;
  };
  // the output of tile `it`, from the state before the CTA's tile
  auto finish = [&](int it, f2 v, const f2 *fn, const f2 *fe, const Marks &mk) {
    const int t0 = (it * K + rank) * kGatedTile + run * S;
    if (p.kept && threadIdx.x < 16 && t0 < p.tokens) put_pair(p.kept + ((long long)b * p.tiles + it * K + rank) * p.dim, v);
    const auto &map = maps[it % kBuffers];
#pragma unroll
    for (int w = 0; w < kGatedWarps; ++w) {
      if (w < warp) v = through<PACKED>(map[2 * w + 1][l], through<PACKED>(map[2 * w][l], v));
    }
    if (half) v = through<PACKED>(map[2 * warp][l], v);
    if constexpr (TMA) {  // the rows before these have left
      if (lane == 0) stores_read();
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
      v = PACKED && (mk.cut >> j & 1) ? fe[j] : step2(fn[j], v, fe[j]);
      if constexpr (TMA) {
        Two<T, PAIR>::store(&sm.out[warp][half * S + j][2 * l], upk(v), true, true);
      } else {
        if (t0 + j < p.tokens) Two<T, PAIR>::store(out + (t0 + j) * p.so[1], upk(v), ok0, ok1);
      }
      if constexpr (PACKED) {
        if (mk.any >> j & 1) {
          const int r = __shfl_sync(~0u, mk.request, (lane & 16) + j + 1);
          if (mk.last >> j & 1) {
            const int slot = p.slot_map[r];
            if (p.state && slot >= 0 && slot < p.slots) put_pair(p.state + slot * p.state_stride, v);
          }
        }
      }
    }
    if constexpr (TMA) {
      fence_proxy_async();
      __syncwarp();
      if (lane == 0 && t0 < p.tokens) {
        store_rows(&tm.out, sm.out[warp], ct * kGatedCh, t0, b);
        commit_stores();
      }
    }
    return v;
  };

  if constexpr (!CL) {
    for (int it = 0; it < rounds; ++it) {
      gates(it);
      __syncthreads();
      if (TMA && it + kStages < rounds) load(it + kStages);
      h = finish(it, carry[(it & 1) ^ 1][l], n, e, now);
      if (threadIdx.x >= kGatedThreads - 16) carry[it & 1][l] = h;
    }
    if (p.last && threadIdx.x >= kGatedThreads - 16) put_pair(p.last + (long long)b * p.dim, h);
  } else {
    for (int it = 0; it <= rounds; ++it) {
      if (it > 0) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
          pn[j] = n[j];
          pe[j] = e[j];
        }
        past = now;
      }
      if (it < rounds) {
        gates(it);
        __syncthreads();
        if (TMA && it + kStages < rounds) load(it + kStages);
      }
      if (it > 0) cluster_wait();  // the maps of the tiles before are here
      if (it < rounds) {
        if (warp == 0) {  // the whole tile's map, to every CTA: half of them from each half
          const auto &map = maps[it % kBuffers];
          ulonglong2 all = map[0][l];
#pragma unroll
          for (int r = 1; r < kRuns; ++r) {
            const ulonglong2 q = map[r][l];
            const bool cuts = PACKED && (upk(q.x).x == kCut || upk(all.x).x == kCut);
            all.y = through<PACKED>(q, all.y);
            all.x = cuts ? both(kCut) : step2(q.x, all.x, q.x);
          }
          for (int r = half; r < K; r += 2) store_remote(&tiles[it % kBuffers][rank][l], r, all);
        }
        __syncwarp();
        cluster_arrive();
      }
      if (it > 0) {
        f2 start = h;
        for (int r = 0; r < K; ++r) {
          if (r == rank) start = h;
          h = through<PACKED>(tiles[(it - 1) % kBuffers][r][l], h);
        }
        finish(it - 1, start, pn, pe, past);
      }
    }
    if (p.last && rank == 0 && threadIdx.x < 16) put_pair(p.last + (long long)b * p.dim, h);
    cluster_sync();  // nobody leaves while its shared memory is written to
  }
  if constexpr (TMA) {
    if (lane == 0) stores_done();
    if (!fine && threadIdx.x == 0) {  // a wait gave up: the copies under way land before the CTA leaves
      for (int s = 0; s < kStages && s < rounds; ++s) {
        const int it = (rounds - 1 - s) / kStages * kStages + s;
        mbar_wait(&sm.full[s], (it / kStages) & 1, p.err, kErrWaitFull);
      }
    }
  }
}

template <typename T, int ROWS, bool IG, bool PACKED, bool CL>
cudaError_t launch(const GatedScanParams &p, const ScanMaps &tm, cudaStream_t s) {
  const auto kernel = ss_gated_scan_kernel<T, ROWS, IG, PACKED, CL>;
  const int smem = ROWS == kTma ? sizeof(ScanSmem<T>) : 0;
  if (smem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((long long)p.batch * p.channel_tiles * p.cluster));
  cfg.blockDim = dim3(kGatedThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = CL;
  return cudaLaunchKernelEx(&cfg, kernel, p, tm);
}
template <typename T, int ROWS, bool IG>
cudaError_t form(const GatedScanParams &p, const ScanMaps &tm, cudaStream_t s) {
  if (p.token_request) return p.cluster > 1 ? launch<T, ROWS, IG, true, true>(p, tm, s) : launch<T, ROWS, IG, true, false>(p, tm, s);
  return p.cluster > 1 ? launch<T, ROWS, IG, false, true>(p, tm, s) : launch<T, ROWS, IG, false, false>(p, tm, s);
}
template <typename T>
cudaError_t pick(int rows, TensorMapEncode enc, GatedScanParams &p, int sms, cudaStream_t s) {
  p.cluster = gated_cluster((long long)p.batch * p.channel_tiles, p.tiles, sms, kResident);
  ScanMaps tm;
  if (rows == kTma) {
    auto map = [&](CUtensorMap *m, const void *base, const long long *st, int box) {
      return rows_map(enc, m, sizeof(T), base, p.dim, p.tokens, p.batch, st, box);
    };
    if (!map(&tm.x, p.x, p.sx, kGatedTile) || !map(&tm.gate, p.gate, p.sg, kGatedTile) ||
        !map(&tm.igate, p.igate ? p.igate : p.x, p.igate ? p.si : p.sx, kGatedTile) || !map(&tm.out, p.out, p.so, 2 * kRun))
      return cudaErrorInvalidValue;
    return p.igate ? form<T, kTma, true>(p, tm, s) : form<T, kTma, false>(p, tm, s);
  }
  if (rows == kPairs) return p.igate ? form<T, kPairs, true>(p, tm, s) : form<T, kPairs, false>(p, tm, s);
  return p.igate ? form<T, kSingles, true>(p, tm, s) : form<T, kSingles, false>(p, tm, s);
}

}  // namespace

cudaError_t launch_gated_scan(int dtype, int rows, TensorMapEncode enc, GatedScanParams p, int sms, cudaStream_t s) {
  return dtype == 0   ? pick<float>(rows, enc, p, sms, s)
         : dtype == 1 ? pick<__half>(rows, enc, p, sms, s)
                      : pick<__nv_bfloat16>(rows, enc, p, sms, s);
}

}  // namespace ssk
