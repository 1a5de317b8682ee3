// Gated linear recurrence, forward, on dense batches and on packed requests
// (include/ssfwd_layer.h):
//   h_t = h_{t-1} + (n_t h_{t-1} + b_t),  n = a - 1 and b from the gates (ss_gated.cuh).
//
// A step is a linear map of h, and maps compose: (N, E) of a run of tokens and then
// (n, b) is (N + n + n N, E + n E + b). A warp takes 8 tokens of 64 channels, two
// channels a lane, and keeps their n and b in registers; its map goes to shared memory;
// every warp then starts from the tile's first state taken through the maps before its
// own and runs its 8 tokens once more. So inputs are read once and the gates'
// arithmetic, which is most of the work, is spread over all warps, whatever the chain.
// Where sequences and channels alone leave SMs idle, the CTAs of a cluster take
// consecutive tiles and hand on their tiles' maps through distributed shared memory:
// nothing is read twice, no workspace, and no wait on memory.
//
// A packed request's first token takes the request's start state in its b, and cuts:
// what comes out of it does not depend on what came before, NaN or not. A map with a
// cut in it has N = kCut.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kSteps = 8;                      // tokens of a warp
constexpr int kWarps = kGatedTile / kSteps;
constexpr int kThreads = kWarps * 32;
constexpr float kCut = 1.f;                    // no decay's n, which lies in [-1, 0]

// The map q = (N, E) applied to h; a cut leaves nothing of it (PACKED).
template <bool PACKED>
__device__ __forceinline__ f2 through(ulonglong2 q, f2 h) {
  f2 r = step2(q.x, h, q.y);
  if constexpr (PACKED)
    if (upk(q.x).x == kCut) r = q.y;
  return r;
}

template <typename T, bool PAIR, bool IG, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) ss_gated_scan_kernel(const __grid_constant__ GatedScanParams p) {
  __shared__ ulonglong2 maps[2][kWarps][32];                // (N, E) of the lane's channels, by warp
  __shared__ ulonglong2 tiles[2][kGatedMostCluster][32];    // the same by CTA of the cluster
  __shared__ f2 carry[2][32];                               // the state after the cluster's last tile
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
  T *const out = static_cast<T *>(p.out) + b * p.so[0] + c0;
  auto pair_at = [&](const float *q) { return pk(ok0 ? q[c0] : 0.f, ok1 ? q[c1] : 0.f); };
  auto put_pair = [&](float *q, f2 v) {
    const float2 w = upk(v);
    if (ok0) q[c0] = w.x;
    if (ok1) q[c1] = w.y;
  };

  Two<T, PAIR> rx[kSteps], rg[kSteps], ri[IG ? kSteps : 1];
  int request = -1;  // PACKED: lane j has the request of the warp's token j - 1
  auto load = [&](int tile) {
    const int t0 = tile * kGatedTile + warp * kSteps;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const bool in = t0 + j < p.tokens;
      const long long t = t0 + j;
      rx[j].load(x + t * p.sx[1], ok0 && in, ok1 && in);
      rg[j].load(gate + t * p.sg[1], ok0 && in, ok1 && in);
      if constexpr (IG) ri[j].load(igate + t * p.si[1], ok0 && in, ok1 && in);
    }
    if constexpr (PACKED) {
      const int t = t0 + lane - 1;
      request = lane < kSteps + 2 && t >= 0 && t < p.tokens ? p.token_request[t] : -1;
    }
  };
  load(rank);

  f2 h = 0;
  if (p.init) h = pair_at(p.init + (long long)b * p.dim);
  if (K > 1) cluster_sync();  // every CTA's shared memory is there
  const int rounds = (p.tiles + K - 1) / K;
  for (int it = 0; it < rounds; ++it) {
    const int buf = it & 1, tile = it * K + rank, t0 = tile * kGatedTile + warp * kSteps;
    f2 n[kSteps], e[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      n[j] = decay2(mul2(open, sigmoid2(rg[j].widen())), near);
      f2 inverse, u = rx[j].widen();
      if constexpr (IG) u = mul2(u, sigmoid2(ri[j].widen()));
      e[j] = mul2(root2(n[j], inverse), u);
      if (t0 + j >= p.tokens) n[j] = e[j] = 0;  // past the end: the state stays
    }
    // PACKED: bit j + 1 is token j
    uint32_t cut = 0, last = 0;
    int req = -1;
    if constexpr (PACKED) {
      req = request;
      const int before = __shfl_up_sync(~0u, req, 1), after = __shfl_down_sync(~0u, req, 1);
      const bool mine = lane >= 1 && lane <= kSteps;
      const uint32_t first = __ballot_sync(~0u, mine && req >= 0 && before != req);
      last = __ballot_sync(~0u, mine && req >= 0 && after != req);
      cut = first | __ballot_sync(~0u, mine && req < 0);  // past the last request: zeros
      if (cut) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          if (first >> (j + 1) & 1) {
            const int r = __shfl_sync(~0u, req, j + 1);
            const int slot = p.slot_map[r];
            if (p.state && p.context && p.context[r] > 0 && slot >= 0 && slot < p.slots)
              e[j] = step2(n[j], pair_at(p.state + slot * p.state_stride), e[j]);
          } else if (cut >> (j + 1) & 1) {
            e[j] = 0;
          }
        }
      }
    }
    if (it + 1 < rounds) load(tile + K);
    auto run = [&](int j, f2 v) { return PACKED && (cut >> (j + 1) & 1) ? e[j] : step2(n[j], v, e[j]); };
    ulonglong2 m = make_ulonglong2(n[0], e[0]);
#pragma unroll
    for (int j = 1; j < kSteps; ++j) {
      m.x = step2(n[j], m.x, n[j]);
      m.y = run(j, m.y);
    }
    if (PACKED && cut) m.x = both(kCut);
    maps[buf][warp][lane] = m;
    __syncthreads();
    if (K > 1) {
      if (warp == kWarps - 1) {  // the whole tile's map, to every CTA
        ulonglong2 all = maps[buf][0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const ulonglong2 q = maps[buf][w][lane];
          const bool cuts = PACKED && (upk(q.x).x == kCut || upk(all.x).x == kCut);
          all.y = through<PACKED>(q, all.y);
          all.x = cuts ? both(kCut) : step2(q.x, all.x, q.x);
        }
        for (int r = 0; r < K; ++r) store_remote(&tiles[buf][rank][lane], r, all);
      }
      cluster_sync();
    }
    if (it > 0) h = carry[buf ^ 1][lane];
    for (int r = 0; r < rank; ++r) h = through<PACKED>(tiles[buf][r][lane], h);
    if (p.kept && warp == 0 && tile < p.tiles) put_pair(p.kept + ((long long)b * p.tiles + tile) * p.dim, h);
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) h = through<PACKED>(maps[buf][w][lane], h);
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      h = run(j, h);
      if (t0 + j < p.tokens) Two<T, PAIR>::store(out + (long long)(t0 + j) * p.so[1], upk(h), ok0, ok1);
      if constexpr (PACKED) {
        if (last >> (j + 1) & 1) {
          const int slot = p.slot_map[__shfl_sync(~0u, req, j + 1)];
          if (p.state && slot >= 0 && slot < p.slots) put_pair(p.state + slot * p.state_stride, h);
        }
      }
    }
    if (warp == kWarps - 1) {
      if (K == 1) {
        carry[buf][lane] = h;
      } else if (rank == K - 1) {
        for (int r = 0; r < K; ++r) store_remote(&carry[buf][lane], r, h);
      }
    }
  }
  if (p.last && rank == K - 1 && warp == kWarps - 1) put_pair(p.last + (long long)b * p.dim, h);
  if (K > 1) cluster_sync();  // nobody leaves while its shared memory is written to
}

template <typename T, bool PAIR, bool IG, bool PACKED>
cudaError_t launch(const GatedScanParams &p, cudaStream_t s) {
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
  return cudaLaunchKernelEx(&cfg, ss_gated_scan_kernel<T, PAIR, IG, PACKED>, p);
}
template <typename T>
cudaError_t pick(bool pair, const GatedScanParams &p, cudaStream_t s) {
  const bool packed = p.token_request != nullptr, ig = p.igate != nullptr;
  if (packed) {
    if (pair) return ig ? launch<T, true, true, true>(p, s) : launch<T, true, false, true>(p, s);
    return ig ? launch<T, false, true, true>(p, s) : launch<T, false, false, true>(p, s);
  }
  if (pair) return ig ? launch<T, true, true, false>(p, s) : launch<T, true, false, false>(p, s);
  return ig ? launch<T, false, true, false>(p, s) : launch<T, false, false, false>(p, s);
}

}  // namespace

cudaError_t launch_gated_scan(int dtype, bool pair, const GatedScanParams &p, cudaStream_t s) {
  return dtype == 0 ? pick<float>(pair, p, s) : dtype == 1 ? pick<__half>(pair, p, s) : pick<__nv_bfloat16>(pair, p, s);
}

// Clusters of the fewest CTAs that give every SM two, as far as there are tiles.
int gated_cluster(long long units, int tiles, int sms) {
  int k = 1;
  while (k < kGatedMostCluster && units * k < 2LL * sms && 2 * k <= tiles) k *= 2;
  return k;
}

}  // namespace ssk
