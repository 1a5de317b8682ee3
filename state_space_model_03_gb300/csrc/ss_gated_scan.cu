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
// the chain. Tiles come and go by TMA, the loads two tiles ahead.
//
// Where sequences and channels alone leave SMs idle, the CTAs of a cluster take
// consecutive tiles and send one another their tiles' maps (st.async, counted by the
// receiver's mbarrier): nothing is read twice, no workspace, no wait on memory. Where
// there are too few of them for that too, a first launch reduces segments of a sequence
// to their maps, and the second starts each from those before it (gated_plan).
//
// A packed request's first token takes the request's start state in its b, and cuts:
// what comes out of it does not depend on what came before, NaN or not. A map with a
// cut in it has N = kCut.
//
// 8 x 2048 x 2560 bf16 64 us, 5.2 TB/s (77% of the copy); 65536 x 2048 in clusters 278
// us, 3.9 TB/s; 16384 packed tokens x 2560 113 us. Nothing is at its rate (issue 0.59,
// special functions 0.37, DRAM 0.58): what bounds the first is latency at the 17 warps an
// SM that 640 CTAs make, and their share, five CTAs on 32 SMs and four on the others, which
// are idle for up to a fifth of the time; in clusters the exchange of each round besides.
// 63 instructions a token and pair of channels: 32 for the gates, the sigmoids' and the
// root's 10 on the special-function unit among them, 7 for the scan, 6 to widen 16 bits,
// the rest for tiles and maps. Tiles of 64 channels (320 CTAs, 2 or 3 an SM) 78 us; loads
// into registers instead of TMA (103 instructions, half of them for addresses and ends) 128.
#include "ss_gated.cuh"

namespace ssk {
namespace {

constexpr int kStages = 2;
constexpr int G = 4;          // tokens whose gates are taken side by side
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
// request; of cut, that it starts one or is past the last. from, to: the slots of the first
// request that starts (-1: it starts from 0; kKept: from the state that the workspace has)
// and of the first that ends in the run, looked up a tile ahead; a run rarely has more.
constexpr int kKept = -2;
struct Marks {
  uint32_t cut, first, last;
  int from, to;
  bool any;  // whether either half has any of these
};

// q after m, as one map.
template <bool PACKED>
__device__ __forceinline__ ulonglong2 then(ulonglong2 m, ulonglong2 q) {
  const bool cuts = PACKED && (upk(q.x).x == kCut || upk(m.x).x == kCut);
  return make_ulonglong2(cuts ? both(kCut) : step2(q.x, m.x, q.x), through<PACKED>(q, m.y));
}

// PACKED: a run's requests and marks. ids: lane j + 1 of a half has the request of its
// run's token j.
struct Requests {
  const GatedScanParams &p;
  int l, half;
  int over;  // a request that goes on after the segment (-1: none): another CTA may already have replaced its state
  __device__ __forceinline__ int ids(int t0) const {
    const int t = t0 + l - 1;
    return l < kRun + 2 && t >= 0 && t < p.tokens ? p.token_request[t] : -1;
  }
  __device__ __forceinline__ int slot_of(int r) const {
    const int slot = r >= 0 && p.state ? p.slot_map[r] : -1;
    return slot < p.slots ? slot : -1;
  }
  __device__ __forceinline__ int start_of(int r) const {
    if (r >= 0 && r == over) return kKept;
    return r >= 0 && p.context && p.context[r] > 0 ? slot_of(r) : -1;
  }
  __device__ __forceinline__ Marks marks(int ids) const {
    // mostly all of a warp's tokens, and those beside them, are of one request
    const int one = __shfl_sync(~0u, ids, 16 * half);
    if (!__any_sync(~0u, one < 0 || (l < kRun + 2 && ids != one))) return Marks{0, 0, 0, -1, -1, false};
    const int before = __shfl_up_sync(~0u, ids, 1), after = __shfl_down_sync(~0u, ids, 1);
    const bool mine = l >= 1 && l <= kRun;
    const uint32_t first = __ballot_sync(~0u, mine && ids >= 0 && before != ids);
    const uint32_t last = __ballot_sync(~0u, mine && ids >= 0 && after != ids);
    const uint32_t none = __ballot_sync(~0u, mine && ids < 0);
    Marks m;
    m.first = first >> (16 * half + 1) & 0xffu;
    m.last = last >> (16 * half + 1) & 0xffu;
    m.cut = m.first | (none >> (16 * half + 1) & 0xffu);
    m.any = (first | last | none) != 0;
    const int r0 = __shfl_sync(~0u, ids, 16 * half + __ffs(m.first)), r1 = __shfl_sync(~0u, ids, 16 * half + __ffs(m.last));
    m.from = start_of(m.first ? r0 : -1);
    m.to = slot_of(m.last ? r1 : -1);
    return m;
  }
};

// n and b of a run's tokens, from their x, gate and input gate.
template <bool IG, typename Get>
__device__ __forceinline__ void run_gates(f2 open, bool near, Get get, f2 *n, f2 *e) {
#pragma unroll
  for (int k = 0; k < kRun; k += G) {
    f2 L[G], root[G], inverse[G], part[G];
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
      root[j] = mul2(root[j], get(0, k + j));
    }
    if constexpr (IG) {
      f2 u[G];
#pragma unroll
      for (int j = 0; j < G; ++j) u[j] = get(2, k + j);
      sigmoid2(u);
#pragma unroll
      for (int j = 0; j < G; ++j) root[j] = mul2(root[j], u[j]);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) e[k + j] = root[j];
  }
}
// PACKED: start states into b where requests start, zeros past the last. start: the first
// one's, afterwards the last one's; of: the state of a slot, or the kept one.
template <typename Of>
__device__ __forceinline__ void run_starts(const Requests &req, const Marks &m, int t0, f2 &start, Of of, const f2 *n, f2 *e) {
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    if (m.first >> j & 1) {
      if (m.first & ((1u << j) - 1)) start = of(req.start_of(req.p.token_request[t0 + j]));
      e[j] = step2(n[j], start, e[j]);
    } else if (m.cut >> j & 1) {
      e[j] = 0;
    }
  }
}
// A run's tokens after the map m.
template <bool PACKED>
__device__ __forceinline__ ulonglong2 run_map(ulonglong2 m, const Marks &marks, const f2 *n, const f2 *e) {
  const f2 before = m.y;
#pragma unroll
  for (int j = 0; j < kRun; ++j) {
    m.x = step2(n[j], m.x, n[j]);
    m.y = step2(n[j], m.y, e[j]);
  }
  if constexpr (PACKED) {
    if (marks.any) {  // again, with the cuts
      m.y = before;
#pragma unroll
      for (int j = 0; j < kRun; ++j) m.y = marks.cut >> j & 1 ? e[j] : step2(n[j], m.y, e[j]);
      if (marks.cut) m.x = both(kCut);
    }
  }
  return m;
}

// What a thread's lane has: two channels of a unit.
template <bool PAIR>
struct Lane {
  int l, half, c0, c1;
  bool ok0, ok1, near;
  f2 open;  // L of an open gate
  __device__ __forceinline__ Lane(const GatedScanParams &p, int ct) {
    l = threadIdx.x & 15;
    half = threadIdx.x >> 4 & 1;
    c0 = ct * kGatedCh + (PAIR ? 2 * l : l);
    c1 = c0 + (PAIR ? 1 : 16);
    ok0 = c0 < p.dim;
    ok1 = c1 < p.dim;
    const float2 most = make_float2(ok0 ? -p.rate * softplus_f(p.decay[c0]) : 0.f, ok1 ? -p.rate * softplus_f(p.decay[c1]) : 0.f);
    near = __all_sync(~0u, most.x >= -0.5f && most.y >= -0.5f);
    open = pk(most);
  }
  __device__ __forceinline__ f2 pair_at(const float *q) const { return pk(ok0 ? q[c0] : 0.f, ok1 ? q[c1] : 0.f); }
  __device__ __forceinline__ void put_pair(float *q, f2 v) const {
    const float2 w = upk(v);
    if (ok0) q[c0] = w.x;
    if (ok1) q[c1] = w.y;
  }
};

__device__ __forceinline__ f2 *segment_starts(const GatedScanParams &p, long long unit, int seg) {
  const long long units = (long long)p.batch * p.channel_tiles;
  return reinterpret_cast<f2 *>(segment_maps(p.maps, units, p.plan.segs, 0)) + (unit * p.plan.segs + seg) * 16;
}

// The maps of all segments but the last: each half warp takes a part of the segment's
// tokens that no other comes between. PACKED: only the request that goes on after the
// segment has to be carried over its end, from its first token or the segment's; its
// start state is kept besides, because the CTA of the segment that it ends in replaces it.
template <typename T, bool PAIR, bool IG, bool PACKED>
__global__ void __launch_bounds__(kGatedThreads, 4) ss_gated_maps_kernel(const __grid_constant__ GatedScanParams p) {
  __shared__ ulonglong2 maps[kRuns][16];
  let_next_start();
  const int segs = p.plan.segs - 1, seg = blockIdx.x % segs, unit = blockIdx.x / segs;
  const int ct = unit % p.channel_tiles, b = unit / p.channel_tiles;
  const Lane<PAIR> me(p, ct);
  const int run = threadIdx.x >> 4, end = (seg + 1) * p.plan.seg_tiles * kGatedTile;
  int begin = end - p.plan.seg_tiles * kGatedTile;
  ulonglong2 m = make_ulonglong2(0, 0);
  if constexpr (PACKED) {
    const int r = p.token_request[end - 1];
    bool starts = true;
    f2 start = 0;
    if (r < 0 || p.token_request[end] != r) {
      begin = end;  // what follows starts by itself
    } else if (p.offsets[r] >= begin) {
      begin = p.offsets[r];
      const int slot = p.state && p.context && p.context[r] > 0 ? p.slot_map[r] : -1;
      if (slot >= 0 && slot < p.slots) start = me.pair_at(p.state + slot * p.state_stride);
    } else {
      starts = false;
    }
    if (starts && run == 0) m = make_ulonglong2(both(kCut), start);
    if (threadIdx.x < 16) *(segment_starts(p, unit, seg) + me.l) = start;
  }
  const T *const x = static_cast<const T *>(p.x) + b * p.sx[0] + me.c0;
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + me.c0;
  const T *const igate = IG ? static_cast<const T *>(p.igate) + b * p.si[0] + me.c0 : nullptr;
  const int steps = (end - begin + kGatedTile - 1) / kGatedTile, first = begin + run * steps * kRun;
  Two<T, PAIR> rx[kRun] = {}, rg[kRun] = {}, ri[kRun] = {};
  auto load = [&](int t0) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool in = t0 + j < end;
      const long long t = t0 + j;
      rx[j].load(x + t * p.sx[1], me.ok0 && in, me.ok1 && in);
      rg[j].load(gate + t * p.sg[1], me.ok0 && in, me.ok1 && in);
      if constexpr (IG) ri[j].load(igate + t * p.si[1], me.ok0 && in, me.ok1 && in);
    }
  };
  if (steps > 0) load(first);
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    const int t0 = first + k * kRun;
    f2 n[kRun], e[kRun];
    run_gates<IG>(me.open, me.near, [&](int which, int j) { return which == 0 ? rx[j].widen() : which == 1 ? rg[j].widen() : ri[j].widen(); }, n, e);
    if (k + 1 < steps) load(t0 + kRun);
    if (t0 + kRun > end) {
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (t0 + j >= end) n[j] = e[j] = 0;
    }
    const bool cut = PACKED && upk(m.x).x == kCut;
    m = run_map<false>(m, Marks{}, n, e);
    if (cut) m.x = both(kCut);
  }
  maps[run][me.l] = m;
  __syncthreads();
  if (threadIdx.x < 16) {
    m = maps[0][me.l];
#pragma unroll
    for (int r = 1; r < kRuns; ++r) m = then<PACKED>(m, maps[r][me.l]);
    *(segment_maps(p.maps, unit, p.plan.segs, seg) + me.l) = m;
  }
}

// CL: a cluster's CTAs take consecutive tiles. Single values of three tensors are addresses
// enough for 150 registers, so three CTAs an SM; four, at 128, spilled: 16384 tokens x 1301
// in bf16 117 us against 83, fp32 192 against 84, 6000 packed tokens x 2561 133 against 98;
// 6000 packed x 333, where the CTAs are few, 16.5 against 17.9.
template <typename T, int ROWS, bool IG, bool PACKED, bool CL>
__global__ void __launch_bounds__(kGatedThreads, ROWS == kSingles && IG ? 3 : ROWS != kTma ? 4 : CL ? 6 : sizeof(T) == 4 ? 4 : 6)
    ss_gated_scan_kernel(const __grid_constant__ GatedScanParams p, const __grid_constant__ ScanMaps tm) {
  constexpr int S = kRun;
  constexpr bool TMA = ROWS == kTma, PAIR = ROWS != kSingles;
  extern __shared__ __align__(128) unsigned char dyn[];
  ScanSmem<T> &sm = *reinterpret_cast<ScanSmem<T> *>(dyn);
  __shared__ ulonglong2 maps[2][kRuns][16];                                // (N, E) of the lane's channels, by run
  __shared__ ulonglong2 tiles[CL ? 2 : 1][kGatedMostCluster][16];          // CL: the same by CTA
  __shared__ uint64_t here[2];                                             // CL: the tiles' maps have come
  __shared__ int asked;  // thread 0's: rounds whose copies it has asked for
  __shared__ f2 carry[2][16];                                              // !CL: the state after a tile
  const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x >> 5, 0);
  // CL: a unit's CTAs are a cluster; else they have a segment each
  const int K = CL ? p.plan.cluster : 1, share = CL ? K : p.plan.segs, rank = blockIdx.x % share, unit = blockIdx.x / share;
  const int ct = unit % p.channel_tiles, b = unit / p.channel_tiles;
  const Lane<PAIR> me(p, ct);
  const int l = me.l, half = me.half, run = 2 * warp + half, c0 = me.c0;
  const bool ok0 = me.ok0, ok1 = me.ok1;
  auto pair_at = [&](const float *q) { return me.pair_at(q); };
  const int rounds = CL ? (p.tiles + K - 1) / K : min(p.plan.seg_tiles, p.tiles - rank * p.plan.seg_tiles);
  auto tile_of = [&](int it) { return CL ? it * K + rank : rank * p.plan.seg_tiles + it; };

  // rows: by TMA two tiles ahead, or into registers one tile ahead
  constexpr int H = TMA ? 1 : S;
  Two<T, PAIR> rx[H] = {}, rg[H] = {}, ri[H] = {};
  const T *const x = static_cast<const T *>(p.x) + b * p.sx[0] + c0;
  const T *const gate = static_cast<const T *>(p.gate) + b * p.sg[0] + c0;
  const T *const igate = IG ? static_cast<const T *>(p.igate) + b * p.si[0] + c0 : nullptr;
  T *const out = static_cast<T *>(p.out) + b * p.so[0] + c0;
  bool fine = true;  // no wait has given up; after one has, nothing more is asked of a barrier
  auto load = [&](int it) {
    const int first = tile_of(it) * kGatedTile;
    if constexpr (TMA) {
      if (threadIdx.x == 0 && fine) {
        const int s = it % kStages;
        asked = it + 1;
        mbar_arrive_expect_tx(&sm.full[s], (IG ? 3 : 2) * sizeof(sm.rows[0][0]));
        if (it == p.wait.copy) return;
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
  int over = -1;
  if (PACKED && !CL && rank < share - 1) {
    const int end = (rank + 1) * p.plan.seg_tiles * kGatedTile;
    const int r = p.token_request[end - 1];
    over = r == p.token_request[end] ? r : -1;
  }
  const Requests req{p, l, half, over};
  f2 kept_start = 0;
  auto of = [&](int slot) { return slot >= 0 ? pair_at(p.state + slot * p.state_stride) : PACKED && !CL && slot == kKept ? kept_start : 0; };
  Marks next{};  // of the next tile; ids: of the one after
  int ids = -1;
  auto expect_maps = [&](int it) { mbar_arrive_expect_tx(&here[it & 1], K * sizeof(tiles[0][0])); };
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
  } else {
    load(0);
  }
  if constexpr (PACKED) {
    next = req.marks(req.ids(tile_of(0) * kGatedTile + run * S));
    if (rounds > 1) ids = req.ids(tile_of(1) * kGatedTile + run * S);
  }

  f2 h = p.init ? pair_at(p.init + (long long)b * p.dim) : 0;  // CL: the state before the cluster's tiles; else what a run ends in
  if constexpr (CL) {
    cluster_sync();  // every CTA's shared memory is there
  } else {
    if (threadIdx.x < 16) carry[1][l] = h;
    __syncthreads();
  }

  // n, e and the map of a run's tokens in tile `it`
  auto gates = [&](int it, f2 *n, f2 *e, Marks &now) {
    const int t0 = tile_of(it) * kGatedTile + run * S;
    f2 start = 0;  // PACKED: what the first request that starts in the run starts from
    if constexpr (PACKED) {
      now = next;
      start = of(now.from);
    }
    if constexpr (TMA) {
      fine = mbar_wait(&sm.full[it % kStages], (it / kStages) & 1, p.err, kErrWaitFull, fine ? p.wait.limit : 1) && fine;
    }
    auto get = [&](int which, int j) {
      Two<T, PAIR> v;
      if constexpr (TMA) {
        v.load(&sm.rows[it % kStages][which][run * S + j][2 * l], true, true);
      } else {
        v = which == 0 ? rx[j] : which == 1 ? rg[j] : ri[j];
      }
      return v.widen();
    };
    run_gates<IG>(me.open, me.near, get, n, e);
    if ((tile_of(it) + 1) * kGatedTile > p.tokens) {  // past the end a finite state stays
#pragma unroll
      for (int j = 0; j < S; ++j)
        if (t0 + j >= p.tokens) n[j] = e[j] = 0;
    }
    if constexpr (PACKED) {
      if (now.any) run_starts(req, now, t0, start, of, n, e);
      if (it + 1 < rounds) {
        next = req.marks(ids);
        ids = it + 2 < rounds ? req.ids(tile_of(it + 2) * kGatedTile + run * S) : -1;
      }
    }
    if constexpr (!TMA) {
      if (it + 1 < rounds) load(it + 1);
    }
    maps[it & 1][run][l] = run_map<PACKED>(make_ulonglong2(0, 0), now, n, e);
  };
  // the output of tile `it`, from the state before the CTA's tile
  auto finish = [&](int it, f2 v, const f2 *fn, const f2 *fe, const Marks &mk) {
    const int t0 = tile_of(it) * kGatedTile + run * S;
    if (p.kept && threadIdx.x < 16 && t0 < p.tokens) me.put_pair(p.kept + ((long long)b * p.tiles + tile_of(it)) * p.dim, v);
    const auto &map = maps[it & 1];
#pragma unroll
    for (int w = 0; w < kGatedWarps; ++w) {
      if (w < warp) v = through<PACKED>(map[2 * w + 1][l], through<PACKED>(map[2 * w][l], v));
    }
    if (half) v = through<PACKED>(map[2 * warp][l], v);
    if constexpr (TMA) {  // the rows before these have left
      if (lane == 0) stores_read();
      __syncwarp();
    }
    auto put = [&](int j) {
      if constexpr (TMA) {
        Two<T, PAIR>::store(&sm.out[warp][half * S + j][2 * l], upk(v), true, true);
      } else {
        if (t0 + j < p.tokens) Two<T, PAIR>::store(out + (t0 + j) * p.so[1], upk(v), ok0, ok1);
      }
    };
    if (PACKED && mk.any) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        v = mk.cut >> j & 1 ? fe[j] : step2(fn[j], v, fe[j]);
        put(j);
        if (mk.last >> j & 1) {
          const int slot = (mk.last & ((1u << j) - 1)) == 0 ? mk.to : req.slot_of(p.token_request[t0 + j]);
          if (slot >= 0) me.put_pair(p.state + slot * p.state_stride, v);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < S; ++j) {
        v = step2(fn[j], v, fe[j]);
        put(j);
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

  // !CL: what the launch before this one has left: the state that the segment starts from,
  // through the maps of the segments before it, a part of them for each half warp
  auto enter = [&] {
    wait_for_previous();
    if (PACKED && rank < share - 1) kept_start = segment_starts(p, unit, rank)[l];
    const int per = (rank + kRuns - 1) / kRuns, from = run * per, to = min(rank, from + per);
    const ulonglong2 *seg = segment_maps(p.maps, unit, p.plan.segs, 0) + l;
    ulonglong2 m = make_ulonglong2(0, 0);
#pragma unroll 4
    for (int k = from; k < to; ++k) m = then<PACKED>(m, seg[k * 16]);
    maps[1][run][l] = m;  // not written again before the second tile
    __syncthreads();
    if (threadIdx.x < 16) {
#pragma unroll
      for (int r = 0; r < kRuns; ++r) h = through<PACKED>(maps[1][r][l], h);
      carry[1][l] = h;
    }
    __syncthreads();
  };
  // after the first tile's gates, unless a request starts there from what is left
  bool entered = CL || share == 1 || (!PACKED && rank == 0);
  if (PACKED && !entered && over >= 0 && p.offsets[over] < (tile_of(0) + 1) * kGatedTile) {
    enter();
    entered = true;
  }
  f2 n[S], e[S];
  Marks now{};
#pragma unroll 1
  for (int it = 0; it < rounds; ++it) {
    gates(it, n, e, now);
    if (!CL && !entered) {
      enter();
      entered = true;
    } else {
      __syncthreads();
    }
    if (TMA && it + kStages < rounds) load(it + kStages);
    if constexpr (!CL) {
      h = finish(it, carry[(it & 1) ^ 1][l], n, e, now);
      if (threadIdx.x >= kGatedThreads - 16) carry[it & 1][l] = h;
    } else {
      // the whole tile's map, to every CTA, half of them from each half. The place that it
      // takes there was read two rounds ago, before the maps of the last round were sent.
      if (warp == 0) {
        const auto &map = maps[it & 1];
        ulonglong2 all = map[0][l];
#pragma unroll
        for (int r = 1; r < kRuns; ++r) all = then<PACKED>(all, map[r][l]);
        for (int r = it == p.wait.maps ? K : half; r < K; r += 2) send(&tiles[it & 1][rank][l], &here[it & 1], r, all);
      }
      fine = mbar_wait_cluster(&here[it & 1], (it >> 1) & 1, p.err, kErrWaitReady, fine ? p.wait.limit : 1) && fine;
      if (threadIdx.x == 0 && fine && it + 2 < rounds) expect_maps(it + 2);
      f2 start = h;
      for (int r = 0; r < K; ++r) {
        if (r == rank) start = h;
        h = through<PACKED>(tiles[it & 1][r][l], h);
      }
      finish(it, start, n, e, now);
    }
  }
  if constexpr (CL) cluster_sync();  // nobody leaves while its shared memory is written to
  if constexpr (!PACKED) {
    // The last token's state, from the half warp that has the token. Over tokens past the
    // end an infinite state does not stay (0 * inf): there the output has it.
    const int left = p.tokens - (tile_of(rounds - 1) * kGatedTile + run * S);
    if (p.last && left > 0 && left <= S) {
      Two<T, PAIR> o;
      if constexpr (TMA) {
        o.load(&sm.out[warp][half * S + left - 1][2 * l], true, true);
      } else {
        o.load(out + (p.tokens - 1) * p.so[1], ok0, ok1);
      }
      const float2 w = upk(h), q = upk(o.widen());
      me.put_pair(p.last + (long long)b * p.dim, pk(w.x == w.x ? w.x : q.x, w.y == w.y ? w.y : q.y));
    }
  }
  if constexpr (TMA) {
    if (lane == 0) stores_done();
    if (!fine && threadIdx.x == 0) {  // a wait gave up: the copies under way land before the CTA leaves
      for (int it = max(asked - kStages, 0); it < asked; ++it)
        mbar_wait(&sm.full[it % kStages], (it / kStages) & 1, p.err, kErrWaitFull, p.wait.limit);
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
  const long long units = (long long)p.batch * p.channel_tiles;
  if (!CL) {
    if (p.plan.segs > 1) {
      ss_gated_maps_kernel<T, ROWS != kSingles, IG, PACKED><<<(unsigned)(units * (p.plan.segs - 1)), kGatedThreads, 0, s>>>(p);
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
template <typename T, int ROWS, bool IG>
cudaError_t form(const GatedScanParams &p, const ScanMaps &tm, cudaStream_t s) {
  const bool cl = p.plan.cluster > 1;
  if (p.token_request) return cl ? launch<T, ROWS, IG, true, true>(p, tm, s) : launch<T, ROWS, IG, true, false>(p, tm, s);
  return cl ? launch<T, ROWS, IG, false, true>(p, tm, s) : launch<T, ROWS, IG, false, false>(p, tm, s);
}
template <typename T>
cudaError_t pick(int rows, TensorMapEncode enc, const GatedScanParams &p, cudaStream_t s) {
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

// Clusters read everything once, but have 8 CTAs at most. Wider ones, which not every
// device runs, gain forward where sequences are long (64 units of 1024 tiles 7%) and lose
// in shorter ones (48 units of 63 tiles 46%) and backward (64 units of 128 tiles 16%). With
// few units they leave SMs idle, and segments, which read the rows a second time, are
// faster from two rounds of a cluster on. Forward / forward and backward in us, bf16:
//                                            clusters    segments
//   16 units, 1024 tiles                    192 / 522   111 / 276
//   32 units, 256 tiles                      54 / 143    59 / 140
//   48 units, 63 tiles                       19 / 50     25 / 55
//   64 units, 128 tiles                      40 / 108    58 / 139
//   80 units, 256 tiles                      86 / 241   139 / 344
//   11 units, 94 tiles, packed, 17 requests  35          18
//   32 units, 256 tiles, packed, 40          85          54
//   48 units, 256 tiles, packed, 40          90          71
//   80 units, 256 tiles, packed, 40         114         104
//   the same, one request                   104         143
//   the same, one of 40 with most tokens    110         141
// A packed segment reduces only the request that goes on after it, so segments gain for
// more units there, but lose a third where one request has most of the tokens. The host,
// which has to choose, does not know the lengths: the same 40 units.
// All CTAs of a cluster run at once: as many of them as leave all clusters resident. The
// kernel's registers leave room for a sixth CTA an SM, without which clusters of 8 or 7 do
// not all find a place (90 units 32 us, 38 with five; packed 40, 54).
GatedPlan gated_plan(int dtype, long long units, int tiles) {
  constexpr int kSms = 152, kSegCtas = 6;           // segments that an SM holds
  const int kClusterCtas = dtype == 0 ? 3 : 5;      // CTAs of clusters that it holds, by shared memory
  GatedPlan plan{1, 1, tiles};
  if (units < 1 || tiles < 2) return plan;
  if (units < 40 && tiles > 2 * kGatedMostCluster) {
    const long long segs = std::min<long long>(std::min<long long>(kSms * kSegCtas / units, kGatedMostSegs), tiles);
    plan.seg_tiles = (int)((tiles + segs - 1) / segs);
    plan.segs = (tiles + plan.seg_tiles - 1) / plan.seg_tiles;
    return plan;
  }
  const long long k = std::min<long long>(std::min<long long>(kSms * kClusterCtas / units, kGatedMostCluster), tiles);
  if (k > 1) plan.cluster = (int)k;
  return plan;
}

cudaError_t launch_gated_scan(int dtype, int rows, TensorMapEncode enc, const GatedScanParams &given, cudaStream_t s) {
  GatedScanParams p = given;
  p.wait = wait_hook();
  return dtype == 0   ? pick<float>(rows, enc, p, s)
         : dtype == 1 ? pick<__half>(rows, enc, p, s)
                      : pick<__nv_bfloat16>(rows, enc, p, s);
}

}  // namespace ssk
