// Request tables of a packed batch: offsets, token -> request and position maps,
// block table and slot map from the request lengths (include/ssfwd_packed.h).
//
// One launch. Every CTA sums the lengths by itself (requests are few against
// tokens: 4 bytes each, out of L2 after the first CTA) and keeps the offsets in
// shared memory, then writes its own share of the token maps and of the block
// table, each entry found by bisection. A second launch, or a hand-over from CTA to
// CTA, would cost more than the sums. Bound by latency: 7.5 us for 66 requests and
// 1100 tokens, 8.9 for 1000 and 200000 (cold; two sums and one bisection each); 5.0
// and 6.0 in a captured graph.
#include <atomic>

#include "ss_packed.h"
#include "ssfwd_packed.h"

namespace ssk {
namespace {

// Shared memory of three tables over the requests.
constexpr int table_bytes(int requests) { return 3 * (requests + 1) * (int)sizeof(int); }

constexpr int kThreads = 512;
constexpr int kTokensPerCta = kThreads * 4;

// Exclusive sums over the CTA's threads; returns the sum of all in `total`.
__device__ __forceinline__ long long block_exclusive(long long v, long long *sm, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();  // sm may still be read from an earlier call
  if (lane == 31) sm[warp] = inc;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm[w];
    all += sm[w];
  }
  total = all;
  return before + inc - v;
}

// The last index r in [0, n) with starts[r] <= v (starts ascend, starts[0] <= v).
__device__ __forceinline__ int last_at_or_before(const int *starts, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) ss_request_tables_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ int sm_tab[];
  int *off = sm_tab;                    // requests + 1
  int *bst = sm_tab + p.requests + 1;   // requests + 1: first block of each request
  int *nst = bst + p.requests + 1;      // requests + 1: requests before it that have tokens
  __shared__ long long sums[kThreads / 32];
  const int tid = threadIdx.x;
  const int per = (p.requests + kThreads - 1) / kThreads;
  const int r0 = min(tid * per, p.requests), r1 = min(r0 + per, p.requests);

  // offsets, cut at the number of tokens; lengths are added in 64 bits
  long long mine = 0, total;
  int negative = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = p.lengths[r];
    negative |= n < 0;
    mine += max(n, 0);
  }
  long long run = block_exclusive(mine, sums, total);
  for (int r = r0; r < r1; ++r) {
    off[r] = (int)min(run, (long long)p.tokens);
    run += max(p.lengths[r], 0);
  }
  if (tid == 0) off[p.requests] = (int)min(total, (long long)p.tokens);
  int errors = total > p.tokens ? 1 : 0;
  __syncthreads();
  // first block of each request (low half), requests before it that need a slot
  // (upper 16 bits) and that have tokens (16 bits below)
  mine = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = off[r + 1] - off[r];
    mine += (n + p.block - 1) / p.block;
    if (n > 0) mine += 1ll << 32;
    if (p.slots && p.slots[r] < 0) mine += 1ll << 48;
  }
  run = block_exclusive(mine, sums, total);
  const int nblocks = (int)(total & 0xffffffff), wanted = (int)(total >> 48);
  for (int r = r0; r < r1; ++r) {
    bst[r] = (int)(run & 0xffffffff);
    nst[r] = (int)((run >> 32) & 0xffff);
    run += (off[r + 1] - off[r] + p.block - 1) / p.block + (off[r + 1] > off[r] ? 1ll << 32 : 0ll);
    if (blockIdx.x == 0) {
      int slot = r;
      if (p.slots) {
        slot = p.slots[r];
        if (slot < 0) {
          const int k = (int)(run >> 48);
          slot = p.free_slots && k < p.free ? p.free_slots[k] : -1;
          run += 1ll << 48;
        }
      }
      p.slot_map[r] = slot;
      p.offsets[r] = off[r];
    }
  }
  if (wanted > p.free || (wanted > 0 && !p.free_slots)) errors |= 4;
  if (__syncthreads_or(negative)) errors |= 2;
  const int live = off[p.requests];
  if (blockIdx.x == 0 && tid == 0) {
    p.offsets[p.requests] = live;
    p.counts[0] = live;
    p.counts[1] = nblocks;
    p.counts[2] = min(wanted, p.free_slots ? p.free : 0);
    p.counts[3] = errors;
  }

  const int step = gridDim.x * kThreads;
  for (int i = blockIdx.x * kThreads + tid; i < p.max_blocks; i += step) {
    int4 row = make_int4(-1, 0, 0, 0);
    if (i < nblocks) {
      const int r = last_at_or_before(bst, p.requests, i);
      const int k = i - bst[r];
      const int first = off[r] + k * p.block;
      row = make_int4(r, first, min(off[r + 1] - first, p.block), k);
    }
    reinterpret_cast<int4 *>(p.blocks)[i] = row;
    // each request before this one has one last block, which is not listed
    if (row.x >= 0 && row.y + row.z < off[row.x + 1]) p.carried[i - nst[row.x]] = i;
  }
  const int carried = nblocks - (int)((total >> 32) & 0xffff);
  for (int i = carried + blockIdx.x * kThreads + tid; i < p.tokens / p.block; i += step) p.carried[i] = -1;

  // four tokens a thread: one bisection, then on along the offsets
  for (long long t0 = ((long long)blockIdx.x * kThreads + tid) * 4; t0 < p.tokens; t0 += (long long)step * 4) {
    int r = last_at_or_before(off, p.requests, (int)t0);
    int req[4], pos[4];
    int at = off[r], ctx = p.context ? p.context[r] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = (int)t0 + k;
      if (t >= live) {
        req[k] = -1;
        pos[k] = 0;
        continue;
      }
      if (t >= off[r + 1]) {
        do ++r; while (t >= off[r + 1]);
        at = off[r];
        ctx = p.context ? p.context[r] : 0;
      }
      req[k] = r;
      pos[k] = ctx + t - at;
    }
    if (t0 + 4 <= p.tokens) {
      reinterpret_cast<int4 *>(p.token_request)[t0 >> 2] = make_int4(req[0], req[1], req[2], req[3]);
      reinterpret_cast<int4 *>(p.token_position)[t0 >> 2] = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t0 + k < p.tokens) {
          p.token_request[t0 + k] = req[k];
          p.token_position[t0 + k] = pos[k];
        }
    }
  }
}

}  // namespace

cudaError_t launch_request_tables(const TablesParams &p, cudaStream_t s) {
  // at most one CTA per SM, so that the sums are repeated no more often than that
  const long long want = ((long long)p.tokens + kTokensPerCta - 1) / kTokensPerCta;
  const int grid = (int)(want < 1 ? 1 : want > 152 ? 152 : want);
  const int smem = table_bytes(p.requests);
  // Opted in once per device (the attribute is per device), always to what the most
  // requests need: a call's own size could be put in place of another thread's larger
  // one, and the 48 KB that need no opt-in have to hold the kernel's static part too.
  static std::atomic<bool> opted[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !opted[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute((const void *)&ss_request_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             table_bytes(SS_MAX_REQUESTS));
    if (e != cudaSuccess) return e;
    if (dev < 64) opted[dev].store(true, std::memory_order_relaxed);
  }
  ss_request_tables_kernel<<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssk
