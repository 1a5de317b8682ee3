// Selective scan with one decay per head over packed requests, 16-bit operands,
// on the tensor cores (include/ssfwd_packed.h; ss_head_scan.cu has the form for
// every type and size).
//
// Mathematics. With a_t = dt_t A and L_t its running sum, inside a chunk of 128
// tokens of one request that starts with state S (headdim x dstate):
//   Y   = (C B^T * M) X + e^L (C S^T),   M[t,s] = e^(L_t - L_s) dt_s for s <= t, else 0
//   S'  = e^(L_end) S + (w X)^T B,       w_s = e^(L_end - L_s) dt_s
// so a chunk is four products of 128-row matrices, and only S goes from chunk to
// chunk. Exponents are never split so that a factor can exceed 1: M takes the
// exponential of a difference inside its diagonal blocks of 32, and elsewhere
// the product of (row: since the end of the column's block) and (column: to the
// end of its block), each a sum of terms of one sign.
//
// One CTA carries 128 (head, p) columns, two heads of 64 or one of 128, through
// one block of a request. C B^T and the operands C and B are shared by its heads.
//   warps 0 - 15   mask C B^T and scale C S^T by e^L, then finish the output
//                  (thread = row t, a warp one quarter of the columns); some also
//                  prepare the decays of the chunk after the next
//   warps 16 - 23  weigh: S to the chunk's start, X to w X (thread = column p)
//   warp 24        loads the chunks by TMA (boxes of 128 tokens x 64 values),
//                  warp 27 stores the output the same way
//   warp 25        issues the products for Y, warp 26 those for S (tcgen05,
//                  accumulators in tensor memory)
// Both groups run side by side: what is between chunks is only S.
// Tensor memory, 512 columns: C B^T, overlaid block by block by the masked forms
// as the product's A operand (128); Y (128); S (128); w X as A operand (128).
//
// What bounds it: the instructions of the scaling warps. A chunk of two heads of 64
// with 128 states is 56 products (2,500 cycles of the tensor pipe) and about 19,000
// warp instructions, a quarter of them the split of w X into exact terms; it takes
// about 4.1 us (5.2 with the gate). 8 requests x 2048 tokens x 24 heads: 92 us on 96
// CTAs; 65536 tokens x 32 heads: 340 us, of which the summaries take 90. To let the
// row warps weigh a quarter of the next chunk, which shortens the column warps' part,
// changed nothing (91 and 355, against 91 and 347): it is the sum that counts. The
// first form, one group of warps that did all steps in turn with its loops unrolled,
// took 204 and 802 us and spent half of that waiting for instructions.
//
// Rounding. C B^T takes the stored B and C; its masked form and the S that C
// multiplies are rounded to 16 bits, about what rounding the output costs. S
// itself stays in fp32 from chunk to chunk: w X enters in three bf16 terms (24
// bits, exact) or two fp16 terms, with w scaled by a power of two per head and
// chunk (summaries: block) that brings its largest to [1/2, 1). No x then leaves
// fp16, and a term is off by at most 2^-22 of itself or 2^-24 of the largest w.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "ss_fwd_kernel.cuh"
#include "ss_packed.h"

namespace ssk {
namespace {

constexpr int kBox = 16384;      // 128 rows of 128 bytes
constexpr int kBoxes = 10;       // X twice, B (then z) twice, C once, two boxes each
constexpr int kTcThreads = 896;  // 16 row warps, 8 column warps, TMA loads, 2 x MMA, TMA stores
constexpr uint32_t kColG = 0, kColY = 128, kColS = 256, kColX = 384;
constexpr int32_t kErrTcWait = 16;

struct TcMaps {
  CUtensorMap x, B, C, z, out;
};

struct Shared {
  uint64_t full_x[2], full_b[2], full_c, full_z[2];  // loaded
  uint64_t empty_x[2], empty_b[2], empty_c;          // may be loaded again
  uint64_t masked, y_done, y_free, s_ready, gy_done;
  uint64_t weighed[2], gained[2];  // by buffer of w X: written; taken in by S
  // Who waits on these does not hold up who arrives for a chunk or more: one
  // barrier for each chunk that the latter can be ahead.
  uint64_t x_read[2];    // columns -> rows (and products for Y): X's columns are read, its rows may be overwritten
  uint64_t finished[4];  // rows -> storing
  uint64_t prepared[4];  // rows -> rows and columns: the chunk's decays
  uint32_t tmem;
  int dead;
  // of chunk c in stage c % 4, by head of the tile
  alignas(16) float tot[4][2][4];       // log2 decay of each 32 tokens
  float top[4][2][4];                   // largest |colf| of each 32 tokens (fp16)
  alignas(16) float nl[4][2][128];      // minus the log2 decay since the start of the 32
  alignas(16) float dt[4][2][128];
  alignas(16) float colf[4][2][128];    // dt times the decay to the end of the 32
  // pairs of 16 columns on the diagonal that are at or before a row, by the row's
  // place in its 32 and the half of them that the columns are
  alignas(16) uint32_t before[2][32][8];
};

// The code runs once per chunk in several roles at once, so its size counts (the
// first, fully unrolled form spent half of its time waiting for instructions):
// loops over pieces of 16 columns stay rolled, and what a wait does when the
// barrier is not there yet is not inlined.
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *dead, int32_t *err) {
  for (uint32_t i = 0; i < kMaxWaitIters; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
  }
  *dead = 1;
  atomicCAS(err, 0, kErrTcWait);
  return false;
}
__device__ __forceinline__ bool wait_tc(uint64_t *bar, uint32_t parity, volatile int *dead, int32_t *err) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, dead, err);
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
         (2ull << 61);  // 128-byte swizzle
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 16 columns of the warp's 32 lanes (thread = lane). The values of tm_ld16_async
// are there after tm_wait on the same registers.
__device__ __forceinline__ void tm_ld16_async(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_wait(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&v)[16]) {
  tm_ld16_async(addr, v);
  tm_wait(v);
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tm_st4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *tm, const void *src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tm)),
               "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
               : "memory");
}

// Four states of a row, `left` of them in it.
__device__ __forceinline__ float4 get4(const float *src, int left, bool vec) {
  if (vec) return *reinterpret_cast<const float4 *>(src);
  return make_float4(src[0], left > 1 ? src[1] : 0.f, left > 2 ? src[2] : 0.f, left > 3 ? src[3] : 0.f);
}
__device__ __forceinline__ void put4(float *dst, float4 v, int left, bool vec) {
  if (vec) {
    *reinterpret_cast<float4 *>(dst) = v;
  } else {
    dst[0] = v.x;
    if (left > 1) dst[1] = v.y;
    if (left > 2) dst[2] = v.z;
    if (left > 3) dst[3] = v.w;
  }
}

// Barrier of the 8 column warps.
__device__ __forceinline__ void sync_weighers() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// One arrival per warp, after all its lanes.
__device__ __forceinline__ void arrive_warp(uint64_t *bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <typename T>
__device__ __forceinline__ float lds_16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  T t;
  memcpy(&t, &v, 2);
  return to_f<T>(t);
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 pku(uint32_t lo, uint32_t hi) { return pk(__uint_as_float(lo), __uint_as_float(hi)); }
template <typename T>
__device__ __forceinline__ f2 wide(uint32_t w) {  // two 16-bit values as a packed fp32 pair
  const float2 v = unpack2<T>(w);
  return pk(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(f2 v) {
  const float2 f = upk(v);
  return pack2<T>(f.x, f.y);
}

// Two fp32 values as 16-bit terms of decreasing size, packed: hi + mid (+ lo).
template <typename T> struct Terms;
template <> struct Terms<__nv_bfloat16> {
  static constexpr int N = 3;  // by truncation, 8 bits each
  static __device__ __forceinline__ void split(f2 v, uint32_t (&t)[3]) {
    const f2 minus = pk(-1.f, -1.f);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const float2 f = upk(v);
      const uint32_t x = __float_as_uint(f.x), y = __float_as_uint(f.y);
      t[k] = __byte_perm(x, y, 0x7632);
      if (k < 2) v = fma2(pku(x & 0xffff0000u, y & 0xffff0000u), minus, v);
    }
  }
};
template <> struct Terms<__half> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void split(f2 v, uint32_t (&t)[2]) {
    t[0] = narrow<__half>(v);
    t[1] = narrow<__half>(fma2(wide<__half>(t[0]), pk(-1.f, -1.f), v));
  }
};

// log2 of a step's decay (the product with A first: A log2(e) may be infinite where
// dt A is not). Below -128 nothing is left (ex2 gives 0); in sums of which differences
// are taken, a larger number would only round away the steps beside it, or make the
// difference one of infinities. Sums over 32 tokens so end at 4096, where a unit is
// 5e-4. NaN stays NaN.
__device__ __forceinline__ float log2_step(float dt, float A) {
  const float l = dt * A * kLog2e;
  return l < -128.f ? -128.f : l;
}

// Instruction descriptor of a product of two T operands into fp32, M = 128.
template <typename T>
constexpr uint32_t kIdesc = (1u << 4) | ((Terms<T>::N == 3 ? 1u : 0u) << 7) | ((Terms<T>::N == 3 ? 1u : 0u) << 10) | (8u << 24);

// What a CTA works on: HT heads of a group through one block of a request.
struct Place {
  int h0, hend, grp, blk;             // first head, end of the group's heads, group, row of the block table
  int r, first, size, index, last;    // request (-1: none), the block's tokens, its index and that of the request's last block
  long long slot;
  bool kept, goes_on;                 // the request has a slot, and starts from it
};
template <int HT, bool CARRIED>  // CARRIED: over the rows of t.carried
__device__ __forceinline__ Place place_of(const HeadScanParams &p) {
  Place w;
  const int tpg = (p.hpg + HT - 1) / HT, tiles = p.heads / p.hpg * tpg, tile = blockIdx.x % tiles;
  w.blk = blockIdx.x / tiles;
  w.grp = tile / tpg;
  w.h0 = w.grp * p.hpg + (tile % tpg) * HT;
  w.hend = (w.grp + 1) * p.hpg;
  w.r = -1;
  if (CARRIED) {
    w.blk = p.t.carried[w.blk];
    if (w.blk < 0) return w;
  } else if (w.blk == p.t.max_blocks) {
    return w;
  }
  const int4 row = reinterpret_cast<const int4 *>(p.t.blocks)[w.blk];
  w.r = row.x;
  w.first = row.y;
  w.size = row.z;
  w.index = row.w;
  if (w.r < 0) return w;
  w.last = (p.t.offsets[w.r + 1] - p.t.offsets[w.r] - 1) / p.t.block;
  w.slot = p.state ? p.t.slot_map[w.r] : -1;
  w.kept = w.slot >= 0 && w.slot < p.slots;
  w.goes_on = w.kept && p.t.context && p.t.context[w.r] > 0;
  return w;
}
// Row pp of head h of a request's kept state, and of its block i's summary.
__device__ __forceinline__ float *cache_row(const HeadScanParams &p, const Place &w, int h, int pp) {
  return p.state + w.slot * p.ss[0] + h * p.ss[1] + (long long)pp * p.dstate;
}
__device__ __forceinline__ long long entry_of(const HeadScanParams &p, const Place &w, int h, int i) {
  return (long long)(w.blk - w.index + i) * p.heads + h;
}
__device__ __forceinline__ float *entry_row(const HeadScanParams &p, const Place &w, int h, int pp, int i) {
  return p.ws_state + (entry_of(p, w, h, i) * p.headdim + pp) * p.dstate;
}

// ---- summaries of a block: the state it ends in ----
//
// Its own gain, with S_0 = 0 but in a request's first block:
// S_end = e^(L_end) S_0 + (w X)^T B over the whole block, w_s = e^(L_end - L_s) dt_s:
// from its last chunk to its first, so that the decay to the block's end is known
// when a chunk is weighed, and S is one sum that no chunk has to scale.
//   warps 0 - 15   weigh (thread = column p, a warpgroup 32 of the chunk's tokens)
//   warps 16 - 23  prepare w (thread = token, a warpgroup per head)
//   warp 24 loads by TMA, warp 25 issues the products
// w X has two buffers of 128 tokens x 3 terms in tensor memory; X and B have
// three places. Bound by the weighing warps' instructions.
constexpr int kSumThreads = 832, kSumStages = 3;

struct SumShared {
  uint64_t full[kSumStages], empty[kSumStages], prepared[2], taken[2], weighed[2], gained[2];
  uint32_t tmem;
  int dead;
  float part[2][2][4], top[2][4];
  float total[2], scale[2];      // by head: log2 decay of the block; scale of w
  alignas(16) float w[2][2][128];
};

template <typename T, int PW, int NS>
__global__ void __launch_bounds__(kSumThreads, 1)
    ss_head_scan_sum_tc_kernel(const __grid_constant__ HeadScanParams p, const __grid_constant__ TcMaps maps) {
  constexpr int HT = 128 / PW, NB = NS / 64, NT = Terms<T>::N, NQ = NS / 4;
  constexpr uint32_t kColSum = 0, kColW = 128;
  extern __shared__ unsigned char raw[];
  unsigned char *ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  SumShared &sh = *reinterpret_cast<SumShared *>(ring + kSumStages * (2 + NB) * kBox);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wq = warp & 3, wg = (warp >> 2) & 3;
  let_next_start();
  const Place at = place_of<HT, true>(p);
  if (at.r < 0) return;
  const int pc = wq * 32 + lane, hs = HT == 2 ? pc >> 6 : 0, pp = HT == 2 ? pc & 63 : pc, h = at.h0 + hs;
  const bool pin = warp < 16 && h < at.hend && pp < p.headdim;
  const int n0 = wg * NQ, nv = min(max(p.dstate - n0, 0), NQ);  // this thread's states of its column
  if (tid == 0) {
    for (int i = 0; i < kSumStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 17);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.prepared[i], 4 * HT);
      mbar_init(&sh.taken[i], 16);
      mbar_init(&sh.weighed[i], 16);
      mbar_init(&sh.gained[i], 1);
    }
    sh.dead = 0;
    fence_barrier_init();
  }
  if (warp == 25) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before();
  }
  __syncthreads();
  fence_after();
  const uint32_t tm = sh.tmem, lane_at = (uint32_t)(wq * 32) << 16;
  volatile int *dead = &sh.dead;
  const int chunks = (at.size + 127) / 128;  // i-th from the end: chunk chunks - 1 - i
  auto xbox = [&](int i, int k) { return ring + ((i % kSumStages) * (2 + NB) + k) * kBox; };
  auto bbox = [&](int i, int k) { return xbox(i, 2 + k); };

  if (warp == 24) {
    // ---- TMA ----
    if (lane == 0) {
      int n = 0;
      for (int i = 0; i < chunks && !*dead; ++i, ++n) {
        const int s = i % kSumStages, t = at.first + (chunks - 1 - i) * 128;
        if (i >= kSumStages && !wait_tc(&sh.empty[s], (i / kSumStages - 1) & 1, dead, p.err)) break;
        mbar_arrive_expect_tx(&sh.full[s], (2 + NB) * kBox);
        for (int k = 0; k < 2; ++k)
          tma_load_3d(xbox(i, k), &maps.x, &sh.full[s], HT == 2 ? 0 : 64 * k, HT == 2 ? at.h0 + k : at.h0, t);
        for (int k = 0; k < NB; ++k) tma_load_3d(bbox(i, k), &maps.B, &sh.full[s], 64 * k, at.grp, t);
      }
      // nothing of this block's copies is left in flight, whatever became of the rest
      for (int i = max(0, n - kSumStages); i < n; ++i)
        for (uint32_t k = 0; k < kMaxWaitIters; ++k)
          if (mbar_try_wait(&sh.full[i % kSumStages], (i / kSumStages) & 1)) break;
      // The tensor cores arrive on these after what the other warps wait for: the CTA
      // stays until they have, or they would write to shared memory that is another's.
      for (int i = max(0, chunks - kSumStages); i < chunks && !*dead; ++i)
        wait_tc(&sh.empty[i % kSumStages], (i / kSumStages) & 1, dead, p.err);
    }
  } else if (warp == 25) {
    // ---- products ----
    constexpr uint32_t id_s = kIdesc<T> | (1u << 16) | ((uint32_t)NS / 8 << 17);  // w X x B: B is N-major
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
      wait_tc(&sh.full[i % kSumStages], (i / kSumStages) & 1, dead, p.err);
      wait_tc(&sh.weighed[i & 1], (i >> 1) & 1, dead, p.err);
      fence_after();
      const uint64_t bd = smem_desc(smem_u32(bbox(i, 0)), kBox, 1024);
      __syncwarp();
      if (elect() && !*dead) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int e = 0; e < NT; ++e)
            mma_ts(tm + kColSum, tm + kColW + 192 * (i & 1) + 64 * e + 8 * k, bd + ((k * 2048) >> 4), id_s, i > 0 || k > 0 || e > 0);
        commit(&sh.gained[i & 1]);
        commit(&sh.empty[i % kSumStages]);
      }
    }
  } else if (warp >= 16) {
    // ---- w: thread = token, warpgroup = head ----
    const int tp = wg, trow = pc;
    if (tp < HT) {
      const int hp = at.h0 + tp < at.hend ? at.h0 + tp : at.h0;
      const float A = p.A[hp], bias = p.bias ? p.bias[hp] : 0.f;
      auto raw_at = [&](int t) -> float {  // token t of the block
        if (t >= at.size) return 0.f;
        const long long k = (long long)(at.first + t) * p.sdt[0] + hp * p.sdt[1];
        return p.dt_f32 ? static_cast<const float *>(p.dt)[k] : to_f<T>(static_cast<const T *>(p.dt)[k]);
      };
      auto load_dt = [&](int i) -> float { return i < chunks ? raw_at((chunks - 1 - i) * 128 + trow) : 0.f; };
      float later = 0.f, scale = 1.f, raw_dt = load_dt(0);  // later: log2 decay of the chunks after this one
      if (NT == 2) {
        // One power of two for the whole block, that brings its largest w to [1/2, 1), as
        // the scan does for a chunk: w X then stays within fp16 for every x. A thread
        // walks a run of the block's tokens from its end; what follows a run is joined
        // afterwards. The margin covers what the order of these sums makes of w.
        float m = 0.f, run = 0.f;  // largest w of the run, with the decay to its end; log2 decay of the run
#pragma unroll 8
        for (int i = chunks - 1; i >= 0; --i) {
          const int t = trow * chunks + i;
          float dt = raw_at(t) + bias;
          if (p.softplus) dt = softplus_f(dt);
          if (t >= at.size) continue;
          m = fmaxf(m, fabsf(dt) * ex2(run));
          run += log2_step(dt, A);
        }
        float to_end = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float dn = __shfl_down_sync(0xffffffffu, to_end, o);
          if (lane + o < 32) to_end += dn;
        }
        const float nx = __shfl_down_sync(0xffffffffu, to_end, 1);
        m *= ex2(lane < 31 ? nx : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) {
          sh.top[tp][wq] = m;
          sh.part[1][tp][wq] = to_end;  // read before the barrier of the first chunk, written after it
        }
        asm volatile("bar.sync %0, 128;" ::"r"(2 + tp) : "memory");
        float after = 0.f;
        m = 0.f;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          m = fmaxf(m, sh.top[tp][k] * ex2(after));
          after += sh.part[1][tp][k];
        }
        const int e = (int)(__float_as_uint(m * 1.015625f) >> 23);
        scale = e < 64 || e > 190 ? 1.f : __uint_as_float((uint32_t)(253 - e) << 23);
      }
#pragma unroll 1
      for (int i = 0; i < chunks; ++i) {
        float dt = raw_dt + bias;
        if (p.softplus) dt = softplus_f(dt);
        const bool in = (chunks - 1 - i) * 128 + trow < at.size;
        if (!in) dt = 0.f;
        raw_dt = load_dt(i + 1);
        float to_end = in ? log2_step(dt, A) : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float dn = __shfl_down_sync(0xffffffffu, to_end, o);
          if (lane + o < 32) to_end += dn;
        }
        if (lane == 0) sh.part[i & 1][tp][wq] = to_end;
        const float nx = __shfl_down_sync(0xffffffffu, to_end, 1);
        asm volatile("bar.sync %0, 128;" ::"r"(2 + tp) : "memory");
        float after = later, total = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float t = sh.part[i & 1][tp][k];
          if (k > wq) after += t;
          total += t;
        }
        later += total;
        float w = dt * ex2(after + (lane < 31 ? nx : 0.f));
        if (i >= 2) wait_tc(&sh.taken[i & 1], ((i >> 1) - 1) & 1, dead, p.err);
        sh.w[i & 1][tp][trow] = w * scale;
        if (trow == 0) {
          sh.total[tp] = later;
          sh.scale[tp] = scale;
        }
        arrive_warp(&sh.prepared[i & 1], lane);
      }
    }
  } else {
    // ---- w X: thread = column, warpgroup = 32 tokens ----
    const int valid = at.size - (chunks - 1) * 128;  // of the first chunk in this order
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
      wait_tc(&sh.full[i % kSumStages], (i / kSumStages) & 1, dead, p.err);
      if (i == 0 && valid < 128) {  // rows of the next request, or of nothing: 0 x anything must be 0
        const int todo = (128 - valid) * 8;
        for (int k = tid; k < todo * (2 + NB); k += 512)
          *reinterpret_cast<uint4 *>(xbox(0, k / todo) + (valid + k % todo / 8) * 128 + (k % 8) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        asm volatile("bar.sync 1, 512;" ::: "memory");
      }
      wait_tc(&sh.prepared[i & 1], (i >> 1) & 1, dead, p.err);
      if (i >= 2) {
        wait_tc(&sh.gained[i & 1], ((i >> 1) - 1) & 1, dead, p.err);
        fence_after();
      }
      uint32_t col = smem_u32(xbox(i, pc >> 6)) + wg * 32 * 128 + (pc & 63) * 2;  // in row 0 of a swizzle atom
      const float *wf = sh.w[i & 1][hs] + wg * 32;
      uint32_t to = tm + lane_at + kColW + 192 * (i & 1) + 16 * wg;
#pragma unroll 1
      for (int j = 0; j < 4; ++j) {
        uint32_t t[NT][4];
        const float4 wa = *reinterpret_cast<const float4 *>(wf), wb = *reinterpret_cast<const float4 *>(wf + 4);
        const f2 w[4] = {pk(wa.x, wa.y), pk(wa.z, wa.w), pk(wb.x, wb.y), pk(wb.z, wb.w)};
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = lds_16<T>((col ^ (k << 4)) + k * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t a[NT];
          Terms<T>::split(mul2(pk(x[2 * k], x[2 * k + 1]), w[k]), a);
#pragma unroll
          for (int e = 0; e < NT; ++e) t[e][k] = a[e];
        }
#pragma unroll
        for (int e = 0; e < NT; ++e) tm_st4(to + 64 * e, t[e]);
        col += 8 * 128;
        wf += 8;
        to += 4;
      }
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.weighed[i & 1]);
        mbar_arrive(&sh.taken[i & 1]);
        mbar_arrive(&sh.empty[i % kSumStages]);
      }
    }
    wait_tc(&sh.gained[(chunks - 1) & 1], ((chunks - 1) >> 1) & 1, dead, p.err);
    fence_after();
    const float keep = ex2(sh.total[hs]);
    const float unscale = __uint_as_float((254u << 23) - __float_as_uint(sh.scale[hs]));  // a power of two
#pragma unroll 1
    for (int n = 0; n < NQ; n += 16) {
      uint32_t v[16];
      tm_ld16(tm + lane_at + kColSum + n0 + n, v);
      if (!pin || *dead) continue;
      const float *start = at.index == 0 && at.goes_on ? cache_row(p, at, h, pp) + n0 : nullptr;
      float *dst = entry_row(p, at, h, pp, at.index) + n0;
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        if (n + k < nv) {
          float4 f = make_float4(__uint_as_float(v[k]) * unscale, __uint_as_float(v[k + 1]) * unscale,
                                 __uint_as_float(v[k + 2]) * unscale, __uint_as_float(v[k + 3]) * unscale);
          if (start) {
            // the last block's entry keeps the start, which the cache loses when that block ends
            const float4 q = get4(start + n + k, nv - n - k, p.vec != 0);
            put4(entry_row(p, at, h, pp, at.last) + n0 + n + k, q, nv - n - k, p.vec != 0);
            f = make_float4(fmaf(keep, q.x, f.x), fmaf(keep, q.y, f.y), fmaf(keep, q.z, f.z), fmaf(keep, q.w, f.w));
          }
          put4(dst + n + k, f, nv - n - k, p.vec != 0);
        }
    }
    if (pin && pp == 0 && wg == 0 && !*dead) p.ws_decay[entry_of(p, at, h, at.index)] = sh.total[hs];
    fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 25) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
  }
}

// ---- the scan of a block ----
// PW: columns of a head in the tile (64: two heads, 128: one). NS: padded dstate.
template <typename T, int PW, int NS, bool GATE>
__global__ void __launch_bounds__(kTcThreads, 1)
    ss_head_scan_tc_kernel(const __grid_constant__ HeadScanParams p, const __grid_constant__ TcMaps maps) {
  constexpr int HT = 128 / PW;
  constexpr int NB = NS / 64;  // boxes of B (and of C)
  constexpr int NT = Terms<T>::N;
  constexpr int NH = NS / 2;                            // states per thread of a column
  extern __shared__ unsigned char raw[];
  unsigned char *ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  unsigned char *s16 = ring + kBoxes * kBox;            // S in 16 bits: [NB][128 p][64 n], swizzled
  Shared &sh = *reinterpret_cast<Shared *>(s16 + NB * kBox);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Place at = place_of<HT, false>(p);
  const int h0 = at.h0, hend = at.hend, first = at.first, size = at.size, index = at.index;
  T *out = static_cast<T *>(p.out);
  if (at.r < 0) wait_for_previous();
  if (at.blk == p.t.max_blocks) {                       // past the last token: zeros
    const int cols = min(HT, hend - h0) * p.headdim;
    for (int t = p.t.counts[0] + warp; t < p.t.tokens; t += kTcThreads / 32)
      for (int i = lane; i < cols; i += 32)
        out[t * p.so[0] + (h0 + i / p.headdim) * p.so[1] + i % p.headdim] = from_f<T>(0.f);
    return;
  }
  if (at.r < 0) return;

  // thread = column: its head, row of the state and half of the states
  const int wg = (warp >> 2) & 1, wq = warp & 3;
  const int pc = wq * 32 + lane, hs = HT == 2 ? pc >> 6 : 0, pp = HT == 2 ? pc & 63 : pc;
  const bool pin = warp >= 16 && warp < 24 && h0 + hs < hend && pp < p.headdim;
  const int n0 = wg * NH, nv = min(max(p.dstate - n0, 0), NH);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.full_x[i], 1);
      mbar_init(&sh.full_b[i], 1);
      mbar_init(&sh.full_z[i], 1);
      mbar_init(&sh.empty_x[i], 1);
      mbar_init(&sh.empty_b[i], 2);  // both kinds of products read B
    }
    mbar_init(&sh.full_c, 1);
    mbar_init(&sh.empty_c, 1);
    mbar_init(&sh.masked, 16);
    mbar_init(&sh.s_ready, 8);
    mbar_init(&sh.y_free, 16);
    mbar_init(&sh.y_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.weighed[i], 8);
      mbar_init(&sh.gained[i], 1);
    }
    mbar_init(&sh.gy_done, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sh.x_read[i], 8);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.finished[i], 16);
      mbar_init(&sh.prepared[i], 4 * HT);
    }
    sh.dead = 0;
    fence_barrier_init();
  }
  if (tid < 512) {
    const int half = tid >> 8, row = (tid >> 3) & 31, c = 16 * half + 2 * (tid & 7);
    sh.before[half][row][tid & 7] = (c <= row ? 0xffffu : 0u) | (c + 1 <= row ? 0xffff0000u : 0u);
  }
  if (warp == 25) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sh.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    fence_before();
  }
  wait_for_previous();  // the start states
  __syncthreads();
  fence_after();
  const uint32_t tm = sh.tmem;
  const uint32_t lane_at = (uint32_t)(wq * 32) << 16;
  volatile int *dead = &sh.dead;
  const int chunks = (size + 127) / 128;
  auto xbox = [&](int c, int k) { return ring + (2 * (c & 1) + k) * kBox; };
  auto bbox = [&](int c, int k) { return ring + (4 + 2 * (c & 1) + k) * kBox; };  // later in the chunk z's
  unsigned char *const cbox = ring + 8 * kBox;
  auto full = [&](uint64_t *bars, int c) { wait_tc(&bars[c & 1], (c >> 1) & 1, dead, p.err); };

  if (warp == 24) {
    // ---- TMA ----
    if (lane == 0) {
      // C has one place: the next chunk's takes it once this chunk's products with
      // it are done. z takes the place of its chunk's B.
      int nx = 0, nb = 0, nc = 0, nz = 0;  // loads under way or done
      auto load_z = [&](int c) {
        if (!wait_tc(&sh.empty_b[c & 1], (c >> 1) & 1, dead, p.err)) return;
        mbar_arrive_expect_tx(&sh.full_z[c & 1], 2 * kBox);
        for (int k = 0; k < 2; ++k)
          tma_load_3d(bbox(c, k), &maps.z, &sh.full_z[c & 1], HT == 2 ? 0 : 64 * k, HT == 2 ? h0 + k : h0, first + c * 128);
        ++nz;
      };
      for (int c = 0; c < chunks && !*dead; ++c) {
        const int t = first + c * 128, before = ((c >> 1) - 1) & 1;
        if (c >= 2 && !wait_tc(&sh.empty_x[c & 1], before, dead, p.err)) break;
        mbar_arrive_expect_tx(&sh.full_x[c & 1], 2 * kBox);
        for (int k = 0; k < 2; ++k)
          tma_load_3d(xbox(c, k), &maps.x, &sh.full_x[c & 1], HT == 2 ? 0 : 64 * k, HT == 2 ? h0 + k : h0, t);
        ++nx;
        if (!GATE && c >= 2 && !wait_tc(&sh.empty_b[c & 1], before, dead, p.err)) break;
        mbar_arrive_expect_tx(&sh.full_b[c & 1], NB * kBox);
        for (int k = 0; k < NB; ++k) tma_load_3d(bbox(c, k), &maps.B, &sh.full_b[c & 1], 64 * k, at.grp, t);
        ++nb;
        if (c >= 1 && !wait_tc(&sh.empty_c, (c - 1) & 1, dead, p.err)) break;
        mbar_arrive_expect_tx(&sh.full_c, NB * kBox);
        for (int k = 0; k < NB; ++k) tma_load_3d(cbox + k * kBox, &maps.C, &sh.full_c, 64 * k, at.grp, t);
        ++nc;
        if (GATE && c >= 1) load_z(c - 1);
      }
      if (GATE && !*dead) load_z(chunks - 1);
      // nothing of this block's copies is left in flight, whatever became of the rest
      auto landed = [&](uint64_t *bar, uint32_t parity) {
        for (uint32_t k = 0; k < kMaxWaitIters; ++k)
          if (mbar_try_wait(bar, parity)) return;
      };
      for (int i = max(0, nx - 2); i < nx; ++i) landed(&sh.full_x[i & 1], (i >> 1) & 1);
      for (int i = max(0, nb - 2); i < nb; ++i) landed(&sh.full_b[i & 1], (i >> 1) & 1);
      for (int i = max(0, nz - 2); i < nz; ++i) landed(&sh.full_z[i & 1], (i >> 1) & 1);
      if (nc > 0) landed(&sh.full_c, (nc - 1) & 1);
      // The tensor cores' last arrivals, after what the other warps wait for (with the
      // gate, load_z has waited for them): they have to find this CTA still there.
      if (!GATE)
        for (int c = max(0, chunks - 2); c < chunks && !*dead; ++c) wait_tc(&sh.empty_b[c & 1], (c >> 1) & 1, dead, p.err);
    }
  } else if (warp == 25) {
    // ---- products for Y ----
    constexpr uint32_t id_g = kIdesc<T> | (128u / 8 << 17);                       // C B^T and C S^T: both K-major, N = 128
    constexpr uint32_t id_y = kIdesc<T> | (1u << 16) | ((uint32_t)PW / 8 << 17);  // masked x X: X is N-major
    const uint64_t sd = smem_desc(smem_u32(s16), 16, 1024);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = c & 1;
      full(sh.full_b, c);
      wait_tc(&sh.full_c, ph, dead, p.err);
      if (c > 0) wait_tc(&sh.y_done, ph ^ 1, dead, p.err);  // the masked forms' columns are free again
      fence_after();
      const uint64_t cd = smem_desc(smem_u32(cbox), 16, 1024), bd = smem_desc(smem_u32(bbox(c, 0)), 16, 1024);
      __syncwarp();
      if (elect() && !*dead) {
#pragma unroll
        for (int k = 0; k < NS / 16; ++k) {
          const uint32_t at = ((k / 4) * kBox + (k % 4) * 32) >> 4;
          mma_ss(tm + kColG, cd + at, bd + at, id_g, k > 0);
        }
      }
      if (c > 0) wait_tc(&sh.y_free, ph ^ 1, dead, p.err);
      wait_tc(&sh.s_ready, ph, dead, p.err);
      fence_after();
      __syncwarp();
      if (elect() && !*dead) {
#pragma unroll
        for (int k = 0; k < NS / 16; ++k) {
          const uint32_t at = ((k / 4) * kBox + (k % 4) * 32) >> 4;
          mma_ss(tm + kColY, cd + at, sd + at, id_g, k > 0);
        }
        commit(&sh.gy_done);
      }
      full(sh.full_x, c);
      if (size - c * 128 < 128) wait_tc(&sh.x_read[c & 1], (c >> 1) & 1, dead, p.err);  // rows past the request's end are cleared
      wait_tc(&sh.masked, ph, dead, p.err);
      fence_after();
      const uint64_t xd = smem_desc(smem_u32(xbox(c, 0)), kBox, 1024);
      __syncwarp();
      if (elect() && !*dead) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int h = 0; h < HT; ++h)
            mma_ts(tm + kColY + 64 * h, tm + kColG + 16 * k + 8 * h, xd + ((h * kBox + k * 2048) >> 4), id_y, true);
        commit(&sh.y_done);
      }
    }
  } else if (warp == 26) {
    // ---- products for S ----
    constexpr uint32_t id_s = kIdesc<T> | (1u << 16) | ((uint32_t)NS / 8 << 17);  // w X x B: B is N-major
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const uint32_t ph = c & 1;
      full(sh.full_b, c);
      wait_tc(&sh.s_ready, ph, dead, p.err);
      const uint64_t bd = smem_desc(smem_u32(bbox(c, 0)), kBox, 1024);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {  // 32 tokens
        wait_tc(&sh.weighed[q & 1], (q >> 1) & 1, dead, p.err);  // a buffer's second use in the chunk
        fence_after();
        __syncwarp();
        if (elect() && !*dead) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < NT; ++e)
              mma_ts(tm + kColS, tm + kColX + 64 * (q & 1) + 16 * e + 8 * k, bd + (((q * 32 + k * 16) * 128) >> 4), id_s, true);
          commit(&sh.gained[q & 1]);
          if (q == 3) commit(&sh.empty_b[c & 1]);
        }
      }
    }
  } else if (warp == 27) {
    // ---- output: whole chunks leave by TMA, a request's last rows have left already ----
    if (lane == 0) {
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        wait_tc(&sh.finished[c & 3], (c >> 2) & 1, dead, p.err);
        if (size - c * 128 >= 128 && !*dead) {
          for (int k = 0; k < 2; ++k)
            if (HT == 1 || h0 + k < hend)
              tma_store_3d(&maps.out, xbox(c, k), HT == 2 ? 0 : 64 * k, HT == 2 ? h0 + k : h0, first + c * 128);
          asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        mbar_arrive(&sh.empty_x[c & 1]);  // and z's place
      }
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
  } else if (warp >= 16) {
    // ---- column warps: thread = column p ----
    float scale = 1.f;  // of w in this chunk
    float fade0 = 0.f, fade1 = 0.f, fade2 = 0.f;  // from the ends of the first 32 tokens, ... to the chunk's end, times scale
#pragma unroll 1
    for (int c = 0; c <= chunks; ++c) {
      const uint32_t ph = c & 1, before = ph ^ 1;
      const bool more = c < chunks;
      const float unscale = __uint_as_float((254u << 23) - __float_as_uint(scale));  // 1 / scale, a power of two
      uint32_t col = 0;              // this column of X, in row 0 of a swizzle atom
      const float *cf = nullptr;
      float keep = 0.f;              // decay of this chunk, times its scale
      if (more) {
        wait_tc(&sh.prepared[c & 3], (c >> 2) & 1, dead, p.err);
        const float *t = sh.tot[c & 3][hs];
        const float t3 = t[3], t2 = t3 + t[2], t1 = t2 + t[1], t0 = t1 + t[0];
        keep = ex2(t0);
        fade0 = ex2(t1);
        fade1 = ex2(t2);
        fade2 = ex2(t3);
        if (NT == 2) {  // the power of two that brings the chunk's largest w to [1/2, 1)
          const float *top = sh.top[c & 3][hs];
          const float m = fmaxf(fmaxf(top[0] * fade0, top[1] * fade1), fmaxf(top[2] * fade2, top[3]));
          const int e = (int)(__float_as_uint(m) >> 23);
          scale = e < 64 || e > 190 ? 1.f : __uint_as_float((uint32_t)(253 - e) << 23);
          keep *= scale;
          fade0 *= scale;
          fade1 *= scale;
          fade2 *= scale;
        }
        const int valid = min(128, size - c * 128);
        full(sh.full_x, c);
        if (valid < 128) {  // rows of the next request, or of nothing: 0 x anything must be 0
          full(sh.full_b, c);
          const int todo = (128 - valid) * 8;
          for (int i = tid - 512; i < todo * (2 + NB); i += 256) {
            const int o = i / todo, k = i % todo;
            unsigned char *b = o < 2 ? xbox(c, o) : bbox(c, o - 2);
            *reinterpret_cast<uint4 *>(b + (valid + k / 8) * 128 + (k % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
          sync_weighers();
        }
        col = smem_u32(xbox(c, pc >> 6)) + wg * 16 * 128 + (pc & 63) * 2;
        cf = sh.colf[c & 3][hs] + wg * 16;
      }
      // Four times 32 tokens of w X, in two buffers: the products take in one while
      // the other is written. The first is weighed before S is handed on, which has
      // to wait for the products of the chunk before.
#pragma unroll 1
      for (int q = more ? 0 : 1; q < 4; ++q) {
        if (q == 1) {
          // S after the chunk before (at first, the block's start): its 16-bit form for
          // this chunk's product, and its decayed, scaled form as the accumulator
          if (c > 0) {
            wait_tc(&sh.gained[1], 1, dead, p.err);  // the chunk's last; and all its columns of X are read
            wait_tc(&sh.gy_done, before, dead, p.err);
            fence_after();
          }
#pragma unroll 1
          for (int n = 0; n < NH; n += 16) {
            float v[16];
            if (c > 0) {
              uint32_t s[16];
              tm_ld16(tm + lane_at + kColS + n0 + n, s);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = NT == 2 ? __uint_as_float(s[i]) * unscale : __uint_as_float(s[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = 0.f;
              auto start = [&](const float *src) {
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  if (n + i < nv) {
                    const float4 f = get4(src + n + i, nv - n - i, p.vec != 0);
                    v[i] = f.x;
                    v[i + 1] = f.y;
                    v[i + 2] = f.z;
                    v[i + 3] = f.w;
                  }
              };
              if (pin) {
                if (index == 0) {
                  if (at.goes_on) start((at.last > 0 ? entry_row(p, at, h0 + hs, pp, at.last) : cache_row(p, at, h0 + hs, pp)) + n0);
                } else {
                  start(entry_row(p, at, h0 + hs, pp, index - 1) + n0);
                }
              }
            }
            if (more) {
#pragma unroll
              for (int i = 0; i < 16; i += 8) {
                uint4 w4;  // a 16-byte piece of the row
                w4.x = pack2<T>(v[i], v[i + 1]);
                w4.y = pack2<T>(v[i + 2], v[i + 3]);
                w4.z = pack2<T>(v[i + 4], v[i + 5]);
                w4.w = pack2<T>(v[i + 6], v[i + 7]);
                *reinterpret_cast<uint4 *>(s16 + ((n0 + n) / 64) * kBox + swz(pc, ((n0 + n + i) % 64) * 2)) = w4;
              }
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const float2 k = upk(mul2(pk(v[i], v[i + 1]), pk(keep, keep)));
                w[i] = __float_as_uint(k.x);
                w[i + 1] = __float_as_uint(k.y);
              }
              tm_st16(tm + lane_at + kColS + n0 + n, w);
            } else if (pin && !*dead && index == at.last && at.kept) {
              float *dst = cache_row(p, at, h0 + hs, pp) + n0 + n;
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                if (n + i < nv) put4(dst + i, make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]), nv - n - i, p.vec != 0);
            }
          }
          if (!more) break;
          fence_proxy_async();
          wait_st();
          fence_before();
          arrive_warp(&sh.s_ready, lane);
        }
        // w X as the product's A operand: thread = column, a warpgroup half of the tokens
        const int use = 2 * c + (q >> 1);
        if (use > 0) {
          wait_tc(&sh.gained[q & 1], (use - 1) & 1, dead, p.err);
          fence_after();
        }
        const float f = q == 0 ? fade0 : q == 1 ? fade1 : q == 2 ? fade2 : scale;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t t[NT][4];
          const float4 wa = *reinterpret_cast<const float4 *>(cf);
          const float4 wb = *reinterpret_cast<const float4 *>(cf + 4);
          const f2 f2f = pk(f, f);
          const f2 w[4] = {mul2(pk(wa.x, wa.y), f2f), mul2(pk(wa.z, wa.w), f2f), mul2(pk(wb.x, wb.y), f2f), mul2(pk(wb.z, wb.w), f2f)};
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = lds_16<T>((col ^ (k << 4)) + k * 128);
          col += 8 * 128;
          cf += 8;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a[NT];
            Terms<T>::split(mul2(pk(x[2 * k], x[2 * k + 1]), w[k]), a);
#pragma unroll
            for (int e = 0; e < NT; ++e) t[e][k] = a[e];
          }
#pragma unroll
          for (int e = 0; e < NT; ++e) tm_st4(tm + lane_at + kColX + 64 * (q & 1) + 16 * e + 8 * wg + 4 * i, t[e]);
        }
        col += 16 * 128;
        cf += 16;
        wait_st();
        fence_before();
        arrive_warp(&sh.weighed[q & 1], lane);
      }
      if (more) arrive_warp(&sh.x_read[ph], lane);
    }
    fence_before();
  } else {
    // ---- row warps: thread = row t; rg: a quarter of the columns, or a head to prepare ----
    const int rg = warp >> 2;
    // The last rows have most columns to mask, and their diagonal ones fall to the
    // first two quarters: the other two prepare.
    const int tp = rg - 2;                                      // the tile's head to prepare
    const bool prepares = tp >= 0 && tp < HT;
    const int hp = prepares && h0 + tp < hend ? h0 + tp : h0;
    const int ho = HT == 2 ? rg >> 1 : 0;                       // the head of the columns in the tile
    const bool hin = h0 + ho < hend;
    const float A = p.A[hp], bias = p.bias ? p.bias[hp] : 0.f, skip = p.D ? p.D[hin ? h0 + ho : h0] : 0.f;
    const int trow = wq * 32 + lane;
    auto load_dt = [&](int c) -> float {
      const int t = c * 128 + trow;
      if (!prepares || t >= size) return 0.f;
      const long long at = (long long)(first + t) * p.sdt[0] + hp * p.sdt[1];
      return p.dt_f32 ? static_cast<const float *>(p.dt)[at] : to_f<T>(static_cast<const T *>(p.dt)[at]);
    };
    // The decays of chunk cp are prepared between masking and finishing chunk cp - 2.
    constexpr int kAhead = 2;
    float raw_dt = load_dt(0);
#pragma unroll 1
    for (int cp = 0; cp < chunks + kAhead; ++cp) {
      const int c = cp - kAhead;
      if (c >= 0) {
        const int st = c & 3;
        wait_tc(&sh.prepared[st], (c >> 2) & 1, dead, p.err);
        wait_tc(&sh.gy_done, c & 1, dead, p.err);
        fence_after();
        if (tid == 0) {
          mbar_arrive(&sh.empty_c);
          mbar_arrive(&sh.empty_b[c & 1]);
        }
        // The masked forms of 16 columns, one per head, in place of C B^T. Of the
        // eight pieces a warp takes rg and 7 - rg: near enough equal work below
        // the diagonal.
#pragma unroll 1
        for (int i2 = 0; i2 < 2; ++i2) {
          const int jb = i2 ? 7 - rg : rg, j = jb >> 1;
          const uint32_t tg = tm + lane_at + kColG + 16 * jb;
          if (j > wq) {
            const uint32_t m[8] = {};
#pragma unroll
            for (int h = 0; h < HT; ++h) tm_st8(tg + 8 * h, m);
            continue;
          }
          uint32_t g[16];
          tm_ld16(tg, g);
#pragma unroll
          for (int h = 0; h < HT; ++h) {
            uint32_t m[8];
            float l = -sh.nl[st][h][trow];
            if (j < wq) {
              const float4 t4 = *reinterpret_cast<const float4 *>(sh.tot[st][h]);  // those between the two
              l += (j < 1 && wq > 1 ? t4.y : 0.f) + (j < 2 && wq > 2 ? t4.z : 0.f);
              l = ex2(l);
              const f2 rf = pk(l, l);
              const float *colf = sh.colf[st][h] + 16 * jb;
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 cf = *reinterpret_cast<const float4 *>(colf + i);
                m[i / 2] = narrow<T>(mul2(mul2(pku(g[i], g[i + 1]), rf), pk(cf.x, cf.y)));
                m[i / 2 + 1] = narrow<T>(mul2(mul2(pku(g[i + 2], g[i + 3]), rf), pk(cf.z, cf.w)));
              }
            } else {
              const float *nl = sh.nl[st][h] + 16 * jb, *dt = sh.dt[st][h] + 16 * jb;
              const uint32_t *before = sh.before[jb & 1][lane];
              const f2 l2 = pk(l, l);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 n4 = *reinterpret_cast<const float4 *>(nl + i), d4 = *reinterpret_cast<const float4 *>(dt + i);
                const float2 a = upk(add2(l2, pk(n4.x, n4.y))), b = upk(add2(l2, pk(n4.z, n4.w)));
                const float2 u = upk(mul2(mul2(pk(ex2(a.x), ex2(a.y)), pk(d4.x, d4.y)), pku(g[i], g[i + 1])));
                const float2 v = upk(mul2(mul2(pk(ex2(b.x), ex2(b.y)), pk(d4.z, d4.w)), pku(g[i + 2], g[i + 3])));
                const uint2 keep = *reinterpret_cast<const uint2 *>(before + i / 2);
                m[i / 2] = pack2<T>(u.x, u.y) & keep.x;
                m[i / 2 + 1] = pack2<T>(v.x, v.y) & keep.y;
              }
            }
            tm_st8(tg + 8 * h, m);
          }
        }
        // Y = e^L (C S^T), 32 columns
        {
          float e = -sh.nl[st][ho][trow];
          const float4 t4 = *reinterpret_cast<const float4 *>(sh.tot[st][ho]);
          e += (wq > 0 ? t4.x : 0.f) + (wq > 1 ? t4.y : 0.f) + (wq > 2 ? t4.z : 0.f);
          e = ex2(e);
          const uint32_t ty = tm + lane_at + kColY + 32 * rg;
          uint32_t y[2][16];
          tm_ld16_async(ty, y[0]);
          tm_ld16_async(ty + 16, y[1]);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            tm_wait(y[q]);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 v = upk(mul2(pku(y[q][i], y[q][i + 1]), pk(e, e)));
              y[q][i] = __float_as_uint(v.x);
              y[q][i + 1] = __float_as_uint(v.y);
            }
            tm_st16(ty + 16 * q, y[q]);
          }
        }
        wait_st();
        fence_before();
        arrive_warp(&sh.masked, lane);
      }
      if (cp < chunks && prepares) {
        const int st = cp & 3;
        float dt = raw_dt + bias;
        if (p.softplus) dt = softplus_f(dt);
        const bool in = cp * 128 + trow < size;
        if (!in) dt = 0.f;
        float l = in ? log2_step(dt, A) : 0.f, to_end = l;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float up = __shfl_up_sync(0xffffffffu, l, o), dn = __shfl_down_sync(0xffffffffu, to_end, o);
          if (lane >= o) l += up;
          if (lane + o < 32) to_end += dn;
        }
        // what follows this token, without the token itself
        const float nx = __shfl_down_sync(0xffffffffu, to_end, 1);
        const float cf = dt * ex2(lane < 31 ? nx : 0.f);
        sh.nl[st][tp][trow] = -l;
        sh.dt[st][tp][trow] = dt;
        sh.colf[st][tp][trow] = cf;
        if (lane == 31) sh.tot[st][tp][wq] = l;
        if (NT == 2) {
          float m = fabsf(cf);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (lane == 0) sh.top[st][tp][wq] = m;
        }
        arrive_warp(&sh.prepared[st], lane);
        raw_dt = load_dt(cp + 1);
      }
      if (c < 0) continue;
      // the output, 32 columns, in place of X's rows
      const int valid = min(128, size - c * 128);
      full(sh.full_x, c);
      wait_tc(&sh.x_read[c & 1], (c >> 1) & 1, dead, p.err);
      wait_tc(&sh.y_done, c & 1, dead, p.err);
      if (GATE) full(sh.full_z, c);
      fence_after();
      unsigned char *xr = xbox(c, rg >> 1);
      const unsigned char *zr = bbox(c, rg >> 1);
      uint32_t y[2][16];
      tm_ld16_async(tm + lane_at + kColY + 32 * rg, y[0]);
      tm_ld16_async(tm + lane_at + kColY + 32 * rg + 16, y[1]);
      tm_wait(y[0]);
      tm_wait(y[1]);
      fence_before();
      arrive_warp(&sh.y_free, lane);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int off = swz(trow, 64 * (rg & 1) + 16 * k);
        const uint4 xq = *reinterpret_cast<const uint4 *>(xr + off);
        const uint32_t xw[4] = {xq.x, xq.y, xq.z, xq.w};
        uint4 zq = make_uint4(0, 0, 0, 0);
        if (GATE) zq = *reinterpret_cast<const uint4 *>(zr + off);
        const uint32_t zw[4] = {zq.x, zq.y, zq.z, zq.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f2 v = fma2(pk(skip, skip), wide<T>(xw[i]), pku(y[k / 2][8 * (k % 2) + 2 * i], y[k / 2][8 * (k % 2) + 2 * i + 1]));
          if (GATE) {
            const f2 zv = wide<T>(zw[i]);
            // z / (1 + e^-z): z/2 + z/2 tanh(z/2) would take one MUFU operation, but it cancels
            // for negative z (tanh's 2^-11 is 1.3% of silu at -4)
            const float2 e = upk(mul2(zv, pk(-kLog2e, -kLog2e)));
            const float2 d = upk(add2(pk(ex2(e.x), ex2(e.y)), pk(1.f, 1.f)));
            v = mul2(v, mul2(zv, pk(rcp(d.x), rcp(d.y))));
          }
          o[i] = narrow<T>(v);
        }
        *reinterpret_cast<uint4 *>(xr + off) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (valid < 128 && hin && !*dead) {  // the request's last rows, as 64-byte pieces
        __syncwarp();
        const int piece = 4 * (rg & 1) + (lane & 3), col = (HT == 2 ? 0 : 64 * (rg >> 1)) + 8 * piece;
        if (col < p.headdim) {
#pragma unroll 1
          for (int t = wq * 32 + (lane >> 2); t < min(valid, wq * 32 + 32); t += 8)
            *reinterpret_cast<uint4 *>(out + (long long)(first + c * 128 + t) * p.so[0] + (h0 + ho) * p.so[1] + col) =
                *reinterpret_cast<const uint4 *>(xr + swz(t, 16 * piece));
        }
      }
      fence_proxy_async();  // before the store, and the next copies into these boxes
      arrive_warp(&sh.finished[c & 3], lane);
    }
    fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 25) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
  }
}

template <typename T, int PW, int NS, bool GATE>
cudaError_t go(const HeadScanParams &p, const TcMaps &maps, cudaStream_t s) {
  constexpr int smem = kBoxes * kBox + NS / 64 * kBox + (int)sizeof(Shared) + 1024;
  constexpr int sum_smem = kSumStages * (2 + NS / 64) * kBox + (int)sizeof(SumShared) + 1024;
  const long long tiles = head_scan_tc_tiles(p), ctas = tiles * (p.t.max_blocks + 1);
  auto sum = ss_head_scan_sum_tc_kernel<T, PW, NS>;
  auto fwd = ss_head_scan_tc_kernel<T, PW, NS, GATE>;
  static std::atomic<bool> set[64];  // the attribute is per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(sum, cudaFuncAttributeMaxDynamicSharedMemorySize, sum_smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fwd, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
  }
  if (p.split) {
    sum<<<(unsigned)(tiles * (p.t.tokens / p.t.block)), kSumThreads, sum_smem, s>>>(p, maps);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_head_scan_carry(p, s);
    if (e != cudaSuccess) return e;  // the scan would start from what no one has written
  }
  return launch_after(fwd, dim3((unsigned)ctas), kTcThreads, smem, s, p.split, p, maps);
}

template <typename T>
cudaError_t by_size(const HeadScanParams &p, const TcMaps &m, cudaStream_t s) {
  if (p.headdim <= 64) {
    if (p.dstate <= 64) return p.z ? go<T, 64, 64, true>(p, m, s) : go<T, 64, 64, false>(p, m, s);
    return p.z ? go<T, 64, 128, true>(p, m, s) : go<T, 64, 128, false>(p, m, s);
  }
  if (p.dstate <= 64) return p.z ? go<T, 128, 64, true>(p, m, s) : go<T, 128, 64, false>(p, m, s);
  return p.z ? go<T, 128, 128, true>(p, m, s) : go<T, 128, 128, false>(p, m, s);
}

bool map3(TensorMapEncode enc, CUtensorMap *m, const void *base, int width, int rows, int tokens, const long long *st) {
  // (width, rows, tokens); a dimension of one element may have any stride
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {rows > 1 ? (cuuint64_t)st[1] * 2 : 16, tokens > 1 ? (cuuint64_t)st[0] * 2 : 16};
  const cuuint32_t bx[3] = {64, 1, 128}, es[3] = {1, 1, 1};
  return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(enc)(
             m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(base), dims, strides, bx, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool head_scan_tc_sizes(int dtype, const HeadScanParams &p) { return dtype != 0 && p.headdim <= 128 && p.dstate <= 128; }

int head_scan_tc_unaligned(const HeadScanParams &p) {
  auto off = [&](const void *base, const long long *st, int n) {
    if (!base) return false;
    return reinterpret_cast<uintptr_t>(base) % 16 != 0 || (n > 1 && (st[1] % 8 != 0 || st[1] == 0)) ||
           (p.t.tokens > 1 && (st[0] % 8 != 0 || st[0] == 0));
  };
  const int groups = p.heads / p.hpg;
  return (off(p.x, p.sx, p.heads) ? kRowsX : 0) | (off(p.B, p.sB, groups) ? kRowsB : 0) | (off(p.C, p.sC, groups) ? kRowsC : 0) |
         (off(p.z, p.sz, p.heads) ? kRowsZ : 0) | (off(p.out, p.so, p.heads) || p.headdim % 8 != 0 ? kRowsOut : 0);
}

namespace {

// One thread: 8 values of a row of the copy.
template <bool TO>
__global__ void __launch_bounds__(256) rows_kernel(uint16_t *strided, long long st0, long long st1, uint4 *rows, int n_rows, int width,
                                                   long long total) {
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= total) return;
  const int per = (width + 7) / 8, w = (int)(i % per) * 8;
  const long long tr = i / per;
  uint16_t *at = strided + tr / n_rows * st0 + tr % n_rows * st1 + w;
  uint32_t v[4] = {};
  if (TO) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (w + k < width) v[k / 2] |= (uint32_t)at[k] << (16 * (k % 2));
    rows[i] = make_uint4(v[0], v[1], v[2], v[3]);
  } else {
    const uint4 q = rows[i];
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (w + k < width) at[k] = (uint16_t)(v[k / 2] >> (16 * (k % 2)));
  }
}
template <bool TO>
cudaError_t copy_rows(void *strided, const long long *st, void *rows, int tokens, int n, int width, cudaStream_t s) {
  const long long total = (long long)tokens * n * ((width + 7) / 8), ctas = copy_rows_ctas(tokens, n, width);
  rows_kernel<TO><<<(unsigned)ctas, 256, 0, s>>>(static_cast<uint16_t *>(strided), st[0], st[1], static_cast<uint4 *>(rows), n, width, total);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_to_rows(const void *src, const long long *st, void *dst, int tokens, int rows, int width, cudaStream_t s) {
  return copy_rows<true>(const_cast<void *>(src), st, dst, tokens, rows, width, s);
}
cudaError_t launch_from_rows(const void *src, void *dst, const long long *st, int tokens, int rows, int width, cudaStream_t s) {
  return copy_rows<false>(dst, st, const_cast<void *>(src), tokens, rows, width, s);
}

cudaError_t launch_head_scan_tc(int dtype, const HeadScanParams &p, TensorMapEncode enc, cudaStream_t s) {
  TcMaps m;
  const int groups = p.heads / p.hpg;
  if (!map3(enc, &m.x, p.x, p.headdim, p.heads, p.t.tokens, p.sx) || !map3(enc, &m.B, p.B, p.dstate, groups, p.t.tokens, p.sB) ||
      !map3(enc, &m.C, p.C, p.dstate, groups, p.t.tokens, p.sC) ||
      !map3(enc, &m.z, p.z ? p.z : p.x, p.headdim, p.heads, p.t.tokens, p.z ? p.sz : p.sx) ||
      !map3(enc, &m.out, p.out, p.headdim, p.heads, p.t.tokens, p.so))
    return cudaErrorInvalidValue;
  return dtype == 1 ? by_size<__half>(p, m, s) : by_size<__nv_bfloat16>(p, m, s);
}

}  // namespace ssk
