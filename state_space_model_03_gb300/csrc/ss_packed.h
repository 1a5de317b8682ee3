// Kernel parameters and launchers of the packed operators (include/ssfwd_packed.h).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssk {

// The library's error word on the current device (nullptr on failure).
int32_t *packed_error_word();

struct TablesParams {
  int requests, tokens, block, max_blocks, free;
  const int32_t *lengths, *context, *slots, *free_slots;
  int32_t *offsets, *token_request, *token_position, *blocks, *carried, *slot_map, *counts;
};
cudaError_t launch_request_tables(const TablesParams &p, cudaStream_t s);

struct Tables {
  int requests, tokens, block, max_blocks;
  const int32_t *offsets, *token_request, *blocks, *carried, *slot_map, *counts, *context;
};

struct PackedConvParams {
  int dim, width, act;
  int vec;  // 16-byte accesses of x, out rows and windows allowed
  long long slots, sx, so, ss;
  const void *x;
  const float *weight, *bias;
  void *state, *out;
  Tables t;
};
cudaError_t launch_packed_conv(int dtype, const PackedConvParams &p, cudaStream_t s);

struct PackedConvUpdateParams {
  int requests, dim, width, act, vec;
  long long slots, sx, so, ss;
  const void *x;
  const float *weight, *bias;
  const int32_t *slot_map;
  void *state, *out;
};
cudaError_t launch_packed_conv_update(int dtype, const PackedConvUpdateParams &p, cudaStream_t s);

struct HeadUpdateParams {
  int requests, heads, headdim, dstate, hpg;  // hpg: heads per group
  int softplus, dt_f32, vec, bcvec;           // vec: 16-byte state accesses; bcvec: 4 B/C values in one access
  long long slots;
  const void *x, *dt, *B, *C, *z;
  const float *A, *D, *bias;
  const int32_t *slot_map;
  float *state;
  void *out;
  long long sx[2], sdt[2], sB[2], sC[2], sz[2], so[2], ss[2];
};
cudaError_t launch_head_update(int dtype, const HeadUpdateParams &p, cudaStream_t s);

struct HeadScanParams {
  int heads, headdim, dstate, hpg;
  int softplus, dt_f32;
  int split;  // a request may have several blocks: ws holds their summaries
  int vec;    // 16-byte accesses of state rows allowed
  long long slots;
  const void *x, *dt, *B, *C, *z;
  const float *A, *D, *bias;
  float *state;
  void *out;
  long long sx[2], sdt[2], sB[2], sC[2], sz[2], so[2], ss[2];
  // Summaries (split): per block of the table and head, the state it ends in,
  // headdim x dstate, and log2 of its whole decay. The first launch leaves a
  // block's own gain (the request's first block: from its start state), the second
  // adds what earlier blocks left, the third starts each block from the entry
  // before its own. The entry of a request's last block, whose end nothing
  // continues, keeps the request's start state. The first two run over the rows
  // of t.carried, tokens / block of them at most.
  float *ws_state, *ws_decay;
  int32_t *err;
  Tables t;
};
cudaError_t launch_head_scan(int dtype, const HeadScanParams &p, cudaStream_t s);
cudaError_t launch_head_scan_carry(const HeadScanParams &p, cudaStream_t s);  // the second launch
inline int head_scan_carry_pieces(const HeadScanParams &p) { return (p.headdim * p.dstate + 1023) / 1024; }  // CTAs of a head's state
inline long long head_scan_carry_ctas(const HeadScanParams &p) {
  return (long long)(p.t.tokens / p.t.block) * p.heads * head_scan_carry_pieces(p);
}

// The same on the tensor cores, for 16-bit operands that TMA can describe.
typedef void *TensorMapEncode;  // the driver's cuTensorMapEncodeTiled
TensorMapEncode packed_map_encode();
// Whether the tensor cores' tiles hold the sizes, and which operands do not lie in
// the 16-byte rows that TMA wants: these are copied to such rows first (and out
// back from them), `p` then has the copies.
bool head_scan_tc_sizes(int dtype, const HeadScanParams &p);
enum { kRowsX = 1, kRowsB = 2, kRowsC = 4, kRowsZ = 8, kRowsOut = 16 };
int head_scan_tc_unaligned(const HeadScanParams &p);
// Tiles of 128 (head, p) columns, two heads of up to 64 or one: a CTA for each and
// for each row of the block table, and one more.
inline long long head_scan_tc_tiles(const HeadScanParams &p) {
  const int ht = p.headdim <= 64 ? 2 : 1;
  return (long long)(p.heads / p.hpg) * ((p.hpg + ht - 1) / ht);
}
inline long long copy_rows_ctas(int tokens, int rows, int width) {
  return ((long long)tokens * rows * ((width + 7) / 8) + 255) / 256;
}
// (tokens, rows, width) in 16-bit values between a strided tensor and contiguous
// rows of `width` rounded up to 8: to_rows zeroes what is past the width.
cudaError_t launch_to_rows(const void *src, const long long *st, void *dst, int tokens, int rows, int width, cudaStream_t s);
cudaError_t launch_from_rows(const void *src, void *dst, const long long *st, int tokens, int rows, int width, cudaStream_t s);
cudaError_t launch_head_scan_tc(int dtype, const HeadScanParams &p, TensorMapEncode enc, cudaStream_t s);

// Programmatic dependent launch of a scan's later launches: each lets the next one
// be scheduled when it starts, and the next one waits for its results where it
// first needs them, so that launches with little to do cost less.
#ifdef __CUDACC__
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t s, bool dependent, const A &...args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace ssk
