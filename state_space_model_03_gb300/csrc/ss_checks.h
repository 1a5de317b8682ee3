// Argument checks that the packed and the layer operators' C ABIs share. Every
// check is made before anything is enqueued.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "ss_packed.h"
#include "ssfwd_packed.h"

namespace {

int elem_size(int dt) { return dt == SS_F32 ? 4 : 2; }
bool bad_dtype(int dt) { return dt < SS_F32 || dt > SS_BF16; }
bool aligned(const void *p, int a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Host-side fault injection for tests, as in the other entry points:
// SSFWD_FAULT=launch makes the launch report a CUDA failure.
bool launch_fault() {
  const char *f = std::getenv("SSFWD_FAULT");
  return f && std::strcmp(f, "launch") == 0;
}

int launched(cudaError_t e) { return e == cudaSuccess ? SS_OK : SS_ERR_CUDA; }

struct Range {
  uintptr_t lo, hi;
};
// The bytes of an operand with the given sizes and strides (outermost first).
Range span(const void *ptr, int64_t esize, std::initializer_list<int64_t> sizes, std::initializer_list<int64_t> strides) {
  if (!ptr) return {0, 0};
  int64_t last = 0;
  auto st = strides.begin();
  for (int64_t n : sizes) {
    if (n == 0) return {0, 0};
    last += (n - 1) * *st++;
  }
  const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
  return {lo, lo + static_cast<uintptr_t>((last + 1) * esize)};
}
bool overlap(Range a, Range b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
// Rows interleaved in one buffer (the parts of a projection's output) have
// overlapping spans and no common element: allowed when both have the same row
// stride and their row parts are disjoint within it.
bool rows_meet(Range a, int64_t row_a, Range b, int64_t row_b, int64_t stride_a, int64_t stride_b) {
  if (!overlap(a, b)) return false;
  if (stride_a != stride_b || stride_a <= 0) return true;
  const int64_t d = static_cast<int64_t>((a.lo > b.lo ? a.lo - b.lo : b.lo - a.lo) % stride_a);
  const int64_t lo = a.lo > b.lo ? row_b : row_a, hi = a.lo > b.lo ? row_a : row_b;
  return d < lo || d + hi > stride_a;
}

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - (int64_t(1) << 20);
constexpr int64_t kMaxBlock = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40;

bool bad_stride(int64_t s) { return s < 0 || s > kMaxStride; }

int64_t most_blocks(int64_t tokens, int64_t block, int64_t requests) {
  return tokens / block + std::min(requests, tokens);
}

int validate_sizes(int64_t requests, int64_t tokens, int64_t block, int64_t max_blocks) {
  if (requests < 1 || tokens < 0 || block < 1) return SS_ERR_SHAPE;
  if (requests > SS_MAX_REQUESTS || tokens >= kMaxTokens || block >= kMaxBlock) return SS_ERR_UNSUPPORTED;
  if (max_blocks != most_blocks(tokens, block, requests)) return SS_ERR_SHAPE;
  return SS_OK;
}

// The tables as an operator's input.
int validate(const ss_packed_tables &t) {
  const int st = validate_sizes(t.requests, t.tokens, t.block, t.max_blocks);
  if (st != SS_OK) return st;
  if (t.tokens == 0) return SS_OK;
  if (!t.offsets || !t.token_request || !t.blocks || !t.slot_map || !t.counts) return SS_ERR_NULL;
  if (t.tokens >= t.block && !t.carried) return SS_ERR_NULL;
  for (const void *q : {(const void *)t.offsets, (const void *)t.token_request, (const void *)t.blocks, (const void *)t.carried,
                        (const void *)t.slot_map, (const void *)t.counts})
    if (!aligned(q, 16)) return SS_ERR_ALIGN;
  if (t.context && !aligned(t.context, 4)) return SS_ERR_ALIGN;
  return SS_OK;
}
ssk::Tables tables_of(const ss_packed_tables &t) {
  return {(int)t.requests, (int)t.tokens, (int)t.block, (int)t.max_blocks, t.offsets, t.token_request, t.blocks,
          t.carried, t.slot_map, t.counts, t.context};
}

}  // namespace
