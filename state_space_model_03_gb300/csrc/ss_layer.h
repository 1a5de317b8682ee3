// Kernel parameters and launchers of the layer operators (include/ssfwd_layer.h).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ss_packed.h"

namespace ssk {

// The recurrence runs in tiles of kGatedTile tokens by kGatedCh channels; the states
// that the backward pass starts from are kept before each tile. How the tiles of a
// (sequence, channel tile) pair, a unit, are shared out:
//   cluster  CTAs that take consecutive tiles together, or
//   segs     segments of seg_tiles tiles, each a CTA's, which one launch reduces to
//            their maps (states in the workspace) before another runs them.
constexpr int kGatedTile = 64;
constexpr int kGatedCh = 32;
constexpr int kGatedMostCluster = 8;
constexpr int kGatedMostSegs = 128;
struct GatedPlan {
  int cluster, segs, seg_tiles;
};
GatedPlan gated_plan(int dtype, long long units, int tiles);
// Of each segment 16 lanes' maps (two pairs), and after all of these 16 lanes' start states.
inline long long gated_map_bytes(long long units, const GatedPlan &plan) { return plan.segs > 1 ? units * plan.segs * 384 : 0; }

// What a test makes of the recurrence's waits: limit: tries of one until it gives up (set
// by the launch); copy, maps: the round whose copies, or whose exchange in a cluster,
// never come (-1: none).
struct WaitHook {
  uint32_t limit;
  int copy = -1, maps = -1;
};

struct GatedScanParams {
  int tokens, dim;      // per sequence
  int batch, channel_tiles;  // sequences; tiles of channels
  int tiles;                 // of tokens
  GatedPlan plan;
  void *maps;  // gated_map_bytes
  float rate;
  int32_t *err;
  WaitHook wait;
  const void *x, *gate, *igate;
  const float *decay, *init;  // init (batch, dim) or NULL
  void *out;
  float *last;  // (batch, dim) or NULL
  float *kept;  // (batch, tiles, dim) or NULL
  long long sx[2], sg[2], si[2], so[2];  // sequence, token
  // packed requests (token_request given): one sequence, states by slot
  const int32_t *token_request, *offsets, *slot_map, *context;
  float *state;
  long long slots, state_stride;
};
// rows: a RowAccess (ss_gated.cuh); enc: the tensor-map encoder, for kTma.
cudaError_t launch_gated_scan(int dtype, int rows, TensorMapEncode enc, const GatedScanParams &p, cudaStream_t s);

struct GatedBwdParams {
  int tokens, dim, batch, channel_tiles, tiles;  // as above
  GatedPlan plan;
  void *maps;
  float rate;
  int32_t *err;
  WaitHook wait;
  const void *x, *gate, *igate, *dout;
  const float *decay, *kept, *dlast;  // dlast (batch, dim) or NULL
  void *dx, *dgate, *digate;          // NULL: not wanted
  float *ddecay, *dinit;
  float *parts;  // (batch * cluster * segs, dim): sums for ddecay
  long long sx[2], sg[2], si[2], sd[2], sdx[2], sdg[2], sdi[2];
};
cudaError_t launch_gated_bwd(int dtype, int rows, TensorMapEncode enc, const GatedBwdParams &p, cudaStream_t s);

struct GatedUpdateParams {
  int rows, dim, vec;  // vec: 16-byte accesses of state rows, and 4 values at once of the others
  float rate;
  long long slots;
  const void *x, *gate, *igate;
  const float *decay;
  const int32_t *slot_map;
  float *state;
  void *out;
  long long sx, sg, si, so, ss;
};
cudaError_t launch_gated_update(int dtype, const GatedUpdateParams &p, cudaStream_t s);

struct NormParams {
  long long rows;
  int dim;
  int weight_f32;
  float eps;
  const void *x, *residual, *weight;  // residual NULL: the sum is x
  void *out, *sum;                    // sum NULL: not wanted
  float *rstd;                        // NULL: not wanted
  long long sx, sr, so, ss;
  // quantised
  int group, e8m0;  // group 0: the row
  void *scale;      // (rows, groups)
  int groups;
};
cudaError_t launch_rms_norm(int dtype, int residual_dtype, bool vec, const NormParams &p, cudaStream_t s);
cudaError_t launch_rms_norm_quant(int dtype, int residual_dtype, bool vec, const NormParams &p, cudaStream_t s);

struct NormBwdParams {
  long long rows;
  int dim;
  int weight_f32;
  const void *dout, *dsum, *sum, *weight;  // dsum NULL: 0
  const float *rstd;
  void *dx, *dresidual, *dweight;  // NULL: not wanted
  float *parts;                    // (ctas, dim): sums for dweight
  int ctas;
  long long sd, sds, ss, sdx, sdr;
};
int norm_bwd_ctas(long long rows, int dim);
cudaError_t launch_rms_norm_bwd(int dtype, int residual_dtype, bool vec, const NormBwdParams &p, cudaStream_t s);

}  // namespace ssk
