// Kernel argument blocks and launch helpers of the block operators (norm and
// rotation of heads, gated products, orthogonalised updates), shared by
// block_api.cpp and their translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"
#include "nvfp4_kernels.hpp"

namespace nvfp4 {

// ---------------------------------------------------------------- rope ----
struct RopeSide {  // the query heads or the key heads
  const void *x;   // x_dtype: what is normalised and rotated; backward: what was (null without a norm)
  uint16_t *y;     // bf16: the result; backward: its gradient
  void *dx;        // x_dtype, backward
  const void *weight;
  float *dweight, *parts;          // backward: [dim], and [workgroups of this side][dim]
  int64_t x_b, x_t, x_h;           // elements between sequences, tokens, heads
  int64_t y_b, y_t, y_h, dx_b, dx_t, dx_h;
  int heads;
  int per;      // heads of one token that a wave takes at a time, a power of two
  int splits;   // waves that share a token's heads
  int groups;   // workgroups of this side
};
struct RopeArgs {
  RopeSide side[2];
  const int64_t *positions;
  const int32_t *cu;
  const double *freqs;
  int64_t total;   // tokens
  int64_t tokens;  // of one sequence (packed: total)
  int batch;
  int dim, rot, interleaved;
  int units;       // lanes of a head that hold elements
  int x_bf16, w_bf16;
  float eps, inv_dim, magnitude;
};

// lanes to a head (a power of two) for this layout, and the heads of a wave
int rope_lanes(int units);
// fills per, splits and groups of both sides from the sizes
void rope_plan(RopeArgs &a);
hipError_t launch_rope(const RopeArgs &a, hipStream_t s);
hipError_t launch_rope_backward(const RopeArgs &a, hipStream_t s);

// --------------------------------------------------------------- gated ----
struct GatedArgs {
  GemmArgs g;  // A, and as B the gate's weights (backward: the weights); M, N, K.  Its output fields are not used
  const uint8_t *u_codes, *u_scales;  // the up projection's weights
  const float *u_S;
  int u_kind;
  int activation;
  uint16_t *h;             // forward: the result
  uint16_t *gate, *up;     // forward: kept products, or null; backward: those of the forward pass
  uint16_t *dgate, *dup;   // backward: the results
  int64_t ld_h, ld_gate, ld_up, ld_dgate, ld_dup;
  unsigned int *amax[2], *rht[2];  // maxima of h, or of dgate and dup (null: not wanted)
};
hipError_t launch_gemm_gated(const GatedArgs &a, hipStream_t s);
hipError_t launch_gemm_gated_backward(const GatedArgs &a, hipStream_t s);

}  // namespace nvfp4
