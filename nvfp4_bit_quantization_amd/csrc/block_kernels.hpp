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
  int per;      // heads of a token that a wave takes at a time: a power of two that divides them
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

// lanes to a head, a power of two
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

// ---------------------------------------------------------------- muon ----
// Matrices are worked on as m x n with m <= n ("turned" ones have more rows than
// columns), padded with zeros to whole tiles.  A value is held times a power of two
// as the sum of two fp16, whose matrices stand one behind the other: 22 bits of it,
// down to 2^-25.  The powers are the largest that keep the values below fp16's 65504.
constexpr float kMuonX = 16384.0f;  // of the iterate, whose singular values stay below 3.5
constexpr float kMuonA = 4096.0f;   // of its square and of the polynomial in it, up to 14
constexpr float kMuonQ = 512.0f;    // of a product of polynomials, up to 64
constexpr int kMuonMats = 30;      // of one launch: what 4 KiB of arguments hold
constexpr int kMuonChunk = 8192;   // elements of a workgroup of the sums and of the update
constexpr int kMuonParts = 512;    // workgroups of a matrix's sum, at most

// Elements between the rows of a matrix of n columns (n a multiple of 64): an odd
// number of 128-byte lines, so that a column of lines is spread over the channels
// of the L2 and of memory.
__host__ __device__ inline int64_t muon_ld(int64_t n) { return (n / 64 | 1) * 64; }

enum MuonFlags : uint32_t { MF_PARAM_BF16 = 1, MF_GRAD_BF16 = 2, MF_TURNED = 4 };

struct MuonMat {
  const void *grad;
  float *m;
  void *param;
  uint16_t *copy, *update;
  float *amax;
  _Float16 *direct, *turned;  // [rp][cp] as the tensor stands, and [cp][rp] (rows muon_ld apart)
  double *parts;
  int rows, cols, rp, cp;     // the tensor's, and padded
  float keep, step;           // 1 - lr * weight_decay, lr * scale
  uint32_t flags, index;
  uint32_t sums;              // workgroups of its sum
};
struct MuonArgs {
  MuonMat mat[kMuonMats];
  uint32_t end[kMuonMats];  // workgroups of a matrix and the earlier ones; past the last: 2^32 - 1
  int count, sr, nesterov;
  float beta, one_minus_beta;
  uint32_t seed_lo, seed_hi, step_lo, tag;
  const float *grad_scale;
};
static_assert(sizeof(MuonMat) == 112 && sizeof(MuonArgs) <= 4096, "kernel arguments");

// The matrix of a workgroup, whose number becomes that within the matrix: all
// ends are loaded at once (one after another, 20 matrices took 2 us).
__device__ __forceinline__ int muon_mat_of(const uint32_t end[kMuonMats], uint32_t &group) {
  int which = 0;
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < kMuonMats; ++i) {
    const bool past = group >= end[i];
    which += past;
    before = past ? end[i] : before;
  }
  group -= before;
  return which;
}

// D = alpha P Q^T + beta E + gamma I of every matrix, P [M][K], Q [N][K], D and E
// [M][N], DT [N][M], rows muon_ld apart; D or DT may be null.  Symmetric: P Q^T is, D = DT, and
// only tiles on and below the diagonal are formed.
struct NsMat {
  const _Float16 *p, *q, *e;
  _Float16 *d, *dt;
  int M, N, K;
};
struct NsArgs {
  NsMat mat[kMuonMats];
  uint32_t end[kMuonMats];  // tiles of a matrix and the earlier ones; past the last: 2^32 - 1
  int count, symmetric;
  float alpha, beta, gamma;
};
// the launches fill the ends
hipError_t launch_muon_sums(MuonArgs &a, hipStream_t s);
hipError_t launch_muon_form(MuonArgs &a, hipStream_t s);
// tile: 64, 128 or 256 rows and columns of a workgroup
hipError_t launch_muon_product(NsArgs &a, int tile, hipStream_t s);
hipError_t launch_muon_update(MuonArgs &a, hipStream_t s);

}  // namespace nvfp4
