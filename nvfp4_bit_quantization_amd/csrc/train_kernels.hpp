// Kernel argument blocks and launch helpers of the training operators (layer
// norm, AdamW, attention), shared by train_api.cpp and their translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4.h"

namespace nvfp4 {

// ---------------------------------------------------------------- norm ----
constexpr int64_t kNormMaxCols = 32768;

hipError_t launch_layernorm(const nvfp4_layernorm_args &a, hipStream_t s);
// workgroups of the gradient kernel = rows of its partial sums [parts][2][cols]
int64_t layernorm_backward_parts(int64_t rows, int64_t cols);
hipError_t launch_layernorm_backward(const nvfp4_layernorm_backward_args &a, float *partials, hipStream_t s);

// --------------------------------------------------------------- adamw ----
constexpr int kAdamThreads = 256;
constexpr int kAdamChunk = 4096;  // elements of one workgroup (a multiple of 8 * kAdamThreads)

enum AdamFlags : uint32_t {
  AF_PARAM_BF16 = 1, AF_GRAD_BF16 = 2, AF_STATE8 = 4,
  AF_EXTRA = 8,       // has an AdamExtra
  AF_EXTRA_SHIFT = 8  // its number, from bit 8 on
};

struct AdamTensor {
  void *param;
  const void *grad;
  void *m, *v;
  int64_t n;
  float keep;      // 1 - lr * weight_decay
  uint32_t flags;
  uint32_t index;  // place in the caller's list
  uint32_t end;    // workgroups of this and the earlier tensors of the launch
};
struct AdamExtra {  // what not every tensor has
  uint8_t *m_scale, *v_scale;
  uint16_t *copy;
  float *amax;
};

// The descriptors travel as kernel arguments: AdamTensors from the front of
// the bytes, AdamExtras from the back, as many as 4 KiB of arguments hold (71
// tensors without extras, 45 with).
constexpr int kAdamBytes = 4000;
struct AdamArgs {
  alignas(8) unsigned char bytes[kAdamBytes];
  int count;
  int sr;
  float lr, beta1, one_minus_beta1, beta2, one_minus_beta2, eps;
  float correct1, correct2;  // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  uint32_t seed_lo, seed_hi, step_lo, tag;
  const float *grad_scale;

  __host__ __device__ const AdamTensor &tensor(int i) const { return ((const AdamTensor *)bytes)[i]; }
  __host__ __device__ const AdamExtra &extra(int i) const { return ((const AdamExtra *)(bytes + kAdamBytes))[-1 - i]; }
};
static_assert(sizeof(AdamTensor) == 56 && sizeof(AdamExtra) == 32 && sizeof(AdamArgs) <= 4096, "kernel arguments");

hipError_t launch_adamw(const AdamArgs &a, hipStream_t s);

// ----------------------------------------------------------- attention ----
struct Heads {
  uint16_t *p;
  int64_t sb, st, sh;  // elements between sequences, tokens, heads
};

// division of a 31-bit n by d as a product: n / d = (n by) >> shift with
// by = ceil(2^shift / d) and shift = 31 + ceil(log2 d), since the excess
// n (by d - 2^shift) / (d 2^shift) < n / 2^31 / d stays below 1 / d
struct Divisor {
  uint32_t d, by, shift;
};
inline Divisor divisor(uint32_t d) {
  Divisor r = {d, 0u, 31u};
  while (((uint64_t)1 << (r.shift - 31)) < d) ++r.shift;
  r.by = (uint32_t)((((uint64_t)1 << r.shift) + d - 1) / d);
  return r;
}

struct AttnArgs {
  Heads q, k, v, o, d_o, dq, dk, dv;
  float *lse;    // [heads][total_q]
  float *minus_delta, *minus_lse;  // gradient: [heads][total_q], -delta and -lse / scale
  // parts of a split pass, in binary32: [part][heads][total_q][D] and
  // [part][heads][total_q]; [part][kv_heads][total_k][D]; D = 64 or 128
  int q_parts, k_parts;
  float *q_part, *lse_part, *k_part, *v_part;
  const int32_t *cu_q, *cu_k;
  int64_t total_q, total_k;
  int window;  // 0: none
  int q_len, k_len;
  int batch, heads, kv_heads, dim;
  int causal;
  float scale;
  int q_tiles, k_tiles;  // tiles of 128 rows
  Divisor by_group, by_batch, by_kv;  // heads of a key head, sequences, key heads
};

// parts that the shape's passes are split into, from its sizes alone
int attention_q_parts(const AttnArgs &a);
int attention_k_parts(const AttnArgs &a);
hipError_t launch_attention(const AttnArgs &a, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs &a, hipStream_t s);

}  // namespace nvfp4
