// Device helpers of the block operators (gfx950).
#pragma once

#include "train_device.hpp"

namespace nvfp4 {

// the largest of a wave's numbers, in each of its lanes
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  const auto top = [](float a, float b) { return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b))); };
  float f = __uint_as_float(v);  // only moved as such
  f = top(f, dpp<0x128>(f));
  f = top(f, dpp<0x124>(f));
  f = top(f, dpp<0x122>(f));
  f = top(f, dpp<0x121>(f));
  f = swapped16(f, top);
  f = swapped32(f, top);
  return __float_as_uint(f);
}

// Raise up to N maxima (null: not wanted) to those of a workgroup of four waves:
// bits[k] of every lane, patterns of floats without their sign, which order as their
// values do, with what is not a number above infinity: as numbers, so that it stays.  Atomics on one address take some 8 ns each, whoever issues them: one
// to a wave made 43 of 71 us of a gated product of 16 rows (5120 waves).  So there
// is one to a workgroup, and only where it raises what stands there; a maximum
// does not depend on the order, nor on reading an older value first.
template <int N>
__device__ __forceinline__ void raise_maxima(unsigned int *const out[N], const uint32_t bits[N]) {
  __shared__ uint32_t tops[N][4];
  const uint32_t wave = threadIdx.x >> 6;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (!out[k]) continue;
    const uint32_t top = wave_top(bits[k]);
    if ((threadIdx.x & 63u) == 0) tops[k][wave] = top;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (out[k] && threadIdx.x == (uint32_t)k) {
      const uint32_t top = max(max(tops[k][0], tops[k][1]), max(tops[k][2], tops[k][3]));
      if (top > __hip_atomic_load(out[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) atomicMax(out[k], top);
    }
}

}  // namespace nvfp4
