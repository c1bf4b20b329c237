// Device helpers of the training operators (gfx950): groups of 8 elements in
// binary32, and reductions over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_device.hpp"

namespace nvfp4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// two values as bf16, nearest-even, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ float round_bf16(float a) { return __uint_as_float(pack_bf16(0.0f, a) & 0xFFFF0000u); }

// 8 consecutive elements, aligned to their own size: global accesses of 16
// bytes need no more on this target (those that are 16-byte aligned are quicker)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) u32x4_at2;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 __attribute__((aligned(4))) f32x4_at4;
__device__ __forceinline__ uint4 load_group(const uint16_t *p) {
  const u32x4 q = *reinterpret_cast<const u32x4_at2 *>(p);
  return make_uint4(q.x, q.y, q.z, q.w);
}
__device__ __forceinline__ void load8(const uint16_t *p, float v[8]) {
  const uint4 q = load_group(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = bf16_at(q, j);
}
__device__ __forceinline__ void load8(const float *p, float v[8]) {
  const f32x4 a = reinterpret_cast<const f32x4_at4 *>(p)[0], b = reinterpret_cast<const f32x4_at4 *>(p)[1];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = a[j];
    v[4 + j] = b[j];
  }
}
__device__ __forceinline__ u32x4 packed8(const float v[8]) {
  return (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
__device__ __forceinline__ void store8(uint16_t *p, const float v[8]) { *reinterpret_cast<u32x4_at2 *>(p) = packed8(v); }
__device__ __forceinline__ void store8(float *p, const float v[8]) {
  reinterpret_cast<f32x4_at4 *>(p)[0] = (f32x4){v[0], v[1], v[2], v[3]};
  reinterpret_cast<f32x4_at4 *>(p)[1] = (f32x4){v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ float load1(const uint16_t *p) { return bf16_lo(*p); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

// v as an element of the type keeps it
template <typename T>
__device__ __forceinline__ float rounded(float v);
template <>
__device__ __forceinline__ float rounded<uint16_t>(float v) { return round_bf16(v); }
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }

// Sum and maximum over the 64 lanes, in every lane: four DPP steps inside the
// rows of 16 lanes, then the row and half swaps (which hand both rows' or
// halves' values to both).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <typename F>
__device__ __forceinline__ float swapped16(float v, F f) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename F>
__device__ __forceinline__ float swapped32(float v, F f) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x128>(v);  // row_ror:8
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  v += dpp<0x121>(v);
  v = swapped16(v, [](float a, float b) { return a + b; });
  v = swapped32(v, [](float a, float b) { return a + b; });
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x128>(v));
  v = fmaxf(v, dpp<0x124>(v));
  v = fmaxf(v, dpp<0x122>(v));
  v = fmaxf(v, dpp<0x121>(v));
  v = swapped16(v, [](float a, float b) { return fmaxf(a, b); });
  v = swapped32(v, [](float a, float b) { return fmaxf(a, b); });
  return v;
}

// fold a wave's maximum of non-negative floats into *out: bit patterns of
// non-negative floats order as their values do, and a maximum does not depend
// on the order of the atomics.  An infinity is kept, a NaN is no maximum: what a
// tensor of finite values cannot hold is not looked for.
__device__ __forceinline__ void fold_max(float *out, float v) {
  v = wave_max(v);
  if ((threadIdx.x & 63) == 0 && v > 0.0f) atomicMax(reinterpret_cast<unsigned int *>(out), __float_as_uint(v));
}

}  // namespace nvfp4
