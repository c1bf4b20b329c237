// One AdamW step over many tensors (include/nvfp4.h: nvfp4_adamw).
//
// Memory-bound: every element's parameter, gradient and two states are read
// and written once.  A workgroup takes one chunk of one tensor; the tensors'
// descriptors travel as kernel arguments, so that a step needs neither a
// device table nor a copy.  A thread holds 8 consecutive elements at a time;
// four neighbouring lanes hold a block of 32 of an 8-bit state, so that block
// maxima need two DPP steps.
//
// Two weights of 5120x20480 take 1083 to 1141 us on several devices with 32-bit
// states and a bf16 copy (5.9 GB, 5.1-5.4 TB/s; a copy of 2 GiB reaches 4.9) and
// 402 to 416 us with 8-bit states (2.1 GB, 5.1-5.3 TB/s, the vector unit busy in
// 94 % of the cycles).  The 8-bit step was bound by vector instructions at
// 623 us while E4M3 was encoded and decoded by integer steps: per 8 elements the
// three Philox draws alone are some 40 multiplications.
#include "train_device.hpp"
#include "train_kernels.hpp"

namespace nvfp4 {
namespace {

// maximum over the 4 lanes that share a block of 32 elements
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));  // quad_perm [1,0,3,2]
  return fmaxf(v, dpp<0x4E>(v));  // quad_perm [2,3,0,1]
}

// 2^k as a float, k in [-126, 127]
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// The block exponent of a maximum: the least e >= -126 with top <= 448 * 2^e.
// 448 = 1.75 * 2^8, so the exponent field counts up where the mantissa passes
// 1.75 (0x600000): 0x600001 + 0x1FFFFF carries.
__device__ __forceinline__ int block_exponent(float top) {
  const int e = (int)((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 135;
  return e > -126 ? e : -126;
}

// 8 state elements: their E4M3 codes under the quad's scale 2^e.  Lanes
// outside the tensor hold zeros.  The gfx950 FP8 conversions round y = x / 2^e
// (|y| <= 448) to nearest, or up iff the place of |y| between its neighbours,
// in 2^-20, and the random operand's upper 20 bits sum to 2^20 or more.  With
// the 16-bit uniform u in the upper half that is floor(|y| / step + u / 65536),
// exactly (the tests compare every binade down to 2^-12).  positive: x >= 0, and what
// is not zero is raised to the least E4M3 value before it is rounded, so that it
// cannot vanish.
template <bool SR>
__device__ __forceinline__ uint2 encode8(const float x[8], const uint32_t w[4], bool positive, int *e) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
  *e = block_exponent(quad_max(top));
  const float inv = pow2(-*e);
  int q[2] = {0, 0};
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = x[j] * inv;
    if (positive) y[j] = x[j] > 0.0f ? fmaxf(y[j], 0.001953125f) : 0.0f;
  }
  if constexpr (SR) {
    q[0] = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], w[0] << 16, q[0], 0);
    q[0] = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], w[0] & 0xFFFF0000u, q[0], 1);
    q[0] = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], w[1] << 16, q[0], 2);
    q[0] = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], w[1] & 0xFFFF0000u, q[0], 3);
    q[1] = __builtin_amdgcn_cvt_sr_fp8_f32(y[4], w[2] << 16, q[1], 0);
    q[1] = __builtin_amdgcn_cvt_sr_fp8_f32(y[5], w[2] & 0xFFFF0000u, q[1], 1);
    q[1] = __builtin_amdgcn_cvt_sr_fp8_f32(y[6], w[3] << 16, q[1], 2);
    q[1] = __builtin_amdgcn_cvt_sr_fp8_f32(y[7], w[3] & 0xFFFF0000u, q[1], 3);
  } else {
    q[0] = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], q[0], false);
    q[0] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], q[0], true);
    q[1] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], q[1], false);
    q[1] = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], q[1], true);
  }
  return make_uint2((uint32_t)q[0], (uint32_t)q[1]);
}

__device__ __forceinline__ void decode8(uint2 q, uint32_t scale, float x[8]) {
  const float s = __builtin_ldexpf(1.0f, (int)scale - 127);
  const f32x2 v[4] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true),
                      __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true)};
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = v[j >> 1][j & 1] * s;
}

// 8 elements, `have` of them in the tensor
template <typename T>
__device__ __forceinline__ void get8(const T *p, int have, float v[8]) {
  if (have == 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < have ? load1(p + j) : 0.0f;
  }
}
// past the caches: 32-bit states and their parameter are not read again before
// the next step (two weights of 5120x20480: 1203 -> 1129 us; with 8-bit states,
// whose traffic is a third, no gain there and 8 % lost on tensors that the
// caches hold)
__device__ __forceinline__ void stream8(uint16_t *p, const float v[8]) {
  __builtin_nontemporal_store(packed8(v), reinterpret_cast<u32x4_at2 *>(p));
}
__device__ __forceinline__ void stream8(float *p, const float v[8]) {
  f32x4_at4 *q = reinterpret_cast<f32x4_at4 *>(p);
  __builtin_nontemporal_store((f32x4){v[0], v[1], v[2], v[3]}, q);
  __builtin_nontemporal_store((f32x4){v[4], v[5], v[6], v[7]}, q + 1);
}
template <bool STREAM, typename T>
__device__ __forceinline__ void put8(T *p, int have, const float v[8]) {
  if (have == 8) {
    if constexpr (STREAM)
      stream8(p, v);
    else
      store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) store1(p + j, v[j]);
  }
}
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 __attribute__((aligned(1))) u32x2_at1;
__device__ __forceinline__ uint2 get_codes(const uint8_t *p, int have) {
  if (have == 8) {
    const u32x2 q = *reinterpret_cast<const u32x2_at1 *>(p);
    return make_uint2(q.x, q.y);
  }
  uint32_t q[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < have) q[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint2(q[0], q[1]);
}
__device__ __forceinline__ void put_codes(uint8_t *p, int have, uint2 q) {
  if (have == 8) {
    *reinterpret_cast<u32x2_at1 *>(p) = (u32x2){q.x, q.y};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < have) p[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
  }
}

// the four words that serve a group of 8 elements (which: 0 m, 1 r, 2 param)
__device__ __forceinline__ void draw(const AdamArgs &a, uint32_t index, uint32_t which, int64_t group, uint32_t w[4]) {
  w[0] = (uint32_t)group;
  w[1] = 4u * index + which;
  w[2] = a.step_lo;
  w[3] = a.tag;
  philox4x32_10(a.seed_lo, a.seed_hi, w);
}

// elements i0 .. i0 + 7 of a tensor; returns the maximum of what is stored
template <typename TP, typename TG, bool S8, bool SR>
__device__ __forceinline__ float step8(const AdamArgs &a, const AdamTensor &t, const AdamExtra &x, float gs, int64_t i0) {
  const int64_t left = t.n - i0;
  const int have = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  float p[8], g[8], m[8], v[8];
  uint32_t w[4];
  get8((const TP *)t.param + i0, have, p);
  get8((const TG *)t.grad + i0, have, g);
  if constexpr (S8) {
    const uint2 qm = get_codes((const uint8_t *)t.m + i0, have), qv = get_codes((const uint8_t *)t.v + i0, have);
    decode8(qm, have ? x.m_scale[i0 >> 5] : 0u, m);
    decode8(qv, have ? x.v_scale[i0 >> 5] : 0u, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= v[j];
  } else {
    get8((const float *)t.m + i0, have, m);
    get8((const float *)t.v + i0, have, v);
  }
  float r[8], least = INFINITY;
  // the square root and reciprocal instructions: 1 unit in the last place
  // each, next to the update's ten other roundings.  Both read subnormal
  // numbers as zero: the reciprocal's is at least eps, which is normal; the
  // root takes such squares (of gradients below some 1e-18) times 2^64
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = g[j] * gs;
    m[j] = m[j] * a.beta1 + y * a.one_minus_beta1;
    v[j] = v[j] * a.beta2 + y * y * a.one_minus_beta2;
    least = fminf(least, v[j]);
    r[j] = __builtin_amdgcn_sqrtf(v[j]);
  }
  if (least < 0x1p-126f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (v[j] < 0x1p-126f) r[j] = __builtin_amdgcn_sqrtf(v[j] * 0x1p64f) * 0x1p-32f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    p[j] = p[j] * t.keep - a.lr * ((m[j] * a.correct1) * __builtin_amdgcn_rcpf(r[j] * a.correct2 + a.eps));
  if constexpr (SR && sizeof(TP) == 2) {
    draw(a, t.index, 2u, i0 >> 3, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = __uint_as_float((__float_as_uint(p[j]) + u16_of(w, j)) & 0xFFFF0000u);
  }
  put8<!S8>((TP *)t.param + i0, have, p);
  if (x.copy) put8<false>(x.copy + i0, have, p);
  if constexpr (S8) {
    int e;
    if (SR) draw(a, t.index, 0u, i0 >> 3, w);
    put_codes((uint8_t *)t.m + i0, have, encode8<SR>(m, w, false, &e));
    const bool leader = have && (threadIdx.x & 3) == 0;
    if (leader) x.m_scale[i0 >> 5] = (uint8_t)(e + 127);
    if (SR) draw(a, t.index, 1u, i0 >> 3, w);
    put_codes((uint8_t *)t.v + i0, have, encode8<SR>(r, w, true, &e));
    if (leader) x.v_scale[i0 >> 5] = (uint8_t)(e + 127);
  } else {
    put8<true>((float *)t.m + i0, have, m);
    put8<true>((float *)t.v + i0, have, v);
  }
  float top = 0.0f;
  if (x.amax) {
    const bool bf16 = x.copy || sizeof(TP) == 2;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(bf16 ? round_bf16(p[j]) : p[j]));
  }
  return top;
}

template <typename TP, typename TG, bool S8, bool SR>
__device__ __forceinline__ void chunk(const AdamArgs &a, const AdamTensor &t, const AdamExtra &x, int64_t first) {
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float top = 0.0f;
  // whole workgroups take part in every step (block maxima cross lanes)
  for (int64_t i = first; i < first + kAdamChunk && i < t.n; i += 8 * kAdamThreads)
    top = fmaxf(top, step8<TP, TG, S8, SR>(a, t, x, gs, i + 8 * threadIdx.x));
  if (x.amax) fold_max(x.amax, top);
}

template <bool SR>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(const AdamArgs a) {
  int i = 0;
  for (int step = 64; step; step >>= 1)  // the first tensor that ends behind this workgroup
    if (i + step <= a.count - 1 && a.tensor(i + step - 1).end <= blockIdx.x) i += step;
  const AdamTensor &t = a.tensor(i);
  const AdamExtra x = t.flags & AF_EXTRA ? a.extra((int)(t.flags >> AF_EXTRA_SHIFT)) : AdamExtra{};
  const int64_t first = (int64_t)(blockIdx.x - (i ? a.tensor(i - 1).end : 0u)) * kAdamChunk;
  switch (t.flags & 7u) {
    case 0: chunk<float, float, false, SR>(a, t, x, first); break;
    case AF_PARAM_BF16: chunk<uint16_t, float, false, SR>(a, t, x, first); break;
    case AF_GRAD_BF16: chunk<float, uint16_t, false, SR>(a, t, x, first); break;
    case AF_PARAM_BF16 | AF_GRAD_BF16: chunk<uint16_t, uint16_t, false, SR>(a, t, x, first); break;
    case AF_STATE8: chunk<float, float, true, SR>(a, t, x, first); break;
    case AF_STATE8 | AF_PARAM_BF16: chunk<uint16_t, float, true, SR>(a, t, x, first); break;
    case AF_STATE8 | AF_GRAD_BF16: chunk<float, uint16_t, true, SR>(a, t, x, first); break;
    default: chunk<uint16_t, uint16_t, true, SR>(a, t, x, first); break;
  }
}

}  // namespace

hipError_t launch_adamw(const AdamArgs &a, hipStream_t s) {
  const unsigned grid = a.tensor(a.count - 1).end;
  if (a.sr)
    adamw_kernel<true><<<grid, kAdamThreads, 0, s>>>(a);
  else
    adamw_kernel<false><<<grid, kAdamThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
