// Norm of every query and key head with the position rotation, and the gradient
// of both (include/nvfp4.h: nvfp4_qk_rope, nvfp4_qk_rope_backward).
//
// A lane holds up to 16 elements of a head as 8 pairs that turn together: with
// half layout 8 consecutive elements of the first half and the 8 that belong to
// them from the second, with interleaved layout 16 consecutive ones.  No element
// leaves its lane; a norm's sum crosses the lanes of one head (8 at head_dim 128)
// in DPP steps.  What is not rotated is held as pairs that turn by nothing.
// The angles' sines are formed once for a token and used for all its heads: the
// angle in turns is reduced in 64 bits (a 32-bit product is off by 0.06 rad at
// position 1000000), the rest in 32.
#include "block_kernels.hpp"
#include "train_device.hpp"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;  // of a workgroup

// the 8 elements of a segment as they stand in memory
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t *p) { q = load_group(p); }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void set(int j, const uint16_t *p) {  // of a zeroed one
    const uint32_t x = (uint32_t)p[j] << (16 * (j & 1));
    ((j >> 1) == 0 ? q.x : (j >> 1) == 1 ? q.y : (j >> 1) == 2 ? q.z : q.w) |= x;
  }
  __device__ __forceinline__ float at(int j) const { return bf16_at(q, j); }
};
template <>
struct Raw<float> {
  float x[8];
  __device__ __forceinline__ void load(const float *p) { load8(p, x); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  }
  __device__ __forceinline__ void set(int j, const float *p) { x[j] = p[j]; }
  __device__ __forceinline__ float at(int j) const { return x[j]; }
};

// A lane's two segments of a head: where they begin and how many elements (0 to
// 8) are theirs.  R: some are shorter than 8.
struct Segments {
  int at[2], len[2];
  int first;  // number of the lane's first pair, or -1: none of its pairs turns
};
__device__ __forceinline__ Segments segments(const RopeArgs &a, int u) {
  Segments s;
  const int half = a.rot / 2, turned = (half + 7) / 8;
  if (!a.interleaved && u < turned) {
    s.at[0] = 8 * u;
    s.at[1] = half + 8 * u;
    s.len[0] = s.len[1] = min(8, half - 8 * u);
    s.first = 8 * u;
    return s;
  }
  s.at[0] = a.interleaved ? 16 * u : a.rot + 16 * (u - turned);
  s.at[1] = s.at[0] + 8;
  s.first = a.interleaved ? 8 * u : -1;
#pragma unroll
  for (int k = 0; k < 2; ++k) s.len[k] = max(0, min(8, a.dim - s.at[k]));
  return s;
}

template <bool R, typename T>
__device__ __forceinline__ void fetch(const T *head, const Segments &s, bool live, Raw<T> r[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    r[k].zero();
    if (!live) continue;
    if (R ? s.len[k] == 8 : s.len[k] > 0) {
      r[k].load(head + s.at[k]);
    } else if (R) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < s.len[k]) r[k].set(j, head + s.at[k]);
    }
  }
}
template <bool R, typename T>
__device__ __forceinline__ void put(T *head, const Segments &s, const float v[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (R ? s.len[k] == 8 : s.len[k] > 0) {
      store8(head + s.at[k], v[k]);
    } else if (R) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < s.len[k]) store1(head + s.at[k] + j, v[k][j]);
    }
  }
}

// sum over the L lanes of a head, in each of them
template <int L>
__device__ __forceinline__ float head_sum(float v) {
  if (L >= 16) v += dpp<0x128>(v);        // row_ror:8
  if (L >= 8) v += dpp<0x141>(v);         // row_half_mirror
  if (L >= 2) v += dpp<0xB1>(v);          // quad_perm 1 0 3 2
  if (L >= 4) v += dpp<0x4E>(v);          // quad_perm 2 3 0 1
  return v;
}

// cos and sin of a number of turns, times `magnitude`: the turns are reduced to
// at most 1/8 around the next quarter, where the Taylor sums to z^9 and z^8 are
// within 2^-25
__device__ __forceinline__ void turn(double turns, float magnitude, float &c, float &s) {
  const float r = (float)(turns - __builtin_rint(turns));
  const float q = __builtin_rintf(4.0f * r);
  const float z = fmaf(-0.25f, q, r) * 6.283185307f, z2 = z * z;
  float ps = fmaf(z2, 2.755731922e-6f, -1.984126984e-4f);
  ps = fmaf(z2, ps, 8.333333333e-3f);
  ps = fmaf(z2, ps, -0.1666666667f);
  ps = fmaf(z2 * z, ps, z);
  float pc = fmaf(z2, 2.480158730e-5f, -1.388888889e-3f);
  pc = fmaf(z2, pc, 4.166666667e-2f);
  pc = fmaf(z2, pc, -0.5f);
  pc = fmaf(z2, pc, 1.0f);
  const int k = (int)q & 3;
  const float a = (k & 1) ? ps : pc, b = (k & 1) ? pc : ps;
  c = (k == 1 || k == 2 ? -a : a) * magnitude;
  s = (k >= 2 ? -b : b) * magnitude;
}

// the place of token t in its sequence; false: it belongs to none
__device__ __forceinline__ bool place_of(const RopeArgs &a, int64_t t, int64_t &b, int64_t &n, double &position) {
  b = 0;
  n = t;
  if (a.cu) {
    int lo = 0, hi = a.batch;  // the last of cu[0 .. batch] that is <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int64_t start = a.cu[lo];
    position = (double)(t - start);
    return lo < a.batch && start <= t;
  }
  if (a.batch > 1) {
    b = (int64_t)((uint32_t)t / (uint32_t)a.tokens);
    n = t - b * a.tokens;
  }
  position = a.positions ? (double)a.positions[t] : (double)n;
  return true;
}

template <typename W>
__device__ __forceinline__ void load_weight(const W *w, const Segments &s, float out[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) out[k][j] = j < s.len[k] ? load1(w + s.at[k] + j) : 0.0f;
}

// v turned by the lane's angles (forward) or back (s of the other sign)
__device__ __forceinline__ void rotate(float v[2][8], const float c[8], const float s[8], bool interleaved, float sign) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float &p = interleaved ? v[j >> 2][2 * (j & 3)] : v[0][j];
    float &q = interleaved ? v[j >> 2][2 * (j & 3) + 1] : v[1][j];
    const float x = p, y = q, t = sign * s[j];
    p = x * c[j] - y * t;
    q = y * c[j] + x * t;
  }
}

// L lanes to a head; I: interleaved pairs; G: the gradient; N: with a norm.
template <typename TX, int L, bool I, bool G, bool N, bool R>
__global__ __launch_bounds__(kWaves * 64) void rope_kernel(RopeArgs a) {
  const bool second = (int)blockIdx.x >= a.side[0].groups;
  const RopeSide &t = a.side[second];
  const int group = (int)blockIdx.x - (second ? a.side[0].groups : 0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int u = lane & (L - 1), slot = lane / L;
  const int per = t.per, at_once = (64 / L) / per;  // tokens of a wave at a time
  const Segments seg = segments(a, u);
  const bool used = u < a.units;
  float w[2][8], dw[2][8];
  if (N) {
    if (a.w_bf16)
      load_weight((const uint16_t *)t.weight, seg, w);
    else
      load_weight((const float *)t.weight, seg, w);
  }
  double f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int p = seg.first + j;
    f[j] = seg.first >= 0 && p < a.rot / 2 ? a.freqs[p] * 0.15915494309189533577 : 0.0;
    if (G && N) dw[0][j] = dw[1][j] = 0.0f;
  }
  const uint32_t item = group * kWaves + wave, items = t.groups * kWaves;
  const int split = item % t.splits;
  for (int64_t base = (int64_t)(item / t.splits) * at_once; base < a.total; base += (int64_t)(items / t.splits) * at_once) {
    const int64_t token = base + slot / per;
    int64_t b, n;
    double position;
    const bool live = used && token < a.total && place_of(a, token, b, n, position);
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.0f;
      s[j] = 0.0f;
      if (live && seg.first >= 0 && seg.first + j < a.rot / 2) turn(position * f[j], a.magnitude, c[j], s[j]);
    }
    const TX *x = (const TX *)t.x + (live ? b * t.x_b + n * t.x_t : 0);
    uint16_t *y = t.y + (live ? b * t.y_b + n * t.y_t : 0);
    TX *dx = G ? (TX *)t.dx + (live ? b * t.dx_b + n * t.dx_t : 0) : nullptr;
    int h = slot % per + split * per;
    const int step = per * t.splits;
    Raw<TX> rx[2];
    Raw<uint16_t> ry[2];
    if (!G || N) fetch<R>(x + h * t.x_h, seg, live && h < t.heads, rx);
    if (G) fetch<R>(y + h * t.y_h, seg, live && h < t.heads, ry);
    for (; __any(live && h < t.heads); h += step) {
      const bool here = live && h < t.heads;
      float v[2][8], g[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!G || N) v[k][j] = rx[k].at(j);
          if (G) g[k][j] = ry[k].at(j);
        }
      const bool next = live && h + step < t.heads;
      if (!G || N) fetch<R>(x + (h + step) * t.x_h, seg, next, rx);
      if (G) fetch<R>(y + (h + step) * t.y_h, seg, next, ry);
      float rstd = 1.0f;
      if (N) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) sum = fmaf(v[k][j], v[k][j], sum);
        rstd = 1.0f / sqrtf(fmaf(head_sum<L>(sum), a.inv_dim, a.eps));
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[k][j] *= rstd;
      }
      if (!G) {
        if (N) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] *= w[k][j];
        }
        rotate(v, c, s, I, 1.0f);
        if (here) put<R>(y + h * t.y_h, seg, v);
        continue;
      }
      rotate(g, c, s, I, -1.0f);
      if (N) {
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            dw[k][j] = fmaf(g[k][j], v[k][j], dw[k][j]);
            g[k][j] *= w[k][j];
            dot = fmaf(g[k][j], v[k][j], dot);
          }
        dot = head_sum<L>(dot) * a.inv_dim;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j) g[k][j] = rstd * fmaf(-dot, v[k][j], g[k][j]);
      }
      if (here) put<R>(dx + h * t.dx_h, seg, g);
    }
  }
  if (!G || !N || !t.dweight) return;
  // the workgroup's part of dweight: over the wave's heads, then over the waves
  __shared__ float sums[kWaves][16 * L];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v = dw[k][j];
#pragma unroll
      for (int o = L; o < 64; o *= 2) v += __shfl_xor(v, o, 64);
      if (lane < L) sums[wave][(k * 8 + j) * L + u] = v;
    }
  __syncthreads();
  if (wave == 0 && lane < L && used) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = 0.0f;
#pragma unroll
        for (int o = 0; o < kWaves; ++o) v += sums[o][(k * 8 + j) * L + u];
        if (j < seg.len[k]) t.parts[(int64_t)group * a.dim + seg.at[k] + j] = v;
      }
  }
}

// dweight of both sides: 8 columns to a workgroup, 32 threads to a column over
// the workgroups' parts, in a fixed order
__global__ __launch_bounds__(256) void rope_reduce_kernel(RopeArgs a) {
  const RopeSide &t = a.side[blockIdx.y];
  if (!t.dweight) return;
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
  float v = 0.0f;
  for (int r = row; r < t.groups; r += 32) v += t.parts[(int64_t)r * a.dim + col];
  __shared__ float sums[256];
  sums[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.0f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += sums[r * 8 + threadIdx.x];
    t.dweight[col] = v;
  }
}

// some segment is shorter than 8
bool ragged(const RopeArgs &a) { return a.interleaved ? false : a.rot % 16 != 0; }

template <typename TX, int L, bool I, bool G>
void launch_of(const RopeArgs &a, dim3 grid, hipStream_t s) {
  const bool n = a.side[0].weight || a.side[1].weight, r = ragged(a);
  const dim3 block(kWaves * 64);
  if (n && r)
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, true, !I>), grid, block, 0, s, a);
  else if (n)
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, true, false>), grid, block, 0, s, a);
  else if (r)
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, false, !I>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, false, false>), grid, block, 0, s, a);
}
template <typename TX, bool G>
hipError_t launch_typed(const RopeArgs &a, hipStream_t s) {
  const dim3 grid(a.side[0].groups + a.side[1].groups);
  const int l = rope_lanes(a.units);
#define NVFP4_ROPE(L)                                                  \
  if (l == L) {                                                        \
    if (a.interleaved)                                                 \
      launch_of<TX, L, true, G>(a, grid, s);                           \
    else                                                               \
      launch_of<TX, L, false, G>(a, grid, s);                          \
  }
  NVFP4_ROPE(4)
  NVFP4_ROPE(8)
  NVFP4_ROPE(16)
#undef NVFP4_ROPE
  return hipGetLastError();
}

}  // namespace

int rope_lanes(int units) { return units <= 4 ? 4 : units <= 8 ? 8 : 16; }

void rope_plan(RopeArgs &a) {
  const int slots = 64 / rope_lanes(a.units);
  for (RopeSide &t : a.side) {
    t.per = 1;
    t.splits = 1;
    t.groups = 0;
    if (!t.heads) continue;
    while (t.per < slots && t.per < t.heads) t.per *= 2;
    const int64_t at_once = slots / t.per, waves = (a.total + at_once - 1) / at_once;
    const int most = (t.heads + t.per - 1) / t.per;
    // few tokens: a wave to each group of heads, so that no load waits for another's
    if (waves * most <= 4096) t.splits = most;
    int64_t groups = (waves * t.splits + kWaves - 1) / kWaves;
    const int64_t cap = 1280;
    if (groups > cap) groups = cap;
    groups = (groups + t.splits - 1) / t.splits * t.splits;  // each split as often
    t.groups = (int)(groups < 1 ? 1 : groups);
  }
}

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  return a.x_bf16 ? launch_typed<uint16_t, false>(a, s) : launch_typed<float, false>(a, s);
}

hipError_t launch_rope_backward(const RopeArgs &a, hipStream_t s) {
  const hipError_t e = a.x_bf16 ? launch_typed<uint16_t, true>(a, s) : launch_typed<float, true>(a, s);
  if (e != hipSuccess || !(a.side[0].dweight || a.side[1].dweight)) return e;
  hipLaunchKernelGGL(rope_reduce_kernel, dim3(a.dim / 8, 2), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
