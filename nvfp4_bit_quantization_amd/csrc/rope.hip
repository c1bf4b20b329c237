// Norm of every query and key head with the position rotation, and the gradient
// of both (include/nvfp4.h: nvfp4_qk_rope, nvfp4_qk_rope_backward).
//
// A lane holds up to 16 elements of a head as 8 pairs that turn together: with
// half layout 8 consecutive elements of the first half and the 8 that belong to
// them from the second, with interleaved layout 16 consecutive ones.  No element
// leaves its lane; a norm's sum crosses the lanes of one head (8 at head_dim 128)
// in DPP steps.  What is not rotated is held as pairs that turn by nothing.
// A wave takes as many neighbouring heads of a token at a time as divide their
// number, up to what fills its lanes (8 at head_dim 128), and as many tokens as
// fill the rest: 40 heads go by eights of one token, 10 by twos of four, 5 of
// eight tokens one by one.  The angles' sines, formed once for a token, serve all
// the heads that the wave goes through.  The angle in turns is reduced in 64 bits
// (a 32-bit product is off by 0.06 rad at position 1000000), the rest in 32.
//
// Both passes are bound by memory: 2 x 8192 tokens of 40 + 8 heads of 128 bf16 move
// 403 MB in 81 us (5.0 TB/s), the gradient 604 MB in 122 (4.9), where a copy of 2 GiB
// reaches 4.9.  Few tokens take what a launch does: 5 us for 16.  4096 tokens are bound
// by a wave's own chain (places, angles, three heads after another): half of it waits.
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

// The places of a wave's tokens base + slot in their sequences; false: in none.
// ends: cu[lane] of every lane, where 64 lanes hold all of cu.
__device__ __forceinline__ bool place_of(const RopeArgs &a, int64_t base, int slot, int slots, int ends, int64_t &b, int64_t &n,
                                         double &position) {
  const int64_t t = base + slot;
  b = 0;
  n = t;
  if (!a.cu) {
    if (a.batch > 1) {
      b = (int64_t)((uint32_t)t / (uint32_t)a.tokens);
      n = t - b * a.tokens;
    }
    position = a.positions && t < a.total ? (double)a.positions[t] : (double)n;
    return true;
  }
  int which = -1, start = 0;  // the last sequence that begins at or before t
  if (a.batch < 64) {
    for (int k = 0; k < slots; ++k) {
      const int begun = __popcll(__ballot((int)(threadIdx.x & 63u) <= a.batch && ends <= base + k)) - 1;
      const int at = __builtin_amdgcn_readlane(ends, begun < 0 ? 0 : begun);
      if (slot == k) {
        which = begun;
        start = at;
      }
    }
  } else {
    int lo = 0, hi = a.batch;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t)
        lo = mid;
      else
        hi = mid - 1;
    }
    start = a.cu[lo];
    which = start <= t ? lo : -1;
  }
  position = (double)(t - start);
  return which >= 0 && which < a.batch;
}

template <typename W>
__device__ __forceinline__ void load_weight(const W *w, const Segments &s, float out[2][8]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (s.len[k] == 8) {
      load8(w + s.at[k], out[k]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) out[k][j] = j < s.len[k] ? load1(w + s.at[k] + j) : 0.0f;
    }
  }
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
__global__ __launch_bounds__(kWaves * 64, G ? 3 : 4) void rope_kernel(RopeArgs a) {
  const bool second = (int)blockIdx.x >= a.side[0].groups;
  const RopeSide &t = a.side[second];
  const int group = (int)blockIdx.x - (second ? a.side[0].groups : 0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = t.per, at_once = 64 / L / per;  // heads and tokens of a wave at a time
  const int u = lane & (L - 1), slot = lane / L / per, sub = lane / L % per;
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
  const int ends = a.cu && a.batch < 64 ? a.cu[min(lane, a.batch)] : 0;
  const uint32_t item = __builtin_amdgcn_readfirstlane(group * kWaves + wave), items = t.groups * kWaves;
  const int rounds = t.heads / per, share = (rounds + t.splits - 1) / t.splits;
  const int h0 = (int)(item % t.splits) * share * per, h1 = min(t.heads, h0 + share * per);
  for (int64_t base = (int64_t)(item / t.splits) * at_once; base < a.total; base += (int64_t)(items / t.splits) * at_once) {
    int64_t b, n;
    double position;
    const bool placed = place_of(a, base, slot, at_once, ends, b, n, position);
    const bool live = used && base + slot < a.total && placed;
    const TX *x = (const TX *)t.x + (live ? b * t.x_b + n * t.x_t + sub * t.x_h : 0);
    uint16_t *y = t.y + (live ? b * t.y_b + n * t.y_t + sub * t.y_h : 0);
    TX *dx = G ? (TX *)t.dx + (live ? b * t.dx_b + n * t.dx_t + sub * t.dx_h : 0) : nullptr;
    Raw<TX> rx[2];  // the first heads are on their way while the angles are formed
    Raw<uint16_t> ry[2];
    if (!G || N) fetch<R>(x + h0 * t.x_h, seg, live, rx);
    if (G) fetch<R>(y + h0 * t.y_h, seg, live, ry);
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = 1.0f;
      s[j] = 0.0f;
      if (live && seg.first >= 0 && seg.first + j < a.rot / 2) turn(position * f[j], a.magnitude, c[j], s[j]);
    }
    for (int h = h0; h < h1; h += per) {
      float v[2][8], g[2][8];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (!G || N) v[k][j] = rx[k].at(j);
          if (G) g[k][j] = ry[k].at(j);
        }
      const int next = h + per < h1 ? h + per : h;
      if (!G || N) fetch<R>(x + next * t.x_h, seg, live, rx);
      if (G) fetch<R>(y + next * t.y_h, seg, live, ry);
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
        if (live) put<R>(y + h * t.y_h, seg, v);
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
      if (live) put<R>(dx + h * t.dx_h, seg, g);
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

// dweight of both sides: 8 columns to a workgroup, 128 threads to a column over
// the workgroups' parts, in a fixed order
__global__ __launch_bounds__(1024) void rope_reduce_kernel(RopeArgs a) {
  const RopeSide &t = a.side[blockIdx.y];
  if (!t.dweight) return;
  const int col = blockIdx.x * 8 + (threadIdx.x & 7);
  float v = 0.0f;
#pragma unroll 8
  for (int r = threadIdx.x >> 3; r < t.groups; r += 128) v += t.parts[(int64_t)r * a.dim + col];
#pragma unroll
  for (int o = 8; o < 64; o *= 2) v += __shfl_xor(v, o, 64);
  __shared__ float sums[16][8];
  if ((threadIdx.x & 63) < 8) sums[threadIdx.x >> 6][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; ++r) v += sums[r][threadIdx.x];
    t.dweight[col] = v;
  }
}

// some segment is shorter than 8 (heads are of multiples of 8)
bool ragged(const RopeArgs &a) { return a.interleaved ? false : a.rot % 16 != 0; }

template <typename TX, int L, bool I, bool G, bool R>
void launch_of(const RopeArgs &a, dim3 grid, hipStream_t s) {
  if (a.side[0].weight || a.side[1].weight)
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, true, R>), grid, dim3(kWaves * 64), 0, s, a);
  else
    hipLaunchKernelGGL((rope_kernel<TX, L, I, G, false, R>), grid, dim3(kWaves * 64), 0, s, a);
}
template <typename TX, bool G>
hipError_t launch_typed(const RopeArgs &a, hipStream_t s) {
  const dim3 grid(a.side[0].groups + a.side[1].groups);
  const int l = rope_lanes(a.units);
  const bool r = ragged(a);
  if (a.interleaved && l == 4)
    launch_of<TX, 4, true, G, false>(a, grid, s);
  else if (a.interleaved)
    launch_of<TX, 8, true, G, false>(a, grid, s);
  else if (l == 4 && r)
    launch_of<TX, 4, false, G, true>(a, grid, s);
  else if (l == 4)
    launch_of<TX, 4, false, G, false>(a, grid, s);
  else if (l == 8 && r)
    launch_of<TX, 8, false, G, true>(a, grid, s);
  else if (l == 8)
    launch_of<TX, 8, false, G, false>(a, grid, s);
  else
    launch_of<TX, 16, false, G, true>(a, grid, s);
  return hipGetLastError();
}

}  // namespace

// Waves that share out heads where tokens are few, and workgroups of a side at most,
// which then go on to further tokens: two to a compute unit keep the weights and
// frequencies that they hold in use and leave no short last round.  In us, by waves
// 512, 1024, 2048, 4096: 10 + 5 float32 heads of 80, backward, 4096 tokens 30.0, 29.8,
// 38.4, 35.9 and 8192 tokens 37.6, 37.7, 48.2, 50.6 (packed 4096: 24.7 for 1024, 28.7,
// 29.9), forward 8192 tokens 19.1, 19.1, 19.3, 22.7; 40 + 8 heads of 128, 64 to 4096
// tokens, the same within 0.5 with any.  By workgroups 256, 384, 512, 768, 1024: 40 + 8
// heads of 128, 16384 tokens 108, 87, 78, 85, 84, backward 130, 129, 122, 127, 131; 65536
// tokens 415, 331, 298, 320, 310, backward 489, 483, 460, 470, 477; 32768 tokens of 10 +
// 5 float32 heads of 80, 84, 71, 59, 57, 58, backward 203, 193, 172, 172, 180; of 32 + 32
// heads of 128, where both sides have as many, 210, 195, 200, 208, 199, backward 297, 304,
// 332, 313, 309: there 512 is up to 12 % off the best.
constexpr int64_t kRopeWaves = 1024, kRopeGroups = 512;

// up to 8 units of 16 elements; a ninth where a head of 128 has a segment cut short
int rope_lanes(int units) { return units <= 4 ? 4 : units <= 8 ? 8 : 16; }

void rope_plan(RopeArgs &a) {
  const int slots = 64 / rope_lanes(a.units);
  for (RopeSide &t : a.side) {
    t.per = t.splits = 1;
    t.groups = 0;
    if (!t.heads) continue;
    while (t.per < slots && t.heads % (2 * t.per) == 0) t.per *= 2;
    const int64_t at_once = slots / t.per, blocks = (a.total + at_once - 1) / at_once, rounds = t.heads / t.per;
    // heads are shared out until there are kRopeWaves waves, or one to a head
    int64_t splits = blocks ? (kRopeWaves + blocks - 1) / blocks : 1;
    if (splits > rounds) splits = rounds;
    const int64_t share = (rounds + splits - 1) / splits;
    t.splits = (int)((rounds + share - 1) / share);
    int64_t groups = (blocks * t.splits + kWaves - 1) / kWaves;
    if (groups > kRopeGroups) groups = kRopeGroups;
    t.groups = (int)((groups + t.splits - 1) / t.splits * t.splits);  // each split as often
    if (t.groups < 1) t.groups = 1;
  }
}

hipError_t launch_rope(const RopeArgs &a, hipStream_t s) {
  return a.x_bf16 ? launch_typed<uint16_t, false>(a, s) : launch_typed<float, false>(a, s);
}

hipError_t launch_rope_backward(const RopeArgs &a, hipStream_t s) {
  const hipError_t e = a.x_bf16 ? launch_typed<uint16_t, true>(a, s) : launch_typed<float, true>(a, s);
  if (e != hipSuccess || !(a.side[0].dweight || a.side[1].dweight)) return e;
  hipLaunchKernelGGL(rope_reduce_kernel, dim3(a.dim / 8, 2), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
