// Layer norm over rows and its gradient (include/nvfp4.h: nvfp4_layernorm,
// nvfp4_layernorm_backward).
//
// A row is held in registers: TPR threads (whole waves) each hold V groups of
// 8 elements, so that mean, centred second moment and the result come from one
// read of the row.  Rows of up to 1024 elements belong to one wave each (no
// LDS), longer ones to up to 16 waves that exchange their sums through LDS.
// Workgroups walk over rows with the weights kept in registers.
//
// Both passes are bound by memory: 8192x5120 bf16 with a residual moves 336 MB
// in 88 us (3.8 TB/s; 159 us before rows were loaded ahead and the two
// exchanges of a row made one), the gradient of 16384x5120 671 MB in 142 us
// (4.7 TB/s; 325 us before; 140-143 on several devices).  Small calls take what a launch does: 3 us for
// 256x256.  Rows need no alignment beyond their elements'.  Above 8192 elements
// neither weights nor the next row fit the registers; above 16384 the gradient's
// sums do not either: 4096x20480 bf16 takes 95 us (161 with all groups' weights
// read at once, which spilled) and its gradient 195 in three kernels, which read
// x and dy twice (611 in two, the sums in scratch memory).
#include "train_device.hpp"
#include "train_kernels.hpp"

namespace nvfp4 {
namespace {

// Where a thread's group v stands: columns base .. base + 7, of which the first
// `lead` are not its own (8: the group is past the end).  At a ragged width (R:
// no multiple of 8) the last group starts at cols - 8, so that its load is one of
// whole 16 bytes; what it repeats of its neighbour counts as zero in sums and is
// not stored.  Widths below 8 have base < 0 and their elements at the end.
// Against an end read element by element, 8192 rows of 5119 bf16 take 59 us
// instead of 73, with a residual 106 instead of 143 (117 with the maximum, too),
// their gradient 70 instead of 120; 16384 rows of 2049, without a residual, 47
// instead of 42.  Widths that are multiples of 8 have kernels without it
// (8192x5120: 48 us, 54 with it).
struct Place {
  int base, lead;
};
template <bool R>
__device__ __forceinline__ Place place(int v, int t, int tpr, int cols) {
  const int c = (v * tpr + t) * 8;
  if (!R) return {c, c < cols ? 0 : 8};
  const int base = c < cols - 8 ? c : cols - 8;
  return {base, c < cols ? c - base : 8};
}
template <bool R>
__device__ __forceinline__ bool own(const Place &p, int j) {
  return R ? j >= p.lead : p.lead == 0;
}

// 8 elements as they stand in memory: what is loaded ahead for the next row
template <typename T>
struct Group;
template <>
struct Group<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t *p) { q = load_group(p); }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load1(int j, const uint16_t *p) {  // into a zeroed group
    const uint32_t x = (uint32_t)*p << (16 * (j & 1));
    ((j >> 1) == 0 ? q.x : (j >> 1) == 1 ? q.y : (j >> 1) == 2 ? q.z : q.w) |= x;
  }
  __device__ __forceinline__ float at(int j) const { return bf16_at(q, j); }
};
template <>
struct Group<float> {
  float x[8];
  __device__ __forceinline__ void load(const float *p) { load8(p, x); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  }
  __device__ __forceinline__ void load1(int j, const float *p) { x[j] = *p; }
  __device__ __forceinline__ float at(int j) const { return x[j]; }
};

// a group of a row, zero past the end; TINY: the width may be below 8
template <bool TINY, typename T>
__device__ __forceinline__ void fetch_group(const T *row, int cols, const Place &p, Group<T> &g) {
  if (p.lead == 8) {
    g.zero();
  } else if (!TINY || cols >= 8) {
    g.load(row + p.base);
  } else {
    g.zero();
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j >= p.lead) g.load1(j, row + p.base + j);
  }
}
// a thread's share of a row
template <int V, bool R, typename T>
__device__ __forceinline__ void fetch_row(const T *row, int cols, int t, int tpr, Group<T> g[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v) fetch_group<(R && V == 1)>(row, cols, place<R>(v, t, tpr, cols), g[v]);
}

template <bool R, typename T>
__device__ __forceinline__ void store_group(T *row, const Place &p, const float in[8]) {
  if (p.lead == 0) {
    store8(row + p.base, in);
  } else if (R && p.lead < 8) {
#pragma unroll
    for (int j = 1; j < 8; ++j)
      if (j >= p.lead) store1(row + p.base + j, in[j]);
  }
}
template <int V, bool R, typename T>
__device__ __forceinline__ void store_row(T *row, int cols, int t, int tpr, const float in[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) store_group<R>(row, place<R>(v, t, tpr, cols), in[v]);
}

// a group of a weight, zero where the elements are not its own
template <bool TINY, bool R, typename T>
__device__ __forceinline__ void load_group_of(const T *w, int cols, const Place &p, float out[8]) {
  Group<T> g;
  fetch_group<TINY>(w, cols, p, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) out[j] = !R || own<R>(p, j) ? g.at(j) : 0.0f;
}
template <int V, bool R>
__device__ __forceinline__ void load_weight_group(const void *w, int bf16, int cols, const Place &p, float out[8]) {
  if (bf16)
    load_group_of<(R && V == 1), R>((const uint16_t *)w, cols, p, out);
  else
    load_group_of<(R && V == 1), R>((const float *)w, cols, p, out);
}
// a thread's share of a weight
template <int V, bool R>
__device__ __forceinline__ void load_weight(const void *w, int bf16, int cols, int t, int tpr, float out[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) load_weight_group<V, R>(w, bf16, cols, place<R>(v, t, tpr, cols), out[v]);
}
// Workgroups of up to 512 threads keep the weights in registers and load the
// next row ahead.  Those of 1024 have 128 registers to a thread, which a row
// of more than 8192 elements takes up: they read both when they are due.
constexpr bool holds(int nt) { return nt <= 512; }
// Above 16384 elements weights are read group by group, and the gradient's sums
// over rows are a kernel's own: beside a row their registers would spill.  bf16
// rows then fit (their ragged forward puts 8 to 24 bytes of a lane in scratch);
// float32 rows still spill, 40 to 76 bytes forward and 24 to 108 in the gradient.
constexpr bool by_group(int v) { return v > 2; }

// blockDim = (TPR, rows per workgroup); more than one row only when TPR = 64.
// The next row is loaded while this one is worked on.  Each wave takes the mean
// of its part and the sum of squares about that; one exchange joins them (n_w
// elements, mean_w, q_w to a wave):
//   mean = sum n_w mean_w / n,  q = sum q_w + n_w (mean_w - mean)^2
template <typename TX, typename TY, int V, int NT, bool R>
__global__ __launch_bounds__(NT) void layernorm_kernel(nvfp4_layernorm_args a) {
  __shared__ float2 slots[2][16];
  __shared__ float counts[16];
  int t = threadIdx.x;
  const int tpr = blockDim.x, waves = tpr >> 6, wave = t >> 6;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  constexpr bool kHold = holds(NT);
  const bool w_bf16 = a.w_dtype == NVFP4_BF16;
  Group<TX> gx[V], gr[V];
  if (kHold && r < a.rows) {
    fetch_row<V, R>((const TX *)a.x + r * a.ld_x, cols, t, tpr, gx);
    if (a.residual) fetch_row<V, R>((const TX *)a.residual + r * a.ld_residual, cols, t, tpr, gr);
  }
  float w[V][8], b[V][8], top = 0.0f;
  const auto weights = [&] {
    load_weight<V, R>(a.weight, w_bf16, cols, t, tpr, w);
    if (a.bias) load_weight<V, R>(a.bias, w_bf16, cols, t, tpr, b);
  };
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
  if (kHold) weights();
  int mine = 0;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) mine += own<R>(place<R>(v, t, tpr, cols), j);
  const float count = wave_sum((float)mine), inv_w = count > 0.0f ? 1.0f / count : 0.0f;
  if (waves > 1 && (t & 63) == 0) counts[wave] = count;
  int turn = 0;
  for (; r < a.rows; r += step) {
    if (by_group(V)) asm volatile("" : "+v"(t));  // what is formed of it stays out of registers between rows
    float x[V][8];
    if (!kHold) {
      fetch_row<V, R>((const TX *)a.x + r * a.ld_x, cols, t, tpr, gx);
      if (a.residual) fetch_row<V, R>((const TX *)a.residual + r * a.ld_residual, cols, t, tpr, gr);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = gx[v].at(j);
    if (a.residual) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = rounded<TX>(x[v][j] + gr[v].at(j));
    }
    if (kHold && r + step < a.rows) {
      fetch_row<V, R>((const TX *)a.x + (r + step) * a.ld_x, cols, t, tpr, gx);
      if (a.residual) fetch_row<V, R>((const TX *)a.residual + (r + step) * a.ld_residual, cols, t, tpr, gr);
    }
    if (a.residual) store_row<V, R>((TX *)a.sum + r * a.ld_sum, cols, t, tpr, x);
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += !R || own<R>(place<R>(v, t, tpr, cols), j) ? x[v][j] : 0.0f;
    float mean = wave_sum(s) * inv_w, q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = own<R>(place<R>(v, t, tpr, cols), j) ? x[v][j] - mean : 0.0f;
        q = fmaf(d, d, q);
      }
    q = wave_sum(q);
    if (waves > 1) {
      // two sets of slots in turn: a set is written again only after a barrier
      // that every wave passed with its reads of it done
      if ((t & 63) == 0) slots[turn][wave] = make_float2(mean, q);
      __syncthreads();
      mean = q = 0.0f;
      for (int i = 0; i < waves; ++i) mean = fmaf(counts[i], slots[turn][i].x, mean);
      mean *= inv;
      for (int i = 0; i < waves; ++i) {
        const float d = slots[turn][i].x - mean;
        q += fmaf(counts[i] * d, d, slots[turn][i].y);
      }
      turn ^= 1;
    }
    const float rstd = 1.0f / sqrtf(fmaf(q, inv, a.eps));
    if (t == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
    if (!kHold && !by_group(V)) weights();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Place at = place<R>(v, t, tpr, cols);
      if (by_group(V)) {
        load_weight_group<V, R>(a.weight, w_bf16, cols, at, w[v]);
        if (a.bias) load_weight_group<V, R>(a.bias, w_bf16, cols, at, b[v]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = rounded<TY>(fmaf((x[v][j] - mean) * rstd, w[v][j], b[v][j]));
        x[v][j] = y;
        if (a.amax && own<R>(at, j)) top = fmaxf(top, fabsf(y));
      }
      if (by_group(V)) {
        store_group<R>((TY *)a.y + r * a.ld_y, at, x[v]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!by_group(V)) store_row<V, R>((TY *)a.y + r * a.ld_y, cols, t, tpr, x);
  }
  if (a.amax) fold_max(a.amax, top);
}

// The gradient: a row's two sums in one exchange; h and dy * weight are formed
// twice from the row as it was loaded, before and after that, which keeps fewer
// registers than holding them.  The sums over rows stay in registers and are
// written once per workgroup, [blockIdx][dweight, dbias][cols].
template <typename TX, typename TY, int V, int NT, bool R>
__global__ __launch_bounds__(NT) void layernorm_backward_kernel(nvfp4_layernorm_backward_args a, float *partials) {
  __shared__ float2 slots[2][16];
  __shared__ float both[NT == 1024 ? 1 : 4][8][64];
  constexpr bool kHold = holds(NT);
  int t = threadIdx.x;
  const int tpr = blockDim.x, waves = tpr >> 6;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  const bool w_bf16 = a.w_dtype == NVFP4_BF16;
  float w[V][8], dw[V][8], db[V][8], top = 0.0f;
  if (kHold) load_weight<V, R>(a.weight, w_bf16, cols, t, tpr, w);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  Group<TX> gx[V], next_x[V], gd[V];
  Group<TY> gy[V], next_y[V];
  float mean = 0.0f, rstd = 0.0f, next_mean = 0.0f, next_rstd = 0.0f;
  const auto fetch = [&](int64_t row, Group<TX> *x, Group<TY> *y, float &m, float &s) {
    fetch_row<V, R>((const TX *)a.x + row * a.ld_x, cols, t, tpr, x);
    fetch_row<V, R>((const TY *)a.dy + row * a.ld_dy, cols, t, tpr, y);
    m = a.mean[row];
    s = a.rstd[row];
  };
  if (kHold && r < a.rows) fetch(r, next_x, next_y, next_mean, next_rstd);
  int turn = 0;
  for (; r < a.rows; r += step) {
    if (by_group(V)) asm volatile("" : "+v"(t));  // what is formed of it stays out of registers between rows
    if (kHold) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        gx[v] = next_x[v];
        gy[v] = next_y[v];
      }
      mean = next_mean;
      rstd = next_rstd;
      if (a.dsum) fetch_row<V, R>((const TX *)a.dsum + r * a.ld_dsum, cols, t, tpr, gd);
      if (r + step < a.rows) fetch(r + step, next_x, next_y, next_mean, next_rstd);
    } else {
      fetch(r, gx, gy, mean, rstd);
      if (!by_group(V)) load_weight<V, R>(a.weight, w_bf16, cols, t, tpr, w);
    }
    const auto weights = [&](int v) {
      __builtin_amdgcn_sched_barrier(0);
      load_weight_group<V, R>(a.weight, w_bf16, cols, place<R>(v, t, tpr, cols), w[v]);
    };
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (by_group(V)) weights(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // elements that are not its own: w = 0, and dw, db are not stored
        const float h = (gx[v].at(j) - mean) * rstd, dy = gy[v].at(j), q = dy * w[v][j];
        if (!by_group(V)) {
          dw[v][j] = fmaf(dy, h, dw[v][j]);
          db[v][j] += dy;
        }
        s1 += q;
        s2 = fmaf(q, h, s2);
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (waves > 1) {
      // two sets of slots in turn: a set is written again only after a barrier
      // that every wave passed with its reads of it done
      if ((t & 63) == 0) slots[turn][t >> 6] = make_float2(s1, s2);
      __syncthreads();
      s1 = s2 = 0.0f;
      for (int i = 0; i < waves; ++i) {
        s1 += slots[turn][i].x;
        s2 += slots[turn][i].y;
      }
      turn ^= 1;
    }
    const float c1 = s1 * inv, c2 = s2 * inv;
    if (!kHold && !by_group(V)) {
      if (a.dsum) fetch_row<V, R>((const TX *)a.dsum + r * a.ld_dsum, cols, t, tpr, gd);
      load_weight<V, R>(a.weight, w_bf16, cols, t, tpr, w);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Place at = place<R>(v, t, tpr, cols);
      if (by_group(V)) {
        if (v == 0) asm volatile("" : "+v"(t));
        weights(v);
        if (a.dsum) fetch_group<false>((const TX *)a.dsum + r * a.ld_dsum, cols, at, gd[v]);
      }
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = (gx[v].at(j) - mean) * rstd;
        x[j] = rstd * (gy[v].at(j) * w[v][j] - fmaf(h, c2, c1));
      }
      if (a.dsum) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] += gd[v].at(j);
      }
      store_group<R>((TX *)a.dx + r * a.ld_dx, at, x);
      if (a.amax) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (own<R>(at, j)) top = fmaxf(top, fabsf(rounded<TX>(x[j])));
      }
    }
  }
  if (a.amax) fold_max(a.amax, top);
  if (by_group(V) || !partials) return;
  float *out = partials + (int64_t)blockIdx.x * 2 * cols;
  if (blockDim.y == 1) {
    store_row<V, R>(out, cols, t, tpr, dw);
    store_row<V, R>(out + cols, cols, t, tpr, db);
    return;
  }
  // the rows of the workgroup's four waves, added in their order: each wave
  // joins two of the eight elements of every thread's group
  if constexpr (NT != 1024) {
#pragma unroll
    for (int k = 0; k < 2; ++k, out += cols)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (k || v) __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) both[threadIdx.y][j][t] = k ? db[v][j] : dw[v][j];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 2 * threadIdx.y + i;
          const Place at = place<R>(v, t, tpr, cols);
          const float s = (both[0][j][t] + both[1][j][t]) + (both[2][j][t] + both[3][j][t]);
          if (own<R>(at, j)) out[at.base + j] = s;
        }
      }
  }
}

// The partial sums of rows above 16384 elements: 8 columns to a thread, every
// gridDim.x-th row, several rows' loads in flight.
template <typename TX, typename TY, bool R>
__global__ __launch_bounds__(256) void layernorm_columns_kernel(nvfp4_layernorm_backward_args a, float *partials) {
  const int cols = (int)a.cols;
  const Place at = place<R>(0, (int)(blockIdx.y * 256 + threadIdx.x), 0, cols);
  if (at.lead == 8) return;
  float dw[8] = {}, db[8] = {};
#pragma unroll 4
  for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    Group<TX> x;
    Group<TY> y;
    x.load((const TX *)a.x + r * a.ld_x + at.base);
    y.load((const TY *)a.dy + r * a.ld_dy + at.base);
    const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float dy = y.at(j);
      dw[j] = fmaf(dy, (x.at(j) - mean) * rstd, dw[j]);
      db[j] += dy;
    }
  }
  float *out = partials + (int64_t)blockIdx.x * 2 * cols;
  store_group<R>(out, at, dw);
  store_group<R>(out + cols, at, db);
}

// dweight and dbias from the partial sums: a workgroup adds 64 columns, 16
// threads to a column, in a fixed order, eight loads in flight (512 parts of
// 5120 columns: 14 -> 5.7 us)
__global__ __launch_bounds__(1024) void layernorm_reduce_kernel(const float *partials, int64_t parts, int64_t cols,
                                                               float *dweight, float *dbias) {
  __shared__ float sums[16][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  float s = 0.0f;
  if (c < 2 * cols) {
    int64_t p = threadIdx.y;
    for (; p + 7 * 16 < parts; p += 8 * 16) {  // eight loads in flight
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = partials[(p + i * 16) * 2 * cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; p < parts; p += 16) s += partials[p * 2 * cols + c];
  }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += sums[i][threadIdx.x];
  float *out = c < cols ? dweight : dbias;
  if (out) out[c < cols ? c : c - cols] = s;
}

// How a row of `cols` elements is split: groups of 8 per thread, the workgroup
// size the kernel is built for, and threads per row and rows per workgroup.
struct Split {
  int v, nt;
  dim3 block;
  int waves() const { return (int)(block.x * block.y) / 64; }
};
Split split_of(int64_t cols) {
  if (cols <= 512) return {1, 256, dim3(64, 4)};
  if (cols <= 1024) return {2, 512, dim3(64, 4)};
  if (cols <= 16384) return {2, cols <= 8192 ? 512 : 1024, dim3((unsigned)((cols + 1023) / 1024 * 64))};
  return {4, 1024, dim3((unsigned)((cols + 2047) / 2048 * 64))};
}
// Workgroups: what the 256 compute units hold at a time (16 waves each, 12 of the
// gradient's), so that all run from the start and each walks over its share of
// the rows.  That is what the registers of bf16 rows admit; of gradients with
// float32 rows between 513 and 8192 elements they admit 8 waves, so that a part of
// the grid waits for the others' end (16384 rows float32 all the same: of 1024
// elements 43.5 us, 4.6 TB/s, of 5120 192 us, 5.2 TB/s).
int64_t resident(const Split &p, int64_t rows, int waves) {
  const int64_t groups = (rows + p.block.y - 1) / p.block.y, most = 256 * (waves / p.waves() > 1 ? waves / p.waves() : 1);
  return groups < most ? groups : most;
}

template <typename TX, typename TY, int V, int NT, bool R>
void run(const nvfp4_layernorm_args &a, float *, unsigned grid, dim3 block, hipStream_t s) {
  layernorm_kernel<TX, TY, V, NT, R><<<grid, block, 0, s>>>(a);
}
template <typename TX, typename TY, int V, int NT, bool R>
void run(const nvfp4_layernorm_backward_args &a, float *partials, unsigned grid, dim3 block, hipStream_t s) {
  if (by_group(V) && partials)  // first: dx may stand where dy or x does
    layernorm_columns_kernel<TX, TY, R><<<dim3((unsigned)layernorm_backward_parts(a.rows, a.cols),
                                            (unsigned)((a.cols + 2047) / 2048)), 256, 0, s>>>(a, partials);
  layernorm_backward_kernel<TX, TY, V, NT, R><<<grid, block, 0, s>>>(a, partials);
}

template <typename TX, typename TY, bool R, typename A>
void pick_split(const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (p.v == 1)
    run<TX, TY, 1, 256, R>(a, partials, grid, p.block, s);
  else if (p.v == 2 && p.nt == 512)
    run<TX, TY, 2, 512, R>(a, partials, grid, p.block, s);
  else if (p.v == 2)
    run<TX, TY, 2, 1024, R>(a, partials, grid, p.block, s);
  else
    run<TX, TY, 4, 1024, R>(a, partials, grid, p.block, s);
}
template <typename TX, typename TY, typename A>
void pick_width(const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (a.cols % 8)
    pick_split<TX, TY, true>(p, a, partials, grid, s);
  else
    pick_split<TX, TY, false>(p, a, partials, grid, s);
}
template <typename A>
void pick(const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (a.x_dtype == NVFP4_BF16 && a.y_dtype == NVFP4_BF16)
    pick_width<uint16_t, uint16_t>(p, a, partials, grid, s);
  else if (a.x_dtype == NVFP4_BF16)
    pick_width<uint16_t, float>(p, a, partials, grid, s);
  else if (a.y_dtype == NVFP4_BF16)
    pick_width<float, uint16_t>(p, a, partials, grid, s);
  else
    pick_width<float, float>(p, a, partials, grid, s);
}

}  // namespace

hipError_t launch_layernorm(const nvfp4_layernorm_args &a, hipStream_t s) {
  const Split p = split_of(a.cols);
  pick(p, a, nullptr, (unsigned)resident(p, a.rows, 16), s);
  return hipGetLastError();
}

// of the gradient: at least four rows to a workgroup beyond one to a compute
// unit, since each adds a row to what the second kernel reads; of the columns'
// kernel 16 rows, up to 128 parts
int64_t layernorm_backward_parts(int64_t rows, int64_t cols) {
  const Split p = split_of(cols);
  if (by_group(p.v)) return rows > 2048 ? 128 : (rows + 15) / 16;
  const int64_t most = resident(p, rows, 12), few = (rows / p.block.y + 3) / 4;
  return most <= 256 || most < few ? most : few > 256 ? few : 256;
}

hipError_t launch_layernorm_backward(const nvfp4_layernorm_backward_args &a, float *partials, hipStream_t s) {
  const Split p = split_of(a.cols);
  const int64_t parts = layernorm_backward_parts(a.rows, a.cols);
  pick(p, a, partials, (unsigned)(by_group(p.v) ? resident(p, a.rows, 16) : parts), s);
  if (partials)
    layernorm_reduce_kernel<<<(unsigned)((2 * a.cols + 63) / 64), dim3(64, 16), 0, s>>>(partials, parts, a.cols,
                                                                                      a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace nvfp4
