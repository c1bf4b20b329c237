// Layer norm over rows and its gradient (include/nvfp4.h: nvfp4_layernorm,
// nvfp4_layernorm_backward).
//
// A row is held in registers: TPR threads (whole waves) each hold V groups of
// 8 elements, so that mean, centred second moment and the result come from one
// read of the row.  Rows of up to 2048 elements belong to one wave each (no
// LDS), longer ones to up to 16 waves that exchange their sums through LDS.
// Workgroups walk over rows with the weights kept in registers.
#include "train_device.hpp"
#include "train_kernels.hpp"

namespace nvfp4 {
namespace {

// element j of a thread's group v: groups of 8 consecutive elements when rows
// can be read 16 bytes at a time, else elements TPR apart, which keeps single
// element accesses of a wave contiguous
template <bool VEC, int V>
__device__ __forceinline__ int64_t column(int v, int j, int t, int tpr) {
  return VEC ? (int64_t)(v * tpr + t) * 8 + j : (int64_t)(v * 8 + j) * tpr + t;
}

// a thread's share of a row, zero outside [0, cols)
template <bool VEC, int V, typename T>
__device__ __forceinline__ void load_row(const T *row, int cols, int t, int tpr, float out[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      const int64_t c = column<true, V>(v, 0, t, tpr);
      if (c < cols) {
        load8(row + c, out[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) out[v][j] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = column<false, V>(v, j, t, tpr);
        out[v][j] = c < cols ? load1(row + c) : 0.0f;
      }
    }
  }
}

template <bool VEC, int V, typename T>
__device__ __forceinline__ void store_row(T *row, int cols, int t, int tpr, const float in[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (VEC) {
      const int64_t c = column<true, V>(v, 0, t, tpr);
      if (c < cols) store8(row + c, in[v]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = column<false, V>(v, j, t, tpr);
        if (c < cols) store1(row + c, in[v][j]);
      }
    }
  }
}

template <bool VEC, int V>
__device__ __forceinline__ void load_weight(const void *w, int bf16, int cols, int t, int tpr, float out[V][8]) {
  if (bf16)
    load_row<VEC, V>((const uint16_t *)w, cols, t, tpr, out);
  else
    load_row<VEC, V>((const float *)w, cols, t, tpr, out);
}

// the sum of v over the waves of a row; `slot`: LDS of 16 floats
__device__ __forceinline__ float row_sum(float v, int waves, float *slot) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < waves; ++w) v += slot[w];
  return v;
}

// blockDim = (TPR, rows per workgroup); more than one row only when TPR = 64
template <typename TX, typename TY, bool VEC, int V, int NT>
__global__ __launch_bounds__(NT) void layernorm_kernel(nvfp4_layernorm_args a) {
  __shared__ float slots[2][16];
  const int t = threadIdx.x, tpr = blockDim.x, waves = tpr >> 6;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  float w[V][8], b[V][8], top = 0.0f;
  load_weight<VEC, V>(a.weight, a.w_dtype == NVFP4_BF16, cols, t, tpr, w);
  if (a.bias) {
    load_weight<VEC, V>(a.bias, a.w_dtype == NVFP4_BF16, cols, t, tpr, b);
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) b[v][j] = 0.0f;
  }
  for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < a.rows; r += (int64_t)gridDim.x * blockDim.y) {
    float x[V][8];
    load_row<VEC, V>((const TX *)a.x + r * a.ld_x, cols, t, tpr, x);
    if (a.residual) {
      float q[V][8];
      load_row<VEC, V>((const TX *)a.residual + r * a.ld_residual, cols, t, tpr, q);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] = rounded<TX>(x[v][j] + q[v][j]);
      store_row<VEC, V>((TX *)a.sum + r * a.ld_sum, cols, t, tpr, x);
    }
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += x[v][j];
    const float mean = row_sum(s, waves, slots[0]) * inv;
    s = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = column<VEC, V>(v, j, t, tpr) < cols ? x[v][j] - mean : 0.0f;
        x[v][j] = d;
        s = fmaf(d, d, s);
      }
    const float rstd = 1.0f / sqrtf(row_sum(s, waves, slots[1]) * inv + a.eps);
    if (t == 0) {
      a.mean[r] = mean;
      a.rstd[r] = rstd;
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = rounded<TY>(fmaf(x[v][j] * rstd, w[v][j], b[v][j]));
        x[v][j] = y;
        top = fmaxf(top, fabsf(y));  // columns past the end hold 0
      }
    store_row<VEC, V>((TY *)a.y + r * a.ld_y, cols, t, tpr, x);
  }
  if (a.amax) fold_max(a.amax, top);
}

// The gradient: a row's two sums in one exchange; the sums over rows stay in
// registers and are written once per workgroup, [blockIdx][dweight, dbias][cols].
template <typename TX, typename TY, bool VEC, int V, int NT>
__global__ __launch_bounds__(NT) void layernorm_backward_kernel(nvfp4_layernorm_backward_args a, float *partials) {
  __shared__ float2 slots[2][16];
  __shared__ float both[4][64 * 8];
  const int t = threadIdx.x, tpr = blockDim.x, waves = tpr >> 6;
  const int cols = (int)a.cols;
  const float inv = 1.0f / (float)cols;
  float w[V][8], dw[V][8], db[V][8], top = 0.0f;
  load_weight<VEC, V>(a.weight, a.w_dtype == NVFP4_BF16, cols, t, tpr, w);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = db[v][j] = 0.0f;
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < a.rows; r += (int64_t)gridDim.x * blockDim.y) {
    float x[V][8], g[V][8];
    load_row<VEC, V>((const TX *)a.x + r * a.ld_x, cols, t, tpr, x);
    load_row<VEC, V>((const TY *)a.dy + r * a.ld_dy, cols, t, tpr, g);
    const float mean = a.mean[r], rstd = a.rstd[r];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // past the end: dy = w = 0
        const float h = (x[v][j] - mean) * rstd, dy = g[v][j];
        dw[v][j] = fmaf(dy, h, dw[v][j]);
        db[v][j] += dy;
        const float q = dy * w[v][j];
        s1 += q;
        s2 = fmaf(q, h, s2);
        x[v][j] = h;
        g[v][j] = q;
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
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = rstd * (g[v][j] - fmaf(x[v][j], c2, c1));
    if (a.dsum) {
      load_row<VEC, V>((const TX *)a.dsum + r * a.ld_dsum, cols, t, tpr, g);
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[v][j] += g[v][j];
    }
    store_row<VEC, V>((TX *)a.dx + r * a.ld_dx, cols, t, tpr, x);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (column<VEC, V>(v, j, t, tpr) < cols) top = fmaxf(top, fabsf(rounded<TX>(x[v][j])));
  }
  if (a.amax) fold_max(a.amax, top);
  if (!partials) return;
  float *out = partials + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
  for (int k = 0; k < 2; ++k, out += cols) {
    if (blockDim.y == 1) {
      store_row<VEC, V>(out, cols, t, tpr, k ? db : dw);
      continue;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {  // the rows of the workgroup's waves, added in their order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) both[threadIdx.y][j * 64 + t] = k ? db[v][j] : dw[v][j];
      __syncthreads();
      if (threadIdx.y == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float s = 0.0f;
          for (int y = 0; y < (int)blockDim.y; ++y) s += both[y][j * 64 + t];
          const int64_t c = column<VEC, V>(v, j, t, tpr);
          if (c < cols) out[c] = s;
        }
      }
    }
  }
}

// dweight and dbias from the partial sums: a workgroup adds 64 columns, 16
// threads to a column, in a fixed order
__global__ __launch_bounds__(1024) void layernorm_reduce_kernel(const float *partials, int64_t parts, int64_t cols,
                                                               float *dweight, float *dbias) {
  __shared__ float sums[16][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
  float s = 0.0f;
  if (c < 2 * cols)
    for (int64_t p = threadIdx.y; p < parts; p += 16) s += partials[p * 2 * cols + c];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0 || c >= 2 * cols) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += sums[i][threadIdx.x];
  float *out = c < cols ? dweight : dbias;
  if (out) out[c < cols ? c : c - cols] = s;
}

bool at16(const void *p, int64_t ld, int32_t dtype) {
  return ((uintptr_t)p & 15u) == 0 && ld % (dtype == NVFP4_BF16 ? 8 : 4) == 0;
}

// How a row of `cols` elements is split: groups of 8 per thread, threads per
// row and rows per workgroup, and the workgroup size the kernel is built for.
struct Split {
  int v, nt;
  dim3 block;
};
Split split_of(int64_t cols) {
  if (cols <= 512) return {1, 256, dim3(64, 4)};
  if (cols <= 1024) return {2, 512, dim3(64, 4)};
  if (cols <= 2048) return {4, 256, dim3(64, 4)};
  if (cols <= 8192) return {2, 512, dim3((unsigned)((cols + 1023) / 1024 * 64))};
  return {4, 1024, dim3((unsigned)((cols + 2047) / 2048 * 64))};
}

template <typename TX, typename TY, bool VEC, int V, int NT>
void run(const nvfp4_layernorm_args &a, float *, unsigned grid, dim3 block, hipStream_t s) {
  layernorm_kernel<TX, TY, VEC, V, NT><<<grid, block, 0, s>>>(a);
}
template <typename TX, typename TY, bool VEC, int V, int NT>
void run(const nvfp4_layernorm_backward_args &a, float *partials, unsigned grid, dim3 block, hipStream_t s) {
  layernorm_backward_kernel<TX, TY, VEC, V, NT><<<grid, block, 0, s>>>(a, partials);
}

template <typename TX, typename TY, bool VEC, typename A>
void pick_split(const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (p.v == 1)
    run<TX, TY, VEC, 1, 256>(a, partials, grid, p.block, s);
  else if (p.v == 2)
    run<TX, TY, VEC, 2, 512>(a, partials, grid, p.block, s);
  else if (p.nt == 256)
    run<TX, TY, VEC, 4, 256>(a, partials, grid, p.block, s);
  else
    run<TX, TY, VEC, 4, 1024>(a, partials, grid, p.block, s);
}
template <typename TX, typename TY, typename A>
void pick_vec(bool vec, const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (vec)
    pick_split<TX, TY, true>(p, a, partials, grid, s);
  else
    pick_split<TX, TY, false>(p, a, partials, grid, s);
}
template <typename A>
void pick(bool vec, const Split &p, const A &a, float *partials, unsigned grid, hipStream_t s) {
  if (a.x_dtype == NVFP4_BF16 && a.y_dtype == NVFP4_BF16)
    pick_vec<uint16_t, uint16_t>(vec, p, a, partials, grid, s);
  else if (a.x_dtype == NVFP4_BF16)
    pick_vec<uint16_t, float>(vec, p, a, partials, grid, s);
  else if (a.y_dtype == NVFP4_BF16)
    pick_vec<float, uint16_t>(vec, p, a, partials, grid, s);
  else
    pick_vec<float, float>(vec, p, a, partials, grid, s);
}

}  // namespace

hipError_t launch_layernorm(const nvfp4_layernorm_args &a, hipStream_t s) {
  const Split p = split_of(a.cols);
  const bool vec = a.cols % 8 == 0 && at16(a.x, a.ld_x, a.x_dtype) && at16(a.y, a.ld_y, a.y_dtype) &&
                   at16(a.weight, 0, a.w_dtype) && at16(a.bias, 0, a.w_dtype) &&
                   (!a.residual || (at16(a.residual, a.ld_residual, a.x_dtype) && at16(a.sum, a.ld_sum, a.x_dtype)));
  const int64_t groups = (a.rows + p.block.y - 1) / p.block.y;
  const unsigned grid = (unsigned)(groups < 2048 ? groups : 2048);
  pick(vec, p, a, nullptr, grid, s);
  return hipGetLastError();
}

int64_t layernorm_backward_parts(int64_t rows, int64_t cols) {
  const Split p = split_of(cols);
  const int64_t groups = (rows + p.block.y - 1) / p.block.y;
  return groups < 512 ? groups : 512;
}

hipError_t launch_layernorm_backward(const nvfp4_layernorm_backward_args &a, float *partials, hipStream_t s) {
  const Split p = split_of(a.cols);
  const bool vec = a.cols % 8 == 0 && at16(a.x, a.ld_x, a.x_dtype) && at16(a.dy, a.ld_dy, a.y_dtype) &&
                   at16(a.weight, 0, a.w_dtype) && at16(a.dx, a.ld_dx, a.x_dtype) &&
                   (!a.dsum || at16(a.dsum, a.ld_dsum, a.x_dtype));
  const int64_t parts = layernorm_backward_parts(a.rows, a.cols);
  pick(vec, p, a, partials, (unsigned)parts, s);
  if (partials)
    layernorm_reduce_kernel<<<(unsigned)((2 * a.cols + 63) / 64), dim3(64, 16), 0, s>>>(partials, parts, a.cols,
                                                                                      a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace nvfp4
