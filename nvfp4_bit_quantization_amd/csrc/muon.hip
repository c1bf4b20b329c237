// Steps of matrices by orthogonalised updates (include/nvfp4.h: nvfp4_muon).
//
// The iterate is X <- (a I + b A + c A^2) X with A = X X^T, three products of
// which two are symmetric: of those only tiles on and below the diagonal are
// formed, and stored twice.  The polynomial takes a I in, so that the third
// product needs nothing but its operands.  Long matrices chain steps (muon_chained):
// products of m x m take the place of those with the long side.  All products are
// "TN" (both operands contiguous in K), for which X is kept as it is and
// transposed: the epilogue writes both.
//
// A value is held as the sum of two fp16 (22 bits), a product formed of three:
// both first parts and the two mixed ones, summed in binary32.  The iteration brings
// weak directions to the size of strong ones, up to 485 times in five steps, and
// with them what rounding the strong ones left there: with one fp16 to a value the
// result was off by 1e-3 of its norm at best, by 2e-2 with one direction over noise
// of a hundredth or singular values that fall off as 1 / i^2, by 0.15 over noise of a
// ten thousandth.  So it is as an iteration in binary32 throughout, against 64 bits:
// 5120 x 20480 normal, over noise of a hundredth and of a ten thousandth 3.9e-6, 4.9e-5
// and 3.3e-4 (binary32: 1.1e-5, 8.3e-5, 6.0e-4); 2048 x 4096 with 1 / i^2 2.9e-5 (4.9e-5).
//
// Large products are bound by the matrix instructions: of 5120 x 20480, X X^T runs
// at 1.19 PFLOP/s of them, the product with X at 1.24 with 76 % of all cycles theirs,
// where a library's product of 8192^3 in fp16 reaches 1.49; the passes over momentum,
// gradient and parameter move 5 TB/s.  Steps of two matrices of 5120 x 20480 take 27.7 ms
// (without chains 45), 1.5 of them in those passes.  Small ones are bound by their
// launches, 8 to 21 us each: 290 us for 20 matrices of 256 x 1024.
#include "block_device.hpp"
#include "block_kernels.hpp"
#include "gemm_device.hpp"

namespace nvfp4 {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------- products ----
// Tiles of 64 T x 64 T by four waves, 2 x 2 of them, T x T blocks of 32 x 32 to a
// wave.  K-tiles of 64: a row's slice is a whole 128-byte line (slices of 64 bytes
// had each line fetched twice).  Its eight 16-byte chunks stand permuted by the
// row, so that 16 rows' reads of one chunk fall on different banks.
//
// A slot of LDS holds one operand's rows of a K-tile; kSlots of them are filled in
// turn, P's and Q's alternating, by direct transfers.  A wave reads fragments two
// sub-steps (of 16 k) ahead, so that a K-tile's slots are free after half of its
// products, and spreads the two slots' transfers over the next K-tile's worth of
// them, one to a row of products: in bursts they held the waves up.
constexpr int slab_stride(int t) { return 32 * t + 8; }  // floats between rows of an epilogue slab
template <int T, int SLOTS>
struct Ns {
  static constexpr int kTile = 64 * T;
  static constexpr int kSlots = SLOTS;
  static constexpr int kSlotBytes = kTile * 128;
  static constexpr int kMoves = 2 * T;                 // transfers of a wave to a slot
  static constexpr int kStride = slab_stride(T);
  static constexpr int kSlab = 32 * kStride;
  static constexpr int kLds = kSlots * kSlotBytes;
  static_assert(4 * kSlab * 4 <= kLds, "the epilogue's slabs");
};

template <int T>
struct NsFrags {
  half8 a[T], b[T];
};
// One sub-step: its products, with the fragments of the one after the next read
// and a slot's transfers issued beneath them, row by row (left to itself, the
// compiler puts reads right before their first use).
template <int T, typename Move>
__device__ __forceinline__ void multiply(f32x16 acc[T][T], const NsFrags<T> &f, NsFrags<T> &ahead, const uint8_t *p, const uint8_t *q,
                                         Move move) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    ahead.a[i] = *reinterpret_cast<const half8 *>(p + i * 4096);
    ahead.b[i] = *reinterpret_cast<const half8 *>(q + i * 4096);
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
    move(i);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// a value as the sum of two fp16: off by 2^-22 of it at most (2^-25, where that is more)
__device__ __forceinline__ void two_parts(float v, half8 parts[2], int j) {
  parts[0][j] = (_Float16)v;
  parts[1][j] = (_Float16)(v - (float)parts[0][j]);
}

__device__ __forceinline__ void slab_fence() { asm volatile("" ::: "memory"); }

// One orientation of a wave's results: 32 rows at a time through its slab, from
// which a lane takes 8 neighbouring columns.  E's elements at the same places are
// read a slab ahead (in turn with the stores, and of one fp16, they made the square
// of a 5120 x 5120 matrix 22 us longer).  write(i) puts rows row0 + 32 i onwards into the slab.
// plane: elements from a value's first part to its second, of D and E.
template <int T, bool E, typename Write>
__device__ __forceinline__ void store_rows(const NsArgs &a, _Float16 *d, const _Float16 *e, int64_t plane, int64_t ld, int64_t row0,
                                           int64_t col0, const float *slab, uint32_t lane, Write write) {
  constexpr int LANES = 4 * T, ROWS = 64 / LANES, TIMES = 32 / ROWS;
  const int c = lane % LANES * 8, first = lane / LANES;
  // where the wave's elements begin, and the lane's from there on (with all of an
  // address formed by lane, the large tiles of E spilled)
  const int64_t at = row0 * ld + col0;
  const uint32_t mine = (uint32_t)(first * ld) + c;
  const int diagonal = (int)(row0 - col0) + first - c;  // of the lane's 8 columns, in its first row
  half8 x[TIMES][2];
  const auto fetch = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < TIMES; ++k)
#pragma unroll
      for (int part = 0; part < 2; ++part)
        x[k][part] = *reinterpret_cast<const half8 *>(e + (at + part * plane + (i * 32 + k * ROWS) * ld) + mine);
  };
  if (E) fetch(0);
#pragma unroll
  for (int i = 0; i < T; ++i) {
    write(i);
    slab_fence();
    float v[TIMES][8];
#pragma unroll
    for (int k = 0; k < TIMES; ++k)
#pragma unroll
      for (int b = 0; b < 8; ++b) v[k][b] = a.alpha * slab[(k * ROWS + first) * slab_stride(T) + c + b];
    slab_fence();
    if (E) {
#pragma unroll
      for (int k = 0; k < TIMES; ++k)
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          v[k][b] = fmaf(a.beta, (float)x[k][0][b] + (float)x[k][1][b], v[k][b]);
          if (diagonal + i * 32 + k * ROWS == b) v[k][b] += a.gamma;
        }
      if (i + 1 < T) fetch(i + 1);
    }
#pragma unroll
    for (int k = 0; k < TIMES; ++k) {
      half8 y[2];
#pragma unroll
      for (int b = 0; b < 8; ++b) two_parts(v[k][b], y, b);
#pragma unroll
      for (int part = 0; part < 2; ++part)
        *reinterpret_cast<half8 *>(d + (at + part * plane + (i * 32 + k * ROWS) * ld) + mine) = y[part];
    }
  }
}

template <int T, int SLOTS, bool E>
__global__ __launch_bounds__(256, T == 4 ? 1 : 2) void ns_product_kernel(NsArgs a) {
  using N = Ns<T, SLOTS>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[N::kLds];
  // the matrix and the tile
  uint32_t tile = xcd_tile(blockIdx.x, gridDim.x);
  const NsMat &t = a.mat[muon_mat_of(a.end, tile)];
  int64_t m0, n0;
  if (a.symmetric) {  // tile = I (I + 1) / 2 + J, J <= I
    uint32_t i = (uint32_t)((sqrtf(8.0f * (float)tile + 1.0f) - 1.0f) * 0.5f);
    while (i * (i + 1) / 2 > tile) --i;
    while ((i + 1) * (i + 2) / 2 <= tile) ++i;
    m0 = (int64_t)i * N::kTile;
    n0 = (int64_t)(tile - i * (i + 1) / 2) * N::kTile;
  } else {
    const uint32_t tiles_m = t.M / N::kTile, tiles_n = t.N / N::kTile;
    const uint32_t group = tile / (kGroupM * tiles_n), first_m = group * kGroupM;
    const uint32_t gm = tiles_m - first_m < kGroupM ? tiles_m - first_m : kGroupM;
    const uint32_t local = tile - group * kGroupM * tiles_n;
    m0 = (int64_t)(first_m + local % gm) * N::kTile;
    n0 = (int64_t)(local / gm) * N::kTile;
  }
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t wm = wave >> 1, wn = wave & 1, lr = lane & 31, h = lane >> 5;

  // transfers: every wave a quarter of a slot
  const int64_t ld = muon_ld(t.K);
  const uint8_t *base_p = reinterpret_cast<const uint8_t *>(t.p + m0 * ld), *base_q = reinterpret_cast<const uint8_t *>(t.q + n0 * ld);
  uint32_t off[N::kMoves];
#pragma unroll
  for (int i = 0; i < N::kMoves; ++i) {
    const uint32_t q = (wave * N::kMoves + i) * 64 + lane, row = q >> 3;
    off[i] = row * (uint32_t)(ld * 2) + ((q ^ (row >> 1)) & 7u) * 16u;
  }
  // fragments: lane half h takes chunk 2 s + h of its row in sub-step s; a wave's
  // blocks are 32 rows apart, so their permutations are one
  uint32_t at_p[4], at_q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t chunk = ((2 * k + h) ^ ((lr >> 1) & 7u)) * 16;
    at_p[k] = (wm * (32 * T) + lr) * 128 + chunk;
    at_q[k] = (wn * (32 * T) + lr) * 128 + chunk;
  }
  f32x16 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  // Each K-tile is taken three times: both first parts, P's first with Q's second,
  // P's second with Q's first (both second ones are 2^-22 of the first's).  Past the
  // end the last again, into slots that nobody reads.
  const uint32_t lds0 = lds_addr(lds), KT = 3u * (uint32_t)(t.K / 64), last = KT - 1;
  const uint64_t second_p = (uint64_t)t.M * ld * 2, second_q = (uint64_t)t.N * ld * 2;
  const auto from_p = [&](uint32_t kt) {
    const uint32_t k = kt < last ? kt : last;
    return base_p + (uint64_t)(k / 3u) * 128u + (k % 3u == 2u ? second_p : 0u);
  };
  const auto from_q = [&](uint32_t kt) {
    const uint32_t k = kt < last ? kt : last;
    return base_q + (uint64_t)(k / 3u) * 128u + (k % 3u == 1u ? second_q : 0u);
  };
  // transfer i of one operand's K-tile, which begins at `at`, into a slot
  const auto move = [&](const uint8_t *at, uint32_t slot, int i) {
    dma16(uniform_ptr(at), off[i], __builtin_amdgcn_readfirstlane(lds0 + slot * N::kSlotBytes + (wave * N::kMoves + i) * 1024u));
  };
  const auto after = [](uint32_t slot, uint32_t by) { return slot + by >= N::kSlots ? slot + by - N::kSlots : slot + by; };
#pragma unroll
  for (int u = 0; u < N::kSlots - 1; ++u)
#pragma unroll
    for (int i = 0; i < N::kMoves; ++i) move(u & 1 ? from_q(u / 2) : from_p(u / 2), u, i);
  NVFP4_WAIT_VMCNT((N::kSlots - 3) * N::kMoves);  // this wave's part of K-tile 0 is in LDS
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  NsFrags<T> f[4];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < T; ++i) {
      f[k].a[i] = *reinterpret_cast<const half8 *>(lds + at_p[k] + i * 4096);
      f[k].b[i] = *reinterpret_cast<const half8 *>(lds + N::kSlotBytes + at_q[k] + i * 4096);
    }
  // At the top of K-tile kt all slots but one, where Q's part of the K-tile before
  // was, are full or on their way: it gets P's part of K-tile kt + kSlots / 2.
  // Where P's part of this one is, Q's follows.
  uint32_t slot = 0;
  for (uint32_t kt = 0; kt < KT; ++kt) {
    const uint32_t slot_q = after(slot, 1), free_q = after(slot, N::kSlots - 1);
    const uint8_t *p = lds + slot * N::kSlotBytes, *q = lds + slot_q * N::kSlotBytes;
    const uint8_t *far_p = from_p(kt + N::kSlots / 2), *far_q = from_q(kt + N::kSlots / 2);
    multiply<T>(acc, f[0], f[2], p + at_p[2], q + at_q[2], [&](int i) { move(far_p, free_q, i); });
    multiply<T>(acc, f[1], f[3], p + at_p[3], q + at_q[3], [&](int i) { move(far_p, free_q, T + i); });
    NVFP4_WAIT_LGKM0();                             // this wave's reads of the two slots are complete
    NVFP4_WAIT_VMCNT((N::kSlots - 4) * N::kMoves);  // its part of K-tile kt + 1 is in LDS
    __builtin_amdgcn_s_barrier();                   // every wave's: K-tile kt + 1 is there, these slots are free
    asm volatile("" ::: "memory");
    const uint32_t next = after(slot, 2), next_q = after(slot, 3);
    p = lds + next * N::kSlotBytes;  // after the last K-tile: what is read is not used
    q = lds + next_q * N::kSlotBytes;
    multiply<T>(acc, f[2], f[0], p + at_p[0], q + at_q[0], [&](int i) { move(far_q, slot, i); });
    multiply<T>(acc, f[3], f[1], p + at_p[1], q + at_q[1], [&](int i) { move(far_q, slot, T + i); });
    slot = next;
  }
  NVFP4_WAIT_VMCNT(0);
  __syncthreads();  // no wave reads the slots, and no transfer writes them, any more

  float *slab = reinterpret_cast<float *>(lds) + wave * N::kSlab;
  const int64_t mw = m0 + wm * (32 * T), nw = n0 + wn * (32 * T);
  if (t.d)
    store_rows<T, E>(a, t.d, t.e, t.M * muon_ld(t.N), muon_ld(t.N), mw, nw, slab, lane, [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) slab[((r >> 2) * 8 + h * 4 + (r & 3)) * N::kStride + j * 32 + lr] = acc[i][j][r];
    });
  if (t.dt && !(a.symmetric && m0 == n0))
    store_rows<T, E>(a, t.dt, t.e, t.N * muon_ld(t.M), muon_ld(t.M), nw, mw, slab, lane, [&](int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<f32x4 *>(&slab[lr * N::kStride + i * 32 + q * 8 + h * 4]) =
              (f32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    });
}

// ---------------------------------------------------------- elementwise ----
// up to 8 elements from p, zero past `n`
template <typename T>
__device__ __forceinline__ void load_some(const T *p, int64_t n, float v[8]) {
  if (n >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? load1(p + j) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store_some(T *p, int64_t n, const float v[8]) {
  if (n >= 8) {
    store8(p, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) store1(p + j, v[j]);
  }
}
__device__ __forceinline__ void load_grad(const MuonMat &t, int64_t i, int64_t n, float scale, float g[8]) {
  if (t.flags & MF_GRAD_BF16)
    load_some((const uint16_t *)t.grad + i, n, g);
  else
    load_some((const float *)t.grad + i, n, g);
#pragma unroll
  for (int j = 0; j < 8; ++j) g[j] *= scale;
}
// the update's direction from the gradient and the new momentum
__device__ __forceinline__ float direction(const MuonArgs &a, float g, float m) {
  return a.nesterov ? fmaf(a.beta, m, a.one_minus_beta * g) : m;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// the new momentum, and the sum of squares of the direction by workgroup
__global__ __launch_bounds__(256) void muon_sums_kernel(MuonArgs a) {
  uint32_t group = blockIdx.x;
  const MuonMat &t = a.mat[muon_mat_of(a.end, group)];
  const int64_t n = (int64_t)t.rows * t.cols;
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  double sum = 0.0;
  for (int64_t i = ((int64_t)group * 256 + threadIdx.x) * 8; i < n; i += (int64_t)t.sums * 2048) {
    float g[8];
    load_grad(t, i, n - i, scale, g);
    if (t.m) {
      float m[8];
      load_some(t.m + i, n - i, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = fmaf(a.beta, m[j], a.one_minus_beta * g[j]);
        g[j] = direction(a, g[j], m[j]);
      }
      store_some(t.m + i, n - i, m);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fma((double)g[j], (double)g[j], sum);
  }
  __shared__ double sums[4];
  sum = wave_sum64(sum);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) t.parts[group] = sums[0] + sums[1] + sums[2] + sums[3];
}

// X and its transpose in two parts, 64 x 64 elements to a workgroup, zeros beyond the tensor
__global__ __launch_bounds__(256) void muon_form_kernel(MuonArgs a) {
  uint32_t group = blockIdx.x;
  const MuonMat &t = a.mat[muon_mat_of(a.end, group)];
  __shared__ double sums[4];
  __shared__ __attribute__((aligned(16))) _Float16 tile[2][64][72];
  double sum = 0.0;
  for (uint32_t i = threadIdx.x; i < t.sums; i += 256) sum += t.parts[i];
  sum = wave_sum64(sum);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = sums[0] + sums[1] + sums[2] + sums[3];
  const double by = sum > 0.0 ? (double)kMuonX / sqrt(sum) : 0.0;
  const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
  const uint32_t across = t.cp / 64;
  const int r0 = (int)(group / across) * 64, c0 = (int)(group % across) * 64;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (threadIdx.x >> 3) + 32 * k, c = (threadIdx.x & 7) * 8;
    const int n = r0 + r < t.rows ? t.cols - (c0 + c) : 0;
    const int64_t i = (int64_t)(r0 + r) * t.cols + c0 + c;
    half8 x[2] = {(half8)(_Float16)0.0f, (half8)(_Float16)0.0f};
    if (n > 0) {
      float g[8], m[8];
      if (t.m) {
        load_some(t.m + i, n, m);
        if (a.nesterov) load_grad(t, i, n, scale, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = direction(a, g[j], m[j]);
      } else {
        load_grad(t, i, n, scale, g);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) two_parts((float)((double)g[j] * by), x, j);
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      *reinterpret_cast<half8 *>(t.direct + (part * t.rp + r0 + r) * muon_ld(t.cp) + c0 + c) = x[part];
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[part][c + j][r] = x[part][j];
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (threadIdx.x >> 3) + 32 * k, c = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int part = 0; part < 2; ++part)
      *reinterpret_cast<half8 *>(t.turned + (part * t.cp + c0 + r) * muon_ld(t.rp) + r0 + c) =
          *reinterpret_cast<const half8 *>(&tile[part][r][c]);
  }
}

// what the last product left, as update and applied to the parameter
__global__ __launch_bounds__(256) void muon_update_kernel(MuonArgs a) {
  uint32_t group = blockIdx.x;
  const MuonMat &t = a.mat[muon_mat_of(a.end, group)];
  const int64_t n = (int64_t)t.rows * t.cols, start = (int64_t)group * kMuonChunk;
  const int64_t row0 = start / t.cols, plane = t.rp * muon_ld(t.cp);
  const uint32_t col0 = (uint32_t)(start - row0 * t.cols);
  uint32_t top = 0;
#pragma unroll 2
  for (uint32_t o = threadIdx.x * 8; o < kMuonChunk; o += 2048) {
    const int64_t i = start + o;
    if (i >= n) break;
    const uint32_t down = (col0 + o) / (uint32_t)t.cols;
    uint32_t c = col0 + o - down * t.cols;
    const _Float16 *x = t.direct + (row0 + down) * muon_ld(t.cp);
    float u[8];
    if (c + 8 <= (uint32_t)t.cols) {
      typedef half8 __attribute__((aligned(2))) half8_at2;
      const half8 q = *reinterpret_cast<const half8_at2 *>(x + c), q2 = *reinterpret_cast<const half8_at2 *>(x + plane + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = ((float)q[j] + (float)q2[j]) * (1.0f / kMuonX);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = i + j < n ? ((float)x[c] + (float)x[plane + c]) * (1.0f / kMuonX) : 0.0f;
        if (++c == (uint32_t)t.cols) {
          c = 0;
          x += muon_ld(t.cp);
        }
      }
    }
    if (t.update) store_some(t.update + i, n - i, u);
    if (!t.param) continue;
    float p[8];
    if (t.flags & MF_PARAM_BF16)
      load_some((const uint16_t *)t.param + i, n - i, p);
    else
      load_some((const float *)t.param + i, n - i, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = fmaf(-t.step, u[j], p[j] * t.keep);
    if (t.flags & MF_PARAM_BF16) {
      if (a.sr) {
        uint32_t w[4] = {(uint32_t)(i >> 3), t.index, a.step_lo, a.tag};
        philox4x32_10(a.seed_lo, a.seed_hi, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __uint_as_float((__float_as_uint(p[j]) + u16_of(w, j)) & 0xFFFF0000u);
      }
      store_some((uint16_t *)t.param + i, n - i, p);
    } else {
      store_some((float *)t.param + i, n - i, p);
    }
    if (t.copy) store_some(t.copy + i, n - i, p);
    if (t.amax) {
      const bool rounds = t.copy || (t.flags & MF_PARAM_BF16);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n - i) top = max(top, __float_as_uint(rounds ? round_bf16(p[j]) : p[j]) & 0x7FFFFFFFu);
    }
  }
  if (t.amax) {
    unsigned int *const out[1] = {reinterpret_cast<unsigned int *>(t.amax)};
    const uint32_t bits[1] = {top};
    raise_maxima<1>(out, bits);
  }
}

}  // namespace

namespace {

template <typename Args, typename Count>
uint32_t fill_ends(Args &a, Count count) {
  uint32_t end = 0;
  for (int i = 0; i < kMuonMats; ++i) a.end[i] = i < a.count ? end += count(a.mat[i]) : ~0u;
  return end;
}
template <int T, int SLOTS>
void launch_product(const NsArgs &a, uint32_t n, hipStream_t s) {
  if (a.mat[0].e)
    hipLaunchKernelGGL((ns_product_kernel<T, SLOTS, true>), dim3(n), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((ns_product_kernel<T, SLOTS, false>), dim3(n), dim3(256), 0, s, a);
}
uint32_t chunks(const MuonMat &t) { return (uint32_t)(((int64_t)t.rows * t.cols + kMuonChunk - 1) / kMuonChunk); }

}  // namespace

hipError_t launch_muon_sums(MuonArgs &a, hipStream_t s) {
  const uint32_t n = fill_ends(a, [](MuonMat &t) { return t.sums = chunks(t) < kMuonParts ? chunks(t) : kMuonParts; });
  hipLaunchKernelGGL(muon_sums_kernel, dim3(n), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_muon_form(MuonArgs &a, hipStream_t s) {
  const uint32_t n = fill_ends(a, [](const MuonMat &t) { return (uint32_t)(t.rp / 64) * (uint32_t)(t.cp / 64); });
  hipLaunchKernelGGL(muon_form_kernel, dim3(n), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_muon_update(MuonArgs &a, hipStream_t s) {
  const uint32_t n = fill_ends(a, [](const MuonMat &t) { return chunks(t); });
  hipLaunchKernelGGL(muon_update_kernel, dim3(n), dim3(256), 0, s, a);
  return hipGetLastError();
}
hipError_t launch_muon_product(NsArgs &a, int tile, hipStream_t s) {
  const uint32_t n = fill_ends(a, [&](const NsMat &t) {
    const uint32_t down = t.M / tile, across = t.N / tile;
    return a.symmetric ? down * (down + 1) / 2 : down * across;
  });
  // Tiles of 128 that are no more than the compute units have all of LDS for
  // transfers ahead, more share it by twos: 2048 x 2048 takes 54 and 56 us for the 136
  // tiles of a square, 7 matrices of 1024 x 1152 61 and 54 for the 504 of the last product.
  // Tiles of 64 likewise, by twos and fours.
  if (tile == 256)
    launch_product<4, 5>(a, n, s);
  else if (tile == 128 && n > 256)
    launch_product<2, 5>(a, n, s);
  else if (tile == 128)
    launch_product<2, 9>(a, n, s);
  else if (n > 512)
    launch_product<1, 5>(a, n, s);
  else
    launch_product<1, 9>(a, n, s);
  return hipGetLastError();
}

}  // namespace nvfp4
