// The gated feed-forward products on 4-bit operands and their gradient
// (include/nvfp4.h: nvfp4_gemm_gated, nvfp4_gemm_gated_backward).
//
// Forward, a workgroup's tile is 256 rows by 128 columns of both products: its B
// rows are, for each of the two wave columns, 64 of the gate's weights and the 64
// of the up projection's that belong to them.  A lane then holds gate and up of
// the same elements in its accumulators, and the epilogue forms act(gate) * up
// without either leaving the registers.  Backward, dh is a plain product whose
// epilogue reads gate and up and writes their gradients; dh itself is not stored.
// The pipeline is the plain GEMM's (gemm_tile.hpp); rows past M or N repeat the
// last one and are not stored, so that only K has to fill its tiles there.
//
// Large calls are bound by the matrix instructions at the power the chip holds:
// 16384 tokens, 5120 -> 2 x 20480 with h, gate and up stored, 4.87 to 5.14 ms (1.34 to
// 1.41 PFLOP/s; the same products by themselves 1.27 at 5120 x 5120 x 8192, a
// library's bf16 product of 8192^3 1.55), their gradient 2.7 to 2.8 ms (1.22 to 1.27: its
// epilogue moves 2.7 GB).  16 tokens are bound by reading the weights: 106 MB in 24
// to 39 us.  What fills few tiles (1008 x 2736 x 1040: 27 us, gradient 20) by a
// compute unit's way through K, 1.2 us a workgroup and K-tile of 128, behind a launch.
#include "block_device.hpp"
#include "block_kernels.hpp"
#include "gemm_tile.hpp"

namespace nvfp4 {
namespace {

// e^x and 1 / x as the hardware has them, within some 2^-22: their results are
// rounded to bf16
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.442695041f); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-x)); }

constexpr float kTanhScale = 1.595769122f;  // 2 sqrt(2 / pi): (1 + tanh(z)) / 2 = sigmoid(2 z)
constexpr float kCubic = 0.044715f;

// P(N > -x) for a normal N, with e = e^(-x^2 / 2): by symmetry from the upper tail at
// a = |x|, which is e t poly(t) with t = 1 / (1 + 0.33 a).  The polynomial is a fit to
// the tail's quotient by e t (over all a, of the relative error): within 2^-19 of the
// tail up to a = 4, 2^-18 up to 8, where the exponent's rounding grows.  With the
// library's erfcf, whose ranges a wave takes one after another, 1008 x 2736 x 1040 took 31
// us for 27, its gradient 24 for 19, that of 16384 tokens, 5120 -> 20480, 3.14 ms for 2.78.
__device__ __forceinline__ float normal_cdf(float x, float &e) {
  const float a = fabsf(x), t = __builtin_amdgcn_rcpf(fmaf(0.33f, a, 1.0f));
  e = __builtin_amdgcn_exp2f(-0.7213475204f * a * a);
  float r = fmaf(t, 0.0332857408f, -0.105665021f);
  r = fmaf(r, t, 0.0674313828f);
  r = fmaf(r, t, 0.0334286168f);
  r = fmaf(r, t, 0.0910049751f);
  r = fmaf(r, t, 0.117216729f);
  r = fmaf(r, t, 0.131646991f);
  r = fmaf(r, t, 0.131651074f);
  const float tail = e * (t * r);
  return x > 0.0f ? 1.0f - tail : tail;
}

// the activation of x, and its derivative
template <int ACT>
__device__ __forceinline__ float act(float x) {
  if (ACT == NVFP4_SILU) return x * sigmoid(x);
  if (ACT == NVFP4_RELU) return x <= 0.0f ? 0.0f : x;  // (a NaN stays one)
  if (ACT == NVFP4_GELU) {
    float e;
    return x * normal_cdf(x, e);
  }
  return x * sigmoid(kTanhScale * x * fmaf(kCubic * x, x, 1.0f));
}
template <int ACT>
__device__ __forceinline__ void act_grad(float x, float &f, float &df) {
  if (ACT == NVFP4_SILU) {
    const float p = sigmoid(x);
    f = x * p;
    df = p * fmaf(x, 1.0f - p, 1.0f);
  } else if (ACT == NVFP4_RELU) {
    f = x <= 0.0f ? 0.0f : x;
    df = x > 0.0f ? 1.0f : 0.0f;
  } else if (ACT == NVFP4_GELU) {
    float e;
    const float p = normal_cdf(x, e);
    f = x * p;
    df = fmaf(x * 0.3989422804f, e, p);
  } else {
    const float p = sigmoid(kTanhScale * x * fmaf(kCubic * x, x, 1.0f));
    const float y = fminf(fmaxf(x, -64.0f), 64.0f);  // beyond, p (1 - p) is zero
    f = x * p;
    df = fmaf(p * (1.0f - p) * y, kTanhScale * fmaf(3.0f * kCubic * y, y, 1.0f), p);
  }
}

// the same for an activation that is known only at run time
__device__ __forceinline__ float act_of(int kind, float x) {
  return kind == NVFP4_SILU ? act<NVFP4_SILU>(x) : kind == NVFP4_GELU ? act<NVFP4_GELU>(x) : kind == NVFP4_RELU ? act<NVFP4_RELU>(x)
                                                                                                               : act<NVFP4_GELU_TANH>(x);
}
__device__ __forceinline__ void act_grad_of(int kind, float x, float &f, float &df) {
  if (kind == NVFP4_SILU)
    act_grad<NVFP4_SILU>(x, f, df);
  else if (kind == NVFP4_GELU)
    act_grad<NVFP4_GELU>(x, f, df);
  else if (kind == NVFP4_RELU)
    act_grad<NVFP4_RELU>(x, f, df);
  else
    act_grad<NVFP4_GELU_TANH>(x, f, df);
}

// A's rows m0 onwards, and TN * 16 rows of the gate's and of the up projection's
// weights to each of the two wave columns
template <int TN>
struct GatedRows {
  const GatedArgs &a;
  int64_t m0, n0;
  static constexpr bool kTwo = true;
  __device__ __forceinline__ int64_t K() const { return a.g.K; }
  template <int A_ROWS>
  __device__ __forceinline__ RowRef ref(int r) const {
    if (r < A_ROWS) return {a.g.a_codes, a.g.a_scales, a.g.a_kind, m0 + r, a.g.M};
    const int b = r - A_ROWS, in = b % (TN * 32);
    const bool up = in >= TN * 16;
    return {up ? a.u_codes : a.g.b_codes, up ? a.u_scales : a.g.b_scales, up ? a.u_kind : a.g.b_kind,
            n0 + b / (TN * 32) * (TN * 16) + in % (TN * 16), a.g.N};
  }
  __device__ __forceinline__ const uint8_t *codes(uint32_t wave, bool second) const {
    return wave < 2 ? a.g.a_codes : second ? a.u_codes : a.g.b_codes;
  }
  __device__ __forceinline__ const uint8_t *scales(uint32_t wave, bool second) const {
    return wave < 2 ? a.g.a_scales : second ? a.u_scales : a.g.b_scales;
  }
  __device__ __forceinline__ uint32_t row(uint32_t r) const {
    const int64_t m = m0 + r, n = n0 + ((r >> 7) & 1u) * 64 + (r & 63u);
    return (uint32_t)(r < 256 ? (m < a.g.M ? m : a.g.M - 1) : (n < a.g.N ? n : a.g.N - 1));
  }
  __device__ __forceinline__ int kind(uint32_t r) const { return r < 256 ? a.g.a_kind : (r & 64u) ? a.u_kind : a.g.b_kind; }
};
// the plain rows, those past the end as the last one
struct EndedRows : PlainRows {
  __device__ __forceinline__ uint32_t row(uint32_t r) const {
    const int64_t m = m0 + r, n = n0 + (r - 256);
    return (uint32_t)(r < 256 ? (m < g.M ? m : g.M - 1) : (n < g.N ? n : g.N - 1));
  }
};

__device__ __forceinline__ EpiScale scale_of(const float *a_S, const float *b_S) {
  GemmArgs g;
  g.a_S = a_S;
  g.b_S = b_S;
  return epi_scale(g);
}

// The epilogue of a tile with TM x TN blocks of 32 x 32 to a wave: block row by
// block row, the accumulators go through a slab of LDS of the wave's own, from
// which a lane takes 8 neighbouring columns of a row, so that loads and stores
// are of 16 bytes, and the loop over rows is short code.  A slab's rows are 32
// banks apart every 4, as the accumulators' lane halves write them.
// What lies past M or N is zero in the maxima.
template <int TN>
struct Slab {
  static constexpr int kStride = 32 * TN + 8;  // floats between rows
  static constexpr int kFloats = 32 * kStride; // of a wave
};

// a slab is read as another type than it was written as, by other lanes of the
// wave: the wave's accesses to LDS keep their order, the compiler has to, too
__device__ __forceinline__ void slab_fence() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void store_past_caches(uint16_t *p, const u32x4 &v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(p));
}
__device__ __forceinline__ uint32_t top_of(uint32_t top, const u32x4 &v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7FFFu, v[k] >> 16 & 0x7FFFu));
  return top;
}
// the maximum of 32 x 32 rounded values and of their transform, a column to a lane
__device__ __forceinline__ void slab_max(FusedMax &f, const GemmArgs &o, const uint16_t *at, int stride, uint32_t lane) {
  uint32_t hb[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) hb[r] = at[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * stride + (lane & 31)];
  fused_max_block(f, o, hb);
}

template <int ACT, int TM, int TN>
__device__ __forceinline__ void gated_store(const GatedArgs &a, int64_t m0, int64_t n0, const float16v acc[TM][TN], float *lds) {
  constexpr int S = Slab<TN>::kStride, LANES = 2 * TN, ROWS = 64 / LANES;  // lanes of a row, rows at a time
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float *slab = lds + wave * Slab<TN>::kFloats;
  const EpiScale eg = scale_of(a.g.a_S, a.g.b_S), eu = scale_of(a.g.a_S, a.u_S);
  GemmArgs o = a.g;
  o.amax_plain = a.amax[0];
  o.amax_rht = a.rht[0];
  FusedMax fm;
  fused_max_init(fm, o, lane);
  const int c = lane % LANES * 8, first = lane / LANES;
  const int64_t n = n0 + (wave & 1) * (TN * 16) + c;
  const int64_t m = m0 + (wave >> 1) * (TM * 32);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        slab[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * S + j * 32 + (lane & 31)] = acc[i][j][r];
    slab_fence();
#pragma unroll 2
    for (int r = first; r < 32; r += ROWS) {
      const int64_t row = m + i * 32 + r;
      float g[8], u[8], h[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[k] = epi_apply(slab[r * S + c + k], eg);
        u[k] = epi_apply(slab[r * S + TN * 16 + c + k], eu);
        h[k] = act<ACT>(g[k]) * u[k];
      }
      u32x4 hb = packed8(h);
      if (row < a.g.M && n < a.g.N) {
        store_past_caches(a.h + row * a.ld_h + n, hb);
        if (a.gate) store_past_caches(a.gate + row * a.ld_gate + n, packed8(g));
        if (a.up) store_past_caches(a.up + row * a.ld_up + n, packed8(u));
      } else {
        hb = (u32x4){0, 0, 0, 0};
      }
      fm.plain = top_of(fm.plain, hb);
      if (o.amax_rht) *reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(slab + r * S) + c) = hb;
    }
    slab_fence();
    if (o.amax_rht) {
#pragma unroll
      for (int j = 0; j < TN / 2; ++j) slab_max(fm, o, reinterpret_cast<const uint16_t *>(slab) + j * 32, 2 * S, lane);
      slab_fence();
    }
  }
  if (o.amax_plain || o.amax_rht) {
    unsigned int *const out[2] = {a.amax[0], a.rht[0]};
    const uint32_t bits[2] = {fm.plain << 16, __float_as_uint(fm.rht * 0.25f)};
    raise_maxima<2>(out, bits);
  }
}

template <int ACT, int TM, int TN>
__device__ __forceinline__ void grad_store(const GatedArgs &a, int64_t m0, int64_t n0, const float16v acc[TM][TN], float *lds) {
  constexpr int S = Slab<TN>::kStride, LANES = 4 * TN, ROWS = 64 / LANES;
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float *slab = lds + wave * Slab<TN>::kFloats;
  const EpiScale es = scale_of(a.g.a_S, a.g.b_S);
  GemmArgs o[2] = {a.g, a.g};
  FusedMax fm[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    o[k].amax_plain = a.amax[k];
    o[k].amax_rht = a.rht[k];
    fused_max_init(fm[k], o[k], lane);
  }
  const bool rht = a.rht[0] || a.rht[1];
  const int c = lane % LANES * 8, first = lane / LANES;
  const int64_t n = n0 + (wave & 1) * (TN * 32) + c;
  const int64_t m = m0 + (wave >> 1) * (TM * 32);
  // gate and up are read four rows of a lane ahead: one after another, 5120 x 20480
  // outputs of 16384 rows took 3.15 ms instead of 2.71
  constexpr int AT_ONCE = 4, PARTS = 32 / (ROWS * AT_ONCE);
  uint4 gate[AT_ONCE], up[AT_ONCE];
  const auto fetch = [&](int part) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int64_t row = m + (part * AT_ONCE + k) * ROWS + first;
      gate[k] = up[k] = make_uint4(0, 0, 0, 0);
      if (row < a.g.M && n < a.g.N) {
        gate[k] = load_group(a.gate + row * a.ld_gate + n);
        up[k] = load_group(a.up + row * a.ld_up + n);
      }
    }
  };
  fetch(0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        slab[((r >> 2) * 8 + (lane >> 5) * 4 + (r & 3)) * S + j * 32 + (lane & 31)] = acc[i][j][r];
    slab_fence();
#pragma unroll 1
    for (int part = 0; part < PARTS; ++part) {
      uint4 g[AT_ONCE], u[AT_ONCE];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        g[k] = gate[k];
        u[k] = up[k];
      }
      if (i * PARTS + part + 1 < TM * PARTS) fetch(i * PARTS + part + 1);
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k) {
        const int r = (part * AT_ONCE + k) * ROWS + first;
        const int64_t row = m + i * 32 + r;
        const bool here = row < a.g.M && n < a.g.N;
        float dg[8], du[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dh = epi_apply(slab[r * S + c + e], es);
          float f, df;
          act_grad<ACT>(bf16_at(g[k], e), f, df);
          dg[e] = dh * bf16_at(u[k], e) * df;
          du[e] = dh * f;
        }
        u32x4 gb = packed8(dg), ub = packed8(du);
        if (here) {
          store_past_caches(a.dgate + row * a.ld_dgate + n, gb);
          store_past_caches(a.dup + row * a.ld_dup + n, ub);
        } else {
          gb = ub = (u32x4){0, 0, 0, 0};
        }
        fm[0].plain = top_of(fm[0].plain, gb);
        fm[1].plain = top_of(fm[1].plain, ub);
        if (rht) {
          uint16_t *at = reinterpret_cast<uint16_t *>(slab + r * S) + c;
          *reinterpret_cast<u32x4 *>(at) = gb;
          *reinterpret_cast<u32x4 *>(at + TN * 32) = ub;
        }
      }
    }
    slab_fence();
    if (rht) {
#pragma unroll
      for (int j = 0; j < 2 * TN; ++j)
        slab_max(fm[j / TN], o[j / TN], reinterpret_cast<const uint16_t *>(slab) + j * 32, 2 * S, lane);
      slab_fence();
    }
  }
  if (a.amax[0] || a.amax[1] || rht) {
    unsigned int *const out[4] = {a.amax[0], a.rht[0], a.amax[1], a.rht[1]};
    const uint32_t bits[4] = {fm[0].plain << 16, __float_as_uint(fm[0].rht * 0.25f), fm[1].plain << 16, __float_as_uint(fm[1].rht * 0.25f)};
    raise_maxima<4>(out, bits);
  }
}

// lds: as many floats as the four waves' slabs, which no wave reads any more
template <bool BACK, int TM, int TN>
__device__ __forceinline__ void store_tile(const GatedArgs &a, int64_t m0, int64_t n0, const float16v acc[TM][TN], float *lds) {
#define NVFP4_STORE(ACT)                              \
  case ACT:                                           \
    if (BACK)                                         \
      grad_store<ACT, TM, TN>(a, m0, n0, acc, lds);   \
    else                                              \
      gated_store<ACT, TM, TN>(a, m0, n0, acc, lds);  \
    break;
  switch (a.activation) {
    NVFP4_STORE(NVFP4_SILU)
    NVFP4_STORE(NVFP4_GELU)
    NVFP4_STORE(NVFP4_GELU_TANH)
    NVFP4_STORE(NVFP4_RELU)
  }
#undef NVFP4_STORE
}

// origin of a workgroup's tile of BM x BN outputs: as tile_origin, but for a last
// row and column of tiles that need not be whole
template <int BM, int BN>
__device__ __forceinline__ void origin(const GatedArgs &a, uint32_t tile, int64_t &m0, int64_t &n0) {
  const uint32_t tiles_m = (uint32_t)((a.g.M + BM - 1) / BM), tiles_n = (uint32_t)((a.g.N + BN - 1) / BN);
  const uint32_t group = tile / (kGroupM * tiles_n), first_m = group * kGroupM;
  const uint32_t gm = tiles_m - first_m < kGroupM ? tiles_m - first_m : kGroupM;
  const uint32_t local = tile - group * kGroupM * tiles_n;
  m0 = (int64_t)(first_m + local % gm) * BM;
  n0 = (int64_t)(local / gm) * BN;
}

// Tiles of 256 x 256 products (256 x 128 columns of both weights): one workgroup to
// a compute unit, 64 KiB of accumulators to a wave; 1.2 to 1.4 PFLOP/s.
template <bool BACK>
__global__ __launch_bounds__(kGThreads) void gated_fast_kernel(GatedArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFStages * kFStageBytes];
  int64_t m0, n0;
  origin<256, BACK ? 256 : 128>(a, xcd_tile(blockIdx.x, gridDim.x), m0, n0);
  float16v acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  if constexpr (BACK)
    fast_tile(EndedRows{a.g, m0, n0}, 0, (uint32_t)(a.g.K / kFBK), acc, lds);
  else
    fast_tile(GatedRows<4>{a, m0, n0}, 0, (uint32_t)(a.g.K / kFBK), acc, lds);
  __syncthreads();  // no wave reads the stages any more
  store_tile<BACK, 4, 4>(a, m0, n0, acc, reinterpret_cast<float *>(lds));
}

// Any K, and what fits no 32-bit offset: tiles of 64 T + 64 T operand rows and
// K-tiles of 128, through registers three K-tiles ahead, in the LDS layout of the fast
// path (codes in chunks permuted by row, then two scale dwords of each row).  Two
// workgroups to a compute unit, whose waits overlap: 1008 x 2736 x 1040 has 344 tiles
// forward and takes 26 us (with operands expanded to fp16 in LDS, shared by the waves,
// 1008 x 2736 x 4112 took 77 us for 70).
// Rows past the end repeat the last one.  A K that is no multiple of 128 ends in
// a K-tile of zeros beyond it: only that one is loaded piece by piece.
typedef uint4 __attribute__((aligned(8))) uint4_at8;
typedef uint2 __attribute__((aligned(1))) uint2_at1;

template <int T>
struct Ragged {
  static constexpr int kRows = 128 * T;
  static constexpr int kCodes = kRows * 4 / kGThreads;   // 16-byte chunks of a thread
  static constexpr int kScales = kRows / kGThreads;      // rows whose scales a thread loads
  static constexpr int kBytes = kRows * 72;              // of a stage
  struct Held {  // a thread's part of a K-tile
    uint4 code[kCodes];
    uint2 scale[kScales];
  };
  const uint8_t *code_at[kCodes], *scale_at[kScales];

  template <typename Rows>
  __device__ __forceinline__ explicit Ragged(const Rows &src) {
    const int64_t pitch = src.K() / 2, kblocks = src.K() / 16;
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int c = threadIdx.x + i * kGThreads;
      const RowRef r = src.template ref<64 * T>(c >> 2);
      code_at[i] = r.codes + (r.row < r.rows ? r.row : r.rows - 1) * pitch + (c & 3) * 16;
    }
#pragma unroll
    for (int i = 0; i < kScales; ++i) {
      const RowRef r = src.template ref<64 * T>(threadIdx.x + i * kGThreads);
      const int64_t row = r.row < r.rows ? r.row : r.rows - 1;
      scale_at[i] = r.scales + (r.kind == 0 ? row : row / 16) * kblocks;
    }
  }
  __device__ __forceinline__ void load(Held &d, int64_t kt) const {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) d.code[i] = *reinterpret_cast<const uint4_at8 *>(code_at[i] + kt * 64);
#pragma unroll
    for (int i = 0; i < kScales; ++i) d.scale[i] = *reinterpret_cast<const uint2_at1 *>(scale_at[i] + kt * 8);
  }
  // the last K-tile, of which `blocks` < 8 blocks of 16 k are there
  __device__ __forceinline__ void load_end(Held &d, int64_t kt, int blocks) const {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const uint8_t *p = code_at[i] + kt * 64;
      const int left = blocks - 2 * (int)((threadIdx.x + i * kGThreads) & 3);
      const uint2 lo = left > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
      const uint2 hi = left > 1 ? *reinterpret_cast<const uint2 *>(p + 8) : make_uint2(0u, 0u);
      d.code[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
#pragma unroll
    for (int i = 0; i < kScales; ++i) {
      const uint8_t *p = scale_at[i] + kt * 8;
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int b = 0; b < 8; ++b)
        if (b < blocks) w[b >> 2] |= (uint32_t)p[b] << (8 * (b & 3));
      d.scale[i] = make_uint2(w[0], w[1]);
    }
  }
  static __device__ __forceinline__ void store(uint8_t *stage, const Held &d) {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const uint32_t c = threadIdx.x + i * kGThreads, row = c >> 2;
      *reinterpret_cast<uint4 *>(stage + (row * 4 + ((c & 3u) ^ swz(row))) * 16) = d.code[i];
    }
#pragma unroll
    for (int i = 0; i < kScales; ++i) {
      const uint32_t row = threadIdx.x + i * kGThreads;
      uint32_t *p = reinterpret_cast<uint32_t *>(stage + kRows * 64 + row * 8);
      p[(row >> 4) & 1u] = d.scale[i].x;
      p[((row >> 4) & 1u) ^ 1u] = d.scale[i].y;
    }
  }
};

template <bool BACK, int T>
__global__ __launch_bounds__(kGThreads, 2) void gated_generic_kernel(GatedArgs a) {
  using S = Ragged<T>;
  constexpr int kSlabs = kGThreads / 64 * Slab<T>::kFloats * 4;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * S::kBytes > kSlabs ? 2 * S::kBytes : kSlabs];
  int64_t m0, n0;
  origin<64 * T, BACK ? 64 * T : 32 * T>(a, xcd_tile(blockIdx.x, gridDim.x), m0, n0);
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t wm = wave >> 1, wn = wave & 1, lr = lane & 31, h = lane >> 5;
  float16v acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const S src = [&] {
    if constexpr (BACK)
      return S(PlainRows{a.g, m0, n0});
    else
      return S(GatedRows<T>{a, m0, n0});
  }();
  const int64_t kblocks = a.g.K / 16, KT = (kblocks + 7) / 8, whole = kblocks / 8;
  const auto load = [&](typename S::Held &d, int64_t kt) {
    if (kt < whole)
      src.load(d, kt);
    else if (kt < KT)
      src.load_end(d, kt, (int)(kblocks & 7));
  };
  typename S::Held held[3];  // K-tiles kt + 1 .. kt + 3
  load(held[0], 0);
  S::store(lds, held[0]);
  load(held[0], 1);
  load(held[1], 2);
  load(held[2], 3);
  __syncthreads();
  const auto step = [&](int64_t kt, typename S::Held &next) {
    const uint8_t *stage = lds + (kt & 1) * S::kBytes;
    if (kt + 1 < KT) S::store(lds + (~kt & 1) * S::kBytes, next);  // read by no wave since the last barrier
    load(next, kt + 4);
    uint4 qa[T][2], qb[T][2];
    half2v sa[T][2], sb[T][2];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t ra = wm * (32 * T) + i * 32 + lr, rb = 64 * T + wn * (32 * T) + i * 32 + lr;
        qa[i][k] = *reinterpret_cast<const uint4 *>(stage + (ra * 4 + ((2 * h + k) ^ swz(ra))) * 16);
        qb[i][k] = *reinterpret_cast<const uint4 *>(stage + (rb * 4 + ((2 * h + k) ^ swz(rb))) * 16);
        const uint32_t wa = *reinterpret_cast<const uint32_t *>(stage + S::kRows * 64 + (ra * 2 + (h ^ ((ra >> 4) & 1u))) * 4);
        const uint32_t wb = *reinterpret_cast<const uint32_t *>(stage + S::kRows * 64 + (rb * 2 + (h ^ ((rb >> 4) & 1u))) * 4);
        sa[i][k] = k ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(wa, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(wa, 1.0f, false);
        sb[i][k] = k ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(wb, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(wb, 1.0f, false);
      }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int k = s >> 2, d = s & 3;
      half8v fa[T], fb[T];
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const uint4 &x = qa[i][k], &y = qb[i][k];
        fa[i] = expand8(d == 0 ? x.x : d == 1 ? x.y : d == 2 ? x.z : x.w, sa[i][k][d >> 1]);
        fb[i] = expand8(d == 0 ? y.x : d == 1 ? y.y : d == 2 ? y.z : y.w, sb[i][k][d >> 1]);
      }
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  };
  for (int64_t kt = 0; kt < KT; kt += 3) {
    step(kt, held[0]);
    if (kt + 1 < KT) step(kt + 1, held[1]);
    if (kt + 2 < KT) step(kt + 2, held[2]);
  }
  store_tile<BACK, T, T>(a, m0, n0, acc, reinterpret_cast<float *>(lds));
}

// Few rows: the weights are read once, and that is all that counts.  A workgroup
// takes 16 columns (forward: of both weights) and up to 16 MT rows; its four waves
// share K, each straight from memory to registers, and add up in LDS.  In a K-tile
// of 128, lane l holds row l % 16 of an operand and k = 32 (l / 16) + 8 s + [0, 8) in
// sub-step s, as 16 bytes of codes under two scales.
// codes and scales of a K-tile, and those of the last one, of which `left` blocks
// of 16 k are there from this lane's first on
__device__ __forceinline__ u32x4 skinny_codes(const uint8_t *p) { return *reinterpret_cast<const u32x4_at2 *>(p); }
__device__ __forceinline__ uint32_t skinny_scales(const uint8_t *p) {
  typedef uint16_t __attribute__((aligned(1))) uint16_at1;
  return *reinterpret_cast<const uint16_at1 *>(p);
}
__device__ __forceinline__ u32x4 skinny_codes_end(const uint8_t *p, int left) {
  const uint2 lo = left > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0u, 0u);
  const uint2 hi = left > 1 ? *reinterpret_cast<const uint2 *>(p + 8) : make_uint2(0u, 0u);
  return (u32x4){lo.x, lo.y, hi.x, hi.y};
}
__device__ __forceinline__ uint32_t skinny_scales_end(const uint8_t *p, int left) {
  return (left > 0 ? p[0] : 0u) | (left > 1 ? p[1] : 0u) << 8;
}

template <int MT, bool BACK>
__global__ __launch_bounds__(kGThreads) void gated_skinny_kernel(GatedArgs a) {
  constexpr int OPS = BACK ? 1 : 2, N = OPS + MT;
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t pitch = a.g.K / 2, kblocks = a.g.K / 16, KT = (kblocks + 7) / 8;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  // Four neighbouring lanes load a row's 64 bytes (with a row to a lane, as the
  // products want it, each lane's 16 bytes were an access of their own); LDS of
  // the wave's own turns that round.
  const uint32_t load_row = lane >> 2, load_part = lane & 3, row = lane & 15, part = lane >> 4;
  const uint8_t *codes[N], *scales[N];  // the weights', then those of MT times 16 rows
#pragma unroll
  for (int o = 0; o < OPS; ++o) {
    const int64_t n = n0 + load_row;
    const int kind = o ? a.u_kind : a.g.b_kind;
    codes[o] = (o ? a.u_codes : a.g.b_codes) + n * pitch + load_part * 16;
    scales[o] = (o ? a.u_scales : a.g.b_scales) + (kind == 0 ? n : n / 16) * kblocks + load_part * 2;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = i * 16 + load_row < a.g.M ? i * 16 + load_row : a.g.M - 1;
    codes[OPS + i] = a.g.a_codes + m * pitch + load_part * 16;
    scales[OPS + i] = a.g.a_scales + (a.g.a_kind == 0 ? m : m / 16) * kblocks + load_part * 2;
  }
  __shared__ u32x4 turn_q[4][N][64];
  __shared__ uint32_t turn_w[4][N][64];
  __shared__ float sums[4][OPS][16 * MT][17];
  __shared__ uint16_t done[2][16 * MT][16];
  // chunk `part` of row r stands at 4 r + (part ^ (r / 4 % 4)): reads of one part meet all banks
  const uint32_t put = load_row * 4 + (load_part ^ (load_row >> 2)), get = row * 4 + (part ^ (row >> 2));
  f32x4 acc[OPS][MT];
#pragma unroll
  for (int o = 0; o < OPS; ++o)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[o][i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  const auto work = [&]() __attribute__((always_inline)) {
    u32x4 q[N];
    half2v sc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = turn_q[wave][i][get];
      sc[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(turn_w[wave][i][get], 1.0f, false);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      half8v f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = expand8(s == 0 ? q[i].x : s == 1 ? q[i].y : s == 2 ? q[i].z : q[i].w, sc[i][s >> 1]);
#pragma unroll
      for (int o = 0; o < OPS; ++o)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[o][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f[OPS + i], f[o], acc[o][i], 0, 0, 0);
    }
  };
  // whole K-tiles two ahead (past the last one: it again, and not used)
  const int64_t whole = kblocks / 8, mine = whole > wave ? (whole - wave + 3) / 4 : 0;
  const auto at = [&](int64_t i) { return wave + 4 * (i < mine ? i : mine - 1); };
  u32x4 q0[N], q1[N];
  uint32_t w0[N], w1[N];
#define NVFP4_LOAD(q, w, kt)                     \
  _Pragma("unroll") for (int i = 0; i < N; ++i) { \
    q[i] = skinny_codes(codes[i] + (kt) * 64);    \
    w[i] = skinny_scales(scales[i] + (kt) * 8);   \
  }
#define NVFP4_TURN(q, w)                          \
  _Pragma("unroll") for (int i = 0; i < N; ++i) { \
    turn_q[wave][i][put] = q[i];                  \
    turn_w[wave][i][put] = w[i];                  \
  }
  if (mine > 0) {
    NVFP4_LOAD(q0, w0, at(0))
    NVFP4_LOAD(q1, w1, at(1))
  }
  for (int64_t k = 0; k < mine; k += 2) {
    NVFP4_TURN(q0, w0)
    NVFP4_LOAD(q0, w0, at(k + 2))
    work();
    if (k + 1 < mine) {
      NVFP4_TURN(q1, w1)
      NVFP4_LOAD(q1, w1, at(k + 3))
      work();
    }
  }
  if (whole < KT && whole % 4 == wave) {
    const int left = (int)(kblocks & 7) - 2 * (int)load_part;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      turn_q[wave][i][put] = skinny_codes_end(codes[i] + whole * 64, left);
      turn_w[wave][i][put] = skinny_scales_end(scales[i] + whole * 8, left);
    }
    work();
  }
#undef NVFP4_LOAD
#undef NVFP4_TURN
  // [wave][weight][row][column]: lane l holds rows 4 (l / 16) .. + 3 of column l % 16
#pragma unroll
  for (int o = 0; o < OPS; ++o)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][o][i * 16 + part * 4 + r][row] = acc[o][i][r];
  __syncthreads();
  const EpiScale es = scale_of(a.g.a_S, a.g.b_S), eu = scale_of(a.g.a_S, BACK ? a.g.b_S : a.u_S);
  uint32_t top[2] = {0, 0};
  for (int e = threadIdx.x; e < 256 * MT; e += kGThreads) {
    const int r = e >> 4, c = e & 15;
    const int64_t m = r, n = n0 + c;
    const auto total = [&](int o) { return sums[0][o][r][c] + sums[1][o][r][c] + sums[2][o][r][c] + sums[3][o][r][c]; };
    uint32_t out[2] = {0, 0};
    if (m < a.g.M) {
      if constexpr (BACK) {
        const float dh = epi_apply(total(0), es), g = bf16_lo(a.gate[m * a.ld_gate + n]), u = bf16_lo(a.up[m * a.ld_up + n]);
        float f, df;
        act_grad_of(a.activation, g, f, df);
        out[0] = bf16_rne_bits(dh * u * df);
        out[1] = bf16_rne_bits(dh * f);
        a.dgate[m * a.ld_dgate + n] = (uint16_t)out[0];
        a.dup[m * a.ld_dup + n] = (uint16_t)out[1];
      } else {
        const float g = epi_apply(total(0), es), u = epi_apply(total(OPS - 1), eu);
        out[0] = bf16_rne_bits(act_of(a.activation, g) * u);
        a.h[m * a.ld_h + n] = (uint16_t)out[0];
        if (a.gate) a.gate[m * a.ld_gate + n] = (uint16_t)bf16_rne_bits(g);
        if (a.up) a.up[m * a.ld_up + n] = (uint16_t)bf16_rne_bits(u);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      top[k] = max(top[k], out[k] & 0x7FFFu);
      if (a.rht[k]) done[k][r][c] = (uint16_t)out[k];
    }
  }
  float most[2] = {0.0f, 0.0f};
  if (a.rht[0] || a.rht[1]) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!a.rht[k] || threadIdx.x >= 16 * MT) continue;  // a column of 16 rows to a thread
      const int g = threadIdx.x >> 4, c = threadIdx.x & 15;
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float x = bf16_lo(done[k][g * 16 + r][c]);
        v[r] = (a.g.rht_mask >> r) & 1u ? -x : x;
      }
      fwht16(v);
#pragma unroll
      for (int r = 0; r < 16; ++r) most[k] = fmaxf(most[k], fabsf(v[r]));
    }
  }
  if (a.amax[0] || a.rht[0] || a.amax[1] || a.rht[1]) {
    unsigned int *const out[4] = {a.amax[0], a.rht[0], a.amax[1], a.rht[1]};
    const uint32_t bits[4] = {top[0] << 16, __float_as_uint(most[0] * 0.25f), top[1] << 16, __float_as_uint(most[1] * 0.25f)};
    raise_maxima<4>(out, bits);
  }
}

int64_t tiles(const GatedArgs &a, int64_t bm, int64_t bn) { return (a.g.M + bm - 1) / bm * ((a.g.N + bn - 1) / bn); }

// Which kernel.  Up to 64 rows the one that reads the weights once (20480 columns,
// K 5120, forward: 16, 32, 64 rows in 24, 30, 46 us with the weights in the last-level
// cache, 32, 42, 56 without; in tiles of 128 rows 77 and 80).  Else
// the pipeline, where K fits its K-tiles and its large tiles leave few compute
// units idle: a round of 256 of them takes as long as 640 of the small ones (two
// to a compute unit).  Forward, K 5120: 256 x 20480 105 us against 126, 768 x 20480
// 250 against 329, 128 x 20480 106 against 81; K 2048: 4096 x 2048 61 against 75,
// 2048 x 2048 50 against 40, 1024 x 2048 48 against 24.  Backward, K 2048: 8192 x
// 2048 82 against 107, 4096 x 2048 70 against 55.
template <bool BACK>
hipError_t launch(const GatedArgs &a, hipStream_t s) {
  const GemmArgs &g = a.g;
  const dim3 block(kGThreads);
  if (g.M <= 64) {
    const dim3 grid((uint32_t)(g.N / 16));
    if (g.M <= 16)
      hipLaunchKernelGGL((gated_skinny_kernel<1, BACK>), grid, block, 0, s, a);
    else if (g.M <= 32)
      hipLaunchKernelGGL((gated_skinny_kernel<2, BACK>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((gated_skinny_kernel<4, BACK>), grid, block, 0, s, a);
    return hipGetLastError();
  }
  const int64_t large = tiles(a, 256, BACK ? 256 : 128), small = tiles(a, 128, BACK ? 128 : 64);
  // the pipeline's offsets have 32 bits, and it moves scales by dwords
  const bool fit = scales_fit(g.a_scales) && scales_fit(g.b_scales) && (BACK || scales_fit(a.u_scales));
  if (g.K % kFBK == 0 && fit && g.K / 2 * (g.M > g.N ? g.M : g.N) < (1ll << 32) && (large + 255) / 256 * 640 <= small)
    hipLaunchKernelGGL((gated_fast_kernel<BACK>), dim3((uint32_t)large), block, 0, s, a);
  else
    hipLaunchKernelGGL((gated_generic_kernel<BACK, 2>), dim3((uint32_t)small), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_gated(const GatedArgs &a, hipStream_t s) { return launch<false>(a, s); }
hipError_t launch_gemm_gated_backward(const GatedArgs &a, hipStream_t s) { return launch<true>(a, s); }

}  // namespace nvfp4
