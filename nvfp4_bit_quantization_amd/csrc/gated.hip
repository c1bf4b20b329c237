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
#include "block_kernels.hpp"
#include "gemm_tile.hpp"
#include "train_device.hpp"

namespace nvfp4 {
namespace {

// e^x and 1 / x as the hardware has them, within some 2^-22: their results are
// rounded to bf16
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.442695041f); }
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-x)); }

constexpr float kTanhScale = 1.595769122f;  // 2 sqrt(2 / pi): (1 + tanh(z)) / 2 = sigmoid(2 z)
constexpr float kCubic = 0.044715f;

// the activation of x, and its derivative
template <int ACT>
__device__ __forceinline__ float act(float x) {
  if (ACT == NVFP4_SILU) return x * sigmoid(x);
  if (ACT == NVFP4_RELU) return fmaxf(x, 0.0f);
  if (ACT == NVFP4_GELU) return x * (0.5f * erfcf(-0.7071067812f * x));
  return x * sigmoid(kTanhScale * x * fmaf(kCubic * x, x, 1.0f));
}
template <int ACT>
__device__ __forceinline__ void act_grad(float x, float &f, float &df) {
  if (ACT == NVFP4_SILU) {
    const float p = sigmoid(x);
    f = x * p;
    df = p * fmaf(x, 1.0f - p, 1.0f);
  } else if (ACT == NVFP4_RELU) {
    f = fmaxf(x, 0.0f);
    df = x > 0.0f ? 1.0f : 0.0f;
  } else if (ACT == NVFP4_GELU) {
    const float p = 0.5f * erfcf(-0.7071067812f * x);
    f = x * p;
    df = fmaf(x * 0.3989422804f, exp_of(-0.5f * x * x), p);
  } else {
    const float p = sigmoid(kTanhScale * x * fmaf(kCubic * x, x, 1.0f));
    const float y = fminf(fmaxf(x, -64.0f), 64.0f);  // beyond, p (1 - p) is zero
    f = x * p;
    df = fmaf(p * (1.0f - p) * y, kTanhScale * fmaf(3.0f * kCubic * y, y, 1.0f), p);
  }
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
  if (o.amax_plain || o.amax_rht) fused_max_flush(fm, o);
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
      const bool here = row < a.g.M && n < a.g.N;
      uint4 g = make_uint4(0, 0, 0, 0), u = g;
      if (here) {
        g = load_group(a.gate + row * a.ld_gate + n);
        u = load_group(a.up + row * a.ld_up + n);
      }
      float dg[8], du[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float dh = epi_apply(slab[r * S + c + k], es);
        float f, df;
        act_grad<ACT>(bf16_at(g, k), f, df);
        dg[k] = dh * bf16_at(u, k) * df;
        du[k] = dh * f;
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
    slab_fence();
    if (rht) {
#pragma unroll
      for (int j = 0; j < 2 * TN; ++j)
        slab_max(fm[j / TN], o[j / TN], reinterpret_cast<const uint16_t *>(slab) + j * 32, 2 * S, lane);
      slab_fence();
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (a.amax[k] || a.rht[k]) fused_max_flush(fm[k], o[k]);
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

// any K: tiles of 64 TM x 64 TN operand rows through registers, a K-tile ahead
template <bool BACK, int TM, int TN>
__global__ __launch_bounds__(kGThreads) void gated_generic_kernel(GatedArgs a) {
  constexpr int BM = GemmTile<TM, TN>::BM, ROWS = GemmTile<TM, TN>::ROWS;
  union Shared {
    struct {
      uint8_t codes[2][ROWS * kRowBytes];
      uint32_t scales[2][ROWS];
    } stage;
    float slabs[kGThreads / 64 * Slab<TN>::kFloats];
  };
  __shared__ __attribute__((aligned(16))) Shared lds;
  auto &lcodes = lds.stage.codes;
  auto &lscales = lds.stage.scales;
  int64_t m0, n0;
  origin<BM, BACK ? 64 * TN : 32 * TN>(a, xcd_tile(blockIdx.x, gridDim.x), m0, n0);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  const int lrow = lane & 31, half = lane >> 5;
  float16v acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int64_t KT = (a.g.K + kBK - 1) / kBK;
  Stage<TM, TN> st;
  const auto load = [&](int64_t kt) {
    if constexpr (BACK)
      stage_load<TM, TN>(PlainRows{a.g, m0, n0}, kt, st);
    else
      stage_load<TM, TN>(GatedRows<TN>{a, m0, n0}, kt, st);
  };
  load(0);
  stage_store<TM, TN>(lcodes[0], lscales[0], st);
  __syncthreads();
  for (int64_t kt = 0; kt < KT; ++kt) {
    const int buf = (int)(kt & 1);
    if (kt + 1 < KT) load(kt + 1);
    uint4 qa[TM], qb[TN];
    uint32_t sa[TM], sb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int row = wm * (TM * 32) + i * 32 + lrow;
      qa[i] = *reinterpret_cast<const uint4 *>(&lcodes[buf][row * kRowBytes + half * 16]);
      sa[i] = lscales[buf][row];
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int row = BM + wn * (TN * 32) + j * 32 + lrow;
      qb[j] = *reinterpret_cast<const uint4 *>(&lcodes[buf][row * kRowBytes + half * 16]);
      sb[j] = lscales[buf][row];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int blk = 2 * half + (s >> 1);
      half8v fa[TM], fb[TN];
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[i] = expand8(s == 0 ? qa[i].x : s == 1 ? qa[i].y : s == 2 ? qa[i].z : qa[i].w, scale_f16(sa[i], blk));
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fb[j] = expand8(s == 0 ? qb[j].x : s == 1 ? qb[j].y : s == 2 ? qb[j].z : qb[j].w, scale_f16(sb[j], blk));
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < KT) stage_store<TM, TN>(lcodes[buf ^ 1], lscales[buf ^ 1], st);
    __syncthreads();
  }
  store_tile<BACK, TM, TN>(a, m0, n0, acc, lds.slabs);
}

int64_t tiles(const GatedArgs &a, int64_t bm, int64_t bn) { return (a.g.M + bm - 1) / bm * ((a.g.N + bn - 1) / bn); }

template <bool BACK>
hipError_t launch(const GatedArgs &a, hipStream_t s) {
  const GemmArgs &g = a.g;
  const dim3 block(kGThreads);
  // the pipeline's K-tiles are whole and its offsets have 32 bits
  const bool fast = g.K % kFBK == 0 && g.K / 2 * (g.M > g.N ? g.M : g.N) < (1ll << 32);
  if (fast)
    hipLaunchKernelGGL((gated_fast_kernel<BACK>), dim3((uint32_t)tiles(a, 256, BACK ? 256 : 128)), block, 0, s, a);
  else
    hipLaunchKernelGGL((gated_generic_kernel<BACK, 2, 2>), dim3((uint32_t)tiles(a, 128, BACK ? 128 : 64)), block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_gated(const GatedArgs &a, hipStream_t s) { return launch<false>(a, s); }
hipError_t launch_gemm_gated_backward(const GatedArgs &a, hipStream_t s) { return launch<true>(a, s); }

}  // namespace nvfp4
