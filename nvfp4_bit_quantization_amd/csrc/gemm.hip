// NVFP4-operand GEMM for gfx950: C[m][n] = (sum_k A^[m][k] B^[n][k]) / (S_A S_B)
// with A^ = e(code) * s_b, both operands stored K-contiguous ("TN").
//
// Method: NVFP4 pretraining news page (zubnet.ai), paragraphs 1-2 -- the 4-bit
// GEMMs consume E2M1 codes with E4M3 block scales and FP32 per-tensor scales.
//
// Design.  Packed codes (4 bits/element) and scale bytes are staged in LDS, so
// a K-tile costs 0.5625 B/element of global and LDS traffic.  Each wave reads
// its MFMA fragments straight from the packed tile and expands them in
// registers: the gfx950 FP4->FP16 conversion gives e(code), one packed FP16
// multiply applies the block scale.  e * s_b has at most 6 significant bits
// and lies in [2^-10, 2688], so the FP16 operand is exact and the
// v_mfma_f32_32x32x16_f16 products are exact; accumulation is FP32 and the
// per-tensor scales are applied once in the epilogue.
//
// Fragment/K mapping: within a 64-wide K-tile, lane-half h (lane / 32) of an
// MFMA in sub-step s holds the 8 consecutive k = 32h + 8s + [0, 8), i.e. one
// dword of codes at byte 16h + 4s of the row's 32-byte K-tile slice, under the
// block scale of k-block 2h + s/2.  A and B use the same mapping, so every k
// of the tile is summed exactly once.
#include "gemm_tile.hpp"

#include <stdlib.h>

namespace nvfp4 {

constexpr int kBK = 64;         // K per tile
constexpr int kRowBytes = 48;   // LDS bytes per row: 32 bytes of codes + 16 pad (bank spread)

__device__ __forceinline__ _Float16 scale_f16(uint32_t scales4, int blk) {
  // E4M3 byte -> fp32 (exact) -> fp16 (exact: 2^-9 .. 448 are fp16 normals)
  const uint32_t b = (scales4 >> (8 * blk)) & 0xFFu;
  return (_Float16)e4m3_value(b);
}

// Each wave folds its maxima with one device-scope atomic maximum per tensor (bit
// patterns of non-negative floats order like the values).
__device__ __forceinline__ void fused_max_flush(const FusedMax &f, const GemmArgs &g) {
  uint32_t mp = f.plain;
  float mr = f.rht;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    mp = max(mp, (uint32_t)__shfl_xor((int)mp, off, 64));
    mr = fmaxf(mr, __shfl_xor(mr, off, 64));
  }
  if ((threadIdx.x & 63u) == 0) {
    if (g.amax_plain) atomicMax(g.amax_plain, mp << 16);
    if (g.amax_rht) atomicMax(g.amax_rht, __float_as_uint(mr * 0.25f));  // the exact 1/4 of the transform
  }
}

template <int TM, int TN>
struct GemmTile {
  static constexpr int BM = 64 * TM;
  static constexpr int BN = 64 * TN;
  static constexpr int ROWS = BM + BN;
};

// Global -> register staging of one K-tile: 32 bytes of codes and 4 scale bytes
// for each of the BM + BN rows.  Rows past M/N and k-blocks past K read as 0.
template <int TM, int TN>
struct Stage {
  static constexpr int ROWS = GemmTile<TM, TN>::ROWS;
  static constexpr int CHUNKS = ROWS * 4;  // 8-byte chunks of codes
  static constexpr int CPT = CHUNKS / kGThreads;
  static constexpr int SPT = (ROWS + kGThreads - 1) / kGThreads;
  uint2 code[CPT];
  uint32_t scale[SPT];
};

template <int TM, int TN, typename Rows>
__device__ __forceinline__ void stage_load(const Rows &src, int64_t kt, Stage<TM, TN> &st) {
  constexpr int BM = GemmTile<TM, TN>::BM, ROWS = GemmTile<TM, TN>::ROWS;
  const int64_t K = src.K(), kblocks = K / 16;
#pragma unroll
  for (int i = 0; i < Stage<TM, TN>::CPT; ++i) {
    const int c = threadIdx.x + i * kGThreads;
    const int row = c >> 2, part = c & 3;  // part = k-block within the tile
    const RowRef ref = src.template ref<BM>(row);
    const int64_t kb = kt * 4 + part;
    uint2 v = make_uint2(0u, 0u);
    if (ref.row < ref.rows && kb < kblocks) v = *reinterpret_cast<const uint2 *>(ref.codes + ref.row * (K / 2) + kb * 8);
    st.code[i] = v;
  }
#pragma unroll
  for (int i = 0; i < Stage<TM, TN>::SPT; ++i) {
    const int row = threadIdx.x + i * kGThreads;
    uint32_t w = 0;
    if (row < ROWS) {
      const RowRef ref = src.template ref<BM>(row);
      if (ref.row < ref.rows) {
        const uint8_t *p = ref.kind == 0 ? ref.scales + ref.row * kblocks : ref.scales + (ref.row / 16) * kblocks;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int64_t kb = kt * 4 + b;
          if (kb < kblocks) w |= (uint32_t)p[kb] << (8 * b);
        }
      }
    }
    st.scale[i] = w;
  }
}

template <int TM, int TN>
__device__ __forceinline__ void stage_store(uint8_t *lcodes, uint32_t *lscales, const Stage<TM, TN> &st) {
  constexpr int ROWS = GemmTile<TM, TN>::ROWS;
#pragma unroll
  for (int i = 0; i < Stage<TM, TN>::CPT; ++i) {
    const int c = threadIdx.x + i * kGThreads;
    const int row = c >> 2, part = c & 3;
    *reinterpret_cast<uint2 *>(lcodes + row * kRowBytes + part * 8) = st.code[i];
  }
#pragma unroll
  for (int i = 0; i < Stage<TM, TN>::SPT; ++i) {
    const int row = threadIdx.x + i * kGThreads;
    if (row < ROWS) lscales[row] = st.scale[i];
  }
}

template <int TM, int TN>
__global__ __launch_bounds__(kGThreads) void gemm_generic_kernel(GemmArgs g) {
  constexpr int BM = GemmTile<TM, TN>::BM, BN = GemmTile<TM, TN>::BN, ROWS = GemmTile<TM, TN>::ROWS;
  __shared__ __attribute__((aligned(16))) uint8_t lcodes[2][ROWS * kRowBytes];
  __shared__ uint32_t lscales[2][ROWS];

  const int64_t tiles_n = (g.N + BN - 1) / BN;
  const uint32_t tile = xcd_tile(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(tile / tiles_n) * BM;
  const int64_t n0 = (int64_t)(tile % tiles_n) * BN;

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

  const int64_t KT = (g.K + kBK - 1) / kBK;
  const PlainRows rows = {g, m0, n0};
  Stage<TM, TN> st;
  stage_load<TM, TN>(rows, 0, st);
  stage_store<TM, TN>(lcodes[0], lscales[0], st);
  __syncthreads();

  for (int64_t kt = 0; kt < KT; ++kt) {
    const int buf = (int)(kt & 1);
    if (kt + 1 < KT) stage_load<TM, TN>(rows, kt + 1, st);

    // fragments of this wave for the whole K-tile: 16 bytes of codes per row tile
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
      for (int i = 0; i < TM; ++i) {
        const uint32_t q = s == 0 ? qa[i].x : s == 1 ? qa[i].y : s == 2 ? qa[i].z : qa[i].w;
        fa[i] = expand8(q, scale_f16(sa[i], blk));
      }
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const uint32_t q = s == 0 ? qb[j].x : s == 1 ? qb[j].y : s == 2 ? qb[j].z : qb[j].w;
        fb[j] = expand8(q, scale_f16(sb[j], blk));
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }

    if (kt + 1 < KT) stage_store<TM, TN>(lcodes[buf ^ 1], lscales[buf ^ 1], st);
    __syncthreads();
  }

  // epilogue: C = acc / (S_A S_B); outputs past M or N are zero (zero
  // operands), so they do not change the fused maxima
  const EpiScale es = epi_scale(g);
  const bool fused = g.c_bf16 && (g.amax_plain || g.amax_rht);
  FusedMax fm;
  if (fused) fused_max_init(fm, g, lane);
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int64_t n = n0 + wn * (TN * 32) + j * 32 + lrow;
      uint32_t hb[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t m = m0 + wm * (TM * 32) + i * 32 + (r >> 2) * 8 + half * 4 + (r & 3);
        const float v = epi_apply(acc[i][j][r], es);
        hb[r] = bf16_rne_bits(v);
        if (m < g.M && n < g.N) {
          if (g.c_bf16)
            reinterpret_cast<uint16_t *>(g.c)[m * g.ldc + n] = (uint16_t)hb[r];
          else
            reinterpret_cast<float *>(g.c)[m * g.ldc + n] = v;
        }
      }
      if (fused) fused_max_block(fm, g, hb);
    }
  if (fused) fused_max_flush(fm, g);
}

// C tile = acc / (S_A S_B), 32-bit offsets from the tile origin
// C is written with non-temporal stores.  Written back through the caches,
// a large C leaves dirty lines in the memory-side cache, and the next kernel
// pays for their write-back while it reads: a 20480x5120 weight quantise
// took 110 us right after a 16384x20480 bf16 GEMM output against 88 us
// alone.  With non-temporal stores C reaches HBM while the GEMM, which is
// bound by the MFMA and not by HBM, still runs (the quantise then took 95 us,
// the GEMM's own time unchanged), and the Wgrad step ran 1 % faster.
__device__ __forceinline__ void fast_store_c(const GemmArgs &g, int64_t m0, int64_t n0, const float16v acc[4][4]) {
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t lr = lane & 31, h = lane >> 5;
  const EpiScale es = epi_scale(g);
  uint32_t ldc = (uint32_t)g.ldc;
  asm volatile("" : "+s"(ldc));  // per-element offsets are formed here, not hoisted and kept live
  if (g.c_bf16) {
    uint16_t *ct = reinterpret_cast<uint16_t *>(g.c) + m0 * g.ldc + n0;
    asm volatile("" : "+s"(ct));  // keep the address arithmetic in the epilogue
    const bool fused = g.amax_plain || g.amax_rht;
    FusedMax fm;
    if (fused) fused_max_init(fm, g, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t hb[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint32_t m = wm * 128 + i * 32 + (r >> 2) * 8 + h * 4 + (r & 3);
          const uint32_t n = wn * 128 + j * 32 + lr;
          hb[r] = bf16_rne_bits(epi_apply(acc[i][j][r], es));
          __builtin_nontemporal_store((uint16_t)hb[r], &ct[m * ldc + n]);
        }
        if (fused) fused_max_block(fm, g, hb);
      }
    if (fused) fused_max_flush(fm, g);
  } else {
    float *ct = reinterpret_cast<float *>(g.c) + m0 * g.ldc + n0;
    asm volatile("" : "+s"(ct));  // keep the address arithmetic in the epilogue
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint32_t m = wm * 128 + i * 32 + (r >> 2) * 8 + h * 4 + (r & 3);
          const uint32_t n = wn * 128 + j * 32 + lr;
          __builtin_nontemporal_store(epi_apply(acc[i][j][r], es), &ct[m * ldc + n]);
        }
  }
}

template <int TM, int TN>
__global__ __launch_bounds__(kGThreads) void gemm_fast_kernel(GemmArgs g) {
  static_assert(TM == 4 && TN == 4, "fast path is laid out for 256x256 tiles");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFStages * kFStageBytes];
  // Each XCD takes a contiguous range of the tile sequence, and the sequence
  // runs down groups of kGroupM tile rows column by column, so the workgroups
  // that one XCD runs at a time cover a compact block of C: they share the A
  // and B K-slices in that XCD's L2 instead of each streaming its own.
  int64_t m0, n0;
  tile_origin(g.M, g.N, xcd_tile(blockIdx.x, gridDim.x), m0, n0);
  float16v acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  fast_tile(PlainRows{g, m0, n0}, 0, (uint32_t)(g.K / kFBK), acc, lds);
  fast_store_c(g, m0, n0, acc);
}

// ===========================================================================
// Stream-K (fast path shapes whose tile count leaves compute units idle in
// the last round): one persistent workgroup per compute unit, all resident
// (the LDS admits one per CU).  The first dp_tiles tiles (whole rounds) are done
// as whole tiles, round by round, so that the workgroups of one XCD start
// their tiles together and share K-slices in L2.  The remaining tiles' units
// (tile, K-tile) are numbered tile by tile in the grouped order and dealt out
// as G contiguous ranges.  A workgroup whose range starts inside a tile
// computes that part first, writes its fp32 partial to workspace slot w and
// raises flag w.  The workgroup that holds the tile's first K-tile (the head,
// at the end of its range) computes its part last, then for each following
// workgroup whose range starts inside the tile waits for its flag (normally
// long raised), adds its partial (in workgroup order, so the sum does not
// depend on timing) and lowers the flag, leaving every flag zero for the next
// launch; then it writes C.  Partials and flags use device-coherent (sc1)
// accesses; a partial's writes complete (vmcnt) before its flag is raised.
// Each wait is bounded (about a second); on time-out `err` is set, that
// tile's result is invalid and the late partial is neither added nor its flag
// lowered, but the launch always ends.
// ===========================================================================
struct StreamK {
  uint32_t *flags;  // [G]
  uint32_t *err;
  float *slots;     // [G][65536]
  uint32_t tiles, KT;
  uint32_t dp_tiles;  // tiles done whole before the stream-K part (a multiple of G)
};

// The partial moves 64 values at a time (a compiler memory barrier between
// groups): four round trips to memory for the loads, and no more than 64
// extra registers live next to the 256 accumulators.
__device__ __forceinline__ void store_partial(float *slot, const float16v acc[4][4]) {
  asm volatile("" : "+s"(slot));  // keep the address arithmetic here (not hoisted and kept live)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        __hip_atomic_store(slot + ((i * 4 + j) * 16 + r) * kGThreads + threadIdx.x, acc[i][j][r], __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");
  }
}

__device__ __forceinline__ void add_partial(float16v acc[4][4], const float *slot) {
  asm volatile("" : "+s"(slot));  // keep the address arithmetic here (not hoisted and kept live)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float p[4][16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        p[j][r] = __hip_atomic_load(slot + ((i * 4 + j) * 16 + r) * kGThreads + threadIdx.x, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] += p[j][r];
  }
}

__device__ __forceinline__ void zero_acc(float16v acc[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
}

__global__ __launch_bounds__(kGThreads) void gemm_streamk_kernel(GemmArgs g, StreamK sk) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kFStages * kFStageBytes];
  const uint32_t G = gridDim.x, w = xcd_tile(blockIdx.x, G);
  float16v acc[4][4];
  int64_t m0, n0;

  for (uint32_t t = w; t < sk.dp_tiles; t += G) {  // whole tiles, round by round
    tile_origin(g.M, g.N, t, m0, n0);
    zero_acc(acc);
    fast_tile(PlainRows{g, m0, n0}, 0, sk.KT, acc, lds);
    fast_store_c(g, m0, n0, acc);
  }

  const uint64_t U = (uint64_t)(sk.tiles - sk.dp_tiles) * sk.KT;
  uint64_t u = U * w / G;
  const uint64_t uend = U * (w + 1) / G;
  while (u < uend) {
    const uint32_t ts = (uint32_t)(u / sk.KT), ka = (uint32_t)(u - (uint64_t)ts * sk.KT);
    const uint64_t tend = (uint64_t)(ts + 1) * sk.KT;
    const uint32_t kb = (uint32_t)((uend < tend ? uend : tend) - (uint64_t)ts * sk.KT);
    tile_origin(g.M, g.N, sk.dp_tiles + ts, m0, n0);
    zero_acc(acc);
    fast_tile(PlainRows{g, m0, n0}, ka, kb, acc, lds);
    if (ka > 0) {  // this range starts inside the tile: hand the partial to its head
      store_partial(sk.slots + (size_t)w * 65536, acc);
      NVFP4_WAIT_VMCNT(0);
      __syncthreads();
      if (threadIdx.x == 0) __hip_atomic_store(sk.flags + w, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      // head: add the partials of the following workgroups whose (non-empty)
      // ranges start inside the tile
      __shared__ uint32_t timed_out;
      for (uint32_t v = w + 1; v < G && U * v / G < tend; ++v) {
        if (U * (v + 1) / G == U * v / G) continue;  // an empty range wrote no partial
        if (threadIdx.x == 0) {
          uint32_t late = 0;
          for (uint32_t spins = 0;
               __hip_atomic_load(sk.flags + v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0u;) {
            __builtin_amdgcn_s_sleep(8);
            if (++spins == (1u << 22)) {
              __hip_atomic_store(sk.err, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              late = 1;
              break;
            }
          }
          timed_out = late;
        }
        __syncthreads();
        // On a time-out the slot holds no finished partial and the flag is
        // left alone (workgroup v raises it later): the tile is invalid, the
        // error word says so, and the caller zero-fills the workspace again
        // before its next use.
        if (!timed_out) {
          add_partial(acc, sk.slots + (size_t)v * 65536);
          __syncthreads();
          if (threadIdx.x == 0) __hip_atomic_store(sk.flags + v, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();  // timed_out is read by every thread before it is written again
      }
      fast_store_c(g, m0, n0, acc);
    }
    u += kb - ka;
  }
}

bool gemm_fast_ok(const GemmArgs &g) {
  return g.M % 256 == 0 && g.N % 256 == 0 && g.K % kFBK == 0 && g.K / 2 * (g.M > g.N ? g.M : g.N) < (1ll << 32) &&
         g.ldc * 256 < (1ll << 31) && scales_fit(g.a_scales) && scales_fit(g.b_scales);
}

size_t gemm_workspace_bytes(int cus) { return kGemmWsSlots + (size_t)cus * kGemmSlotBytes; }

hipError_t launch_gemm(const GemmArgs &g, void *workspace, size_t workspace_bytes, hipStream_t s) {
  constexpr int TM = 4, TN = 4;
  constexpr int BM = GemmTile<TM, TN>::BM, BN = GemmTile<TM, TN>::BN;
  const int64_t tiles = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
  if (!gemm_fast_ok(g) || getenv("NVFP4_GEMM_GENERIC")) {
    hipLaunchKernelGGL((gemm_generic_kernel<TM, TN>), dim3((uint32_t)tiles), dim3(kGThreads), 0, s, g);
    return hipGetLastError();
  }
  // Stream-K when a workspace is given, there are more than two rounds of
  // tiles and the last round would leave more than a tenth of the compute
  // units idle.  (With fewer rounds the split tiles' pipeline refills and
  // partial sums cost more than the idle units of one short last round, which
  // also runs at a higher clock: measured on 5120x5120x8192.)
  // A stream being captured into a graph gets whole tiles: a replay must not
  // depend on every workgroup of the persistent grid being resident.
  hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
  if (hipStreamIsCapturing(s, &capture) != hipSuccess) {
    (void)hipGetLastError();
    capture = hipStreamCaptureStatusActive;  // unknown: take the whole-tile path
  }
  int dev = 0, cus = 0;
  if (workspace && capture == hipStreamCaptureStatusNone && !getenv("NVFP4_GEMM_DATA_PARALLEL") &&
      hipGetDevice(&dev) == hipSuccess &&
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && cus > 0 &&
      cus <= kGemmMaxCUs && tiles > 2 * (int64_t)cus && workspace_bytes >= gemm_workspace_bytes(cus)) {
    const int64_t rounds = (tiles + cus - 1) / cus;
    if (10 * tiles < 9 * rounds * cus) {
      StreamK sk;
      sk.flags = (uint32_t *)workspace;
      sk.err = (uint32_t *)workspace + kGemmMaxCUs;
      sk.slots = (float *)((char *)workspace + kGemmWsSlots);
      sk.tiles = (uint32_t)tiles;
      sk.KT = (uint32_t)(g.K / kFBK);
      sk.dp_tiles = (uint32_t)((tiles / cus) * cus);  // whole rounds first
      // One workgroup per compute unit, launched as an ordinary kernel: its
      // 108 KiB of LDS admits one per CU, so on a GPU that runs nothing
      // else all are resident together.  A workgroup only ever waits for
      // workgroups with a larger index, and each wait is bounded, so the
      // launch ends even if some were held back (then the error word is set).
      // (A cooperative launch would guarantee residency but costs 15-22 us
      // per call, measured on the Wgrad and linear-step shapes.)
      int per_cu = 0;
      if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, gemm_streamk_kernel, kGThreads, 0) == hipSuccess &&
          per_cu >= 1) {
        hipLaunchKernelGGL(gemm_streamk_kernel, dim3((uint32_t)cus), dim3(kGThreads), 0, s, g, sk);
        return hipGetLastError();
      }
      (void)hipGetLastError();  // occupancy unknown: whole tiles
    }
  }
  hipLaunchKernelGGL((gemm_fast_kernel<TM, TN>), dim3((uint32_t)tiles), dim3(kGThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace nvfp4
