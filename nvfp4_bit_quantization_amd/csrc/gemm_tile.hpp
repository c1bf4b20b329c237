// Device code of the NVFP4-operand products (gfx950) that the plain GEMM and the
// gated products share: operand expansion, per-tensor scales, producer-fused
// maxima, where a tile's rows come from and the pipelined 256x256 tile.
#pragma once

#include "gemm_device.hpp"
#include "nvfp4_device.hpp"
#include "nvfp4_kernels.hpp"

namespace nvfp4 {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr int kGThreads = 256;  // 4 waves as 2 x 2

// 8 codes in `q` with block scale `s` -> 8 exact fp16 operand values
__device__ __forceinline__ half8v expand8(uint32_t q, _Float16 s) {
  const half2v sv = {s, s};
  const half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0) * sv;
  const half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1) * sv;
  const half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2) * sv;
  const half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3) * sv;
  half8v r;
  r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
  r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
  return r;
}

// The epilogue's division by S_A S_B, without forming that product in
// binary32: it overflows when both per-tensor maxima are small (about 1e-16
// each) and underflows when both are large, although C itself is
// representable.  S_A S_B = m 2^e with m = ma mb in [1/4, 1) (frexp), so
// C = ldexp(acc * (1/m), -e): one rounded multiply (1/m lies in (1, 4]), then
// an exact power-of-two scaling whenever C is a normal binary32.
struct EpiScale {
  float inv_m;
  int neg_e;
};

__device__ __forceinline__ EpiScale epi_scale(const GemmArgs &g) {
  int ea, eb;
  const float ma = frexpf(*g.a_S, &ea), mb = frexpf(*g.b_S, &eb);
  EpiScale s;
  s.inv_m = 1.0f / (ma * mb);
  s.neg_e = -(ea + eb);
  return s;
}

__device__ __forceinline__ float epi_apply(float acc, const EpiScale &s) { return ldexpf(acc * s.inv_m, s.neg_e); }

// ---------------------------------------------------------------------------
// Producer-fused maxima of a bf16 output (nvfp4_gemm_amax): the per-tensor
// maxima the quantisation of C needs, taken from the rounded outputs while
// they are in registers, so that the quantiser need not read C for them.
//   plain: max |c| over the stored bf16 values;
//   RHT along rows: max |H16 D c| / 4 over the aligned 16-row groups (the
//   transform a column-blocked quantisation of C applies; D from the mask).
// The transform of a 32x32 accumulator block is one product Z = T C on the
// bf16 MFMA (two 16-deep K-steps), T block-diagonal with two copies of H16 D.
// The accumulator layout (lane half h holds rows (r >> 2) 8 + 4h + (r & 3))
// serves directly as the K order of the B operand: K-step s takes r = 8s ..
// 8s + 7, i.e. the rows rho(k) = (k & 3) | (h << 2) | ((k >> 2) << 3) of
// group s, k = 8h + kk, and T's columns are permuted to match.  Products with
// +-1 are exact; the sums are fp32.  How lanes' maxima are joined is the
// launch's own.
// ---------------------------------------------------------------------------
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t bf16_rne_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// A operand of K-step s: lane l supplies row i = l % 32 of Z and k = 8 (l/32) + kk
__device__ __forceinline__ bf16x8v rht_rows_operand(uint32_t mask, uint32_t s, uint32_t lane) {
  const uint32_t i = lane & 31u, hh = lane >> 5;
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t pair = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t kk = 2 * q + e;
      const uint32_t rho = (kk & 3u) | (hh << 2) | ((kk >> 2) << 3);  // row of the 16-row group
      const uint32_t neg = (__builtin_popcount((i & 15u) & rho) + ((mask >> rho) & 1u)) & 1u;
      const uint32_t v = (i >> 4) == s ? (neg ? 0xBF80u : 0x3F80u) : 0u;
      pair |= v << (16 * e);
    }
    w[q] = pair;
  }
  return __builtin_bit_cast(bf16x8v, make_uint4(w[0], w[1], w[2], w[3]));
}

struct FusedMax {
  bf16x8v t0, t1;     // the transform's A operands (K-steps 0 and 1)
  uint32_t plain;     // max of |c| as bf16 magnitude bits
  float rht;          // max |H16 D c| (unnormalised)
};

__device__ __forceinline__ void fused_max_init(FusedMax &f, const GemmArgs &g, uint32_t lane) {
  f.plain = 0;
  f.rht = 0.0f;
  if (g.amax_rht) {
    f.t0 = rht_rows_operand(g.rht_mask, 0, lane);
    f.t1 = rht_rows_operand(g.rht_mask, 1, lane);
  }
}

// fold one 32x32 block's 16 rounded values (bf16 bit patterns) of this lane
__device__ __forceinline__ void fused_max_block(FusedMax &f, const GemmArgs &g, const uint32_t hb[16]) {
#pragma unroll
  for (int r = 0; r < 16; ++r) f.plain = max(f.plain, hb[r] & 0x7FFFu);
  if (g.amax_rht) {
    const bf16x8v b0 = __builtin_bit_cast(
        bf16x8v, make_uint4(hb[0] | (hb[1] << 16), hb[2] | (hb[3] << 16), hb[4] | (hb[5] << 16), hb[6] | (hb[7] << 16)));
    const bf16x8v b1 = __builtin_bit_cast(bf16x8v, make_uint4(hb[8] | (hb[9] << 16), hb[10] | (hb[11] << 16),
                                                              hb[12] | (hb[13] << 16), hb[14] | (hb[15] << 16)));
    float16v z;
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r] = 0.0f;
    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.t0, b0, z, 0, 0, 0);
    z = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.t1, b1, z, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 16; ++r) f.rht = fmaxf(f.rht, fabsf(z[r]));
  }
}

// Where the rows of a tile's stage come from: its first A_ROWS rows are A's, the
// others B's (PlainRows: rows m0 and n0 onwards of one A and one B).
struct RowRef {
  const uint8_t *codes, *scales;
  int kind;
  int64_t row, rows;  // the tensor has `rows`: what stands for those beyond is the caller's to say (the
                      // plain product takes zeros, the gated ones the last row, which they do not store)
};
struct PlainRows {
  const GemmArgs &g;
  int64_t m0, n0;
  static constexpr bool kTwo = false;  // B's rows come from one tensor
  __device__ __forceinline__ int64_t K() const { return g.K; }
  template <int A_ROWS>
  __device__ __forceinline__ RowRef ref(int r) const {
    const bool isA = r < A_ROWS;
    return {isA ? g.a_codes : g.b_codes, isA ? g.a_scales : g.b_scales, isA ? g.a_kind : g.b_kind,
            isA ? m0 + r : n0 + (r - A_ROWS), isA ? g.M : g.N};
  }
  // of the fast path's 256 + 256 rows: the tensors that a wave transfers, the row and scale kind of stage row r
  __device__ __forceinline__ const uint8_t *codes(uint32_t wave, bool) const { return wave < 2 ? g.a_codes : g.b_codes; }
  __device__ __forceinline__ const uint8_t *scales(uint32_t wave, bool) const { return wave < 2 ? g.a_scales : g.b_scales; }
  __device__ __forceinline__ uint32_t row(uint32_t r) const { return (uint32_t)(r < 256 ? m0 + r : n0 + (r - 256)); }
  __device__ __forceinline__ int kind(uint32_t r) const { return r < 256 ? g.a_kind : g.b_kind; }
};

// ===========================================================================
// Fast path (K a multiple of 128; M and N multiples of 256, or a row() that keeps to
// the tensors' rows, as the gated products'): 256x256x128 tiles, three LDS stages
// filled by direct global->LDS transfers.
//
// LDS stage layout (36 KiB): codes of the 256 A rows then the 256 B rows,
// 64 bytes (one 128-wide K slice) per row in four 16-byte chunks stored in
// the order chunk ^ swz(row), then 8 scale bytes per row as two dwords stored
// in the order half ^ ((row >> 4) & 1).  The swizzles make the fragment reads
// (ds_read_b128 of one row per lane, ds_read_b32 of its scales) free of bank
// conflicts for 32- and 64-bank LDS.  The transfers write consecutive 16-byte
// (4-byte for scales) slots per lane, so the swizzle is applied by choosing
// which global chunk each lane fetches.
//
// K mapping inside a 128-wide K-tile: lane-half h of the MFMA in sub-step s
// (0..7) holds k = 64h + 8s + [0, 8): dword s of the 32 bytes at byte 32h of
// the row slice, under block scale 4h + s/2 (byte s/2 of scale dword h).
// ===========================================================================
constexpr int kFBK = 128;
constexpr int kFStageCodes = 512 * 64;         // bytes of codes per stage
constexpr int kFStageBytes = kFStageCodes + 512 * 8;
constexpr int kFStages = 3;

// Whether the fast path may take a tensor's scales, which it transfers by dwords: a
// row has K / 16 of them, a multiple of 8, so that all rows are aligned as the first
// is.  (Codes are 16-byte aligned in every call.)
inline bool scales_fit(const uint8_t *scales) { return ((uintptr_t)scales & 3u) == 0; }

struct FastCtx {
  const uint8_t *cbase;  // codes of the operand this wave transfers (A: waves 0-1, B: waves 2-3)
  const uint8_t *sbase;  // its scales
  const uint8_t *cbase2, *sbase2;  // of the second half of its rows, where B's rows come from two tensors
  // per-lane global offsets (bytes) of this lane's 8 code chunks and 4 scale dwords at kt = 0
  uint32_t coff[8];
  uint32_t soff[4];
};

// Each wave issues exactly 12 transfers per K-tile (8 x 1 KiB of codes, 4 x
// 256 B of scales), which the vmcnt waits of the main loop count on.  Waves 0-1
// fill the A half of the stage (code slots 0..1023, scale slots 0..511), waves
// 2-3 the B half.  Transfers [FIRST, FIRST + COUNT) of the 12 are issued here
// (0-7 codes, 8-11 scales), so that a tile's transfers can be spread over
// several MFMA sub-steps.  `wave` must be wave-uniform.
// The K-tile's offset moves the scalar base address (two scalar adds per
// operand), so the per-lane offsets stay fixed: adding it to each transfer's
// per-lane offset took twelve VALU adds per K-tile from the MFMA shadow
// (measured: the 5120 x 5120 x 8192 GEMM 1.5 % faster this way).
// TWO: transfers 4-7 and 10, 11 (the second 64 of a wave's 128 rows) have a base
// of their own.
template <int FIRST, int COUNT, bool TWO>
__device__ __forceinline__ void fast_issue(const FastCtx &c, uint32_t lds_stage, uint32_t kt, uint32_t wave) {
  if constexpr (TWO && COUNT > 2) {  // by pairs, which do not cross from one base to the other
    fast_issue<FIRST, 2, TWO>(c, lds_stage, kt, wave);
    fast_issue<FIRST + 2, COUNT - 2, TWO>(c, lds_stage, kt, wave);
  } else {
    const bool two = TWO && (FIRST < 8 ? FIRST >= 4 : FIRST >= 10);
    const uint8_t *cb = uniform_ptr((two ? c.cbase2 : c.cbase) + (uint64_t)kt * 64u);
    const uint8_t *sb = uniform_ptr((two ? c.sbase2 : c.sbase) + (uint64_t)kt * 8u);
#pragma unroll
    for (int t = FIRST; t < FIRST + COUNT; ++t) {
      if (t < 8)
        dma16(cb, c.coff[t], __builtin_amdgcn_readfirstlane(lds_stage + (wave * 8 + t) * 1024u));
      else
        dma4(sb, c.soff[t - 8], __builtin_amdgcn_readfirstlane(lds_stage + kFStageCodes + (wave * 4 + (t - 8)) * 256u));
    }
  }
}

// The fp16 MFMA operands of one sub-step (16 k): 4 A and 4 B fragments.
struct Frags {
  half8v a[4], b[4];
};

// Expand sub-step s (0..3) of one half of a K-tile: dword s of this lane's
// 16 code bytes of each row, under block scale element s/2 of the pair.
template <int S>
__device__ __forceinline__ void expand_step(Frags &f, const uint4 qa[4], const uint4 qb[4], const half2v sa[4],
                                            const half2v sb[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = S == 0 ? qa[i].x : S == 1 ? qa[i].y : S == 2 ? qa[i].z : qa[i].w;
    f.a[i] = expand8(w, (S >> 1) ? sa[i][1] : sa[i][0]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t w = S == 0 ? qb[j].x : S == 1 ? qb[j].y : S == 2 ? qb[j].z : qb[j].w;
    f.b[j] = expand8(w, (S >> 1) ? sb[j][1] : sb[j][0]);
  }
}

__device__ __forceinline__ void mfma_step(float16v acc[4][4], const Frags &f) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Instruction order of one sub-step: each MFMA followed by four VALU
// instructions of the next sub-step's expansion (64 of them per 16 MFMAs), so
// the expansion runs in the shadow of the 8-pass MFMAs instead of between them.
__device__ __forceinline__ void interleave_step() {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // VALU
  }
}

// Accumulate K-tiles [ka, kb) of the 256x256 C tile at (m0, n0) into acc.
// Every wave of the workgroup calls it with the same arguments; it owns the
// whole LDS pipeline while it runs (it starts with a barrier, so the stages
// may be reused from one call to the next, and ends with no transfer in
// flight).
template <typename Rows>
__device__ __forceinline__ void fast_tile(const Rows &src, uint32_t ka, uint32_t kb, float16v acc[4][4], uint8_t *lds) {
  constexpr bool TWO = Rows::kTwo;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wm = wave >> 1, wn = wave & 1;
  const uint32_t lr = lane & 31, h = lane >> 5;
  const uint32_t kbytes = (uint32_t)(src.K() / 2), kblocks = (uint32_t)(src.K() / 16);

  // which global bytes this lane transfers (the same for every K-tile up to the K offset)
  FastCtx c;
  c.cbase = src.codes(wave, false);
  c.sbase = src.scales(wave, false);
  if (TWO) {
    c.cbase2 = src.codes(wave, true);
    c.sbase2 = src.scales(wave, true);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t q = (wave * 8 + i) * 64 + lane;  // 16-byte slot of the stage
    const uint32_t row = q >> 2;                      // 0..511: A rows then B rows
    const uint32_t chunk = (q & 3u) ^ swz(row);
    const uint32_t grow = src.row(row);
    c.coff[i] = grow * kbytes + chunk * 16u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t d = (wave * 4 + i) * 64 + lane;  // scale dword slot
    const uint32_t row = d >> 1;
    const uint32_t half = (d & 1u) ^ ((row >> 4) & 1u);
    const uint32_t grow = src.row(row);
    const uint32_t srow = src.kind(row) == 0 ? grow : (grow >> 4);
    c.soff[i] = srow * kblocks + half * 4u;
  }

  // LDS byte offsets (within a stage) of this lane's fragments: [i][0] holds
  // the k of the first half of the K-tile (sub-steps 0-3), [i][1] the second
  uint32_t aoff[4][2], boff[4][2], asoff[4], bsoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = wm * 128 + i * 32 + lr;
    aoff[i][0] = (r * 4 + ((2 * h) ^ swz(r))) * 16;
    aoff[i][1] = (r * 4 + ((2 * h + 1) ^ swz(r))) * 16;
    asoff[i] = kFStageCodes + (r * 2 + (h ^ ((r >> 4) & 1u))) * 4;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t r = 256 + wn * 128 + j * 32 + lr;
    boff[j][0] = (r * 4 + ((2 * h) ^ swz(r))) * 16;
    boff[j][1] = (r * 4 + ((2 * h + 1) ^ swz(r))) * 16;
    bsoff[j] = kFStageCodes + (r * 2 + (h ^ ((r >> 4) & 1u))) * 4;
  }

  // Pipeline.  Transfers run up to three K-tiles ahead of the MFMAs; every
  // iteration issues exactly one tile's transfers (the index clamped to the
  // last tile, so the vmcnt bookkeeping is the same in every iteration; the
  // clamped copies land in stages nobody reads again), two per sub-step: the
  // first six of tile kt+3 after the barrier of iteration kt, the other six
  // in the first half of iteration kt+1, before its barrier.  The barrier of tile
  // kt+1 sits between the two halves of tile kt, and the fp16 fragments are
  // expanded one MFMA sub-step ahead, so MFMAs are ready on both sides of it.
  const uint32_t lds0 = lds_addr(lds);
  const uint32_t klast = kb - 1;
  NVFP4_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();  // no wave still reads the stages (a previous tile's)
  asm volatile("" ::: "memory");
  fast_issue<0, 12, TWO>(c, lds0, ka, wave);
  fast_issue<0, 12, TWO>(c, lds0 + kFStageBytes, ka + 1 < klast ? ka + 1 : klast, wave);
  fast_issue<0, 6, TWO>(c, lds0 + 2 * kFStageBytes, ka + 2 < klast ? ka + 2 : klast, wave);
  NVFP4_WAIT_VMCNT(18);  // this wave's transfers of tile ka are done
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");

  // first-half codes and the tile's scales (E4M3 -> fp16 pairs: lo = blocks
  // (4h, 4h+1) of the first half, hi = (4h+2, 4h+3) of the second)
  uint4 qlo_a[4], qlo_b[4];
  half2v sal[4], sah[4], sbl[4], sbh[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    qlo_a[i] = *reinterpret_cast<const uint4 *>(lds + aoff[i][0]);
    const uint32_t sw = *reinterpret_cast<const uint32_t *>(lds + asoff[i]);
    sal[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, false);
    sah[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, true);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qlo_b[j] = *reinterpret_cast<const uint4 *>(lds + boff[j][0]);
    const uint32_t sw = *reinterpret_cast<const uint32_t *>(lds + bsoff[j]);
    sbl[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, false);
    sbh[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sw, 1.0f, true);
  }
  Frags f, fn;
  expand_step<0>(f, qlo_a, qlo_b, sal, sbl);

  uint32_t stage = 0;
  for (uint32_t kt = ka; kt < kb; ++kt) {
    // Each sub-step is a scheduling region of its own (sched_barrier), in
    // which the MFMAs of one sub-step interleave with the expansion of the next.
    const uint8_t *base = lds + stage * kFStageBytes;
    const uint32_t pstage = stage == 0 ? 2 : stage - 1;  // (kt + 2) % 3
    const uint32_t plds = lds0 + pstage * kFStageBytes, ptile = kt + 2 < klast ? kt + 2 : klast;
    uint4 qhi_a[4], qhi_b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) qhi_a[i] = *reinterpret_cast<const uint4 *>(base + aoff[i][1]);
#pragma unroll
    for (int j = 0; j < 4; ++j) qhi_b[j] = *reinterpret_cast<const uint4 *>(base + boff[j][1]);

    // first half: sub-steps 0-3 (sub-step 0's fragments are ready)
    expand_step<1>(fn, qlo_a, qlo_b, sal, sbl);
    mfma_step(acc, f);
    __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);  // the second-half code reads first
    interleave_step();
    fast_issue<6, 2, TWO>(c, plds, ptile, wave);
    __builtin_amdgcn_sched_barrier(0);
    expand_step<2>(f, qlo_a, qlo_b, sal, sbl);
    mfma_step(acc, fn);
    interleave_step();
    fast_issue<8, 2, TWO>(c, plds, ptile, wave);
    __builtin_amdgcn_sched_barrier(0);
    expand_step<3>(fn, qlo_a, qlo_b, sal, sbl);
    mfma_step(acc, f);
    interleave_step();
    fast_issue<10, 2, TWO>(c, plds, ptile, wave);
    __builtin_amdgcn_sched_barrier(0);
    expand_step<0>(f, qhi_a, qhi_b, sah, sbh);
    mfma_step(acc, fn);
    interleave_step();
    __builtin_amdgcn_sched_barrier(0);

    half2v cah[4], cbh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) cah[i] = sah[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) cbh[j] = sbh[j];

    NVFP4_WAIT_LGKM0();    // this wave's reads of the stage are complete
    NVFP4_WAIT_VMCNT(12);  // this wave's transfers of tile kt+1 are done (kt+2's may be in flight)
    __builtin_amdgcn_s_barrier();  // every wave's: tile kt+1 is in LDS, this stage is free
    asm volatile("" ::: "memory");
    const uint32_t dlds = lds_addr(base), dtile = kt + 3 < klast ? kt + 3 : klast;
    const uint32_t nstage = stage == 2 ? 0 : stage + 1;
    const uint8_t *nbase = lds + nstage * kFStageBytes;
    uint32_t swa[4], swb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qlo_a[i] = *reinterpret_cast<const uint4 *>(nbase + aoff[i][0]);
      swa[i] = *reinterpret_cast<const uint32_t *>(nbase + asoff[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qlo_b[j] = *reinterpret_cast<const uint4 *>(nbase + boff[j][0]);
      swb[j] = *reinterpret_cast<const uint32_t *>(nbase + bsoff[j]);
    }
    stage = nstage;

    // second half: sub-steps 4-7, then sub-step 0 of tile kt+1 is expanded
    // (on the last tile from a stale stage; those fragments are not used)
    expand_step<1>(fn, qhi_a, qhi_b, cah, cbh);
    mfma_step(acc, f);
    interleave_step();
    fast_issue<0, 2, TWO>(c, dlds, dtile, wave);
    __builtin_amdgcn_sched_barrier(0);
    expand_step<2>(f, qhi_a, qhi_b, cah, cbh);
    mfma_step(acc, fn);
    interleave_step();
    fast_issue<2, 2, TWO>(c, dlds, dtile, wave);
    __builtin_amdgcn_sched_barrier(0);
    expand_step<3>(fn, qhi_a, qhi_b, cah, cbh);
    mfma_step(acc, f);
    interleave_step();
    fast_issue<4, 2, TWO>(c, dlds, dtile, wave);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sal[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(swa[i], 1.0f, false);
      sah[i] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(swa[i], 1.0f, true);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sbl[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(swb[j], 1.0f, false);
      sbh[j] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(swb[j], 1.0f, true);
    }
    expand_step<0>(f, qlo_a, qlo_b, sal, sbl);
    mfma_step(acc, fn);
    interleave_step();
    __builtin_amdgcn_sched_barrier(0);
  }
  NVFP4_WAIT_VMCNT(0);  // the clamped transfers of the last iterations

}

}  // namespace nvfp4
