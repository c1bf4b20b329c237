// Attention over the keys in sight and its gradient (include/nvfp4.h:
// nvfp4_attention, nvfp4_attention_backward).
//
// All products run on the 32x32x16 bf16 MFMA, of which lane l (n = l & 31,
// h = l >> 5) holds: of A, row n, and of B, column n, the eight inner indices
// 8 h .. 8 h + 7; of the result, column n and the rows 8 (i / 4) + 4 h + i % 4,
// i = 0 .. 15.  Every product is laid out so that its result is the next one's
// B operand without crossing lanes: scores are formed with the index the next
// product sums over in their rows, and that product's A operand is read from
// LDS in the same order of that index (4 h .. 4 h + 3, then 8 + 4 h .. 11 + 4 h
// of each 16) by the transposing LDS read.
//
// Operands have the 8 significant bits of bf16, the inputs' type: probabilities
// and their gradients are rounded to it for their products, sums of both stay in
// binary32.  A product in binary32 has a sixteenth of the rate.  o is then off by
// 0.0020 of its norm, where rounding it alone costs 0.0016, the gradients by
// 0.0023 to 0.0025 instead of 0.0017 to 0.0019 (1024 random tokens, 64 bits but
// for these roundings, and the kernels alike).
//
// The gradient recomputes scores and dP in each of its two passes, dQ and
// dK + dV: seven products instead of five, but no sums by atomics, whose order
// would change results, and no binary32 buffer for dQ.
#include "gemm_device.hpp"
#include "train_device.hpp"
#include "train_kernels.hpp"

namespace nvfp4 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

constexpr int kThreads = 256;
constexpr int kTile = 64;               // rows of a staged tile
// instruction classes of sched_group_barrier
constexpr int kValu = 0x2, kMfma = 0x8, kDsRead = 0x100;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLow = -3e38f;          // below every score; finite, so that differences stay numbers

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}
// row of result register i in half h
__device__ __forceinline__ int row_of(int i, int h) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// ------------------------------------------------------------ sequences ----
struct Seq {
  int64_t q0, k0;  // first tokens
  int nq, nk;
  int64_t bq, bk;  // sequence index for the batch stride (0 when packed)
};
__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t lo, int64_t hi) { return v < lo ? lo : v > hi ? hi : v; }
__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b) {
  Seq s;
  if (a.cu_q) {
    s.q0 = clamp64(a.cu_q[b], 0, a.total_q);
    s.k0 = clamp64(a.cu_k[b], 0, a.total_k);
    s.nq = (int)clamp64(clamp64(a.cu_q[b + 1], s.q0, a.total_q) - s.q0, 0, a.q_len);
    s.nk = (int)clamp64(clamp64(a.cu_k[b + 1], s.k0, a.total_k) - s.k0, 0, a.k_len);
    s.bq = s.bk = 0;
  } else {
    s.q0 = s.k0 = 0;
    s.nq = a.q_len;
    s.nk = a.k_len;
    s.bq = s.bk = b;
  }
  return s;
}
// token index over all sequences of a sequence's first query
__device__ __forceinline__ int64_t first_row(const AttnArgs &a, const Seq &s, int b) {
  return a.cu_q ? s.q0 : (int64_t)b * a.q_len;
}
__device__ __forceinline__ uint16_t *at(const Heads &t, int64_t seq, int64_t token, int head) {
  return t.p + seq * t.sb + token * t.st + (int64_t)head * t.sh;
}

// keys [lo, hi) that query i sees; off = nk - nq.  Lengths and the window are
// at most 2^30, which keeps these sums in 32 bits.
__device__ __forceinline__ int within(int v, int hi) { return v < 0 ? 0 : v > hi ? hi : v; }
__device__ __forceinline__ void sight(const AttnArgs &a, int i, int nk, int off, int &lo, int &hi) {
  lo = 0;
  hi = nk;
  if (a.causal) {
    hi = within(i + off + 1, nk);
    if (a.window) lo = within(i + off + 1 - a.window, nk);
  }
}

// ---------------------------------------------------------------- tiles ----
// A tile of 64 rows of D elements in LDS.  It is filled by direct transfers of
// 1024 bytes, whose lanes' 16 bytes land next to each other: a segment of 4
// (D = 128) or 8 (D = 64) rows.  Chunks (16 bytes) are permuted within a row by
// which address each lane reads, chunk c of row r standing at c ^ spread(r),
// and segments are 16 (D = 128) or 32 (D = 64) bytes further apart than they
// are long.  Both reads below then meet every group of banks equally, the plain
// one (32 rows at one chunk; the rows that meet in a cycle are four groups of
// four, 0, 3, 5, 6 or 1, 2, 4, 7, which 16 bytes do not keep apart for D = 64)
// and the transposing one (4 rows at 4 neighbouring chunks), and all reads of a
// lane stand at fixed distances from D / 32 addresses each, as the
// instructions' immediate offsets.  (16 bytes for D = 64: 5 % of the
// gradient of 2 x 4096 tokens, 40 heads of 64, 8 key heads, causal, now 609 us.)
template <int D>
struct Tile {
  static constexpr int kChunks = D / 8, kSegRows = 64 / kChunks;
  static constexpr uint32_t kSeg = 1024 + (D == 128 ? 16 : 32);
  static constexpr uint32_t bytes(int rows) { return (uint32_t)(rows / kSegRows) * kSeg; }
  static __device__ __forceinline__ uint32_t spread(uint32_t r) {
    return D == 128 ? (r & 3u) << 2 : ((r >> 1) & 1u) << 2 | ((r >> 2) & 1u);
  }
};

// Transfer rows row0 .. row0 + R - 1 of a head (rows past `rows` repeat the
// last one, chunks past head_dim the first: their products are masked, or meet
// zeros) into the tile at LDS address lds.  Each of four waves fills a quarter
// of its segments.
template <int D, int R>
__device__ __forceinline__ void fetch_tile(const uint16_t *head, int64_t stride, int row0, int rows, int chunks,
                                           uint32_t lds, int wave, int lane) {
  typedef Tile<D> T;
  const uint8_t *base = uniform_ptr((const uint8_t *)(head + (int64_t)row0 * stride));
  asm volatile("" : "+v"(lane));  // the offsets are formed here, not kept in registers
  const uint32_t r = (uint32_t)lane / T::kChunks, pitch = (uint32_t)stride * 2u;
  uint32_t c = ((uint32_t)lane % T::kChunks) ^ T::spread(r);
  c = (int)c < chunks ? c * 16u : 0u;
  const int left = rows - row0 - 1;
  constexpr int kSegs = R / T::kSegRows / 4;
#pragma unroll
  for (int i = 0; i < kSegs; ++i) {
    const int seg = wave * kSegs + i, row = seg * T::kSegRows + (int)r;
    dma16(base, __umul24((uint32_t)(row < left ? row : left), pitch) + c,
          __builtin_amdgcn_readfirstlane(lds + (uint32_t)seg * T::kSeg));
  }
}

// a lane's addresses within a tile
template <int D>
struct Reads {
  uint32_t row[D / 32], col[D / 32];
  __device__ __forceinline__ Reads(int lane, uint32_t at) {
    typedef Tile<D> T;
    const uint32_t n = lane & 31, h = lane >> 5, i = lane & 15, g = lane >> 4;
#pragma unroll
    for (uint32_t k = 0; k < D / 32; ++k) {
      const uint32_t c = 4 * k + h;
      row[k] = n / T::kSegRows * T::kSeg + n % T::kSegRows * (2 * D) + (c ^ T::spread(n)) * 16 + at;
    }
#pragma unroll
    for (uint32_t dt = 0; dt < D / 32; ++dt) {
      const uint32_t r = 4 * (g >> 1) + (i >> 2), c = dt * 4 + (g & 1) * 2 + ((i & 3) >> 1);
      col[dt] = r / T::kSegRows * T::kSeg + r % T::kSegRows * (2 * D) + (c ^ T::spread(r)) * 16 + (i & 1) * 8 + at;
    }
  }
  // to the tile `by` bytes on
  __device__ __forceinline__ void move(uint32_t by) {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) row[k] += by;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) col[k] += by;
  }
  // A operand from rows r0 .. r0 + 31 (r0 = 0, 32) as they stand: row n,
  // elements 16 c + 8 h ..; `tile`: bytes to another tile
  __device__ __forceinline__ bf16x8 rows(uint32_t tile, int r0, int c) const {
    const uint32_t a = row[c >> 1] + tile + (uint32_t)(r0 / Tile<D>::kSegRows) * Tile<D>::kSeg + (c & 1) * 32u;
    return *(const __attribute__((address_space(3))) bf16x8 *)a;
  }
  __device__ __forceinline__ void set_row(int c, bf16x8 v) const {
    *(__attribute__((address_space(3))) bf16x8 *)(row[c >> 1] + (c & 1) * 32u) = v;
  }
  // A operand from the transposed tile: row = element 32 dt + n, inner index =
  // tile rows r0 + 4 h .. and r0 + 8 + 4 h .. (r0 = 0, 16, 32, 48)
  __device__ __forceinline__ bf16x8 cols(uint32_t tile, int r0, int dt) const {
    typedef short i16x8 __attribute__((ext_vector_type(8)));
    constexpr uint32_t k8 = 8 / Tile<D>::kSegRows * Tile<D>::kSeg;
    const uint32_t a = col[dt] + tile + (uint32_t)(r0 / 8) * k8;
    const i16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)a);
    const i16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(a + k8));
    const i16x8 v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
};

// Scores out of sight: of 32 rows from r0 on (register i of half h is row
// row_of(i, h)) those below lo and from hi on become -inf.  Which of the two
// limits falls within the rows is uniform over the wave.
template <int N>
__device__ __forceinline__ void hide(f32x16 (&p)[N], int lo, int hi, bool below, bool above, int h) {
  if (above) {
    const int n = hi - 4 * h;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) p[u][i] = n > 32 * u + row_of(i, 0) ? p[u][i] : -INFINITY;
  }
  if (below) {
    const int n = lo - 4 * h;
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) p[u][i] = n <= 32 * u + row_of(i, 0) ? p[u][i] : -INFINITY;
  }
}

// B operands of a row held by its lane: elements 16 c + 8 h .. of `row`, zero
// from head_dim on
template <int D>
__device__ __forceinline__ void load_row(const uint16_t *row, int chunks, int h, bf16x8 out[D / 16]) {
  uint4 q[D / 16];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) q[c] = *reinterpret_cast<const uint4 *>(row + 8 * (2 * c + h < chunks ? 2 * c + h : 0));
  if (chunks < D / 8) {
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      if (2 * c + h >= chunks) q[c] = make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int c = 0; c < D / 16; ++c) out[c] = __builtin_bit_cast(bf16x8, q[c]);
}

// eight result registers as a B operand
__device__ __forceinline__ bf16x8 pack8(const f32x16 &v, int first) {
  uint4 q;
  q.x = pack_bf16(v[first], v[first + 1]);
  q.y = pack_bf16(v[first + 2], v[first + 3]);
  q.z = pack_bf16(v[first + 4], v[first + 5]);
  q.w = pack_bf16(v[first + 6], v[first + 7]);
  return __builtin_bit_cast(bf16x8, q);
}

// result columns as rows of memory: lane n's column, its elements times f
template <int D>
__device__ __forceinline__ void store_cols(uint16_t *row, const f32x16 *acc, float f, int dim, int h) {
  const bool whole = dim == D;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = dt * 32 + 8 * g + 4 * h;
      if (whole || d < dim)
        *reinterpret_cast<uint2 *>(row + d) = make_uint2(pack_bf16(acc[dt][4 * g] * f, acc[dt][4 * g + 1] * f),
                                                         pack_bf16(acc[dt][4 * g + 2] * f, acc[dt][4 * g + 3] * f));
    }
}

__device__ __forceinline__ void tile_barrier() {
  NVFP4_WAIT_VMCNT(0);
  NVFP4_WAIT_LGKM0();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// workgroup -> (head, sequence, tile).  Key heads are innermost, so that with
// a multiple of 8 of them each stays on one XCD (workgroups are dealt to the 8
// XCDs in turn), and a tile's level outermost, heaviest first: what a compute
// unit gets then adds up alike.  Against heads outermost, a range of them to
// each XCD: gradient of 23 packed documents (4096 tokens, 16 heads of 64) 62 ->
// 51 us, of 8 x 1024 tokens 116 -> 95, of 16384 tokens, 20 heads of 128, 4518 ->
// 4187, forward of these 1422 -> 1329; without a causal mask 2565 -> 2581.
// Where all workgroups are resident at once, in up to three rounds of one to a
// compute unit, the second round goes backwards, so that it gives the lightest
// to the units that have the heaviest (gradient of 8192 tokens, 12 heads of 64,
// 409 -> 396 us).
struct Work {
  int b, head, level, part;
};
// n / d and n % d
__device__ __forceinline__ uint32_t split_off(uint32_t &n, const Divisor &d) {
  const uint32_t q = (uint32_t)(((uint64_t)n * d.by) >> d.shift), r = n - q * d.d;
  n = q;
  return r;
}
__device__ __forceinline__ Work work_of(const AttnArgs &a, int parts, bool by_group) {
  uint32_t w = blockIdx.x;
  if (gridDim.x <= 768 && (w | 255) < gridDim.x && (w >> 8 & 1)) w ^= 0xF8;
  Work r;
  r.head = (int)split_off(w, a.by_kv);
  if (by_group) r.head = r.head * (int)a.by_group.d + (int)split_off(w, a.by_group);
  r.part = (int)(w % (uint32_t)parts);
  w /= (uint32_t)parts;
  r.b = (int)split_off(w, a.by_batch);
  r.level = (int)w;
  return r;
}
// the steps [lo, hi) of part `part` of `parts`
__device__ __forceinline__ void part_of(int part, int parts, int &lo, int &hi) {
  const int n = hi - lo, at = lo;
  if (parts == 1) return;
  lo = at + (int)((uint32_t)(n * part) / (uint32_t)parts);  // below 2^26 steps, at most 16 parts
  hi = at + (int)((uint32_t)(n * (part + 1)) / (uint32_t)parts);
}

// a row of a part's binary32 results, [part][head][row][D]
template <int D>
__device__ __forceinline__ float *part_row(float *p, int part, int heads, int head, int64_t rows, int64_t row) {
  return p + (((int64_t)part * heads + head) * rows + row) * D;
}
template <int D>
__device__ __forceinline__ void store_part(float *row, const f32x16 *acc, float f, int dim, int h) {
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int d = dt * 32 + 8 * g + 4 * h;
      if (d < dim)
        *reinterpret_cast<float4 *>(row + d) =
            make_float4(acc[dt][4 * g] * f, acc[dt][4 * g + 1] * f, acc[dt][4 * g + 2] * f, acc[dt][4 * g + 3] * f);
    }
}

// -------------------------------------------------------------- forward ----
constexpr int kQueries = 128;  // queries of a workgroup: 32 per wave

// One wave holds 32 queries as columns: scores^T = K Q^T, o^T = V^T p^T.
// Running maximum and sum per query stay in its two lanes.  Two waves per SIMD:
// while one waits or takes exponentials the other multiplies.
// 8192 tokens, 40 heads of 128, 8 key heads, causal: 650-711 us on several devices, 0.97-1.06
// PFLOP/s, the MFMA busy in 57 % of the cycles at 1.82 GHz.  Power bounds it: 8 % fewer
// cycles (operands read ahead) left the time as it was and lowered the clock.
// Eight waves to a workgroup, which halves the transfers, took the same time;
// 64 queries to a wave at one wave per SIMD, which halves the LDS reads, 807 us.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attention_kernel(AttnArgs a) {
  __shared__ __align__(16) uint8_t lds[4 * Tile<D>::bytes(kTile)];
  constexpr uint32_t kB = Tile<D>::bytes(kTile);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const Work w = work_of(a, a.q_parts, true);
  const Seq s = sequence(a, w.b);
  const int first = (a.q_tiles - 1 - w.level) * kQueries;  // the later, the more keys in sight
  if (first >= s.nq) return;
  const int last = (first + kQueries < s.nq ? first + kQueries : s.nq) - 1, off = s.nk - s.nq;
  uint32_t of_head = (uint32_t)w.head;
  split_off(of_head, a.by_group);
  const int hk = (int)of_head, chunks = a.dim / 8;
  const uint16_t *kh = at(a.k, s.bk, s.k0, hk), *vh = at(a.v, s.bk, s.k0, hk);

  const int mine = first + wave * 32 + (lane & 31), qi = mine < s.nq ? mine : s.nq - 1;
  bf16x8 q[D / 16];
  const uint16_t *qrow = at(a.q, s.bq, s.q0 + qi, w.head);
  load_row<D>(qrow, chunks, h, q);

  int lo, hi, unused, begin, end;
  sight(a, qi, s.nk, off, lo, hi);
  sight(a, first, s.nk, off, begin, unused);
  sight(a, last, s.nk, off, unused, end);
  // what all, and what any, of the wave's queries see
  const int w0 = first + wave * 32 < s.nq ? first + wave * 32 : s.nq - 1, w1 = w0 + 31 < s.nq ? w0 + 31 : s.nq - 1;
  int any_lo, all_lo, any_hi, all_hi;
  sight(a, w0, s.nk, off, any_lo, all_hi);
  sight(a, w1, s.nk, off, all_lo, any_hi);

  f32x16 o[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) o[dt] = zero16();
  float top = kLow, sum = 0.0f;
  const float c2 = a.scale * kLog2e;
  Reads<D> in(lane, lds_addr(lds));

  int t0 = begin / kTile, t1 = end > begin ? (end + kTile - 1) / kTile : t0;
  part_of(w.part, a.q_parts, t0, t1);
  if (t0 < t1) {
    fetch_tile<D, kTile>(kh, a.k.st, t0 * kTile, s.nk, chunks, lds_addr(lds), wave, lane);
    fetch_tile<D, kTile>(vh, a.v.st, t0 * kTile, s.nk, chunks, lds_addr(lds) + kB, wave, lane);
  }
  for (int t = t0; t < t1; ++t) {
    const int stage = (t - t0) & 1, k0 = t * kTile;
    if (t > t0) in.move(stage ? 2 * kB : 0u - 2 * kB);
    tile_barrier();  // this tile is in LDS, and every wave has read the previous one
    if (t + 1 < t1) {
      fetch_tile<D, kTile>(kh, a.k.st, k0 + kTile, s.nk, chunks, lds_addr(lds) + (uint32_t)(stage ^ 1) * 2 * kB, wave, lane);
      fetch_tile<D, kTile>(vh, a.v.st, k0 + kTile, s.nk, chunks, lds_addr(lds) + (uint32_t)(stage ^ 1) * 2 * kB + kB, wave, lane);
    }
    if (k0 >= any_hi || k0 + kTile <= any_lo) continue;  // nothing in the wave's sight
    f32x16 p[2] = {zero16(), zero16()};
    bf16x8 kf[2 * (D / 16)];
#pragma unroll
    for (int c = 0; c < 2 * (D / 16); ++c) kf[c] = in.rows(0, (c & 1) * 32, c >> 1);
#pragma unroll
    for (int c = 0; c < 2 * (D / 16); ++c) p[c & 1] = mfma(kf[c], q[c >> 1], p[c & 1]);
    // half of the operands ahead of the products, the others between them
    __builtin_amdgcn_sched_group_barrier(kDsRead, D / 16, 0);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, D / 16, 0);
    hide(p, lo - k0, hi - k0, k0 < all_lo, k0 + kTile > all_hi, h);
    float m = fmaxf(p[0][0], p[1][0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) m = fmaxf(m, fmaxf(p[0][i], p[1][i]));
    m = swapped32(m, [](float x, float y) { return fmaxf(x, y); }) * c2;
    // The exponents' reference follows the maximum only when that has risen by
    // more than 8 (a factor of 256 in p): results do not depend on it
    if (__any(m > top + 8.0f)) {
      const float next = fmaxf(top, m), f = __builtin_amdgcn_exp2f(top - next);
      top = next;
      sum *= f;
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[dt][i] *= f;
    }
    bf16x8 vf[4][D / 32];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) vf[c][dt] = in.cols(kB, c * 16, dt);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int i = 8 * (c & 1); i < 8 * (c & 1) + 8; ++i) {
        p[c >> 1][i] = __builtin_amdgcn_exp2f(fmaf(p[c >> 1][i], c2, -top));
        sum += p[c >> 1][i];
      }
      const bf16x8 b = pack8(p[c >> 1], 8 * (c & 1));  // sum has them unrounded
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) o[dt] = mfma(vf[c][dt], b, o[dt]);
    }
    // the first 16 keys' operands and probabilities, then each 16 keys'
    // products between the next ones'
    __builtin_amdgcn_sched_group_barrier(kDsRead, D / 16, 0);
    __builtin_amdgcn_sched_group_barrier(kValu, 28, 0);
#pragma unroll
    for (int c = 0; c < 3; ++c) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) {
        __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kValu, 28 / (D / 32), 0);
      }
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, D / 32, 0);
  }
  sum = swapped32(sum, [](float x, float y) { return x + y; });
  if (mine >= s.nq) return;
  const bool none = sum == 0.0f;
  const float f = none ? 0.0f : 1.0f / sum, lse = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
  const int64_t row = first_row(a, s, w.b) + mine;
  if (a.q_parts > 1) {
    store_part<D>(part_row<D>(a.q_part, w.part, a.heads, w.head, a.total_q, row), o, f, a.dim, h);
    if (h == 0) a.lse_part[((int64_t)w.part * a.heads + w.head) * a.total_q + row] = lse;
    return;
  }
  store_cols<D>(at(a.o, s.bq, s.q0 + mine, w.head), o, f, a.dim, h);
  if (h == 0) a.lse[(int64_t)w.head * a.total_q + row] = lse;
}

// Parts joined: 16 rows of a head to a workgroup, 16 threads to a row, four
// parts' loads in flight.
// WHAT = kJoinO: o = sum_p exp(lse_p - lse) o_p, lse = log sum_p exp(lse_p);
// else sums over the parts in their order: dQ, or dK (blockIdx.y = 0) and dV.
enum { kJoinO, kJoinQ, kJoinKV };
constexpr int kJoinRows = kThreads / 16;
template <int D, int WHAT>
__global__ __launch_bounds__(kThreads) void attention_join_kernel(AttnArgs a) {
  const bool kv = WHAT == kJoinKV, v = kv && blockIdx.y;
  const int heads = kv ? a.kv_heads : a.heads, parts = kv ? a.k_parts : a.q_parts;
  const int64_t rows = kv ? a.total_k : a.total_q;
  const int tiles = ((kv ? a.k_len : a.q_len) + kJoinRows - 1) / kJoinRows, c = (int)threadIdx.x & 15;
  uint32_t w = blockIdx.x;
  const int i = (int)(w % (uint32_t)tiles) * kJoinRows + (int)(threadIdx.x >> 4);
  w /= (uint32_t)tiles;
  const int b = (int)(w % (uint32_t)a.batch), head = (int)(w / (uint32_t)a.batch);
  const Seq s = sequence(a, b);
  const int n = kv ? s.nk : s.nq;
  if (i >= n || c * 8 >= a.dim) return;
  const int64_t row = (!a.cu_q ? (int64_t)b * n : kv ? s.k0 : s.q0) + i;
  float *from = kv ? (v ? a.v_part : a.k_part) : a.q_part, sum[8] = {};
  if constexpr (WHAT == kJoinO) {
    const float *lse = a.lse_part + (int64_t)head * rows + row;
    const int64_t pitch = (int64_t)heads * rows;
    float top = -INFINITY, total = 0.0f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) top = fmaxf(top, lse[p * pitch]);
    if (top > -INFINITY) {
#pragma unroll 4
      for (int p = 0; p < parts; ++p) {
        const float f = __builtin_amdgcn_exp2f((lse[p * pitch] - top) * kLog2e);
        float x[8];
        load8(part_row<D>(from, p, heads, head, rows, row) + c * 8, x);
        total += f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = fmaf(f, x[j], sum[j]);
      }
    }
    const float f = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] *= f;
    if (c == 0) a.lse[(int64_t)head * a.total_q + row] = total > 0.0f ? top + __builtin_amdgcn_logf(total) * kLn2 : -INFINITY;
  } else {
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      float x[8];
      load8(part_row<D>(from, p, heads, head, rows, row) + c * 8, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += x[j];
    }
  }
  const Heads &to = kv ? (v ? a.dv : a.dk) : WHAT == kJoinO ? a.o : a.dq;
  store8(at(to, kv ? s.bk : s.bq, (kv ? s.k0 : s.q0) + i, head) + c * 8, sum);
}

// ------------------------------------------------------------- gradient ----
// dQ (2 x 4096 tokens, 40 heads of 128, 8 key heads, causal: 477-506 us, 1.02-1.08
// PFLOP/s over its three products, the MFMA busy in 60 % of the cycles: power).
// A wave holds 32 queries as columns; scores^T = K Q^T, dP^T = V dO^T,
// dQ^T = K^T dS^T.  It forms delta = sum_d do * o on the way, and leaves
// -delta and -lse / scale, from which the accumulators of the dK, dV pass start.
template <int D>
__global__ __launch_bounds__(kThreads, 2) void attention_dq_kernel(AttnArgs a) {
  __shared__ __align__(16) uint8_t lds[4 * Tile<D>::bytes(kTile)];
  constexpr uint32_t kB = Tile<D>::bytes(kTile);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const Work w = work_of(a, a.q_parts, true);
  const Seq s = sequence(a, w.b);
  const int first = (a.q_tiles - 1 - w.level) * kQueries;  // the later, the more keys in sight
  if (first >= s.nq) return;
  const int last = (first + kQueries < s.nq ? first + kQueries : s.nq) - 1, off = s.nk - s.nq;
  uint32_t of_head = (uint32_t)w.head;
  split_off(of_head, a.by_group);
  const int hk = (int)of_head, chunks = a.dim / 8;
  const uint16_t *kh = at(a.k, s.bk, s.k0, hk), *vh = at(a.v, s.bk, s.k0, hk);

  const int mine = first + wave * 32 + (lane & 31), qi = mine < s.nq ? mine : s.nq - 1;
  bf16x8 q[D / 16], g[D / 16];
  const uint16_t *qrow = at(a.q, s.bq, s.q0 + qi, w.head), *grow = at(a.d_o, s.bq, s.q0 + qi, w.head);
  load_row<D>(qrow, chunks, h, q);
  load_row<D>(grow, chunks, h, g);
  const uint16_t *orow = at(a.o, s.bq, s.q0 + qi, w.head);
  float delta = 0.0f;
  bf16x8 o[D / 16];
  load_row<D>(orow, chunks, h, o);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    const uint4 x = __builtin_bit_cast(uint4, o[c]), y = __builtin_bit_cast(uint4, g[c]);
#pragma unroll
    for (int j = 0; j < 8; ++j) delta = fmaf(bf16_at(x, j), bf16_at(y, j), delta);
  }
  delta = swapped32(delta, [](float x, float y) { return x + y; });
  const int64_t stat = (int64_t)w.head * a.total_q + first_row(a, s, w.b) + qi;
  const float lse = a.lse[stat], start = lse == -INFINITY ? 0.0f : -lse * kLog2e;  // all of such a row is masked
  if (h == 0 && mine < s.nq && w.part == 0) {
    a.minus_delta[stat] = -delta;
    a.minus_lse[stat] = lse == -INFINITY ? 0.0f : -lse / a.scale;
  }

  int lo, hi, unused, begin, end;
  sight(a, qi, s.nk, off, lo, hi);
  sight(a, first, s.nk, off, begin, unused);
  sight(a, last, s.nk, off, unused, end);
  const int w0 = first + wave * 32 < s.nq ? first + wave * 32 : s.nq - 1, w1 = w0 + 31 < s.nq ? w0 + 31 : s.nq - 1;
  int any_lo, all_lo, any_hi, all_hi;
  sight(a, w0, s.nk, off, any_lo, all_hi);
  sight(a, w1, s.nk, off, all_lo, any_hi);

  f32x16 acc[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) acc[dt] = zero16();
  const float c2 = a.scale * kLog2e;
  Reads<D> in(lane, lds_addr(lds));
  int t0 = begin / kTile, t1 = end > begin ? (end + kTile - 1) / kTile : t0;
  part_of(w.part, a.q_parts, t0, t1);
  if (t0 < t1) {
    fetch_tile<D, kTile>(kh, a.k.st, t0 * kTile, s.nk, chunks, lds_addr(lds), wave, lane);
    fetch_tile<D, kTile>(vh, a.v.st, t0 * kTile, s.nk, chunks, lds_addr(lds) + kB, wave, lane);
  }
  for (int t = t0; t < t1; ++t) {
    const int stage = (t - t0) & 1, k0 = t * kTile;
    if (t > t0) in.move(stage ? 2 * kB : 0u - 2 * kB);
    tile_barrier();
    if (t + 1 < t1) {
      fetch_tile<D, kTile>(kh, a.k.st, k0 + kTile, s.nk, chunks, lds_addr(lds) + (uint32_t)(stage ^ 1) * 2 * kB, wave, lane);
      fetch_tile<D, kTile>(vh, a.v.st, k0 + kTile, s.nk, chunks, lds_addr(lds) + (uint32_t)(stage ^ 1) * 2 * kB + kB, wave, lane);
    }
    if (k0 >= any_hi || k0 + kTile <= any_lo) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // as in the dK, dV pass: operands two steps ahead, products between the
      // exponentials of the other 16 keys
      constexpr int kN = D / 16, kM = D / 32;
      f32x16 pd[1] = {zero16()}, d = zero16();
      f32x16 &p = pd[0];
      bf16x8 ka[kN], va[kN], t[2 * kM];
      const auto read_step = [&](int c) {
        ka[c] = in.rows(0, u * 32, c);
        va[c] = in.rows(kB, u * 32, c);
      };
      const auto read_cols = [&](int i) { t[i] = in.cols(0, u * 32 + i / kM * 16, i % kM); };
      read_step(0);
      read_step(1);
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (c + 2 < kN)
          read_step(c + 2);
        else
          read_cols(c + 2 - kN);
        p = mfma(ka[c], q[c], p);
        d = mfma(va[c], g[c], d);
        __builtin_amdgcn_sched_barrier(0);
      }
      hide(pd, lo - k0 - u * 32, hi - k0 - u * 32, k0 + u * 32 < all_lo, k0 + u * 32 + 32 > all_hi, h);
      const auto element = [&](int i) { p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], c2, start)) * (d[i] - delta); };
#pragma unroll
      for (int i = 0; i < 8; ++i) element(i);
      bf16x8 b = pack8(p, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 2 * kM; ++i) {
        if (i + 2 < 2 * kM) read_cols(i + 2);
        acc[i % kM] = mfma(t[i], b, acc[i % kM]);
        if (i < kM) {
#pragma unroll
          for (int j = 0; j < 8 / kM; ++j) element(8 + i * (8 / kM) + j);
        }
        if (i == kM - 1) b = pack8(p, 8);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (mine >= s.nq) return;
  if (a.q_parts > 1)
    store_part<D>(part_row<D>(a.q_part, w.part, a.heads, w.head, a.total_q, first_row(a, s, w.b) + mine), acc, a.scale,
                  a.dim, h);
  else
    store_cols<D>(at(a.dq, s.bq, s.q0 + mine, w.head), acc, a.scale, a.dim, h);
}

// dK, dV: a wave holds 32 keys as columns; scores = Q K^T, dP = dO V^T,
// dV^T = dO^T P, dK^T = Q^T dS, summed over the query heads of the key head.
// The keys' operands stay in registers and the values' in LDS: with both in
// registers nothing is left of the 256 that two waves per SIMD have each to
// read operands ahead.  Queries come in tiles of 32 rows (D = 128), so that two
// workgroups fit a compute unit's LDS, or 64 (D = 64).
// The same tokens as for dQ: 661-700 us, 0.98-1.04 PFLOP/s over its four
// products, and 25 to join them with the queries in two parts (1254 us as first
// written, one wave per SIMD; 898 with two and both operands in registers; 775
// with values in LDS and one part).
constexpr int kKeys = 128;  // keys of a workgroup

template <int D>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void attention_dkv_kernel(AttnArgs a) {
  constexpr int kRows = D == 128 ? 32 : 64;
  constexpr uint32_t kB = Tile<D>::bytes(kRows), kV = Tile<D>::bytes(kKeys);
  __shared__ __align__(16) uint8_t lds[4 * kB + kV];
  __shared__ __align__(16) float stats[2][2][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
  const int group = (int)a.by_group.d;
  const Work w = work_of(a, a.k_parts, false);
  const int hk = w.head;
  const Seq s = sequence(a, w.b);
  // counted from the sequence's last tile: the earlier, the more queries see it
  const int first = ((s.nk + kKeys - 1) / kKeys - a.k_tiles + w.level) * kKeys;
  if (first < 0 || first >= s.nk) return;
  const int last = (first + kKeys < s.nk ? first + kKeys : s.nk) - 1, off = s.nk - s.nq;
  const int chunks = a.dim / 8;

  const int mine = first + wave * 32 + (lane & 31), ki = mine < s.nk ? mine : s.nk - 1;
  bf16x8 k[D / 16];
  const uint16_t *krow = at(a.k, s.bk, s.k0 + ki, hk), *vrow = at(a.v, s.bk, s.k0 + ki, hk);
  const uint32_t v_at = lds_addr(lds) + 4 * kB + (uint32_t)wave * Tile<D>::bytes(32);
  Reads<D> in(lane, lds_addr(lds));
  const Reads<D> values(lane, v_at);  // the wave's own 32 rows, written and read by it alone
  load_row<D>(krow, chunks, h, k);
  {
    bf16x8 v[D / 16];
    load_row<D>(vrow, chunks, h, v);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) values.set_row(c, v[c]);
  }
  // the queries [lo, hi) that see key j: j - off <= i < j - off + window, with causal
  const auto seen_by = [&](int j, int &lo, int &hi) {
    lo = a.causal ? within(j - off, s.nq) : 0;
    hi = a.window ? within(j - off + a.window, s.nq) : s.nq;
  };
  int begin, end, all_lo, all_hi, unused;
  seen_by(first, begin, unused);
  seen_by(last, unused, end);
  seen_by(first + wave * 32, unused, all_hi);
  seen_by(first + wave * 32 + 31, all_lo, unused);
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) {
    dk[dt] = zero16();
    dv[dt] = zero16();
  }
  const float c2 = a.scale * kLog2e;
  const int t0 = begin / kRows, t1 = end > begin ? (end + kRows - 1) / kRows : t0;
  const int64_t row0 = first_row(a, s, w.b);
  const auto fetch = [&](int head, int t, int stage) {
    const int i0 = t * kRows;
    const uint32_t to = lds_addr(lds) + (uint32_t)stage * 2 * kB;
    fetch_tile<D, kRows>(at(a.q, s.bq, s.q0, head), a.q.st, i0, s.nq, chunks, to, wave, lane);
    fetch_tile<D, kRows>(at(a.d_o, s.bq, s.q0, head), a.d_o.st, i0, s.nq, chunks, to + kB, wave, lane);
    if (wave < 2) {
      const float *src = (wave ? a.minus_delta : a.minus_lse) + (int64_t)head * a.total_q + row0 + i0;
      const int left = s.nq - i0 - 1;
      dma4(uniform_ptr((const uint8_t *)src), (uint32_t)(lane < left ? lane : left) * 4u,
           __builtin_amdgcn_readfirstlane(lds_addr(stats[stage][wave])));
    }
  };
  // steps: the query tiles of each of the query heads in turn
  int step = 0, steps = (t1 - t0) * group;
  part_of(w.part, a.k_parts, step, steps);
  int head = hk * group, t = t0, stage = 0;
  if (step < steps) {
    if (step > 0) {
      head += step / (t1 - t0);
      t += step % (t1 - t0);
    }
    fetch(head, t, 0);
  }
  for (; step < steps; ++step) {
    const int i0 = t * kRows;
    tile_barrier();  // this tile is in LDS, and every wave has read the previous one
    if (++t == t1) {
      t = t0;
      ++head;
    }
    if (step + 1 < steps) fetch(head, t, stage ^ 1);
#pragma unroll
    for (int u = 0; u < kRows / 32; ++u) {
      // the accumulators start from -lse / scale and -delta
      constexpr int kN = D / 16;
      f32x16 pd[1], d;
      f32x16 &p = pd[0];
      int l = lane;
      asm volatile("" : "+v"(l));  // what is formed of it stays out of registers between tiles
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float4 x = *reinterpret_cast<const float4 *>(&stats[stage][0][32 * u + 8 * b + 4 * (l >> 5)]);
        const float4 y = *reinterpret_cast<const float4 *>(&stats[stage][1][32 * u + 8 * b + 4 * (l >> 5)]);
        p[4 * b] = x.x, p[4 * b + 1] = x.y, p[4 * b + 2] = x.z, p[4 * b + 3] = x.w;
        d[4 * b] = y.x, d[4 * b + 1] = y.y, d[4 * b + 2] = y.z, d[4 * b + 3] = y.w;
      }
      // Operands are read two steps ahead of their products.  The order below
      // is the one wanted; scheduling stays within a step.
      bf16x8 qa[kN], ga[kN], va[kN], t[2 * kN];
      const auto read_step = [&](int c) {
        qa[c] = in.rows(0, 32 * u, c);
        ga[c] = in.rows(kB, 32 * u, c);
        va[c] = values.rows(0, 0, c);
      };
      // product 2 dt + w of the 16 queries c: w = 0: dV from dO, 1: dK from Q
      const auto read_cols = [&](int i) { t[i] = in.cols(i & 1 ? 0 : kB, 32 * u + i / kN * 16, i % kN / 2); };
      read_step(0);
      read_step(1);
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (c + 2 < kN)
          read_step(c + 2);
        else
          read_cols(2 * (c + 2 - kN)), read_cols(2 * (c + 2 - kN) + 1);
        p = mfma(qa[c], k[c], p);
        d = mfma(ga[c], va[c], d);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i0 + 32 * u + 32 > all_hi || i0 + 32 * u < all_lo) {
        int lo, hi;
        asm volatile("" : "+v"(l));
        seen_by(first + wave * 32 + (l & 31), lo, hi);
        hide(pd, lo - i0 - 32 * u, hi - i0 - 32 * u, i0 + 32 * u < all_lo, i0 + 32 * u + 32 > all_hi, l >> 5);
      }
      const auto element = [&](int i) {
        p[i] = __builtin_amdgcn_exp2f(p[i] * c2);
        d[i] = p[i] * d[i];
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) element(i);
      bf16x8 b0 = pack8(p, 0), b1 = pack8(d, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 2 * kN; ++i) {
        if (i + 4 < 2 * kN) read_cols(i + 4);
        f32x16 &acc = i & 1 ? dk[i % kN / 2] : dv[i % kN / 2];
        acc = mfma(t[i], i & 1 ? b1 : b0, acc);
        if (i < kN) {
#pragma unroll
          for (int j = 0; j < 8 / kN; ++j) element(8 + i * (8 / kN) + j);
        }
        if (i == kN - 1) {
          b0 = pack8(p, 8);
          b1 = pack8(d, 8);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    in.move(stage ? 0u - 2 * kB : 2 * kB);
    stage ^= 1;
  }
  if (mine >= s.nk) return;
  if (a.k_parts > 1) {
    const int64_t row = (a.cu_q ? s.k0 : (int64_t)w.b * a.k_len) + mine;
    store_part<D>(part_row<D>(a.k_part, w.part, a.kv_heads, hk, a.total_k, row), dk, a.scale, a.dim, h);
    store_part<D>(part_row<D>(a.v_part, w.part, a.kv_heads, hk, a.total_k, row), dv, 1.0f, a.dim, h);
    return;
  }
  store_cols<D>(at(a.dk, s.bk, s.k0 + mine, hk), dk, a.scale, a.dim, h);
  store_cols<D>(at(a.dv, s.bk, s.k0 + mine, hk), dv, 1.0f, a.dim, h);
}

}  // namespace

namespace {

int64_t tiles_of(int64_t n) { return (n + 127) / 128; }

// Workgroups that a pass over the rows of `heads` heads has without parts
// (packed: an estimate, the lengths being on the device).
int64_t units(const AttnArgs &a, int64_t len, int64_t total, int heads) {
  if (!a.cu_q) return heads * a.batch * tiles_of(len);
  const int64_t most = tiles_of(total) > a.batch ? tiles_of(total) : a.batch;
  return heads * (most > 0 ? most : 1);
}
// keys that a query has in sight at most
int64_t sight_of(const AttnArgs &a) { return a.window && a.window < a.k_len ? a.window : a.k_len; }

}  // namespace

// Keys split where the queries' tiles alone leave compute units idle: parts of
// at least 8 tiles of 64 keys, up to 512 workgroups, joined by a second kernel.
// (Parts of 4 tiles: 1 query on 512 keys, 8 heads, 18 us against 15, 7 packed
// documents of 2000 tokens 27 against 20, 1000 tokens with 8 heads 23 against 24.)
int attention_q_parts(const AttnArgs &a) {
  const int64_t n = units(a, a.q_len, a.total_q, a.heads), steps = sight_of(a) / kTile;
  int64_t parts = n >= 256 ? 1 : 512 / n;
  if (parts > steps / 8) parts = steps / 8;
  return (int)(parts < 1 ? 1 : parts > 16 ? 16 : parts);
}
// Queries split for dK and dV: parts of at least 8 steps of 32 queries, up to
// 512 workgroups, what the compute units hold of them (4 x 500 tokens, 20 heads
// of 128, 4 key heads: 63 us against 114 with one part; 2 x 4096 without a
// causal mask: two parts cost the 28 us that joining them takes).  Causal passes
// whose tiles weigh unevenly gain from a second set of workgroups, dealt to
// whichever compute unit is done, where that makes no more than two rounds of
// them and parts are long enough to pay for the join.  Up to 512 tiles of keys,
// heads of 128: 2 x 4096 tokens, 40 heads, 8 key heads (160 steps a part) 1251 ->
// 1182 us, 8192, 8 and 8 (64) 532 -> 527, 4096, 24 and 4 (48) 407 -> 396, but 2 x
// 3200, 24 and 8 (50) 454 -> 462; below 48, 4096, 20 and 4 (40) 350 -> 342, but
// 3000, 16 and 4 (17) 183 -> 193.  More tiles than 512 have a round and a part as
// they are: 6144 tokens, 16 and 16 (48) 528 -> 575 with twice as many, 12288, 8
// and 8 (96) 1010 -> 1044, 14336 (112) 1416 -> 1415.
int attention_k_parts(const AttnArgs &a) {
  const int64_t n = units(a, a.k_len, a.total_k, a.kv_heads);
  const int64_t rows = a.window && a.window < a.q_len ? a.window : a.causal ? (a.q_len + 1) / 2 : a.q_len;
  const int64_t steps = rows / 32 * (a.heads / a.kv_heads), twice = (1024 + n - 1) / n;
  int64_t parts = a.causal && n <= 512 && steps >= 48 * twice ? twice : (512 + n - 1) / n;
  if (parts > steps / 8) parts = steps / 8;
  return (int)(parts < 1 ? 1 : parts > 16 ? 16 : parts);
}

namespace {
unsigned join_groups(const AttnArgs &a, int heads, int len) {
  return (unsigned)((int64_t)a.batch * heads * ((len + kJoinRows - 1) / kJoinRows));
}
template <int D>
hipError_t forward(const AttnArgs &a, unsigned rows, hipStream_t s) {
  attention_kernel<D><<<rows * (unsigned)a.q_parts, kThreads, 0, s>>>(a);
  if (a.q_parts > 1) attention_join_kernel<D, kJoinO><<<join_groups(a, a.heads, a.q_len), kThreads, 0, s>>>(a);
  return hipGetLastError();
}
template <int D>
hipError_t backward(const AttnArgs &a, unsigned rows, unsigned keys, hipStream_t s) {
  // packed sequences may have no queries, or no keys: nothing of theirs to write
  if (rows) attention_dq_kernel<D><<<rows * (unsigned)a.q_parts, kThreads, 0, s>>>(a);
  if (keys) attention_dkv_kernel<D><<<keys * (unsigned)a.k_parts, kThreads, 0, s>>>(a);
  if (rows && a.q_parts > 1) attention_join_kernel<D, kJoinQ><<<join_groups(a, a.heads, a.q_len), kThreads, 0, s>>>(a);
  if (keys && a.k_parts > 1)
    attention_join_kernel<D, kJoinKV><<<dim3(join_groups(a, a.kv_heads, a.k_len), 2), kThreads, 0, s>>>(a);
  return hipGetLastError();
}
}  // namespace

static_assert(kQueries == 128 && kKeys == 128, "tiles_of");

hipError_t launch_attention(const AttnArgs &a, hipStream_t s) {
  const unsigned rows = (unsigned)(a.batch * a.heads * tiles_of(a.q_len));
  return a.dim <= 64 ? forward<64>(a, rows, s) : forward<128>(a, rows, s);
}

hipError_t launch_attention_backward(const AttnArgs &a, hipStream_t s) {
  const unsigned rows = (unsigned)(a.batch * a.heads * tiles_of(a.q_len));
  const unsigned keys = (unsigned)(a.batch * a.kv_heads * tiles_of(a.k_len));
  return a.dim <= 64 ? backward<64>(a, rows, keys, s) : backward<128>(a, rows, keys, s);
}

}  // namespace nvfp4
