// C ABI of the block operators: argument validation on the host, then kernel
// launches on the caller's stream.  The entry points and their contracts are
// declared and documented in include/nvfp4.h.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "block_kernels.hpp"
#include "nvfp4.h"

using namespace nvfp4;

namespace {

bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(int32_t t) { return t == NVFP4_F32 || t == NVFP4_BF16; }
size_t size_of(int32_t t) { return t == NVFP4_BF16 ? 2 : 4; }

// the launches' status; with NVFP4_SYNC_CHECK=1 (read once) also the kernels'
int finish(hipError_t e, hipStream_t s) {
  if (e != hipSuccess) return NVFP4_E_HIP;
  static const bool check = [] {
    const char *v = getenv("NVFP4_SYNC_CHECK");
    return v && v[0] == '1';
  }();
  if (check && (hipStreamSynchronize(s) != hipSuccess || hipGetLastError() != hipSuccess)) return NVFP4_E_HIP;
  return NVFP4_OK;
}

// ---------------------------------------------------------------- rope ----
bool batched(const nvfp4_qk_rope_args &a) { return !a.cu && a.batch > 1; }

int check_rope_heads(const nvfp4_heads &t, const nvfp4_qk_rope_args &a, int64_t heads, bool output) {
  if (!t.data && a.batch * a.tokens) return NVFP4_E_NULL;
  if (t.token_stride < 0 || t.head_stride < 0 || (batched(a) && t.batch_stride < 0)) return NVFP4_E_LD;
  const int64_t d = a.head_dim;
  if (output && (t.token_stride < d || (heads > 1 && t.head_stride < d) || (batched(a) && t.batch_stride < d)))
    return NVFP4_E_LD;
  if (!aligned(t.data, 16) || t.token_stride % 8 || t.head_stride % 8 || (batched(a) && t.batch_stride % 8))
    return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

// whether output o may be written beside t: they begin apart, or every element
// stands in the place of its own
bool rope_fits(const nvfp4_heads &o, int32_t o_type, const nvfp4_heads &t, int32_t t_type, int64_t heads,
               const nvfp4_qk_rope_args &a) {
  if (o.data != t.data || !o.data) return true;
  return o_type == t_type && o.token_stride == t.token_stride && (heads == 1 || o.head_stride == t.head_stride) &&
         (!batched(a) || o.batch_stride == t.batch_stride);
}

int check_rope(const nvfp4_qk_rope_args *a, bool backward) {
  if (!a) return NVFP4_E_NULL;
  const nvfp4_rope_heads *sides[2] = {&a->q, &a->k};
  const int64_t most = (int64_t)1 << 31;
  if (a->batch < 1 || a->batch >= most || a->tokens < 0 || a->tokens >= most) return NVFP4_E_SHAPE;
  if (!a->cu && a->batch * a->tokens >= most) return NVFP4_E_SHAPE;
  for (const nvfp4_rope_heads *t : sides)
    if (t->heads < 0 || t->heads > 65535) return NVFP4_E_SHAPE;
  if (!a->q.heads && !a->k.heads) return NVFP4_E_SHAPE;
  if (a->head_dim < 8 || a->head_dim > 128 || a->head_dim % 8) return NVFP4_E_UNSUPPORTED;
  if (a->rot_dim < 0 || a->rot_dim > a->head_dim || a->rot_dim % 2) return NVFP4_E_UNSUPPORTED;
  if ((a->interleaved != 0 && a->interleaved != 1) || !dtype_ok(a->x_dtype) || !dtype_ok(a->w_dtype))
    return NVFP4_E_UNSUPPORTED;
  if (a->positions && a->cu) return NVFP4_E_UNSUPPORTED;
  const bool norm = a->q.heads ? a->q.weight : a->k.weight;
  if (a->q.heads && a->k.heads && !a->q.weight != !a->k.weight) return NVFP4_E_NULL;
  if (a->rot_dim && !a->freqs) return NVFP4_E_NULL;
  if (!a->rot_dim && !norm) return NVFP4_E_UNSUPPORTED;  // nothing to do
  if (!aligned(a->freqs, 8) || !aligned(a->positions, 8) || !aligned(a->cu, 4)) return NVFP4_E_ALIGN;
  if (!isfinite(a->magnitude)) return NVFP4_E_VALUE;
  if (norm && (!(a->eps >= FLT_MIN) || !isfinite(a->eps))) return NVFP4_E_VALUE;
  for (const nvfp4_rope_heads *t : sides) {
    if (!t->heads) continue;
    if (t->weight && !aligned(t->weight, size_of(a->w_dtype))) return NVFP4_E_ALIGN;
    if (t->dweight && (!backward || !t->weight)) return NVFP4_E_UNSUPPORTED;
    if (!aligned(t->dweight, 4)) return NVFP4_E_ALIGN;
    int st = check_rope_heads(t->y, *a, t->heads, !backward);
    if (!st && (!backward || norm)) st = check_rope_heads(t->x, *a, t->heads, false);
    if (!st && backward) st = check_rope_heads(t->dx, *a, t->heads, true);
    if (st) return st;
  }
  // an element is read by the lane that writes its place
  for (int i = 0; i < 2; ++i) {
    const nvfp4_rope_heads &t = *sides[i], &o = *sides[1 - i];
    if (!t.heads) continue;
    const nvfp4_heads &out = backward ? t.dx : t.y;
    const int32_t type = backward ? a->x_dtype : NVFP4_BF16;
    if ((!backward || norm) && !rope_fits(out, type, t.x, a->x_dtype, t.heads, *a)) return NVFP4_E_UNSUPPORTED;
    if (backward && !rope_fits(out, type, t.y, NVFP4_BF16, t.heads, *a)) return NVFP4_E_UNSUPPORTED;
    if (!o.heads || !out.data) continue;
    if (out.data == (backward ? o.dx : o.y).data) return NVFP4_E_UNSUPPORTED;
    if ((!backward || norm) && out.data == o.x.data) return NVFP4_E_UNSUPPORTED;
    if (backward && out.data == o.y.data) return NVFP4_E_UNSUPPORTED;
    if (t.dweight && t.dweight == o.dweight) return NVFP4_E_UNSUPPORTED;
  }
  return NVFP4_OK;
}

RopeArgs rope_args(const nvfp4_qk_rope_args &a) {
  RopeArgs r = {};
  const nvfp4_rope_heads *sides[2] = {&a.q, &a.k};
  r.positions = a.positions;
  r.cu = a.cu;
  r.freqs = a.freqs;
  r.tokens = a.tokens;
  r.total = a.cu ? a.tokens : a.batch * a.tokens;
  r.batch = (int)a.batch;
  r.dim = a.head_dim;
  r.rot = a.rot_dim;
  r.interleaved = a.interleaved;
  r.units = a.interleaved ? (a.head_dim + 15) / 16 : (a.rot_dim / 2 + 7) / 8 + (a.head_dim - a.rot_dim + 15) / 16;
  r.x_bf16 = a.x_dtype == NVFP4_BF16;
  r.w_bf16 = a.w_dtype == NVFP4_BF16;
  r.eps = a.eps;
  r.inv_dim = 1.0f / (float)a.head_dim;
  r.magnitude = a.magnitude;
  for (int i = 0; i < 2; ++i) {
    const nvfp4_rope_heads &t = *sides[i];
    RopeSide &o = r.side[i];
    o.heads = (int)t.heads;
    if (!t.heads) continue;
    o.x = t.x.data;
    o.y = (uint16_t *)t.y.data;
    o.dx = t.dx.data;
    o.weight = t.weight;
    o.dweight = t.dweight;
    o.x_b = t.x.batch_stride, o.x_t = t.x.token_stride, o.x_h = t.x.head_stride;
    o.y_b = t.y.batch_stride, o.y_t = t.y.token_stride, o.y_h = t.y.head_stride;
    o.dx_b = t.dx.batch_stride, o.dx_t = t.dx.token_stride, o.dx_h = t.dx.head_stride;
  }
  rope_plan(r);
  return r;
}

size_t rope_parts(RopeArgs &r, void *workspace) {
  size_t used = 0;
  for (RopeSide &t : r.side) {
    if (!t.dweight) continue;
    t.parts = workspace ? (float *)workspace + used : nullptr;
    used += (size_t)t.groups * r.dim;
  }
  return used * sizeof(float);
}

// --------------------------------------------------------------- gated ----
int check_operand(const nvfp4_tensor *t) {
  if (!t || !t->codes || !t->scales || !t->global_scale) return NVFP4_E_NULL;
  if (t->rows <= 0 || t->cols <= 0 || t->rows % 16 || t->cols % 16 || t->rows > ((int64_t)1 << 31)) return NVFP4_E_SHAPE;
  if (t->scale_kind != NVFP4_SCALE_1D16 && t->scale_kind != NVFP4_SCALE_2D16) return NVFP4_E_UNSUPPORTED;
  return aligned(t->codes, 16) ? NVFP4_OK : NVFP4_E_ALIGN;
}

int check_matrix(const nvfp4_gated_matrix *t, int64_t cols) {
  if (!t || !t->data) return NVFP4_E_NULL;
  if (t->ld < cols) return NVFP4_E_LD;
  if (!aligned(t->data, 16) || t->ld % 8 || !aligned(t->amax_plain, 4) || !aligned(t->amax_rht_col, 4)) return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

// a launch counts its threads in 32 bits, 256 to a workgroup: of 16 columns (up to
// 64 rows), or of at least 128 x 64 outputs
bool gated_grid_ok(int64_t M, int64_t N) {
  return (M <= 64 ? N / 16 : (M + 127) / 128 * ((N + 63) / 64)) < ((int64_t)1 << 24);
}

GatedArgs gated_args(const nvfp4_tensor *a, const nvfp4_tensor *b, int32_t activation, uint64_t rht_seed) {
  GatedArgs r = {};
  r.g.a_codes = a->codes;
  r.g.a_scales = a->scales;
  r.g.a_S = a->global_scale;
  r.g.b_codes = b->codes;
  r.g.b_scales = b->scales;
  r.g.b_S = b->global_scale;
  r.g.M = a->rows;
  r.g.N = b->rows;
  r.g.K = a->cols;
  r.g.a_kind = a->scale_kind;
  r.g.b_kind = b->scale_kind;
  r.g.c_bf16 = 1;
  r.g.rht_mask = nvfp4_rht_sign_mask(rht_seed);
  r.activation = activation;
  return r;
}

unsigned int *bits(float *p) { return reinterpret_cast<unsigned int *>(p); }

// ---------------------------------------------------------------- muon ----
int check_muon(const nvfp4_muon_tensor &t, bool buffers) {
  const int64_t side = (int64_t)1 << 17;
  if (t.rows < 0 || t.rows > side || t.cols < 0 || t.cols > side || t.rows * t.cols > ((int64_t)1 << 33)) return NVFP4_E_SHAPE;
  if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype)) return NVFP4_E_UNSUPPORTED;
  if (!buffers) return NVFP4_OK;
  if (!(t.weight_decay >= 0.0f) || !isfinite(t.weight_decay) || !isfinite(t.scale)) return NVFP4_E_VALUE;
  if (!t.param && (t.copy || t.amax)) return NVFP4_E_UNSUPPORTED;
  if (!t.rows || !t.cols) return NVFP4_OK;
  if (!t.grad || (!t.param && !t.update)) return NVFP4_E_NULL;
  if (!aligned(t.grad, size_of(t.grad_dtype)) || !aligned(t.param, size_of(t.param_dtype)) || !aligned(t.m, 4) ||
      !aligned(t.copy, 2) || !aligned(t.update, 2) || !aligned(t.amax, 4))
    return NVFP4_E_ALIGN;
  // all of a gradient is read before a parameter, copy or update is written, but not before the momentum
  if (t.m && (t.m == t.grad || t.m == t.param || t.m == t.copy || t.m == t.update)) return NVFP4_E_UNSUPPORTED;
  if (t.param && (t.param == t.copy || t.param == t.update)) return NVFP4_E_UNSUPPORTED;
  if (t.update && t.update == t.copy) return NVFP4_E_UNSUPPORTED;
  return NVFP4_OK;
}

// Whether the iteration's singular values, from [0, 1], stay where fp16 holds its
// matrices: s p(s^2) is extreme at the ends and where its derivative vanishes,
// p(s^2) at the ends and at s^2 = -b / 2 c.  most[k]: the largest |p| of step k.
bool muon_bounded(const nvfp4_muon_config &c, double *most) {
  const auto p = [&](double q) { return c.a + q * (c.b + q * c.c); };
  double top = 1.0;
  for (int k = 0; k < c.steps; ++k) {
    double next = 0.0;
    most[k] = 0.0;
    const auto look = [&](double q, bool turn) {
      if (!(q >= 0.0 && q <= top * top)) return true;
      if (!turn) next = fmax(next, sqrt(q) * fabs(p(q)));
      most[k] = fmax(most[k], fabs(p(q)));
      return fabs(p(q)) <= 14.0;
    };
    bool good = look(0.0, false) && look(top * top, false);
    if (c.c != 0.0) {
      const double d = 9.0 * c.b * c.b - 20.0 * c.a * c.c;
      if (d >= 0.0) good = good && look((-3.0 * c.b - sqrt(d)) / (10.0 * c.c), false) && look((-3.0 * c.b + sqrt(d)) / (10.0 * c.c), false);
      good = good && look(-c.b / (2.0 * c.c), true);
    } else if (c.b != 0.0) {
      good = good && look(-c.a / (3.0 * c.b), false);
    }
    if (!good || !(next <= 3.5)) return false;
    top = next;
  }
  return true;
}

int64_t round_up(int64_t n, int64_t by) { return (n + by - 1) / by * by; }

// What a matrix's sides are padded to multiples of: the largest tile that costs no
// more than a sixteenth over the smallest's padding.
int muon_pad(const nvfp4_muon_tensor &t) {
  for (const int tile : {256, 128})
    if (16 * round_up(t.rows, tile) * round_up(t.cols, tile) <= 17 * round_up(t.rows, 64) * round_up(t.cols, 64)) return tile;
  return 64;
}

// Whether steps of a matrix, m x n with m <= n, are chained.  The polynomials of
// successive steps are all polynomials of the first one's A, so they commute: with
// P = p(A) the next A is P A P, and a chain's steps are one product of X with the
// product of their polynomials.  A step more in a chain costs four products of m x m,
// three of them for A and the iterate's, and saves one of X with X and one with X
// (of three steps of 5120 x 20480 that is half of all operations).  Five steps,
// chained against not, in us: 1024 x 1536 326 against 313, 1024 x 2048 344, 353; 7 of
// 1024 x 4096 1170, 1740; 2048 x 2048 870, 775; 2048 x 3500 1040, 1125; 2048 x 8192 1390,
// 1970; 2 of 5120 x 7680 16500, 19100; 2 of 5120 x 20480 27000, 44800.  A's rounding is
// carried through a chain: 1024 x 1536 and 2048 x 4096 come out off by 2.9e-6 and 3.7e-6
// for normal matrices (single steps 2.1e-6, 2.9e-6; binary32 3.3e-6, 4.6e-6), by 2.1e-5
// and 2.9e-5 (2.4e-5, 3.4e-5; 3.4e-5, 4.9e-5) with 1 / i^2 spectra and by 1.9e-5 and
// 1.1e-5 (9e-6, 7e-6; 6e-6, 6e-6) where half of the directions are empty.  At m = 300
// it is up to 1.9 times single steps' error; those go by single steps.
bool muon_chained(const nvfp4_muon_tensor &t) {
  const int64_t m = t.rows < t.cols ? t.rows : t.cols, n = t.rows < t.cols ? t.cols : t.rows;
  return m >= 1024 && 2 * n >= 3 * m;
}
// The steps from k on that make a chain: three at first, then two (all five in one
// chain carry A's errors past small singular values; two and then three doubled the
// error where these fall off as 1 / i), with a product of at most 64 (kMuonQ).
int muon_chain(int steps, int k, const double *most) {
  int length = 1;
  double top = most[k];
  while (length < (k ? 2 : 3) && k + length < steps && top * most[k + length] <= 64.0) top *= most[k + length++];
  return length;
}

// Tiles of a product of the group: those that take least by these times in us, as
// measured (one product of 7 matrices of 1024 x 1152, 1 of 2048 x 2048, 1 of 4096 x
// 4096 and others at every tile size): a fixed part, and per 64 of K, each taken three
// times, the longer of one tile's own time and what the chip needs for all of them,
// 256 at a time.  E. g. X X^T of 2048 x 2048: 118 us in tiles of 256, 54 of 128, 63 of
// 64; the last product of 4096 x 4096: 322, 386, 638; 20 matrices of 512 x 512: 379 us
// by these tiles, all in 64 399, in 256 696.
int muon_tile(const NsArgs &p, int pad) {
  struct Cost {
    int tile;
    double fixed, own, all;
  };
  constexpr Cost costs[3] = {{256, 8.0, 1.2, 1.7}, {128, 7.5, 0.46, 0.70}, {64, 4.0, 0.25, 0.29}};
  double least = 0.0;
  int best = 0;
  for (const Cost &c : costs) {
    if (c.tile > pad) continue;
    int64_t tiles = 0, k = 0;
    for (int i = 0; i < p.count; ++i) {
      const int64_t down = p.mat[i].M / c.tile, across = p.mat[i].N / c.tile;
      const int64_t n = p.symmetric ? down * (down + 1) / 2 : down * across;
      tiles += n;
      k += n * (p.mat[i].K / 64) * 3;
    }
    // a compute unit holds one of the large tiles, but several of the others
    const double rounds = c.tile == 256 ? (double)((tiles + 255) / 256) : (double)tiles / 256.0;
    const double us = c.fixed + (double)k / (double)tiles * fmax(c.own, rounds * c.all);
    if (!best || us < least) {
      best = c.tile;
      least = us;
    }
  }
  return best;
}

// The matrices of the list with one padding, chained or not, from `from` on, that make
// a group: as many as a launch takes, or 2^27 elements.
struct MuonGroup {
  int64_t index[kMuonMats];
  int count = 0;
  int64_t next = 0;  // where to go on in the list
};
MuonGroup muon_group(const nvfp4_muon_tensor *tensors, int64_t n, int64_t from, int pad, bool chained) {
  MuonGroup g;
  int64_t elements = 0, i = from;
  for (; i < n && g.count < kMuonMats && elements < ((int64_t)1 << 27); ++i) {
    const nvfp4_muon_tensor &t = tensors[i];
    if (!t.rows || !t.cols || muon_pad(t) != pad || muon_chained(t) != chained) continue;
    g.index[g.count++] = i;
    elements += t.rows * t.cols;
  }
  g.next = i;
  return g;
}
struct MuonBuffers {
  double *parts;
  _Float16 *x, *xt[2], *a, *q[2], *p;  // q[1] and p where steps are chained
};
size_t muon_buffers(const nvfp4_muon_tensor &t, int pad, char *base, size_t used, MuonBuffers &o) {
  const int64_t m = round_up(t.rows < t.cols ? t.rows : t.cols, pad), n = round_up(t.rows < t.cols ? t.cols : t.rows, pad);
  const auto take = [&](size_t bytes) {
    char *p = base ? base + used : nullptr;
    used += (bytes + 255) & ~(size_t)255;
    return p;
  };
  o.parts = (double *)take(kMuonParts * sizeof(double));
  const auto matrix = [&](int64_t rows, int64_t cols) { return (_Float16 *)take((size_t)(rows * muon_ld(cols)) * 4); };
  o.x = matrix(m, n);
  o.xt[0] = matrix(n, m);
  o.xt[1] = matrix(n, m);
  o.a = matrix(m, m);
  o.q[0] = matrix(m, m);
  o.q[1] = o.p = nullptr;
  if (muon_chained(t)) {
    o.q[1] = matrix(m, m);
    o.p = matrix(m, m);
  }
  return used;
}
constexpr int kPads[3] = {256, 128, 64};
constexpr int kMuonSteps = 16;

hipError_t muon_run(const nvfp4_muon_tensor *tensors, const MuonGroup &g, int pad, bool chained, const nvfp4_muon_config &c,
                    const double *most, MuonArgs &a, char *base, hipStream_t s) {
  MuonBuffers buf[kMuonMats];
  size_t used = 0;
  for (int i = 0; i < g.count; ++i) {
    const nvfp4_muon_tensor &t = tensors[g.index[i]];
    used = muon_buffers(t, pad, base, used, buf[i]);
    const bool turned = t.rows > t.cols;
    MuonMat &d = a.mat[i];
    d.grad = t.grad;
    d.m = t.m;
    d.param = t.param;
    d.copy = (uint16_t *)t.copy;
    d.update = (uint16_t *)t.update;
    d.amax = t.amax;
    d.direct = turned ? buf[i].xt[0] : buf[i].x;
    d.turned = turned ? buf[i].x : buf[i].xt[0];
    d.parts = buf[i].parts;
    d.rows = (int)t.rows;
    d.cols = (int)t.cols;
    d.rp = (int)round_up(t.rows, pad);
    d.cp = (int)round_up(t.cols, pad);
    d.keep = (float)(1.0 - (double)c.lr * t.weight_decay);
    d.step = (float)((double)c.lr * t.scale);
    d.flags = (t.param_dtype == NVFP4_BF16 ? MF_PARAM_BF16 : 0u) | (t.grad_dtype == NVFP4_BF16 ? MF_GRAD_BF16 : 0u) |
              (turned ? MF_TURNED : 0u);
    d.index = (uint32_t)g.index[i];
  }
  a.count = g.count;
  hipError_t e = launch_muon_sums(a, s);
  if (e == hipSuccess) e = launch_muon_form(a, s);
  NsArgs p = {};
  p.count = g.count;
  const double kx = kMuonX, ka = kMuonA, kq = kMuonQ;
  p.beta = (float)c.b;
  p.gamma = (float)(c.a * ka);
  // one product of every matrix i: operands(buffers, m, n, turned)
  const auto product = [&](bool symmetric, double alpha, const auto &operands) {
    if (e != hipSuccess) return;
    for (int i = 0; i < g.count; ++i) {
      const MuonMat &t = a.mat[i];
      const bool turned = t.flags & MF_TURNED;
      p.mat[i] = operands(buf[i], turned ? t.cp : t.rp, turned ? t.rp : t.cp, turned);
    }
    p.symmetric = symmetric;
    p.alpha = (float)alpha;
    e = launch_muon_product(p, muon_tile(p, pad), s);
  };
  int now = 0;  // the iterate's transpose is in xt[now]
  for (int k = 0; k < c.steps && e == hipSuccess;) {
    const int length = chained ? muon_chain(c.steps, k, most) : 1;
    product(true, ka / (kx * kx), [](const MuonBuffers &b, int m, int n, bool) { return NsMat{b.x, b.x, nullptr, b.a, b.a, m, m, n}; });
    int q = 0;  // the chain's product is in q[q], at first its first polynomial
    for (int l = 0; l < length; ++l) {
      const auto poly = [&](const MuonBuffers &b) { return l ? b.p : b.q[0]; };
      product(true, c.c / ka, [&](const MuonBuffers &b, int m, int, bool) { return NsMat{b.a, b.a, b.a, poly(b), poly(b), m, m, m}; });
      if (l) {
        product(true, (l == 1 ? kq / ka : 1.0) / ka,
                [&](const MuonBuffers &b, int m, int, bool) { return NsMat{b.p, b.q[q], nullptr, b.q[!q], b.q[!q], m, m, m}; });
        q = !q;
      }
      if (l + 1 < length) {  // A = p(A) A p(A)
        product(true, 1.0 / ka,
                [&](const MuonBuffers &b, int m, int, bool) { return NsMat{poly(b), b.a, nullptr, b.q[!q], b.q[!q], m, m, m}; });
        product(true, 1.0 / ka,
                [&](const MuonBuffers &b, int m, int, bool) { return NsMat{poly(b), b.q[!q], nullptr, b.a, b.a, m, m, m}; });
      }
    }
    k += length;
    const bool last = k == c.steps;
    product(false, 1.0 / (length > 1 ? kq : ka), [&](const MuonBuffers &b, int m, int n, bool turned) {
      return NsMat{b.q[q], b.xt[now], nullptr, last && turned ? nullptr : b.x, last && !turned ? nullptr : b.xt[!now], m, n, m};
    });
    now = !now;
  }
  for (int i = 0; i < g.count; ++i)
    if (a.mat[i].flags & MF_TURNED) a.mat[i].direct = buf[i].xt[now];
  return e == hipSuccess ? launch_muon_update(a, s) : e;
}

}  // namespace

extern "C" {

int nvfp4_qk_rope(const nvfp4_qk_rope_args *a, void *stream) {
  if (const int st = check_rope(a, false)) return st;
  const RopeArgs r = rope_args(*a);
  if (!r.total) return NVFP4_OK;  // nothing is written
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_rope(r, s), s);
}

size_t nvfp4_qk_rope_backward_workspace_bytes(const nvfp4_qk_rope_args *a) {
  if (check_rope(a, true) != NVFP4_OK) return 0;
  RopeArgs r = rope_args(*a);
  return rope_parts(r, nullptr);
}

int nvfp4_qk_rope_backward(const nvfp4_qk_rope_args *a, void *workspace, size_t workspace_bytes, void *stream) {
  if (const int st = check_rope(a, true)) return st;
  RopeArgs r = rope_args(*a);
  const size_t need = rope_parts(r, workspace);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4_E_WORKSPACE;
  if (need && !aligned(workspace, 16)) return NVFP4_E_ALIGN;
  if (!r.total && !need) return NVFP4_OK;  // nothing is written
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_rope_backward(r, s), s);
}

int nvfp4_gemm_gated(const nvfp4_tensor *a, const nvfp4_tensor *b_gate, const nvfp4_tensor *b_up, int32_t activation,
                     const nvfp4_gated_matrix *h, const nvfp4_gated_matrix *gate, const nvfp4_gated_matrix *up,
                     uint64_t rht_seed, void *stream) {
  for (const nvfp4_tensor *t : {a, b_gate, b_up})
    if (const int st = check_operand(t)) return st;
  if (a->cols != b_gate->cols || a->cols != b_up->cols || b_gate->rows != b_up->rows) return NVFP4_E_UNSUPPORTED;
  if (activation < NVFP4_SILU || activation > NVFP4_RELU) return NVFP4_E_UNSUPPORTED;
  if (!gated_grid_ok(a->rows, b_gate->rows)) return NVFP4_E_SHAPE;
  if (const int st = check_matrix(h, b_gate->rows)) return st;
  for (const nvfp4_gated_matrix *t : {gate, up}) {
    if (!t) continue;
    if (const int st = check_matrix(t, b_gate->rows)) return st;
    if (t->amax_plain || t->amax_rht_col || t->data == h->data) return NVFP4_E_UNSUPPORTED;
  }
  if (gate && up && gate->data == up->data) return NVFP4_E_UNSUPPORTED;
  GatedArgs r = gated_args(a, b_gate, activation, rht_seed);
  r.u_codes = b_up->codes;
  r.u_scales = b_up->scales;
  r.u_S = b_up->global_scale;
  r.u_kind = b_up->scale_kind;
  r.h = (uint16_t *)h->data;
  r.ld_h = h->ld;
  r.amax[0] = bits(h->amax_plain);
  r.rht[0] = bits(h->amax_rht_col);
  if (gate) r.gate = (uint16_t *)gate->data, r.ld_gate = gate->ld;
  if (up) r.up = (uint16_t *)up->data, r.ld_up = up->ld;
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_gemm_gated(r, s), s);
}

int nvfp4_gemm_gated_backward(const nvfp4_tensor *a, const nvfp4_tensor *b, int32_t activation,
                              const nvfp4_gated_matrix *gate, const nvfp4_gated_matrix *up,
                              const nvfp4_gated_matrix *dgate, const nvfp4_gated_matrix *dup, uint64_t rht_seed,
                              void *stream) {
  for (const nvfp4_tensor *t : {a, b})
    if (const int st = check_operand(t)) return st;
  if (a->cols != b->cols || activation < NVFP4_SILU || activation > NVFP4_RELU) return NVFP4_E_UNSUPPORTED;
  if (!gated_grid_ok(a->rows, b->rows)) return NVFP4_E_SHAPE;
  for (const nvfp4_gated_matrix *t : {gate, up, dgate, dup})
    if (const int st = check_matrix(t, b->rows)) return st;
  if (dgate->data == dup->data) return NVFP4_E_UNSUPPORTED;
  for (const nvfp4_gated_matrix *out : {dgate, dup})  // read by the lane that writes them
    for (const nvfp4_gated_matrix *in : {gate, up})
      if (out->data == in->data && out->ld != in->ld) return NVFP4_E_UNSUPPORTED;
  GatedArgs r = gated_args(a, b, activation, rht_seed);
  r.gate = (uint16_t *)gate->data, r.ld_gate = gate->ld;
  r.up = (uint16_t *)up->data, r.ld_up = up->ld;
  r.dgate = (uint16_t *)dgate->data, r.ld_dgate = dgate->ld;
  r.dup = (uint16_t *)dup->data, r.ld_dup = dup->ld;
  r.amax[0] = bits(dgate->amax_plain), r.rht[0] = bits(dgate->amax_rht_col);
  r.amax[1] = bits(dup->amax_plain), r.rht[1] = bits(dup->amax_rht_col);
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_gemm_gated_backward(r, s), s);
}

size_t nvfp4_muon_workspace_bytes(const nvfp4_muon_tensor *tensors, int64_t n_tensors) {
  if (!tensors || n_tensors < 1 || n_tensors >= ((int64_t)1 << 30)) return 0;
  for (int64_t i = 0; i < n_tensors; ++i)
    if (check_muon(tensors[i], false) != NVFP4_OK) return 0;
  size_t most = 0;
  for (const int pad : kPads)
    for (const bool chained : {false, true})
      for (int64_t at = 0; at < n_tensors;) {
        const MuonGroup g = muon_group(tensors, n_tensors, at, pad, chained);
        size_t used = 0;
        MuonBuffers b;
        for (int i = 0; i < g.count; ++i) used = muon_buffers(tensors[g.index[i]], pad, nullptr, used, b);
        if (used > most) most = used;
        at = g.next;
      }
  return most;
}

int nvfp4_muon(const nvfp4_muon_tensor *tensors, int64_t n_tensors, const nvfp4_muon_config *c, void *workspace,
               size_t workspace_bytes, void *stream) {
  if (!tensors || !c) return NVFP4_E_NULL;
  if (n_tensors < 1 || n_tensors >= ((int64_t)1 << 30)) return NVFP4_E_SHAPE;
  double most[kMuonSteps];
  if ((c->rounding != NVFP4_RTN && c->rounding != NVFP4_SR) || (c->nesterov != 0 && c->nesterov != 1)) return NVFP4_E_UNSUPPORTED;
  if (!(c->lr >= 0.0f) || !isfinite(c->lr) || !(c->momentum >= 0.0 && c->momentum < 1.0) || c->steps < 1 || c->steps > kMuonSteps ||
      c->step < 0 || c->step >= ((int64_t)1 << 47) || !isfinite(c->a) || !isfinite(c->b) || !isfinite(c->c) || !muon_bounded(*c, most))
    return NVFP4_E_VALUE;
  if (!aligned(c->grad_scale, 4)) return NVFP4_E_ALIGN;
  for (int64_t i = 0; i < n_tensors; ++i)
    if (const int st = check_muon(tensors[i], true)) return st;
  const size_t need = nvfp4_muon_workspace_bytes(tensors, n_tensors);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4_E_WORKSPACE;
  if (need && !aligned(workspace, 16)) return NVFP4_E_ALIGN;

  MuonArgs a = {};
  a.sr = c->rounding == NVFP4_SR;
  a.nesterov = c->nesterov;
  a.beta = (float)c->momentum;
  a.one_minus_beta = (float)(1.0 - c->momentum);
  a.seed_lo = (uint32_t)c->seed;
  a.seed_hi = (uint32_t)(c->seed >> 32);
  a.step_lo = (uint32_t)c->step;
  a.tag = 0x4D550000u + (uint32_t)(c->step >> 32);
  a.grad_scale = c->grad_scale;
  hipStream_t s = (hipStream_t)stream;
  for (const int pad : kPads)
    for (const bool chained : {false, true})
      for (int64_t at = 0; at < n_tensors;) {
        const MuonGroup g = muon_group(tensors, n_tensors, at, pad, chained);
        at = g.next;
        if (g.count && muon_run(tensors, g, pad, chained, *c, most, a, (char *)workspace, s) != hipSuccess) return NVFP4_E_HIP;
      }
  return finish(hipSuccess, s);
}

}  // extern "C"
