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

// one workgroup per 128 x 64 outputs at most: the grid counts its threads in 32 bits
bool gated_grid_ok(int64_t M, int64_t N) { return (M / 16 + 1) * (N / 16 + 1) / 32 < ((int64_t)1 << 24); }

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

}  // extern "C"
