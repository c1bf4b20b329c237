// C ABI of the training operators: argument validation on the host, then
// kernel launches on the caller's stream.  The entry points and their
// contracts are declared and documented in include/nvfp4.h.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "nvfp4.h"
#include "train_kernels.hpp"

using namespace nvfp4;

namespace {

// a launch counts its threads in 32 bits, 256 to a workgroup
constexpr int64_t kMaxGroups = ((int64_t)1 << 24) - 1;

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

int norm_shape(int64_t rows, int64_t cols) {
  return rows <= 0 || rows >= ((int64_t)1 << 31) || cols <= 0 || cols > kNormMaxCols ? NVFP4_E_SHAPE : NVFP4_OK;
}

// Whether the rows of output a may be written where those of b are read, each
// only after all of it was read: they begin apart, or are as far apart.
bool rows_fit(const void *a, int64_t ld_a, int32_t type_a, const void *b, int64_t ld_b, int32_t type_b, int64_t rows) {
  return !a || a != b || rows == 1 || ld_a * (int64_t)size_of(type_a) == ld_b * (int64_t)size_of(type_b);
}

// one bf16 tensor of an attention call, of queries or of keys (an empty one may
// have no data); outputs must not overlap themselves
int check_heads(const nvfp4_heads *t, const nvfp4_attention_shape *s, bool queries, bool output) {
  const int32_t heads = queries ? s->heads : s->kv_heads;
  if (!t || (!t->data && (queries ? s->total_q : s->total_k))) return NVFP4_E_NULL;
  const bool batched = !s->cu_q && s->batch > 1;
  if (t->token_stride < 0 || t->token_stride >= ((int64_t)1 << 23) || t->head_stride < 0 ||
      (batched && t->batch_stride < 0))
    return NVFP4_E_LD;
  if (output && (t->token_stride < s->head_dim || (heads > 1 && t->head_stride < s->head_dim) ||
                 (batched && t->batch_stride < s->head_dim)))
    return NVFP4_E_LD;
  if (!aligned(t->data, 16) || t->token_stride % 8 || t->head_stride % 8 || (batched && t->batch_stride % 8))
    return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

// Whether output a may be written beside tensor b: they begin apart, or, where
// b's elements are read before their places are written, stand alike.  (Without
// queries or keys nothing meets.)
bool apart(const nvfp4_heads *a, const nvfp4_heads *b) { return a->data != b->data; }
bool apart_or_alike(const nvfp4_heads *a, const nvfp4_heads *b, const nvfp4_attention_shape *s) {
  return apart(a, b) || (a->token_stride == b->token_stride && a->head_stride == b->head_stride &&
                         (s->cu_q || s->batch == 1 || a->batch_stride == b->batch_stride));
}

// The first pass alone reads o, each row before it writes that of dq; the second
// reads q and d_o anywhere, and a workgroup its keys and values before it writes theirs.
bool gradients_apart(const nvfp4_attention_shape &s, const nvfp4_heads *q, const nvfp4_heads *k, const nvfp4_heads *v,
                     const nvfp4_heads *o, const nvfp4_heads *d_o, const nvfp4_heads *dq, const nvfp4_heads *dk,
                     const nvfp4_heads *dv) {
  for (const nvfp4_heads *t : {q, k, v, d_o, dk, dv})
    if (!apart(dq, t)) return false;
  for (const nvfp4_heads *t : {q, o, d_o})
    if (!apart(dk, t) || !apart(dv, t)) return false;
  for (const nvfp4_heads *t : {k, v})
    if (!apart_or_alike(dk, t, &s) || !apart_or_alike(dv, t, &s)) return false;
  return apart(dk, dv) && apart_or_alike(dq, o, &s);
}

// what a sequence's length cannot exceed (0 only with packed sequences)
int64_t longest(const nvfp4_attention_shape *s, int64_t len, int64_t total) {
  return !s->cu_q || len < total ? len : total;
}

int check_shape(const nvfp4_attention_shape *s) {
  if (!s) return NVFP4_E_NULL;
  const int64_t most = (int64_t)1 << 30, least = s->cu_q ? 0 : 1;
  if (s->batch < 1 || s->batch > most || s->q_len < least || s->q_len > most || s->k_len < least || s->k_len > most ||
      s->heads < 1 || s->heads > 65535 || s->kv_heads < 1 || s->heads % s->kv_heads)
    return NVFP4_E_SHAPE;
  if (s->head_dim < 8 || s->head_dim > 128 || s->head_dim % 8) return NVFP4_E_UNSUPPORTED;
  if (s->causal != 0 && s->causal != 1) return NVFP4_E_UNSUPPORTED;
  if (s->window < 0 || (s->window > 0 && !s->causal)) return NVFP4_E_UNSUPPORTED;
  if (!s->cu_q != !s->cu_k) return NVFP4_E_NULL;
  if (s->cu_q) {
    if (s->total_q < 0 || s->total_k < 0 || s->total_q >= ((int64_t)1 << 31) || s->total_k >= ((int64_t)1 << 31))
      return NVFP4_E_SHAPE;
    if (!aligned(s->cu_q, 4) || !aligned(s->cu_k, 4)) return NVFP4_E_ALIGN;
  } else if (s->total_q != s->batch * s->q_len || s->total_k != s->batch * s->k_len) {
    return NVFP4_E_SHAPE;
  }
  // the gradient forms -lse / scale, all passes scale * log2(e)
  if (!(s->scale >= 0x1p-120f && s->scale <= 0x1p120f)) return NVFP4_E_VALUE;
  // tiles are split into parts only where they are few
  const int64_t q = longest(s, s->q_len, s->total_q), k = longest(s, s->k_len, s->total_k);
  const int64_t tiles = (q > k ? q : k) / 128 + 1;
  if (s->batch > kMaxGroups / tiles / s->heads) return NVFP4_E_SHAPE;
  // and a key tile's steps over its heads' query tiles in 26 bits
  if ((q / 32 + 1) * (s->heads / s->kv_heads) >= (int64_t)1 << 26) return NVFP4_E_SHAPE;
  return NVFP4_OK;
}

Heads heads_of(const nvfp4_heads *t) {
  return Heads{(uint16_t *)t->data, t->batch_stride, t->token_stride, t->head_stride};
}

AttnArgs attn_args(const nvfp4_attention_shape *s) {
  AttnArgs a = {};
  a.cu_q = s->cu_q;
  a.cu_k = s->cu_k;
  a.total_q = s->total_q;
  a.total_k = s->total_k;
  a.window = s->window < ((int64_t)1 << 30) ? (int)s->window : 1 << 30;  // no length exceeds that
  a.q_len = (int)longest(s, s->q_len, s->total_q);
  a.k_len = (int)longest(s, s->k_len, s->total_k);
  a.batch = (int)s->batch;
  a.heads = s->heads;
  a.kv_heads = s->kv_heads;
  a.dim = s->head_dim;
  a.causal = s->causal;
  a.scale = s->scale;
  a.by_group = divisor((uint32_t)(s->heads / s->kv_heads));
  a.by_batch = divisor((uint32_t)s->batch);
  a.by_kv = divisor((uint32_t)s->kv_heads);
  a.q_tiles = (a.q_len + 127) / 128;
  a.k_tiles = (a.k_len + 127) / 128;
  return a;
}

// Buffers of a workspace, one after another in whole 256 bytes.
struct Carver {
  char *base;
  size_t used;
  float *floats(size_t n) {
    float *p = base ? (float *)(base + used) : nullptr;
    used += (n * sizeof(float) + 255) & ~(size_t)255;
    return p;
  }
};
size_t padded_dim(const AttnArgs &a) { return a.dim <= 64 ? 64 : 128; }
size_t carve_forward(AttnArgs &a, void *workspace) {
  Carver c = {(char *)workspace, 0};
  a.q_parts = attention_q_parts(a);
  if (a.q_parts > 1) {
    const size_t rows = (size_t)a.q_parts * a.heads * a.total_q;
    a.q_part = c.floats(rows * padded_dim(a));
    a.lse_part = c.floats(rows);
  }
  return c.used;
}
size_t carve_backward(AttnArgs &a, void *workspace) {
  Carver c = {(char *)workspace, 0};
  const size_t stats = (size_t)a.heads * a.total_q;
  a.minus_delta = c.floats(stats + 1);
  a.minus_lse = c.floats(stats + 1);
  a.q_parts = attention_q_parts(a);
  a.k_parts = attention_k_parts(a);
  if (a.q_parts > 1) a.q_part = c.floats(a.q_parts * stats * padded_dim(a));
  if (a.k_parts > 1) {
    const size_t rows = (size_t)a.k_parts * a.kv_heads * a.total_k;
    a.k_part = c.floats(rows * padded_dim(a));
    a.v_part = c.floats(rows * padded_dim(a));
  }
  return c.used;
}

int check_adamw(const nvfp4_adamw_tensor &t) {
  if (t.n < 0 || t.n > ((int64_t)1 << 34)) return NVFP4_E_SHAPE;
  if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || (t.state_bits != 32 && t.state_bits != 8))
    return NVFP4_E_UNSUPPORTED;
  if (!(t.weight_decay >= 0.0f) || !isfinite(t.weight_decay)) return NVFP4_E_VALUE;
  if (t.n == 0) return NVFP4_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return NVFP4_E_NULL;
  if (t.state_bits == 8 && (!t.m_scale || !t.v_scale)) return NVFP4_E_NULL;
  if (!aligned(t.param, size_of(t.param_dtype)) || !aligned(t.grad, size_of(t.grad_dtype)) ||
      (t.copy && !aligned(t.copy, 2)) || (t.amax && !aligned(t.amax, 4)))
    return NVFP4_E_ALIGN;
  if (t.state_bits == 32 && (!aligned(t.m, 4) || !aligned(t.v, 4))) return NVFP4_E_ALIGN;
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_layernorm(const nvfp4_layernorm_args *a, void *stream) {
  if (!a || !a->x || !a->weight || !a->y || !a->mean || !a->rstd) return NVFP4_E_NULL;
  if (a->residual && !a->sum) return NVFP4_E_NULL;
  if (const int st = norm_shape(a->rows, a->cols)) return st;
  if (!dtype_ok(a->x_dtype) || !dtype_ok(a->y_dtype) || !dtype_ok(a->w_dtype)) return NVFP4_E_UNSUPPORTED;
  if (a->sum && !a->residual) return NVFP4_E_UNSUPPORTED;
  if (a->ld_x < a->cols || a->ld_y < a->cols || (a->residual && (a->ld_residual < a->cols || a->ld_sum < a->cols)))
    return NVFP4_E_LD;
  const size_t xs = size_of(a->x_dtype), ws = size_of(a->w_dtype);
  if (!aligned(a->x, xs) || !aligned(a->y, size_of(a->y_dtype)) || !aligned(a->weight, ws) ||
      (a->bias && !aligned(a->bias, ws)) || (a->residual && (!aligned(a->residual, xs) || !aligned(a->sum, xs))) ||
      !aligned(a->mean, 4) || !aligned(a->rstd, 4) || (a->amax && !aligned(a->amax, 4)))
    return NVFP4_E_ALIGN;
  if (!(a->eps >= 0.0f) || !isfinite(a->eps)) return NVFP4_E_VALUE;
  const int32_t xt = a->x_dtype;
  if (a->y == a->sum || !rows_fit(a->y, a->ld_y, a->y_dtype, a->x, a->ld_x, xt, a->rows) ||
      !rows_fit(a->y, a->ld_y, a->y_dtype, a->residual, a->ld_residual, xt, a->rows) ||
      !rows_fit(a->sum, a->ld_sum, xt, a->x, a->ld_x, xt, a->rows) ||
      !rows_fit(a->sum, a->ld_sum, xt, a->residual, a->ld_residual, xt, a->rows))
    return NVFP4_E_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_layernorm(*a, s), s);
}

size_t nvfp4_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (norm_shape(rows, cols) != NVFP4_OK) return 0;
  return (size_t)layernorm_backward_parts(rows, cols) * 2 * (size_t)cols * sizeof(float);
}

int nvfp4_layernorm_backward(const nvfp4_layernorm_backward_args *a, void *workspace, size_t workspace_bytes,
                             void *stream) {
  if (!a || !a->dy || !a->x || !a->weight || !a->mean || !a->rstd || !a->dx) return NVFP4_E_NULL;
  if (const int st = norm_shape(a->rows, a->cols)) return st;
  if (!dtype_ok(a->x_dtype) || !dtype_ok(a->y_dtype) || !dtype_ok(a->w_dtype)) return NVFP4_E_UNSUPPORTED;
  if (a->ld_x < a->cols || a->ld_dy < a->cols || a->ld_dx < a->cols || (a->dsum && a->ld_dsum < a->cols))
    return NVFP4_E_LD;
  const size_t xs = size_of(a->x_dtype);
  if (!aligned(a->x, xs) || !aligned(a->dx, xs) || (a->dsum && !aligned(a->dsum, xs)) ||
      !aligned(a->dy, size_of(a->y_dtype)) || !aligned(a->weight, size_of(a->w_dtype)) || !aligned(a->mean, 4) ||
      !aligned(a->rstd, 4) || (a->dweight && !aligned(a->dweight, 4)) || (a->dbias && !aligned(a->dbias, 4)) ||
      (a->amax && !aligned(a->amax, 4)))
    return NVFP4_E_ALIGN;
  const bool sums = a->dweight || a->dbias;
  if (sums) {
    if (!workspace || workspace_bytes < nvfp4_layernorm_backward_workspace_bytes(a->rows, a->cols))
      return NVFP4_E_WORKSPACE;
    if (!aligned(workspace, 16)) return NVFP4_E_ALIGN;
  }
  const int32_t xt = a->x_dtype;
  if (!rows_fit(a->dx, a->ld_dx, xt, a->dy, a->ld_dy, a->y_dtype, a->rows) ||
      !rows_fit(a->dx, a->ld_dx, xt, a->x, a->ld_x, xt, a->rows) ||
      !rows_fit(a->dx, a->ld_dx, xt, a->dsum, a->ld_dsum, xt, a->rows))
    return NVFP4_E_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_layernorm_backward(*a, sums ? (float *)workspace : nullptr, s), s);
}

size_t nvfp4_attention_workspace_bytes(const nvfp4_attention_shape *shape) {
  if (check_shape(shape) != NVFP4_OK) return 0;
  AttnArgs a = attn_args(shape);
  return carve_forward(a, nullptr);
}

int nvfp4_attention(const nvfp4_attention_shape *shape, const nvfp4_heads *q, const nvfp4_heads *k,
                    const nvfp4_heads *v, const nvfp4_heads *o, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream) {
  if (const int st = check_shape(shape)) return st;
  if (!lse && shape->total_q) return NVFP4_E_NULL;
  if (!aligned(lse, 4)) return NVFP4_E_ALIGN;
  int st = check_heads(q, shape, true, false);
  if (!st) st = check_heads(k, shape, false, false);
  if (!st) st = check_heads(v, shape, false, false);
  if (!st) st = check_heads(o, shape, true, true);
  if (st) return st;
  const size_t need = nvfp4_attention_workspace_bytes(shape);
  if (need && (!workspace || workspace_bytes < need)) return NVFP4_E_WORKSPACE;
  if (need && !aligned(workspace, 16)) return NVFP4_E_ALIGN;
  // a workgroup reads its queries before it writes their rows; any reads the keys
  if (shape->total_q && shape->total_k && (!apart(o, k) || !apart(o, v) || !apart_or_alike(o, q, shape)))
    return NVFP4_E_UNSUPPORTED;
  AttnArgs a = attn_args(shape);
  a.q = heads_of(q);
  a.k = heads_of(k);
  a.v = heads_of(v);
  a.o = heads_of(o);
  a.lse = lse;
  carve_forward(a, workspace);
  if (a.q_len == 0) return NVFP4_OK;  // nothing is written
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_attention(a, s), s);
}

size_t nvfp4_attention_backward_workspace_bytes(const nvfp4_attention_shape *shape) {
  if (check_shape(shape) != NVFP4_OK) return 0;
  AttnArgs a = attn_args(shape);
  return carve_backward(a, nullptr);
}

int nvfp4_attention_backward(const nvfp4_attention_shape *shape, const nvfp4_heads *q, const nvfp4_heads *k,
                             const nvfp4_heads *v, const nvfp4_heads *o, const float *lse, const nvfp4_heads *d_o,
                             const nvfp4_heads *dq, const nvfp4_heads *dk, const nvfp4_heads *dv, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (const int st = check_shape(shape)) return st;
  if (!lse && shape->total_q) return NVFP4_E_NULL;
  if (!aligned(lse, 4)) return NVFP4_E_ALIGN;
  const nvfp4_heads *by_q[4] = {q, o, d_o, dq}, *by_k[4] = {k, v, dk, dv};
  for (int i = 0; i < 4; ++i) {
    if (const int st = check_heads(by_q[i], shape, true, i == 3)) return st;
    if (const int st = check_heads(by_k[i], shape, false, i >= 2)) return st;
  }
  if (!workspace || workspace_bytes < nvfp4_attention_backward_workspace_bytes(shape)) return NVFP4_E_WORKSPACE;
  if (!aligned(workspace, 16)) return NVFP4_E_ALIGN;
  if (shape->total_q && shape->total_k && !gradients_apart(*shape, q, k, v, o, d_o, dq, dk, dv)) return NVFP4_E_UNSUPPORTED;
  AttnArgs a = attn_args(shape);
  a.q = heads_of(q);
  a.k = heads_of(k);
  a.v = heads_of(v);
  a.o = heads_of(o);
  a.d_o = heads_of(d_o);
  a.dq = heads_of(dq);
  a.dk = heads_of(dk);
  a.dv = heads_of(dv);
  a.lse = const_cast<float *>(lse);
  carve_backward(a, workspace);
  if (a.q_len == 0 && a.k_len == 0) return NVFP4_OK;  // nothing is written
  hipStream_t s = (hipStream_t)stream;
  return finish(launch_attention_backward(a, s), s);
}

int nvfp4_adamw(const nvfp4_adamw_tensor *tensors, int64_t n_tensors, const nvfp4_adamw_config *c, void *stream) {
  if (!tensors || !c) return NVFP4_E_NULL;
  if (n_tensors < 1 || n_tensors >= ((int64_t)1 << 30)) return NVFP4_E_SHAPE;
  if (c->rounding != NVFP4_RTN && c->rounding != NVFP4_SR) return NVFP4_E_UNSUPPORTED;
  if (!(c->lr >= 0.0f) || !isfinite(c->lr) || !(c->beta1 >= 0.0 && c->beta1 < 1.0) ||
      !(c->beta2 >= 0.0 && c->beta2 < 1.0) || !(c->eps >= FLT_MIN) || !isfinite(c->eps) || c->step < 1 ||
      c->step >= ((int64_t)1 << 47))
    return NVFP4_E_VALUE;
  if (c->grad_scale && !aligned(c->grad_scale, 4)) return NVFP4_E_ALIGN;
  for (int64_t i = 0; i < n_tensors; ++i)
    if (const int st = check_adamw(tensors[i])) return st;

  AdamArgs a = {};
  a.sr = c->rounding == NVFP4_SR;
  a.lr = c->lr;
  a.beta1 = (float)c->beta1;
  a.one_minus_beta1 = (float)(1.0 - c->beta1);
  a.beta2 = (float)c->beta2;
  a.one_minus_beta2 = (float)(1.0 - c->beta2);
  a.eps = c->eps;
  a.correct1 = (float)(1.0 / (1.0 - pow(c->beta1, (double)c->step)));
  a.correct2 = (float)(1.0 / sqrt(1.0 - pow(c->beta2, (double)c->step)));
  a.seed_lo = (uint32_t)c->seed;
  a.seed_hi = (uint32_t)(c->seed >> 32);
  a.step_lo = (uint32_t)c->step;
  a.tag = 0x41440000u + (uint32_t)(c->step >> 32);
  a.grad_scale = c->grad_scale;
  hipStream_t s = (hipStream_t)stream;
  uint32_t end = 0;
  int extras = 0;
  for (int64_t i = 0; i <= n_tensors; ++i) {
    const bool more = i < n_tensors, extra = more && (tensors[i].m_scale || tensors[i].copy || tensors[i].amax);
    // a launch counts its threads in 32 bits; a tensor has at most 2^22 workgroups
    const uint32_t groups = more ? (uint32_t)((tensors[i].n + kAdamChunk - 1) / kAdamChunk) : 0u;
    if (a.count && (!more || end + groups > kMaxGroups ||
                    (a.count + 1) * sizeof(AdamTensor) + (extras + extra) * sizeof(AdamExtra) > kAdamBytes)) {
      if (launch_adamw(a, s) != hipSuccess) return NVFP4_E_HIP;
      a.count = extras = 0;
      end = 0;
    }
    if (!more || tensors[i].n == 0) continue;
    const nvfp4_adamw_tensor &t = tensors[i];
    AdamTensor d;
    d.param = t.param;
    d.grad = t.grad;
    d.m = t.m;
    d.v = t.v;
    d.n = t.n;
    d.keep = (float)(1.0 - (double)c->lr * t.weight_decay);
    d.index = (uint32_t)i;
    d.flags = (t.param_dtype == NVFP4_BF16 ? AF_PARAM_BF16 : 0u) | (t.grad_dtype == NVFP4_BF16 ? AF_GRAD_BF16 : 0u) |
              (t.state_bits == 8 ? AF_STATE8 : 0u);
    if (extra) {
      const AdamExtra e = {t.m_scale, t.v_scale, (uint16_t *)t.copy, t.amax};
      d.flags |= AF_EXTRA | (uint32_t)extras << AF_EXTRA_SHIFT;
      memcpy(a.bytes + kAdamBytes - ++extras * sizeof e, &e, sizeof e);
    }
    d.end = end += groups;
    memcpy(a.bytes + a.count++ * sizeof d, &d, sizeof d);
  }
  return finish(hipSuccess, s);
}

}  // extern "C"
