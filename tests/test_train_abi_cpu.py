"""CPU-only checks of the training operators' entry points: every refusal comes
from the host before anything is enqueued (no GPU is touched), through ctypes
and, with both sanitizers on the host code, from a C program."""
import ctypes
import os
import shutil
import subprocess

import pytest

import nvfp4_bit_quantization_amd as nv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nvfp4_bit_quantization_amd", "csrc")
FAKE = 0x10000  # aligned, not null, never dereferenced on the error paths
NULL, SHAPE, LD, ALIGN, UNSUPPORTED, WORKSPACE, VALUE = -1, -2, -3, -4, -5, -6, -8


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantization_amd import build
        build.build()
    return nv.lib()


def _norm(**kw):
    a = dict(x=FAKE, residual=None, weight=FAKE, bias=FAKE, y=FAKE, sum=None, mean=FAKE, rstd=FAKE, amax=None, rows=4,
             cols=64, ld_x=64, ld_residual=0, ld_y=64, ld_sum=0, x_dtype=1, y_dtype=1, w_dtype=0, eps=1e-5)
    a.update(kw)
    return nv.nvfp4_layernorm_args(**a)


NORM = [(dict(x=None), NULL), (dict(weight=None), NULL), (dict(y=None), NULL), (dict(mean=None), NULL),
        (dict(rstd=None), NULL), (dict(residual=FAKE, ld_residual=64), NULL), (dict(rows=0), SHAPE),
        (dict(rows=1 << 31), SHAPE), (dict(cols=0), SHAPE), (dict(cols=32769, ld_x=32769, ld_y=32769), SHAPE),
        (dict(x_dtype=2), UNSUPPORTED), (dict(y_dtype=-1), UNSUPPORTED), (dict(w_dtype=7), UNSUPPORTED),
        (dict(sum=FAKE, ld_sum=64), UNSUPPORTED), (dict(ld_x=63), LD), (dict(ld_y=0), LD),
        (dict(residual=FAKE, sum=FAKE, ld_residual=63, ld_sum=64), LD), (dict(residual=FAKE, sum=FAKE, ld_residual=64, ld_sum=8), LD),
        (dict(x=FAKE + 1), ALIGN), (dict(weight=FAKE + 2), ALIGN), (dict(mean=FAKE + 2), ALIGN), (dict(amax=FAKE + 1), ALIGN),
        (dict(eps=-1e-9), VALUE), (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE)]


@pytest.mark.parametrize("change,status", NORM, ids=str)
def test_layernorm_refusals(L, change, status):
    assert L.nvfp4_layernorm(ctypes.byref(_norm(**change)), None) == status


def test_layernorm_null(L):
    assert L.nvfp4_layernorm(None, None) == NULL
    assert L.nvfp4_layernorm_backward(None, None, 0, None) == NULL


def _norm_grad(**kw):
    a = dict(dy=FAKE, x=FAKE, weight=FAKE, mean=FAKE, rstd=FAKE, dsum=None, dx=FAKE, dweight=FAKE, dbias=FAKE, amax=None,
             rows=4, cols=64, ld_dy=64, ld_x=64, ld_dsum=0, ld_dx=64, x_dtype=1, y_dtype=1, w_dtype=0)
    a.update(kw)
    return nv.nvfp4_layernorm_backward_args(**a)


NORM_GRAD = [(dict(dy=None), NULL), (dict(x=None), NULL), (dict(dx=None), NULL), (dict(mean=None), NULL), (dict(rows=-1), SHAPE),
             (dict(cols=40000, ld_x=40000, ld_dy=40000, ld_dx=40000), SHAPE), (dict(x_dtype=3), UNSUPPORTED),
             (dict(ld_dy=1), LD), (dict(ld_x=1), LD), (dict(ld_dx=1), LD), (dict(dsum=FAKE, ld_dsum=1), LD),
             (dict(dx=FAKE + 1), ALIGN), (dict(dweight=FAKE + 2), ALIGN), (dict(dbias=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("change,status", NORM_GRAD, ids=str)
def test_layernorm_backward_refusals(L, change, status):
    need = L.nvfp4_layernorm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert L.nvfp4_layernorm_backward(ctypes.byref(_norm_grad(**change)), FAKE, need, None) == status


def test_layernorm_backward_workspace(L):
    need = L.nvfp4_layernorm_backward_workspace_bytes(4, 64)
    a = _norm_grad()
    assert L.nvfp4_layernorm_backward(ctypes.byref(a), None, need, None) == WORKSPACE
    assert L.nvfp4_layernorm_backward(ctypes.byref(a), FAKE, need - 1, None) == WORKSPACE
    assert L.nvfp4_layernorm_backward(ctypes.byref(a), FAKE + 8, need, None) == ALIGN
    assert L.nvfp4_layernorm_backward_workspace_bytes(0, 64) == 0
    assert L.nvfp4_layernorm_backward_workspace_bytes(4, 32769) == 0


def _shape(**kw):
    a = dict(batch=2, q_len=16, k_len=32, heads=4, kv_heads=2, head_dim=64, causal=1, window=0, cu_q=None, cu_k=None,
             total_q=32, total_k=64, scale=0.125)
    a.update(kw)
    return nv.nvfp4_attention_shape(**a)


def _heads(**kw):
    a = dict(data=FAKE, batch_stride=16 * 256, token_stride=256, head_stride=64)
    a.update(kw)
    return nv.nvfp4_heads(**a)


def _attention(L, s, lse=FAKE, ws=None, nbytes=0, **kw):
    t = {n: _heads() for n in ("q", "k", "v", "o")}
    t.update(kw)
    return L.nvfp4_attention(ctypes.byref(s), *[None if t[n] is None else ctypes.byref(t[n]) for n in ("q", "k", "v", "o")],
                             lse, ws, nbytes, None)


SHAPES = [(dict(batch=0), SHAPE), (dict(q_len=0, total_q=0), SHAPE), (dict(k_len=0, total_k=0), SHAPE), (dict(heads=0), SHAPE),
          (dict(kv_heads=0), SHAPE), (dict(kv_heads=3), SHAPE), (dict(heads=65536, kv_heads=1), SHAPE), (dict(total_q=31), SHAPE), (dict(total_k=65), SHAPE),
          (dict(head_dim=0), UNSUPPORTED), (dict(head_dim=60), UNSUPPORTED), (dict(head_dim=136), UNSUPPORTED),
          (dict(causal=2), UNSUPPORTED), (dict(window=-1), UNSUPPORTED), (dict(window=5, causal=0), UNSUPPORTED),
          (dict(cu_q=FAKE), NULL), (dict(cu_k=FAKE), NULL), (dict(cu_q=FAKE, cu_k=FAKE, total_q=-1), SHAPE),
          (dict(cu_q=FAKE, cu_k=FAKE, total_k=1 << 31), SHAPE), (dict(cu_q=FAKE + 2, cu_k=FAKE), ALIGN),
          (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=float("nan")), VALUE),
          (dict(scale=float("inf")), VALUE), (dict(q_len=(1 << 30) + 1, total_q=(1 << 31) + 2), SHAPE),
          (dict(batch=1, q_len=1 << 30, k_len=128, heads=2, kv_heads=1, total_q=1 << 30, total_k=128), SHAPE),
          (dict(batch=1 << 29, q_len=64, k_len=64, total_q=1 << 35, total_k=1 << 35), SHAPE)]


@pytest.mark.parametrize("change,status", SHAPES, ids=str)
def test_attention_shape_refusals(L, change, status):
    s = _shape(**change)
    assert _attention(L, s) == status
    assert L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s)) == 0
    h = ctypes.byref(_heads())
    assert L.nvfp4_attention_backward(ctypes.byref(s), h, h, h, h, FAKE, h, h, h, h, FAKE, 1 << 30, None) == status


def test_attention_workgroup_limits(L):
    """A launch of 2^24 workgroups of 256 threads is refused; lengths of packed sequences count up to the tokens there are."""
    need = lambda **kw: L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(_shape(**kw)))
    packed = dict(cu_q=FAKE, cu_k=FAKE, heads=4, kv_heads=4)
    assert need(batch=1 << 16, q_len=8192, k_len=8192, total_q=1 << 17, total_k=1 << 17, **packed) == 0
    assert need(batch=1 << 15, q_len=8192, k_len=8192, total_q=1 << 17, total_k=1 << 17, **packed) > 0
    assert need(batch=1 << 14, q_len=1 << 30, k_len=1 << 30, total_q=1 << 14, total_k=1 << 14, **packed) > 0
    few = dict(batch=3, total_q=1000, total_k=1200, **packed)
    assert need(q_len=1 << 30, k_len=1 << 30, **few) == need(q_len=1000, k_len=1200, **few) > 0
    assert need(batch=3, q_len=5, k_len=5, total_q=0, total_k=0, **packed) > 0
    assert _attention(L, _shape(batch=1 << 16, q_len=8192, k_len=8192, total_q=1 << 17, total_k=1 << 17, **packed)) == SHAPE


TENSORS = [(dict(data=None), NULL), (dict(data=FAKE + 8), ALIGN), (dict(token_stride=260), ALIGN), (dict(head_stride=60), ALIGN),
           (dict(batch_stride=4), ALIGN), (dict(token_stride=-256), LD), (dict(token_stride=1 << 23), LD),
           (dict(head_stride=-64), LD), (dict(batch_stride=-8), LD)]


@pytest.mark.parametrize("change,status", TENSORS, ids=str)
def test_attention_tensor_refusals(L, change, status):
    s = _shape()
    for n in ("q", "k", "v", "o"):
        assert _attention(L, s, **{n: _heads(**change)}) == (LD if n == "o" and change == dict(batch_stride=4) else
                                                             LD if n == "o" and change == dict(head_stride=60) else status)
        assert _attention(L, s, **{n: None}) == NULL
    need = L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s))
    for at in range(8):
        t = [_heads() for _ in range(8)]
        t[at] = _heads(**change)
        r = [ctypes.byref(x) for x in t]
        got = L.nvfp4_attention_backward(ctypes.byref(s), *r[:4], FAKE, *r[4:], FAKE, need, None)
        assert got in (status, LD) and got < 0


def test_attention_outputs_do_not_overlap(L):
    s = _shape()
    for bad in (dict(token_stride=0), dict(head_stride=0), dict(batch_stride=0), dict(head_stride=56)):
        assert _attention(L, s, o=_heads(**bad)) == LD
    assert _attention(L, s, lse=None) == NULL
    assert _attention(L, s, lse=FAKE + 2) == ALIGN


def test_attention_workspace(L):
    """Keys are split, and a workspace is wanted, where few queries meet many keys; not for other shapes."""
    assert L.nvfp4_attention_workspace_bytes(ctypes.byref(_shape())) == 0
    s = _shape(batch=1, q_len=4, k_len=8192, total_q=4, total_k=8192)
    need = L.nvfp4_attention_workspace_bytes(ctypes.byref(s))
    assert need >= 4 * (2 * 4 * 4 * 64)
    assert _attention(L, s) == WORKSPACE
    assert _attention(L, s, ws=FAKE, nbytes=need - 1) == WORKSPACE
    assert _attention(L, s, ws=FAKE + 8, nbytes=need) == ALIGN


def test_attention_backward_workspace(L):
    s, h = _shape(), ctypes.byref(_heads())
    need = L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s))
    assert need >= 4 * 4 * 32
    for ws, size, want in ((None, need, WORKSPACE), (FAKE, need - 1, WORKSPACE), (FAKE + 4, need, ALIGN)):
        assert L.nvfp4_attention_backward(ctypes.byref(s), h, h, h, h, FAKE, h, h, h, h, ws, size, None) == want
    assert L.nvfp4_attention_backward(ctypes.byref(s), h, h, h, h, None, h, h, h, h, FAKE, need, None) == NULL


def _adam(**kw):
    a = dict(param=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=None, v_scale=None, copy=None, amax=None, n=100, param_dtype=0,
             grad_dtype=0, state_bits=32, weight_decay=0.1)
    a.update(kw)
    return nv.nvfp4_adamw_tensor(**a)


def _config(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, rounding=0, step=1, seed=0, grad_scale=None)
    a.update(kw)
    return nv.nvfp4_adamw_config(**a)


ADAM = [(dict(n=-1), SHAPE), (dict(n=(1 << 34) + 1), SHAPE), (dict(param_dtype=2), UNSUPPORTED), (dict(grad_dtype=-1), UNSUPPORTED),
        (dict(state_bits=16), UNSUPPORTED), (dict(weight_decay=-0.1), VALUE), (dict(weight_decay=float("nan")), VALUE),
        (dict(param=None), NULL), (dict(grad=None), NULL), (dict(m=None), NULL), (dict(v=None), NULL),
        (dict(state_bits=8), NULL), (dict(state_bits=8, m_scale=FAKE), NULL), (dict(param=FAKE + 2), ALIGN),
        (dict(param_dtype=1, param=FAKE + 1), ALIGN), (dict(grad=FAKE + 2), ALIGN), (dict(m=FAKE + 1), ALIGN),
        (dict(v=FAKE + 2), ALIGN), (dict(copy=FAKE + 1), ALIGN), (dict(amax=FAKE + 2), ALIGN)]


@pytest.mark.parametrize("change,status", ADAM, ids=str)
def test_adamw_tensor_refusals(L, change, status):
    """A bad tensor refuses the whole step, wherever it stands."""
    bad, c = _adam(**change), _config()
    for at in (0, 2, 59):
        arr = (nv.nvfp4_adamw_tensor * 60)(*[_adam() for _ in range(60)])
        arr[at] = bad
        assert L.nvfp4_adamw(arr, 60, ctypes.byref(c), None) == status


CONFIG = [(dict(lr=-1.0), VALUE), (dict(lr=float("inf")), VALUE), (dict(beta1=1.0), VALUE), (dict(beta1=-0.1), VALUE),
          (dict(beta2=1.0), VALUE), (dict(beta2=float("nan")), VALUE), (dict(eps=0.0), VALUE), (dict(eps=float("inf")), VALUE),
          (dict(step=0), VALUE), (dict(step=1 << 47), VALUE), (dict(rounding=2), UNSUPPORTED), (dict(grad_scale=FAKE + 1), ALIGN)]


@pytest.mark.parametrize("change,status", CONFIG, ids=str)
def test_adamw_config_refusals(L, change, status):
    arr = (nv.nvfp4_adamw_tensor * 1)(_adam())
    assert L.nvfp4_adamw(arr, 1, ctypes.byref(_config(**change)), None) == status


def test_adamw_null_and_counts(L):
    arr, c = (nv.nvfp4_adamw_tensor * 1)(_adam()), _config()
    assert L.nvfp4_adamw(None, 1, ctypes.byref(c), None) == NULL
    assert L.nvfp4_adamw(arr, 1, None, None) == NULL
    assert L.nvfp4_adamw(arr, 0, ctypes.byref(c), None) == SHAPE
    # nothing to do: no launch, with or without buffers
    arr[0] = _adam(n=0, param=None, grad=None, m=None, v=None)
    assert L.nvfp4_adamw(arr, 1, ctypes.byref(c), None) == 0


def test_status_text(L):
    assert nv.nvfp4_status_string(VALUE) == "a scalar argument out of its range"


def test_python_checks():
    """Shapes, types and strides that the pointers could not show are refused by the binding."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64)
    with pytest.raises(ValueError):
        nv.nvfp4_layernorm(x, w, w, 1e-5, x, torch.zeros(4), torch.zeros(4))       # host memory
    with pytest.raises(TypeError):
        nv.attention(x.view(1, 4, 1, 64).half(), x.view(1, 4, 1, 64), x.view(1, 4, 1, 64))
    with pytest.raises(ValueError):
        nv.attention(x.view(4, 1, 64), x.view(4, 1, 64), x.view(4, 1, 64), cu_q=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        nv.adamw_tensor(w, w, state_bits=16)
    with pytest.raises(ValueError):
        nv.AdamWList([])
    with pytest.raises(ValueError):
        nv.AdamWList([nv.AdamWTensor(w, w, w.to(torch.uint8), w.to(torch.uint8))])


DRIVER = r"""
#include <stdio.h>
#include <string.h>
#include <hip/hip_runtime.h>
#include "nvfp4.h"
#include "train_kernels.hpp"
namespace nvfp4 {
int launched = 0;
hipError_t launch_layernorm(const nvfp4_layernorm_args &, hipStream_t) { ++launched; return hipErrorInvalidValue; }
int64_t layernorm_backward_parts(int64_t rows, int64_t) { return rows < 512 ? rows : 512; }
hipError_t launch_layernorm_backward(const nvfp4_layernorm_backward_args &, float *, hipStream_t) { ++launched; return hipErrorInvalidValue; }
int64_t adam_ends = 0, adam_tensors = 0;
hipError_t launch_adamw(const AdamArgs &a, hipStream_t) { ++launched; adam_ends += a.tensor(a.count - 1).end; adam_tensors += a.count; return hipSuccess; }
int attention_q_parts(const AttnArgs &) { return 2; }
int attention_k_parts(const AttnArgs &) { return 3; }
hipError_t launch_attention(const AttnArgs &, hipStream_t) { ++launched; return hipErrorInvalidValue; }
hipError_t launch_attention_backward(const AttnArgs &, hipStream_t) { ++launched; return hipErrorInvalidValue; }
}
#define FAKE ((void *)0x10000)
#define CHECK(c) do { if (!(c)) { printf("check failed line %d\n", __LINE__); return 1; } } while (0)
int main() {
  nvfp4_layernorm_args n; memset(&n, 0, sizeof n);
  CHECK(nvfp4_layernorm(nullptr, nullptr) == NVFP4_E_NULL);
  CHECK(nvfp4_layernorm(&n, nullptr) == NVFP4_E_NULL);
  n.x = n.weight = FAKE; n.y = FAKE; n.mean = n.rstd = (float *)FAKE; n.rows = INT64_MAX; n.cols = INT64_MAX;
  CHECK(nvfp4_layernorm(&n, nullptr) == NVFP4_E_SHAPE);
  n.rows = 4; n.cols = 64; n.ld_x = n.ld_y = INT64_MIN;
  CHECK(nvfp4_layernorm(&n, nullptr) == NVFP4_E_LD);
  CHECK(nvfp4_layernorm_backward_workspace_bytes(INT64_MAX, 64) == 0);
  CHECK(nvfp4_layernorm_backward_workspace_bytes((int64_t)1 << 30, 32768) == (size_t)512 * 2 * 32768 * 4);
  nvfp4_attention_shape s; memset(&s, 0, sizeof s);
  nvfp4_heads h = {FAKE, 0, 64, 64};
  CHECK(nvfp4_attention(nullptr, &h, &h, &h, &h, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_E_NULL);
  CHECK(nvfp4_attention(&s, &h, &h, &h, &h, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_E_SHAPE);
  s.batch = INT64_MAX; s.q_len = INT64_MAX; s.k_len = INT64_MAX; s.heads = s.kv_heads = 1; s.head_dim = 64; s.scale = 1;
  CHECK(nvfp4_attention(&s, &h, &h, &h, &h, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_E_SHAPE);
  s.batch = 1 << 30; s.q_len = s.k_len = 1 << 30; s.total_q = s.total_k = (int64_t)1 << 60; s.heads = s.kv_heads = 65535;
  CHECK(nvfp4_attention(&s, &h, &h, &h, &h, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_E_SHAPE);
  CHECK(nvfp4_attention_backward_workspace_bytes(&s) == 0);
  CHECK(nvfp4::launched == 0);
  /* more tensors than one launch takes, and more workgroups than one grid: cut into launches */
  static nvfp4_adamw_tensor t[1000]; memset(t, 0, sizeof t);
  for (int i = 0; i < 1000; ++i) {
    t[i].param = t[i].m = t[i].v = FAKE; t[i].grad = FAKE; t[i].n = i % 10 == 3 ? 0 : (int64_t)1 << 34; t[i].state_bits = 32;
  }
  nvfp4_adamw_config c; memset(&c, 0, sizeof c);
  c.beta1 = 0.9; c.beta2 = 0.99; c.eps = 1e-8f; c.step = ((int64_t)1 << 47) - 1; c.seed = ~0ull;
  CHECK(nvfp4_adamw(t, 1000, &c, nullptr) == NVFP4_OK);
  CHECK(nvfp4::adam_tensors == 900 && nvfp4::adam_ends == 900 * (((int64_t)1 << 34) / nvfp4::kAdamChunk));
  /* division by a product: at the borders of every quotient, for small, round and large divisors */
  for (uint64_t k = 0; k < 3000; ++k) {
    const uint32_t d = k < 2000 ? (uint32_t)k + 1 : k < 2090 ? (1u << (k - 2000) / 3) + (uint32_t)(k % 3) - 1 : (uint32_t)(k * 2654435761u % 0x7FFFFFFFu) + 1;
    if (d == 0) continue;
    const nvfp4::Divisor v = nvfp4::divisor(d);
    for (uint64_t q = 0, j = 0; j < 200; ++j, q = j < 100 ? j : (0x7FFFFFFFull / d) - (199 - j)) {
      for (uint64_t r = 0; r < 2; ++r) {
        const uint64_t n = r ? q * d + d - 1 : q * d;
        if (n > 0x7FFFFFFF || q > 0x7FFFFFFF) continue;
        CHECK((n * v.by) >> v.shift == n / d);
      }
    }
  }
  printf("ok\n");
  return 0;
}
"""


def test_validation_under_asan_and_ubsan(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    drv, exe = tmp_path / "drv.cpp", tmp_path / "train_abi_san"
    drv.write_text(DRIVER)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]
    r = subprocess.run([hipcc, "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-g"] + san +
                       ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", str(exe), os.path.join(CSRC, "train_api.cpp"),
                        str(drv)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr[-4000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
