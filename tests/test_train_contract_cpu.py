"""CPU-only checks of what the training operators' entry points accept and
refuse at the borders of their contracts."""
import ctypes
import os
import shutil
import subprocess

import pytest

import nvfp4_bit_quantization_amd as nv
from test_train_abi_cpu import ALIGN, CSRC, FAKE, LD, NULL, ROOT, SHAPE, UNSUPPORTED, VALUE, WORKSPACE, _adam, _config, _heads, _norm, _norm_grad, _shape


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nv.LIB_PATH):
        from nvfp4_bit_quantization_amd import build
        build.build()
    return nv.lib()


@pytest.mark.parametrize("eps,status", [(1e-45, VALUE), (1.17e-38, VALUE), (2.0 ** -126, 0), (1e-20, 0)])
def test_adamw_eps_is_normal(L, eps, status):
    """The reciprocal instruction takes subnormal numbers for zero."""
    arr = (nv.nvfp4_adamw_tensor * 1)(_adam(n=0))  # nothing to launch
    assert L.nvfp4_adamw(arr, 1, ctypes.byref(_config(eps=eps)), None) == status


@pytest.mark.parametrize("scale,good", [(1e-45, False), (1.2e-38, False), (7.5e-37, False), (2.0 ** -120, True), (1.0, True),
                                        (2.0 ** 120, True), (1.4e36, False), (3e38, False)])
def test_attention_scale_is_representable(L, scale, good):
    """-lse / scale and scale * log2(e) have to be finite."""
    s, h = _shape(scale=scale), ctypes.byref(_heads())
    assert (L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s)) > 0) == good
    if not good:
        assert L.nvfp4_attention(ctypes.byref(s), h, h, h, h, FAKE, None, 0, None) == VALUE
        assert L.nvfp4_attention_backward(ctypes.byref(s), h, h, h, h, FAKE, h, h, h, h, FAKE, 1 << 30, None) == VALUE


def _distinct(**kw):
    """Tensors of one shape (as many query as key heads), each of its own memory but for those named as another's."""
    t = {n: _heads(data=FAKE * (i + 1)) for i, n in enumerate(("q", "k", "v", "o", "d_o", "dq", "dk", "dv"))}
    for name, (other, change) in kw.items():
        t[name] = _heads(**dict(dict(data=t[other].data), **change))
    return {n: ctypes.byref(x) for n, x in t.items()}


OUTPUTS = [("dq", "q"), ("dq", "k"), ("dq", "v"), ("dq", "d_o"), ("dk", "q"), ("dk", "o"), ("dk", "d_o"), ("dv", "q"),
           ("dv", "o"), ("dv", "d_o"), ("dk", "dq"), ("dv", "dq"), ("dv", "dk")]
IN_PLACE = [("dq", "o"), ("dk", "k"), ("dk", "v"), ("dv", "k"), ("dv", "v")]


@pytest.mark.parametrize("output,other", OUTPUTS + [("o", "k"), ("o", "v")], ids=str)
def test_attention_outputs_keep_off_what_is_still_read(L, output, other):
    s = _shape(heads=2, kv_heads=2)
    t = _distinct(**{output: (other, {})})
    if output == "o":
        assert L.nvfp4_attention(ctypes.byref(s), t["q"], t["k"], t["v"], t["o"], FAKE * 9, None, 0, None) == UNSUPPORTED
        return
    need = L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s))
    order = [t[n] for n in ("q", "k", "v", "o")], [t[n] for n in ("d_o", "dq", "dk", "dv")]
    assert L.nvfp4_attention_backward(ctypes.byref(s), *order[0], FAKE * 9, *order[1], FAKE * 10, need, None) == UNSUPPORTED


@pytest.mark.parametrize("output,other", IN_PLACE + [("o", "q")], ids=str)
def test_attention_in_place_outputs_have_the_strides(L, output, other):
    """What may stand in another tensor's place does so element by element."""
    s = _shape(heads=2, kv_heads=2)
    for change in (dict(token_stride=264), dict(head_stride=72), dict(batch_stride=32 * 256)):
        t = _distinct(**{output: (other, change)})
        if output == "o":
            assert L.nvfp4_attention(ctypes.byref(s), t["q"], t["k"], t["v"], t["o"], FAKE * 9, None, 0, None) == UNSUPPORTED
            continue
        need = L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s))
        order = [t[n] for n in ("q", "k", "v", "o")], [t[n] for n in ("d_o", "dq", "dk", "dv")]
        assert L.nvfp4_attention_backward(ctypes.byref(s), *order[0], FAKE * 9, *order[1], FAKE * 10, need, None) == UNSUPPORTED


def test_workspaces_are_memory():
    """An expanded tensor counts more elements than it has."""
    torch = pytest.importorskip("torch")
    nv._scratch(torch.zeros(64), -1)
    for bad, device in ((torch.zeros(1).expand(64), -1), (torch.zeros(8, 8).t(), -1), (torch.zeros(64), 0)):
        with pytest.raises(ValueError):
            nv._scratch(bad, device)


@pytest.mark.parametrize("change", [
    dict(sum=FAKE * 2, y=FAKE * 2), dict(y=FAKE * 3, ld_y=72), dict(y=FAKE * 4, ld_y=72), dict(y=FAKE * 3, y_dtype=0),
    dict(sum=FAKE * 3, ld_sum=72), dict(sum=FAKE * 4, ld_sum=72)], ids=str)
def test_layernorm_outputs_in_place(L, change):
    """The two outputs stand apart, and what stands in an input's place has its rows as far apart, in bytes."""
    a = dict(x=FAKE * 3, residual=FAKE * 4, y=FAKE * 5, sum=FAKE * 6, ld_residual=64, ld_sum=64)
    assert L.nvfp4_layernorm(ctypes.byref(_norm(**dict(a, **change))), None) == UNSUPPORTED


@pytest.mark.parametrize("change", [dict(dx=FAKE * 2, ld_dx=72), dict(dx=FAKE * 3, ld_dx=72), dict(dx=FAKE * 4, ld_dx=72),
                                    dict(dx=FAKE * 2, y_dtype=0)], ids=str)
def test_layernorm_backward_in_place(L, change):
    a = dict(dy=FAKE * 2, x=FAKE * 3, dsum=FAKE * 4, ld_dsum=64, dx=FAKE * 5)
    need = L.nvfp4_layernorm_backward_workspace_bytes(4, 64)
    assert L.nvfp4_layernorm_backward(ctypes.byref(_norm_grad(**dict(a, **change))), FAKE, need, None) == UNSUPPORTED


@pytest.mark.parametrize("tokens,heads,kv_heads,parts", [
    (6144, 16, 16, 1), (12288, 8, 8, 1), (4096, 16, 16, 1), (8192, 8, 8, 2), (4096, 40, 8, 4), (4096, 20, 4, 4), (4096, 24, 4, 8)])
def test_attention_gradient_parts(L, tokens, heads, kv_heads, parts):
    """How often dK and dV are split goes by the tiles of 128 keys: only up to 512 of them get a second set of
    workgroups.  The parts are what the workspace holds beside two numbers for each query."""
    s = _shape(batch=1, q_len=tokens, k_len=tokens, total_q=tokens, total_k=tokens, heads=heads, kv_heads=kv_heads, head_dim=128)
    stats = 2 * ((4 * (heads * tokens + 1) + 255) // 256 * 256)
    held = 2 * 4 * 128 * kv_heads * tokens
    assert L.nvfp4_attention_backward_workspace_bytes(ctypes.byref(s)) == stats + (parts * held if parts > 1 else 0)


# the entry points' host code with launches that are only counted
DRIVER = r"""
#include <stdio.h>
#include <string.h>
#include <hip/hip_runtime.h>
#include "nvfp4.h"
#include "train_kernels.hpp"
namespace nvfp4 {
int launched = 0;
hipError_t launch_layernorm(const nvfp4_layernorm_args &, hipStream_t) { return hipSuccess; }
int64_t layernorm_backward_parts(int64_t, int64_t) { return 1; }
hipError_t launch_layernorm_backward(const nvfp4_layernorm_backward_args &, float *, hipStream_t) { return hipSuccess; }
int64_t adam_groups = 0, adam_most = 0;
hipError_t launch_adamw(const AdamArgs &a, hipStream_t) {
  const int64_t n = a.tensor(a.count - 1).end;
  ++launched, adam_groups += n;
  if (n > adam_most) adam_most = n;
  return hipSuccess;
}
int attention_q_parts(const AttnArgs &) { return 1; }
int attention_k_parts(const AttnArgs &) { return 1; }
hipError_t launch_attention(const AttnArgs &, hipStream_t) { ++launched; return hipSuccess; }
hipError_t launch_attention_backward(const AttnArgs &, hipStream_t) { ++launched; return hipSuccess; }
}
#define FAKE ((void *)0x10000)
#define CHECK(c) do { if (!(c)) { printf("check failed line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  // a launch of 256 threads to a workgroup counts its threads in 32 bits
  static nvfp4_adamw_tensor t[200];
  memset(t, 0, sizeof t);
  for (int i = 0; i < 200; ++i) {
    t[i].param = t[i].m = t[i].v = FAKE, t[i].grad = FAKE, t[i].state_bits = 32;
    t[i].n = i % 3 ? ((int64_t)1 << 34) - i * 5000 : i * 1000;
  }
  nvfp4_adamw_config c;
  memset(&c, 0, sizeof c);
  c.beta1 = 0.9, c.beta2 = 0.99, c.eps = 1e-8f, c.step = 1;
  CHECK(nvfp4_adamw(t, 200, &c, nullptr) == NVFP4_OK);
  int64_t groups = 0;
  for (int i = 0; i < 200; ++i) groups += (t[i].n + nvfp4::kAdamChunk - 1) / nvfp4::kAdamChunk;
  CHECK(nvfp4::adam_groups == groups);
  CHECK(nvfp4::adam_most < (int64_t)1 << 24);

  // packed sequences: no tokens at all need no buffers, and launch nothing
  nvfp4_attention_shape s;
  memset(&s, 0, sizeof s);
  s.batch = 2, s.heads = 4, s.kv_heads = 2, s.head_dim = 64, s.causal = 1, s.scale = 0.125f;
  s.cu_q = s.cu_k = (const int32_t *)FAKE;
  const nvfp4_heads none = {nullptr, 0, 256, 64}, some = {FAKE, 0, 256, 64}, out = {(void *)0x20000, 0, 256, 64};
  const nvfp4_heads dq = {(void *)0x30000, 0, 256, 64}, dk = {(void *)0x40000, 0, 256, 64}, dv = {(void *)0x50000, 0, 256, 64};
  for (int64_t most = 0; most <= 7; most += 7) {
    s.q_len = most, s.k_len = 9, s.total_q = 0, s.total_k = 20;
    nvfp4::launched = 0;
    CHECK(nvfp4_attention_workspace_bytes(&s) == 0);
    CHECK(nvfp4_attention(&s, &none, &some, &some, &none, nullptr, nullptr, 0, nullptr) == NVFP4_OK);
    CHECK(nvfp4::launched == 0);
    CHECK(nvfp4_attention_backward(&s, &none, &some, &some, &none, nullptr, &none, &none, &dk, &dv, FAKE, 1 << 20, nullptr) == NVFP4_OK);
    CHECK(nvfp4::launched == 1);
    CHECK(nvfp4_attention(&s, &none, &none, &some, &none, nullptr, nullptr, 0, nullptr) == NVFP4_E_NULL);
    CHECK(nvfp4_attention_backward(&s, &none, &some, &some, &none, nullptr, &none, &none, &none, &dv, FAKE, 1 << 20, nullptr) == NVFP4_E_NULL);
    s.q_len = 9, s.k_len = most, s.total_q = 20, s.total_k = 0;
    nvfp4::launched = 0;
    CHECK(nvfp4_attention(&s, &some, &none, &none, &out, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_OK);
    CHECK(nvfp4_attention_backward(&s, &some, &none, &none, &out, (float *)FAKE, &out, &dq, &none, &none, FAKE, 1 << 20, nullptr) == NVFP4_OK);
    CHECK(nvfp4::launched == 2);
    CHECK(nvfp4_attention(&s, &some, &none, &none, &out, nullptr, nullptr, 0, nullptr) == NVFP4_E_NULL);
    CHECK(nvfp4_attention(&s, &some, &none, &none, &none, (float *)FAKE, nullptr, 0, nullptr) == NVFP4_E_NULL);
    s.q_len = s.k_len = most, s.total_q = s.total_k = 0;
    CHECK(nvfp4_attention_backward(&s, &none, &none, &none, &none, nullptr, &none, &none, &none, &none, FAKE, 1 << 20, nullptr) == NVFP4_OK);
    CHECK(nvfp4::launched == 2);
  }
  s.cu_q = s.cu_k = nullptr;
  CHECK(nvfp4_attention(&s, &none, &none, &none, &none, nullptr, nullptr, 0, nullptr) == NVFP4_E_SHAPE);
  printf("ok\n");
  return 0;
}
"""


def test_entry_points_without_a_gpu(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    drv, exe = tmp_path / "drv.cpp", tmp_path / "contract"
    drv.write_text(DRIVER)
    r = subprocess.run([hipcc, "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, "-o", str(exe), os.path.join(CSRC, "train_api.cpp"), str(drv)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr[-4000:]
