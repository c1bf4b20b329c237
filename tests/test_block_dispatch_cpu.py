"""Which kernel the 4-bit products launch, by launches that are only looked at: scales
may stand at any address, but the pipeline's transfers move them by dwords."""
import os
import shutil
import subprocess

import pytest

from nvfp4_bit_quantization_amd import build
from test_train_abi_cpu import CSRC

DRIVER = r"""
#include <stdio.h>
#include <string.h>
#include <map>
#include <string>
#include <hip/hip_runtime.h>
#include "block_kernels.hpp"
static std::map<const void *, std::string> *names;
static std::string launched;
extern "C" {
void **__hipRegisterFatBinary(const void *) { static void *module; return &module; }
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *, void *, void *, void *, int *) {
  if (!names) names = new std::map<const void *, std::string>;
  (*names)[host] = name;
}
hipError_t hipLaunchKernel(const void *f, dim3, dim3, void **, size_t, hipStream_t) {
  launched = names && names->count(f) ? (*names)[f] : "?";
  return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *s) { *s = hipStreamCaptureStatusNone; return hipSuccess; }
}
using namespace nvfp4;
int failed = 0;
void want(const char *what, const char *kernel) {
  if (launched.find(kernel) == std::string::npos) printf("%s: %s, not %s\n", what, launched.c_str(), kernel), failed = 1;
}
int main() {
  const uint8_t *p = (const uint8_t *)0x100000;
  GatedArgs a;
  memset(&a, 0, sizeof a);
  a.g.M = 8192, a.g.N = 2048, a.g.K = 256;
  for (int off = 0; off < 4; ++off)
    for (int which = 0; which < 3; ++which) {
      a.g.a_codes = a.g.b_codes = a.u_codes = p;
      a.g.a_scales = p + (which == 0 ? off : 0);
      a.g.b_scales = p + (which == 1 ? off : 4);
      a.u_scales = p + (which == 2 ? off : 8);
      launch_gemm_gated(a, nullptr);
      want("gated", off ? "gated_generic_kernel" : "gated_fast_kernel");
      launch_gemm_gated_backward(a, nullptr);
      want("gated gradient", off && which < 2 ? "gated_generic_kernel" : "gated_fast_kernel");
      GemmArgs g = a.g;
      g.ldc = g.N;
      launch_gemm(g, nullptr, 0, nullptr);
      want("gemm", off && which < 2 ? "gemm_generic_kernel" : "gemm_fast_kernel");
    }
  a.g.M = 64;
  a.g.a_scales = p + 1;
  launch_gemm_gated(a, nullptr);
  want("gated, few rows", "gated_skinny_kernel");
  if (!failed) printf("ok\n");
  return failed;
}
"""


def test_scales_that_are_not_aligned_go_by_other_kernels(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    drv, exe = tmp_path / "drv.cpp", tmp_path / "dispatch"
    drv.write_text(DRIVER)
    r = subprocess.run([hipcc, "-x", "hip"] + [f for f in build.FLAGS if f not in ("-O3", "-fPIC")] +
                       ["-O1", "-o", str(exe)] + [os.path.join(CSRC, s) for s in ("gated.hip", "gemm.hip")] + [str(drv)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-2000:] + r.stderr[-2000:]
