"""The block operators' host code with launches that are only looked at, under the
host sanitizers: what is launched stays within the workspace that was asked for, and
grids within what a launch counts."""
import os
import shutil
import subprocess

import pytest

from test_train_abi_cpu import CSRC, ROOT

DRIVER = r"""
#include <stdio.h>
#include <string.h>
#include <set>
#include <hip/hip_runtime.h>
#include "nvfp4.h"
#include "block_kernels.hpp"
#define CHECK(c) do { if (!(c)) { printf("check failed line %d: %s\n", __LINE__, #c); failed = 1; } } while (0)
int failed = 0;
static char *const base = (char *)0x100000;
static size_t bytes = 0;
namespace nvfp4 {
int ropes = 0, products = 0, sums = 0, forms = 0, updates = 0, tiles[3] = {0, 0, 0};
int64_t elements = 0;
void inside(const void *p, size_t n) { CHECK((const char *)p >= base && (const char *)p + n <= base + bytes); }
hipError_t launch_rope(const RopeArgs &, hipStream_t) { ++ropes; return hipSuccess; }
hipError_t launch_rope_backward(const RopeArgs &a, hipStream_t) {
  ++ropes;
  for (const RopeSide &t : a.side)
    if (t.dweight) inside(t.parts, (size_t)t.groups * a.dim * 4);
  if (a.side[0].dweight && a.side[1].dweight) CHECK(a.side[1].parts == a.side[0].parts + (size_t)a.side[0].groups * a.dim);
  return hipSuccess;
}
void rope_plan(RopeArgs &a) { for (RopeSide &t : a.side) t.groups = t.heads ? 7 : 0; }
hipError_t launch_gemm_gated(const GatedArgs &, hipStream_t) { return hipSuccess; }
hipError_t launch_gemm_gated_backward(const GatedArgs &, hipStream_t) { return hipSuccess; }
void whole(const MuonArgs &a) {
  CHECK(a.count >= 1 && a.count <= kMuonMats);
  for (int i = 0; i < a.count; ++i) {
    const MuonMat &t = a.mat[i];
    inside(t.direct, (size_t)(t.rp * muon_ld(t.cp)) * 2);
    inside(t.turned, (size_t)(t.cp * muon_ld(t.rp)) * 2);
    inside(t.parts, kMuonParts * sizeof(double));
    CHECK(t.rp >= t.rows && t.cp >= t.cols && t.rp % 64 == 0 && t.cp % 64 == 0);
    for (int j = 0; j < i; ++j) CHECK(a.mat[j].direct != t.direct && a.mat[j].index != t.index);
  }
}
std::set<const _Float16 *> formed;
hipError_t launch_muon_sums(MuonArgs &a, hipStream_t) { whole(a); ++sums; return hipSuccess; }
hipError_t launch_muon_form(MuonArgs &a, hipStream_t) {
  whole(a);
  ++forms;
  formed.clear();
  for (int i = 0; i < a.count; ++i) formed.insert({a.mat[i].direct, a.mat[i].turned});
  return hipSuccess;
}
hipError_t launch_muon_update(MuonArgs &a, hipStream_t) {
  whole(a);
  ++updates;
  int64_t groups = 0;
  for (int i = 0; i < a.count; ++i) {
    CHECK(formed.count(a.mat[i].direct));
    elements += (int64_t)a.mat[i].rows * a.mat[i].cols;
    groups += ((int64_t)a.mat[i].rows * a.mat[i].cols + kMuonChunk - 1) / kMuonChunk;
  }
  CHECK(groups < (1 << 24));
  return hipSuccess;
}
hipError_t launch_muon_product(NsArgs &a, int tile, hipStream_t) {
  ++products;
  ++tiles[tile == 256 ? 0 : tile == 128 ? 1 : 2];
  int64_t groups = 0;
  for (int i = 0; i < a.count; ++i) {
    const NsMat &t = a.mat[i];
    CHECK(t.M % tile == 0 && t.N % tile == 0 && t.K % 64 == 0 && t.M > 0 && t.N > 0 && t.K > 0);
    inside(t.p, (size_t)(t.M * muon_ld(t.K)) * 2);
    inside(t.q, (size_t)(t.N * muon_ld(t.K)) * 2);
    if (t.d) inside(t.d, (size_t)(t.M * muon_ld(t.N)) * 2);
    if (t.dt) inside(t.dt, (size_t)(t.N * muon_ld(t.M)) * 2);
    if (t.e) inside(t.e, (size_t)(t.M * muon_ld(t.N)) * 2);
    CHECK(t.d || t.dt);
    // nothing is written that the same launch reads
    for (const _Float16 *out : {t.d, t.dt}) CHECK(!out || (out != t.p && out != t.q && out != t.e));
    if (a.symmetric) CHECK(t.M == t.N && t.d == t.dt && (t.p == t.q || t.K == t.M));
    // what is read has been formed, and not by another group
    for (const _Float16 *in : {t.p, t.q, t.e}) CHECK(!in || formed.count(in));
    CHECK((t.e != nullptr) == (a.mat[0].e != nullptr));
    groups += (int64_t)(t.M / tile) * (t.N / tile);
  }
  for (int i = 0; i < a.count; ++i)
    for (const _Float16 *out : {a.mat[i].d, a.mat[i].dt})
      if (out) formed.insert(out);
  CHECK(groups < (1 << 24));
  return hipSuccess;
}
}
extern "C" uint16_t nvfp4_rht_sign_mask(uint64_t) { return 0; }
using namespace nvfp4;
int main() {
  static nvfp4_muon_tensor t[120];
  memset(t, 0, sizeof t);
  nvfp4_muon_config c;
  memset(&c, 0, sizeof c);
  c.lr = 0.1f, c.momentum = 0.9, c.nesterov = 1, c.a = 3.4445, c.b = -4.775, c.c = 2.0315;
  uint32_t r = 12345;
  for (int round = 0; round < 60; ++round) {
    const int n = 1 + (int)((r = r * 1664525u + 1013904223u) >> 16) % 120;
    int64_t want = 0;
    for (int i = 0; i < n; ++i) {
      const int big = round % 4 == 0 ? 12 : round % 4 == 1 ? 9 : 6;
      const auto side = [&] { r = r * 1664525u + 1013904223u; return (int64_t)((r >> 8) % (1u << (1 + (r >> 28) % big))); };
      t[i].rows = side(), t[i].cols = side();
      t[i].param = (void *)((uintptr_t)0x10000000 + i * 0x1000);
      t[i].grad = (void *)((uintptr_t)0x20000000 + i * 0x1000);
      t[i].m = i % 3 ? (float *)((uintptr_t)0x30000000 + i * 0x1000) : nullptr;
      want += t[i].rows * t[i].cols;
    }
    c.steps = 1 + round % 6;
    bytes = nvfp4_muon_workspace_bytes(t, n);
    sums = forms = updates = products = 0;
    elements = 0;
    CHECK(nvfp4_muon(t, n, &c, base, bytes, nullptr) == NVFP4_OK);
    CHECK(elements == want && sums == forms && sums == updates && products >= 3 * c.steps * sums && products <= 4 * c.steps * sums);
  }
  // one matrix of the largest sizes
  for (const auto &s : {(int64_t)1 << 17, (int64_t)1 << 16}) {
    t[0].rows = s, t[0].cols = ((int64_t)1 << 33) / s;
    bytes = nvfp4_muon_workspace_bytes(t, 1);
    CHECK(bytes > 0 && nvfp4_muon(t, 1, &c, base, bytes, nullptr) == NVFP4_OK);
  }
  t[0].rows = 1024, t[0].cols = 1536;  // chains of three and two steps
  c.steps = 5;
  bytes = nvfp4_muon_workspace_bytes(t, 1);
  products = 0;
  CHECK(nvfp4_muon(t, 1, &c, base, bytes, nullptr) == NVFP4_OK && products == 18);
  t[0].cols = 1535;
  bytes = nvfp4_muon_workspace_bytes(t, 1);
  products = 0;
  CHECK(nvfp4_muon(t, 1, &c, base, bytes, nullptr) == NVFP4_OK && products == 15);
  t[0].rows = t[0].cols = 2048;  // tiles by what they take
  tiles[0] = tiles[1] = tiles[2] = 0;
  bytes = nvfp4_muon_workspace_bytes(t, 1);
  CHECK(nvfp4_muon(t, 1, &c, base, bytes, nullptr) == NVFP4_OK && tiles[0] == 0 && tiles[1] > 0);
  t[0].rows = 5120, t[0].cols = 20480;
  tiles[0] = tiles[1] = tiles[2] = 0;
  bytes = nvfp4_muon_workspace_bytes(t, 1);
  CHECK(nvfp4_muon(t, 1, &c, base, bytes, nullptr) == NVFP4_OK && tiles[1] == 0 && tiles[2] == 0);

  nvfp4_qk_rope_args a;
  memset(&a, 0, sizeof a);
  for (nvfp4_rope_heads *h : {&a.q, &a.k}) {
    const uintptr_t at = h == &a.q ? 0x1000000 : 0x2000000;
    h->heads = 4;
    h->x = {(void *)at, 0, 256, 64}, h->y = {(void *)(at + 0x100000), 0, 256, 64}, h->dx = {(void *)(at + 0x200000), 0, 256, 64};
    h->weight = (void *)(at + 0x300000), h->dweight = (float *)(at + 0x400000);
  }
  a.batch = 1, a.tokens = 9, a.head_dim = 64, a.rot_dim = 32, a.freqs = (const double *)0x40000, a.eps = 1e-6f, a.magnitude = 1;
  bytes = nvfp4_qk_rope_backward_workspace_bytes(&a);
  CHECK(bytes == 2 * 7 * 64 * 4);
  CHECK(nvfp4_qk_rope_backward(&a, base, bytes, nullptr) == NVFP4_OK && ropes == 1);
  a.k.dweight = nullptr;
  bytes = nvfp4_qk_rope_backward_workspace_bytes(&a);
  CHECK(bytes == 7 * 64 * 4 && nvfp4_qk_rope_backward(&a, base, bytes, nullptr) == NVFP4_OK);
  a.tokens = 0;  // nothing but the weights' gradients, which are zero
  CHECK(nvfp4_qk_rope_backward(&a, base, bytes, nullptr) == NVFP4_OK && ropes == 3);
  a.q.dweight = nullptr;
  CHECK(nvfp4_qk_rope_backward(&a, nullptr, 0, nullptr) == NVFP4_OK && ropes == 3);
  if (!failed) printf("ok\n");
  return failed;
}
"""


def test_host_code_without_a_gpu(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    drv, exe = tmp_path / "drv.cpp", tmp_path / "contract"
    drv.write_text(DRIVER)
    r = subprocess.run([hipcc, "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-g",
                        "-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", str(exe),
                        os.path.join(CSRC, "block_api.cpp"), str(drv)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr[-4000:]
