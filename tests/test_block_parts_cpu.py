"""The second parts of the orthogonalised steps' matrices, which stand behind the first
ones, in the host code's plan: both within the workspace, and no matrix in another's."""
import os
import shutil
import subprocess

import pytest

import test_block_contract_cpu as contract
from test_train_abi_cpu import CSRC, ROOT

# every matrix that a product or the first pass works on, with both its parts, and what it may not share
SEEN = r"""
std::map<const char *, size_t> held;  // of one call: where a matrix begins, and its bytes
void inside(const void *p, size_t n);
void both(const void *p, int64_t rows, int64_t cols) {
  const size_t n = (size_t)(rows * muon_ld(cols)) * 4;
  inside(p, n);
  size_t &was = held[(const char *)p];
  CHECK(was == 0 || was == n);
  was = n;
}
void apart() {
  const char *end = nullptr;
  for (const auto &h : held) {
    CHECK(h.first >= end);
    end = h.first + h.second;
  }
}
"""


def driver():
    text = contract.DRIVER.replace("#include <set>", "#include <map>\n#include <set>")
    for what in ("t.direct, (size_t)(t.rp * muon_ld(t.cp)) * 2", "t.turned, (size_t)(t.cp * muon_ld(t.rp)) * 2",
                 "t.p, (size_t)(t.M * muon_ld(t.K)) * 2", "t.q, (size_t)(t.N * muon_ld(t.K)) * 2", "t.d, (size_t)(t.M * muon_ld(t.N)) * 2",
                 "t.dt, (size_t)(t.N * muon_ld(t.M)) * 2", "t.e, (size_t)(t.M * muon_ld(t.N)) * 2"):
        assert text.count("inside(" + what + ")") == 1
        name, rest = what.split(", (size_t)(")
        rows, cols = rest[:rest.index(")")].split(" * muon_ld(")
        text = text.replace("inside(" + what + ")", "both(%s, %s, %s)" % (name, rows, cols))
    at = "void inside("
    text = text.replace(at, SEEN + at, 1)
    at = "hipError_t launch_muon_sums(MuonArgs &a, hipStream_t) { "
    assert text.count(at) == 1
    text = text.replace(at, at + "held.clear(); ")  # a group's matrices
    at = "hipError_t launch_muon_update(MuonArgs &a, hipStream_t) {"
    assert text.count(at) == 1
    return text.replace(at, at + " apart();")


def test_both_parts_in_the_workspace(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    drv, exe = tmp_path / "drv.cpp", tmp_path / "parts"
    drv.write_text(driver())
    r = subprocess.run([hipcc, "-x", "hip", "--offload-arch=gfx950", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                        "-o", str(exe), os.path.join(CSRC, "block_api.cpp"), str(drv)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout[-2000:] + r.stderr[-2000:]
