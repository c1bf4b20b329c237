"""The wait states that transfers to LDS need, counted in the block operators'
kernels as in the others'."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from nvfp4_bit_quantization_amd import build
from test_wait_states_cpu import FAR, _program, _scalars, _wait_states

SOURCES = ["gated.hip", "muon.hip"]


@pytest.fixture(scope="module")
def transfers(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    folder = tmp_path_factory.mktemp("asm")

    def assembly(src):
        out = str(folder / (src + ".s"))
        r = subprocess.run([hipcc] + build.FLAGS + build.FILE_FLAGS.get(src, []) +
                           ["-x", "hip", "-S", "--offload-device-only", os.path.join(build.CSRC, src), "-o", out],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-4000:]
        return open(out).read()

    found = []
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        for src, text in zip(SOURCES, ex.map(assembly, SOURCES)):
            for m in re.finditer(r"^(_Z\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M):
                ins, before = _program(m.group(2))
                found += [(src, m.group(1), x, i, ins, before) for i, x in enumerate(ins) if "_load_lds_" in x]
    assert {f[0] for f in found} == set(SOURCES)
    return found


def test_transfer_waits_for_m0(transfers):
    for src, kernel, x, i, ins, before in transfers:
        n = _wait_states(i, ins, before, lambda y: re.match(r"s_\w+ m0\b", y))
        assert 1 <= n < FAR, "%s, %s: %d wait states between M0 and %s" % (src, kernel, n, x)


def test_transfer_waits_for_its_base(transfers):
    for src, kernel, x, i, ins, before in transfers:
        base = _scalars(x)
        assert base, x

        def writes(y):
            return y.startswith("v_") and bool(base & _scalars(y.split(None, 1)[1].split(",")[0]))

        n = _wait_states(i, ins, before, writes)
        assert n >= 5, "%s, %s: %d wait states between a vector instruction and %s" % (src, kernel, n, x)
