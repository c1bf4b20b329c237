"""Wait states that the hardware leaves to the program, counted in the built
kernels' assembly.  The transfers from global memory to LDS are written in
inline asm, into which the compiler's own pass for them does not look.

A GFX9 transfer to LDS takes its LDS address from M0 and needs a wait state (an
instruction, or a count of s_nop) after the scalar instruction that wrote it, and
any memory access needs five after a vector instruction wrote its scalar base."""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from nvfp4_bit_quantization_amd import build

SOURCES = ["gemm.hip", "mxfp4.hip", "attention.hip"]
FAR = 9  # wait states that are looked back at most


@pytest.fixture(scope="module")
def transfers(tmp_path_factory):
    """Every transfer to LDS: [(source, kernel, instruction, its index, instructions, their predecessors)]."""
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


def _program(body):
    """A function's instructions, and the indices of those that each may follow."""
    ins, labels = [], {}
    for line in body.splitlines():
        line = line.split(";")[0].strip()
        label = re.match(r"([.\w$]+):", line)
        if label:
            labels[label.group(1)] = len(ins)
        elif line and not line.startswith("."):
            ins.append(line)
    before = [[] for _ in ins]
    for i, x in enumerate(ins):
        if x.split()[0] not in ("s_branch", "s_endpgm") and i + 1 < len(ins):
            before[i + 1].append(i)
        jump = re.match(r"s_c?branch\w*\s+(\S+)", x)
        if jump:
            before[labels[jump.group(1)]].append(i)
    return ins, before


def _wait_states(at, ins, before, writes):
    """The fewest wait states on any way from an instruction that `writes` to instruction `at`."""
    least, seen, todo = FAR, {}, [(at, 0)]
    while todo:
        i, n = todo.pop()
        for j in before[i]:
            if writes(ins[j]):
                least = min(least, n)
                continue
            nop = re.match(r"s_nop (\d+)", ins[j])
            m = n + (int(nop.group(1)) + 1 if nop else 1)
            if m < least and seen.get(j, FAR) > m:
                seen[j] = m
                todo.append((j, m))
    return least


def test_transfer_waits_for_m0(transfers):
    for src, kernel, x, i, ins, before in transfers:
        n = _wait_states(i, ins, before, lambda y: re.match(r"s_\w+ m0\b", y))
        assert 1 <= n < FAR, "%s, %s: %d wait states between M0 and %s" % (src, kernel, n, x)


def _scalars(text):
    """The scalar registers named in some operands."""
    out = set()
    for m in re.finditer(r"\bs(?:(\d+)\b|\[(\d+):(\d+)\])", text):
        out |= {int(m.group(1))} if m.group(1) else set(range(int(m.group(2)), int(m.group(3)) + 1))
    return out


def test_transfer_waits_for_its_base(transfers):
    """A base address that the vector unit wrote (a lane's value, a reload of a spilled one) needs five wait states."""
    for src, kernel, x, i, ins, before in transfers:
        base = _scalars(x)
        assert base, x

        def writes(y):
            return y.startswith("v_") and bool(base & _scalars(y.split(None, 1)[1].split(",")[0]))

        n = _wait_states(i, ins, before, writes)
        assert n >= 5, "%s, %s: %d wait states between a vector instruction and %s" % (src, kernel, n, x)
