"""Loads from global memory straight to LDS, in the library as it is built.

A vector memory instruction may not read a scalar register within five wait
states of a vector instruction's write to it (CDNA3 ISA, manually inserted wait
states; the hardware does not wait by itself).  The compiler keeps this for its
own instructions and not for those written in assembly, whose descriptors come
out of v_readfirstlane, so each such load has to bring its own.  It does not
know either that the assembly writes m0: where it does, nothing else may."""
import os
import re
import shutil
import subprocess
from collections import Counter

import pytest

import combine_get_dispatch_amd as ep
from combine_get_dispatch_amd import _build

WAIT_STATES = 5
LLVM = "/opt/rocm/llvm/bin/llvm-objdump"


def scalars(operand):
    """Numbers of the scalar registers of s7 or s[4:7]; VCC's as -1."""
    if operand.startswith("vcc"):
        return {-1}
    m = re.fullmatch(r"s(\d+)", operand) or re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if not m:
        return set()
    return set(range(int(m[1]), int(m[m.lastindex]) + 1))


def hazards(lines):
    """(kernel, line) of each load to LDS that is too near a vector
    instruction's write to its scalars, and per kernel the numbers of loads and
    of instructions that name m0.  What comes before a branch's target is not
    known: it counts as such a write."""
    found, loads, m0 = [], Counter(), Counter()
    kernel, since, unknown = "", {}, 0  # wait states since a write; since a target
    for line in lines:
        head = re.match(r"[0-9a-f]+ <(.+)>:", line)
        if head:  # of a kernel, or a branch's target
            kernel = kernel if re.fullmatch(r"L\d+", head[1]) else head[1]
            since, unknown = {}, 0
            continue
        text = line.split("//")[0].split()
        if not text or line[:1] not in " \t":
            continue
        op, operands = text[0], [t.rstrip(",") for t in text[1:]]
        if op.startswith("buffer_load") and "lds" in operands:
            loads[kernel] += 1
            reads = set().union(*map(scalars, operands))
            if unknown < WAIT_STATES or any(since.get(s, WAIT_STATES) < WAIT_STATES
                                            for s in reads):
                found.append((kernel, line.strip()))
        if "m0" in operands:
            m0[kernel] += 1
        states = int(operands[0], 0) + 1 if op == "s_nop" else 1
        unknown += states
        since = {s: n + states for s, n in since.items() if n + states < WAIT_STATES}
        if op.startswith("v_"):
            for operand in operands[:2]:  # a result, and a carry or the like
                since.update(dict.fromkeys(scalars(operand), 0))
    return found, loads, m0


def test_hazards_are_seen():
    bad = """0000000000001900 <kernel>:
	v_readfirstlane_b32 s6, v3                                 // 000000001904: 7E0C0503
	s_mov_b32 m0, s9                                           // 000000001908: BEFC0009
	s_nop 0                                                    // 00000000190C: BF800000
	buffer_load_dwordx4 v15, s[4:7], 0 offen lds               // 000000001910: E05D1000
""".splitlines()
    at = "kernel", bad[4].strip()
    assert hazards(["\ts_nop 4"] + bad) == ([at], {"kernel": 1}, {"kernel": 1})
    assert not hazards(bad[:1] + ["\ts_nop 4"] + [bad[1].replace("s6", "s8")] + bad[2:])[0]
    assert hazards([t.replace("s_nop 0", "s_nop 2") for t in bad])[0]
    assert not hazards([t.replace("s_nop 0", "s_nop 3") for t in bad])[0]
    assert hazards(["0000000000001900 <L3>:", "\ts_nop 3"] + bad[4:])[0]


def test_loads_to_lds_wait_for_their_scalars(tmp_path):
    if not os.path.exists(LLVM):
        pytest.skip("llvm-objdump not found")
    ep.lib()
    so = shutil.copy(_build.LIB, tmp_path)
    subprocess.run([LLVM, "--offloading", so], cwd=tmp_path, check=True, capture_output=True)
    some = False
    for name in sorted(os.listdir(tmp_path)):
        if not name.endswith("gfx950"):
            continue
        asm = subprocess.run([LLVM, "-d", "--symbolize-operands", str(tmp_path / name)], check=True,
                             capture_output=True, text=True).stdout
        found, loads, m0 = hazards(asm.splitlines())
        assert not found, (len(found), sum(loads.values()), found[:4])
        for kernel, n in loads.items():
            assert m0[kernel] == n, kernel
            some = True
    assert some
