"""Loads from memory to LDS that are written in inline assembly: the compiler
does not look into them for hazards.  A buffer load may follow a write of its
descriptor by the vector unit by five wait states at the earliest, and a write of
m0 by one (AMD's CDNA3 instruction set guide, manually inserted wait states)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_precision_quantization_amd", "csrc")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def _wait_states(op, args):
    return int(args[0], 0) + 1 if op == "s_nop" else 1


def _lines(text):
    for line in text:
        line = re.split(r"//|;", line)[0].strip()
        if line:
            op, _, rest = line.partition(" ")
            yield op, [a.strip() for a in rest.split(",")]


def test_a_block_is_safe_by_itself():
    """The shared core's asm blocks, whatever stands before them: a load's
    descriptor is written by the scalar unit within the block, which no load has to
    wait for, or the block waits five states; m0 is written two instructions before
    and named as changed."""
    text = open(os.path.join(CSRC, "mx_mm.h")).read()
    blocks = re.findall(r'asm volatile\(((?:\s*"[^"]*")+)([^;]*);', text)
    loads = [(b, rest) for b, rest in blocks if " lds" in b]
    assert len(loads) == 2
    for b, rest in loads:
        code = list(_lines("".join(re.findall(r'"([^"]*)"', b)).replace("\\t", " ").split("\\n")))
        at = next(i for i, (op, _) in enumerate(code) if op.startswith("buffer_load"))
        descriptor = _registers(code[at][1][1])
        copied = set().union(*(_registers(a[0]) for op, a in code[:at] if op.startswith("s_mov_b")))
        states = sum(_wait_states(*c) for c in code[:at])
        assert states >= 5 or (descriptor and descriptor <= copied), b
        assert code[0] == ("s_mov_b32", ["m0", "%0"]) and at >= 2, b
        changed = rest.rsplit(":", 1)[1]
        assert all('"%s"' % r in changed for r in ["m0"] + ["s%d" % r for r in descriptor]), b


def _registers(arg):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", arg)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", arg)
    return {int(m[1])} if m else set()


def _hazards(text):
    """(loads to LDS, those too near a vector write of their descriptor or of m0)."""
    before, loads, bad = [], 0, []
    for op, args in _lines(text):
        if op.startswith("buffer_load") and args[-1].endswith(" lds"):
            loads += 1
            # (after a label or a branch the other way in ran at least as long)
            states = 0
            for o, a in reversed(before):
                if o == "s_mov_b32" and a[0] == "m0" and states < 1:
                    bad.append((o, a, op, args))
                if o.startswith("v_") and any(_registers(x) & _registers(args[1]) for x in a[:1]):
                    bad.append((o, a, op, args))
                states += _wait_states(o, a)
                if states >= 5:
                    break
        before = (before + [(op, args)])[-6:]
    return loads, bad


def test_the_search_finds_what_it_looks_for():
    load = "buffer_load_dwordx4 v1, s[12:15], 0 offen lds"
    assert _hazards(["v_readlane_b32 s13, v2, 1", "s_mov_b32 m0, s2", "s_nop 0", load]) [1]
    assert _hazards(["s_mov_b32 m0, s2", load])[1]
    assert _hazards(["v_readfirstlane_b32 s15, v2", "s_nop 4", "s_mov_b32 m0, s2", "s_nop 0", load]) == (1, [])
    assert _hazards(["v_readlane_b32 s16, v2, 1", "s_mov_b32 m0, s2", "s_nop 0", load]) == (1, [])


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_the_built_library(tmp_path):
    """Every load to LDS in the library that was built here."""
    import fp8_precision_quantization_amd as mx
    from fp8_precision_quantization_amd import build
    if not os.path.exists(mx.LIB_PATH):
        build.build()
    lib = shutil.copy(mx.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", os.path.basename(lib)], cwd=tmp_path, check=True, capture_output=True)
    parts = [p for p in os.listdir(tmp_path) if "gfx950" in p]
    assert parts
    loads = 0
    for p in parts:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", p], cwd=tmp_path, check=True, capture_output=True,
                              text=True).stdout
        n, bad = _hazards(text.splitlines())
        assert not bad, (p, bad[:3])
        loads += n
    assert loads > 0
