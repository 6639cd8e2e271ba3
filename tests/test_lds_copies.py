"""CPU: the copies from memory to LDS in the built library, as the hardware needs
them. They stand in inline assembly, where the compiler does not look for pairs of
instructions that must not follow each other directly. On gfx950 the hardware does
not wait by itself
  - between a scalar write of m0 and a copy to LDS, which takes its place there from
    m0: one wait state;
  - between a vector instruction's write of a scalar register and a memory
    instruction that reads it (descriptor, offset): five.
Every instruction is a wait state, s_nop N is N + 1 of them."""

import os
import re
import struct
import subprocess

import pytest

from newton_schulz_matrix_amd import build

BUNDLE = b"__CLANG_OFFLOAD_BUNDLE__"
M0_STATES, SCALAR_STATES = 1, 5
COPY = re.compile(r"^buffer_load_\w+ v\d+, s\[(\d+):(\d+)\], (\S+) .*\blds\b")


def code_objects(lib):
    with open(lib, "rb") as f:
        data = f.read()
    at = data.find(BUNDLE)
    while at >= 0:
        entries, = struct.unpack_from("<Q", data, at + len(BUNDLE))
        p = at + len(BUNDLE) + 8
        for _ in range(entries):
            offset, size, n = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + n]:
                yield data[at + offset:at + offset + size]
            p += 24 + n
        at = data.find(BUNDLE, at + 1)


def instructions(lib, folder):
    """Lists of instructions, one of each code object."""
    dump = os.path.join(os.path.dirname(os.path.dirname(build.hipcc())), "llvm", "bin", "llvm-objdump")
    for i, code in enumerate(code_objects(lib)):
        path = folder / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([dump, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True,
                              check=True).stdout
        yield [line.split("//")[0].strip() for line in text.splitlines() if line.startswith("\t")]


def states(line):
    nop = re.match(r"s_nop (\d+)", line)
    return int(nop.group(1)) + 1 if nop else 1


def scalars(line, operands):
    """Scalar registers among an instruction's first operands."""
    out = set()
    for operand in line.split(None, 1)[-1].split(",")[:operands]:
        operand = operand.strip()
        if one := re.fullmatch(r"s(\d+)", operand):
            out.add(int(one.group(1)))
        elif many := re.fullmatch(r"s\[(\d+):(\d+)\]", operand):
            out.update(range(int(many.group(1)), int(many.group(2)) + 1))
    return out


def faults(lines):
    """(index, reason) of every copy that follows too soon."""
    for i, line in enumerate(lines):
        copy = COPY.match(line)
        if not copy:
            continue
        reads = set(range(int(copy.group(1)), int(copy.group(2)) + 1))
        if offset := re.fullmatch(r"s(\d+)", copy.group(3)):
            reads.add(int(offset.group(1)))
        passed = 0
        for before in reversed(lines[max(0, i - SCALAR_STATES):i]):
            if passed < M0_STATES and re.match(r"s_\w+ m0,", before):
                yield i, before
            # (the second operand of a vector instruction may be one that it writes)
            if before.startswith("v_") and passed < SCALAR_STATES and scalars(before, 2) & reads:
                yield i, before
            if before.startswith("s_"):   # written by a scalar instruction since: that one waits by itself
                reads -= scalars(before, 1)
            passed += states(before)


def test_the_rule_itself():
    copy = "buffer_load_dwordx4 v3, s[8:11], s4 offen lds"
    assert list(faults(["s_mov_b32 m0, s1", copy])) == [(1, "s_mov_b32 m0, s1")]
    assert not list(faults(["s_mov_b32 m0, s1", "s_nop 0", copy]))
    assert not list(faults(["s_add_i32 s2, s2, 1", "s_mov_b32 s1, m0", copy]))
    late = "v_readfirstlane_b32 s10, v1"
    assert list(faults([late, "s_mov_b32 m0, s1", "s_nop 0", copy])) == [(3, late)]
    assert list(faults(["v_readfirstlane_b32 s4, v1", "s_nop 3", copy]))
    assert not list(faults(["v_readfirstlane_b32 s4, v1", "s_nop 4", copy]))
    assert not list(faults(["v_readfirstlane_b32 s12, v1", copy]))
    assert not list(faults([late, "s_lshl_b32 s10, s10, 6", copy]))


def test_copies_to_lds_in_the_library(tmp_path):
    if not os.path.exists(build.LIB):
        pytest.skip("the library has not been built")
    copies, wrong = 0, []
    for lines in instructions(build.LIB, tmp_path):
        copies += sum(COPY.match(line) is not None for line in lines)
        wrong += [(reason, lines[i]) for i, reason in faults(lines)]
    assert copies > 100, "no copies to LDS found: has their form changed?"
    assert not wrong, f"{len(wrong)} of {copies} copies follow too soon, such as {wrong[:3]}"
