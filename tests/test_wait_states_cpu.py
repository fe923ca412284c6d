"""Wait states around the memory instructions of the built library.

The global -> LDS copies are inline assembly, where the compiler inserts none
of the waits that the hardware leaves to the program. This reads the library's
own gfx950 code and requires them of every copy, along every path that leads to
it:
  * one wait state between a scalar write of m0 and the copy that reads it;
  * five between a vector instruction's write of a scalar register
    (v_readfirstlane and the like) and a buffer instruction that reads it;
and that no 128-bit buffer store takes a scalar register as its offset: the
compiler then sees no hazard between the store and an instruction right after
it that overwrites the store's last data register, and there is one.
"""
import os
import re
import shutil
import subprocess

import pytest

import dense_gemm_04_amd as dg
from dense_gemm_04_amd import build

OBJDUMP = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump")
REG = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc|m0)\b")
TARGET = re.compile(r"<[^>]*\+0x([0-9a-f]+)>\s*$")


def scalars(text):
    """Scalar registers that an operand list names."""
    found = set()
    for lo, hi, one, name in REG.findall(text):
        found |= {name} if name else set(range(int(lo), int(hi) + 1)) if lo else {int(one)}
    return found


def scalar_writes(op, args):
    return scalars(re.split(r",\s*", args)[0]) if op.startswith("s_") else set()


def vector_writes(op, args):
    """Scalar registers that a vector instruction writes: its first operand, and
    the carry of those that have one."""
    if not op.startswith("v_"):
        return set()
    parts = re.split(r",\s*", args)
    return scalars(parts[0]) | (scalars(parts[1]) if "_co_" in op or "div_scale" in op else set())


def parse(line):
    op, _, args = line.split("//")[0].strip().partition(" ")
    return op, args


class Function:
    """One function's instruction lines, and which lines can run right before each."""

    def __init__(self, lines):
        self.lines = lines
        self.jumps = {}                       # line -> lines that jump to it
        self.base = self.at(0)
        for i, line in enumerate(lines):
            if line.startswith(("\ts_cbranch", "\ts_branch")):
                m = TARGET.search(line)
                # A branch to the function's start carries no offset.
                off = int(m.group(1), 16) if m else 0
                self.jumps.setdefault(self.base + off, []).append(i)

    def at(self, i):
        return int(self.lines[i].split("//")[1].split(":")[0], 16)

    def before(self, i):
        if i > 0 and not self.lines[i - 1].startswith(("\ts_branch", "\ts_endpgm", "\ts_setpc")):
            yield i - 1
        yield from self.jumps.get(self.at(i), ())

    def follows_write(self, i, states, writes, reads):
        """True when an instruction that writes one of `reads`, as `writes`
        names an instruction's registers, lies fewer than `states` wait states
        before line i on some path, and nothing writes that register between."""
        for j in self.before(i):
            op, args = parse(self.lines[j])
            if writes(op, args) & reads:
                return True
            kept = reads - scalar_writes(op, args)
            left = states - (int(args, 0) + 1 if op == "s_nop" else 1)
            if left > 0 and kept and self.follows_write(j, left, writes, kept):
                return True
        return False


def too_early(fn):
    """(rule, line) of every instruction of a function that breaks one."""
    bad = []
    for i, line in enumerate(fn.lines):
        if not line.startswith("\tbuffer_"):
            continue
        op, args = parse(line)
        if " lds" in args and fn.follows_write(i, 1, scalar_writes, {"m0"}):
            bad.append(("m0", line))
        if fn.follows_write(i, 5, vector_writes, scalars(args)):
            bad.append(("scalar", line))
        if op == "buffer_store_dwordx4" and re.split(r",\s*", args)[3].startswith("s"):
            bad.append(("store", line))
    return bad


def functions(text):
    lines = []
    for line in text.splitlines():
        if line.startswith("\t"):
            lines.append(line)
        elif lines:
            yield Function(lines)
            lines = []
    if lines:
        yield Function(lines)


def listing(body):
    """Instructions as the disassembler prints them, 4 bytes each."""
    return "".join(f"\t{ins.ljust(40)} // {4 * i:012X}: 00000000{where}\n" for i, (ins, where) in enumerate(body))


@pytest.mark.parametrize("body,rules", [
    (["s_mov_b32 m0, s5", "buffer_load_dwordx4 v3, s[24:27], s16 offen lds"], ["m0"]),
    (["s_mov_b32 m0, s5", "s_nop 0", "buffer_load_dwordx4 v3, s[24:27], s16 offen lds"], []),
    (["v_readfirstlane_b32 s16, v1", "s_mov_b32 m0, s5", "s_nop 0", "s_add_i32 s3, s3, 1", "s_add_i32 s3, s3, 1",
      "buffer_load_dword v3, s[24:27], s16 offen lds"], ["scalar"]),
    (["v_readfirstlane_b32 s25, v1", "s_nop 4", "s_mov_b32 m0, s5", "s_nop 0",
      "buffer_load_dword v3, s[24:27], s16 offen lds"], []),
    # What the copy reads is the scalar unit's result, not the vector unit's.
    (["v_readlane_b32 s16, v1, 3", "s_mul_i32 s16, s4, s16", "s_mov_b32 m0, s5", "s_nop 0",
      "buffer_load_dword v3, s[24:27], s16 offen lds"], []),
    (["v_add_co_u32_e64 v1, s[24:25], v1, v2", "buffer_load_dword v3, v4, s[24:27], 0 offen"], ["scalar"]),
    (["buffer_store_dwordx4 v[0:3], v4, s[24:27], s8 offen"], ["store"]),
    (["buffer_store_dwordx4 v[0:3], v4, s[24:27], 0 offen"], []),
    # The write lies before a branch to the copy, not before it in the listing.
    (["v_readfirstlane_b32 s16, v1", ("s_branch 3", " <f+0x10>"), "s_nop 7", "s_nop 7",
      "buffer_load_dword v3, s[24:27], s16 offen lds", "s_endpgm"], ["scalar"]),
])
def test_the_rules_find_what_they_name(body, rules):
    body = [b if isinstance(b, tuple) else (b, "") for b in body]
    fn, = functions("0000 <f>:\n" + listing(body))
    assert [rule for rule, _ in too_early(fn)] == rules


@pytest.mark.parametrize("check", ["", *build.CHECK_BUILDS])
def test_library(check, tmp_path):
    lib = build.lib_path(check)
    if not os.path.exists(lib):
        build.build(check=check)
    # The tool writes the code objects beside the file it reads.
    shutil.copy(lib, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    copies, bad = 0, []
    objects = sorted(f for f in os.listdir(tmp_path) if f.endswith(build.ARCH))
    assert len(objects) == len(build.sources())
    for name in objects:
        text = subprocess.run([OBJDUMP, "-d", f"--mcpu={build.ARCH}", name], cwd=tmp_path, check=True,
                              capture_output=True, text=True).stdout
        for fn in functions(text):
            copies += sum(" lds" in line for line in fn.lines if line.startswith("\tbuffer_load"))
            bad += too_early(fn)
    assert copies > 1000
    assert not bad, bad[:5]
