"""The norm's gradients in place of an operand: dX may be dY or R, and where a row does
not fill its lanes several of them load and store the same bytes. When these lie in
different waves, every load of the row has to have landed before the barrier that
the waves meet in ahead of the row's stores, and that barrier waits for LDS alone.
This reads the library's own gfx950 code: on no path may a register that a load
was still to fill at a barrier be read on the way to a store before the next one.
"""
import os
import re
import shutil
import subprocess

import pytest

import dense_gemm_04_amd as dg
from dense_gemm_04_amd import build
from test_wait_states_cpu import OBJDUMP, Function, listing, parse

VREG = re.compile(r"\bv\[(\d+):(\d+)\]|\bv(\d+)\b")
# Kernels whose rows several waves share: 128, 256 or 512 lanes to a row.
KERNEL = re.compile(r"norm_gradI[tf]Li(?:128|256|512)ELi\dE")
STORES = ("global_store", "scratch_store", "flat_store", "buffer_store")
LOADS = ("global_load", "flat_load", "buffer_load", "scratch_load")
# A row is read in vectors of 16 bytes (its mean and rstd, and a lane's own memory, are
# no place that another wave stores to).
ROW_LOAD = "global_load_dwordx4"


def vregs(text):
    found = set()
    for lo, hi, one in VREG.findall(text):
        found |= set(range(int(lo), int(hi) + 1)) if lo else {int(one)}
    return frozenset(found)


def late_reads(fn):
    """Lines of stores that follow a read of a register which was in flight at the
    last barrier, on any path through a function."""
    after = {}
    for i in range(len(fn.lines)):
        for j in fn.before(i):
            after.setdefault(j, []).append(i)
    split = []
    for line in fn.lines:
        op, args = parse(line)
        first, _, rest = args.partition(",")
        store = op.startswith(STORES)
        split.append((op, args, vregs("" if store else first), vregs(args if store else rest)))
    bad, seen = set(), set()
    # At a line: what is in flight (a row load's registers, nothing for the rest),
    # registers in flight at the last barrier, and whether one of those was read since.
    todo = [(0, (), frozenset(), False)]
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        i, flight, late, dirty = state
        op, args, writes, reads = split[i]
        if op == "s_waitcnt":
            m = re.search(r"vmcnt\((\d+)\)", args)
            if m and len(flight) > int(m.group(1)):
                flight = flight[len(flight) - int(m.group(1)):] if int(m.group(1)) else ()
        elif op == "s_barrier":
            late, dirty = frozenset().union(*flight), False
        else:
            dirty = dirty or bool(reads & late)
            if op.startswith("global_store") and dirty:
                bad.add(fn.lines[i])
            late = late - writes
            if op == ROW_LOAD:
                flight += (writes,)
            elif op.startswith(LOADS + STORES):
                flight += (frozenset(),)
        todo += [(j, flight, late, dirty) for j in after.get(i, ())]
    return bad


LOAD, SUM, USE = "global_load_dwordx4 v[4:7], v[2:3], off", "v_add_f32 v9, v9, v4", "v_add_f32 v8, v8, v4"
STORE = "global_store_dwordx4 v[2:3], v[8:11], off"


@pytest.mark.parametrize("body,found", [
    ([LOAD, "s_barrier", "s_waitcnt vmcnt(0)", USE, STORE], 1),
    ([LOAD, "s_waitcnt vmcnt(0)", "s_barrier", USE, STORE], 0),
    # What is read on the way to the next barrier, or loaded after this one.
    ([LOAD, "s_barrier", "s_waitcnt vmcnt(0)", SUM, "s_barrier", STORE], 0),
    (["s_barrier", LOAD, "s_waitcnt vmcnt(0)", USE, STORE], 0),
    # The wait leaves the newer of two loads in flight.
    (["global_load_dwordx4 v[12:15], v[2:3], off", LOAD, "s_waitcnt vmcnt(1)", "s_barrier", USE, STORE], 1),
    ([LOAD, "global_load_dwordx4 v[12:15], v[2:3], off", "s_waitcnt vmcnt(1)", "s_barrier", USE, STORE], 0),
    # A branch past the wait.
    ([LOAD, ("s_cbranch_vccnz 1", " <f+0xc>"), "s_waitcnt vmcnt(0)", "s_barrier", USE, STORE], 1),
    # Overwritten before it is read.
    ([LOAD, "s_barrier", "s_waitcnt vmcnt(0)", "v_mov_b32_e32 v4, 0", USE, STORE], 0),
])
def test_the_rule_finds_what_it_names(body, found):
    lines = listing([b if isinstance(b, tuple) else (b, "") for b in body + ["s_endpgm"]]).splitlines()
    assert len(late_reads(Function(lines))) == found


def test_rows_of_several_waves_are_whole_before_their_barrier(tmp_path):
    if not os.path.exists(dg.LIB_PATH):
        build.build()
    shutil.copy(dg.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    checked, bad = 0, {}
    for name in sorted(f for f in os.listdir(tmp_path) if f.endswith(build.ARCH)):
        symbols = subprocess.run([OBJDUMP, "-t", name], cwd=tmp_path, check=True, capture_output=True, text=True).stdout
        if not KERNEL.search(symbols):
            continue
        text = subprocess.run([OBJDUMP, "-d", f"--mcpu={build.ARCH}", name], cwd=tmp_path, check=True,
                              capture_output=True, text=True).stdout
        for head, body in re.findall(r"<([^>\n]+)>:\n((?:\t.*\n)+)", text):
            if KERNEL.search(head):
                checked += 1
                found = late_reads(Function([line for line in body.splitlines() if "//" in line]))
                if found:
                    bad[head] = len(found)
    # 3 to 8 vectors of bf16 (above 4 with 512 lanes alone), 5 to 8 of fp32; with and without R.
    assert checked == 2 * (2 + 2 + 6 + 3 * 4)
    assert not bad, bad


def test_lanes_that_exchange_through_lds_order_it():
    """A barrier of a wave's lanes orders no memory by itself: it stands between a release and an
    acquire of LDS, also where the lanes run in step."""
    fence = r'__builtin_amdgcn_fence\(__ATOMIC_{}, "(?:wavefront|workgroup)", "local"\);\s*'
    whole = re.compile(fence.format("RELEASE") + r"__builtin_amdgcn_wave_barrier\(\);\s*" + fence.format("ACQUIRE"))
    bare = {}
    for name in sorted(os.listdir(build.CSRC)):
        text = open(os.path.join(build.CSRC, name), encoding="utf-8").read()
        left = whole.sub("", text).count("wave_barrier")
        if left != text.count("lds_wave_barrier"):
            bare[name] = left
    assert not bare, bare
