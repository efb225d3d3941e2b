"""The copies from memory to LDS of the fp8 product, in the code built for the
device.  They are written as inline assembly, which the compiler takes as it is:
neither waits nor bounds are its business there, and no result shows a copy
whose data are not used."""
import os
import re
import shutil
import subprocess

import pytest

import tensor_all_reduce_amd as tar

OBJDUMP = shutil.which("llvm-objdump", path="/opt/rocm/llvm/bin" + os.pathsep + os.environ.get("PATH", ""))
pytestmark = pytest.mark.skipif(OBJDUMP is None, reason="llvm-objdump not available")

COPY = re.compile(r"buffer_load_dwordx4 v\d+, s\[(\d+):(\d+)\], (\S+) offen lds")


def instructions(lib, tmp):
    """Instructions of every kernel of the library, in order, without labels."""
    shutil.copy(lib, tmp / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp, check=True, capture_output=True)
    for obj in sorted(tmp.glob("lib.so.*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", obj.name], cwd=tmp, check=True, capture_output=True,
                              text=True).stdout
        for line in text.splitlines():
            line = line.split("//")[0].strip()
            if line and not line.endswith(":"):
                yield line


def scalars(text):
    """Numbers of the scalar registers that `text` names."""
    regs = set()
    for lo, hi, one in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        regs |= {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return regs


def states_before(window, regs):
    """Wait states between a vector instruction's write of one of `regs` and
    what follows `window`; five if there is none nearer."""
    states = 0
    for ins in reversed(window):
        op, _, rest = ins.partition(" ")
        if op.startswith("v_") and scalars(rest.split(",")[0]) & regs:
            return states
        states += int(rest, 0) + 1 if op == "s_nop" else 1
        if states >= 5:
            break
    return 5


def test_plain_state_count():
    assert scalars("v1, s[4:6], s9") == {4, 5, 6, 9}
    assert states_before(["v_readlane_b32 s5, v1, 0", "s_mov_b32 m0, s1", "s_nop 0"], {5}) == 2
    assert states_before(["v_readlane_b32 s5, v1, 0", "s_mov_b32 m0, s1", "s_nop 3"], {5}) == 5
    assert states_before(["v_readlane_b32 s4, v1, 0", "s_nop 0"], {5}) == 5


def test_copies_wait_for_their_scalar_registers(tmp_path):
    """A vector memory instruction that reads a scalar register needs five wait
    states after a vector instruction (v_readlane, v_readfirstlane) wrote it;
    the hardware does not hold it back, and reads an old descriptor or offset."""
    window, copies, early = [], 0, []
    for ins in instructions(tar.lib_path, tmp_path):
        if COPY.search(ins):
            copies += 1
            n = states_before(window, scalars(ins))
            if n < 5:
                early.append((n, ins))
        window = window[-7:] + [ins]
    assert copies > 100
    assert not early, f"{len(early)} of {copies} copies come too early: {early[:3]}"


def test_copies_to_lds_have_no_scalar_offset(tmp_path):
    """A buffer's size bounds what a copy reads: a tile's rows past the last,
    and blocks past a slice of K, lie beyond it and have to read nothing.  The
    check compares the lane's own offset with the size; how a scalar offset takes
    part once it exceeds the size is another matter, so the lane's register
    holds the whole offset."""
    copies = [m.group(3) for m in map(COPY.search, instructions(tar.lib_path, tmp_path)) if m]
    assert len(copies) > 100
    assert set(copies) == {"0"}, f"{sum(c != '0' for c in copies)} of {len(copies)} copies use a scalar offset"
