"""The attention kernels' copies from memory to LDS in the code built for the
device: inline assembly, to which the compiler adds no waits of its own."""
import re

import pytest

import tensor_all_reduce_amd as tar
from test_block_bounds import OBJDUMP, instructions, scalars, states_before

pytestmark = pytest.mark.skipif(OBJDUMP is None, reason="llvm-objdump not available")

COPY = re.compile(r"global_load_lds_dword(?:x4)? v(?:\d+|\[\d+:\d+\]), (off|s\[\d+:\d+\])")


def test_copies_wait_for_their_scalar_registers(tmp_path):
    """A copy's base has been written five wait states before if a vector
    instruction wrote it, and M0 one wait state before."""
    window, copies, based = [], 0, 0
    for ins in instructions(tar.lib_path, tmp_path):
        m = COPY.match(ins)
        if m:
            copies += 1
            assert window[-1].startswith("s_nop") and window[-2].startswith("s_mov_b32 m0,"), window[-3:]
            if m.group(1) != "off":
                based += 1
                assert states_before(window, scalars(m.group(1))) >= 5, window[-8:]
        window = window[-11:] + [ins]
    assert copies > 100 and based > 20
