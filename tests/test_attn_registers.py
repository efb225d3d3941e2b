"""The attention kernels keep everything in registers and LDS.  Results in
scratch memory are right but slow, beyond its traffic: a load from there waits
for the copies to LDS that are under way, which share its counter."""
import os
import re
import shutil
import subprocess

import pytest

import tensor_all_reduce_amd as tar
from test_block_bounds import OBJDUMP

READELF = shutil.which("llvm-readelf", path="/opt/rocm/llvm/bin" + os.pathsep + os.environ.get("PATH", ""))
pytestmark = pytest.mark.skipif(OBJDUMP is None or READELF is None, reason="llvm-objdump, llvm-readelf not available")


def scratch(lib, tmp):
    """Bytes of scratch memory a lane, of every kernel of the library."""
    shutil.copy(lib, tmp / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp, check=True, capture_output=True)
    res = {}
    for obj in sorted(tmp.glob("lib.so.*gfx950")):
        notes = subprocess.run([READELF, "--notes", obj.name], cwd=tmp, check=True, capture_output=True, text=True).stdout
        for part in re.split(r"\n\s*- \.agpr_count", notes)[1:]:
            size = re.search(r"\.private_segment_fixed_size:\s+(\d+)", part)
            names = re.findall(r"\.name:\s+(_Z\S+)", part)
            assert size and names, part[:200]
            res[names[0]] = int(size.group(1))
    return res


def test_attention_uses_no_scratch(tmp_path):
    sizes = {k: v for k, v in scratch(tar.lib_path, tmp_path).items() if "k_attn" in k or "k_rope" in k}
    assert len(sizes) == 18 + 4 + 5 + 8                # prompts, single tokens, gradients, rotation
    assert not {k: v for k, v in sizes.items() if v}
