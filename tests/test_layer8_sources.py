"""What the 8-bit layer's kernels must keep in their source, without a GPU.

A load from tensor memory fills its registers some time after the instruction; the compiler knows
that only if the wait names those registers. Where it does not, the compiler may move their first
use before the wait.
"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sketch_compressed_sparse_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


def source(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_for_tensor_memory_name_registers():
    waits = [w for p in FILES for w in re.findall(r"tcgen05\.wait::ld[^;]*;[^;]*;", source(p))]
    assert waits
    for w in waits:
        assert w.count('"+r"') == 16, w


@pytest.mark.parametrize("path", [p for p in FILES if "tmem_ld16(" in source(p) and not p.endswith("s2_tc.cuh")],
                         ids=os.path.basename)
def test_loads_are_waited_for_before_their_use(path):
    """After tmem_ld16(address, r) the next mention of r is wait_ld16(r)."""
    text = source(path)
    loads = list(re.finditer(r"\btmem_ld16\([^;]*,\s*(\w+)\);", text))
    assert loads
    for m in loads:
        r = m.group(1)
        after = re.search(rf"(\w+\()?\b{r}\b", text[m.end():])
        line = text.count("\n", 0, m.start()) + 1
        assert after and after.group(0) == f"wait_ld16({r}", f"{os.path.basename(path)}:{line}: {m.group(0)}"
