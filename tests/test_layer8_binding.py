"""The Python side of the 8-bit layer without a GPU: import on other builds of torch, and the
refusals of the binding itself."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_import_without_cuda_in_torch():
    """A torch built for the CPU lacks the private functions that name the current stream; what needs no
    device works with it."""
    r = run("import torch\n"
            "for n in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import sketch_compressed_sparse_gb300 as s2\n"
            "assert s2.s2_version() and s2.nwords(33) == 2\n"
            "assert s2._stream(type('Stream', (), {'cuda_stream': 5})) == 5\n"
            "torch.cuda.current_stream = lambda: type('Stream', (), {'cuda_stream': 7})\n"
            "assert s2._stream(None) == 7\n")
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("layout", ["row", "", None, 2, -1, 1 << 32, 1.5])
def test_unknown_layouts(layout):
    """A layout is "rows", "tiles" or their constants; nothing is taken for one of them."""
    import sketch_compressed_sparse_gb300 as s2

    with pytest.raises(ValueError, match="layout"):
        s2.alloc_pack8(4, 4, layout, device="cpu")
    for known in ("rows", "tiles", s2.S2_SCALE_ROWS, s2.S2_SCALE_TILES):
        s2.alloc_pack8(4, 4, known, device="cpu")
