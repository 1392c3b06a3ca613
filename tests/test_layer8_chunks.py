"""The division of a long sum's stages into chunks, without a GPU (csrc/s2_chunks.h compiled by itself)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sketch_compressed_sparse_gb300", "csrc")


@pytest.fixture(scope="module")
def ends(tmp_path_factory):
    """ends(stages, most): the ends of all chunks."""
    d = tmp_path_factory.mktemp("chunks")
    src, lib = str(d / "c.cpp"), str(d / "c.so")
    with open(src, "w") as f:
        f.write('#include "s2_chunks.h"\n'
                'extern "C" uint32_t count(uint32_t stages, uint32_t most) { return s2::chunk_count(stages, most); }\n'
                'extern "C" void ends(uint32_t stages, uint32_t chunks, uint32_t* e) {\n'
                '    for (uint32_t c = 0; c < chunks; ++c) e[c] = s2::chunk_end(stages, chunks, c);\n}\n')
    subprocess.run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.count.restype = ctypes.c_uint32

    def f(stages, most):
        e = np.zeros(so.count(stages, most), dtype=np.uint32)
        so.ends(stages, len(e), e.ctypes.data_as(ctypes.c_void_p))
        return e.astype(np.int64)

    return f


# 2^25 stages of 64 tokens are the 2^31 - 1 tokens that a call takes
@pytest.mark.parametrize("stages", [1, 10, 11, 12, 32, 33, 128, 1000, 217_000, 218_000, 262_144, 375_000, 1 << 22, (1 << 25) - 1, 1 << 25])
@pytest.mark.parametrize("most", [11, 32])
def test_chunks_cover_all_stages(ends, stages, most):
    """Every chunk has at least one stage and at most `most`, and the last ends with the stages."""
    e = ends(stages, most)
    sizes = np.diff(np.concatenate([[0], e]))
    assert sizes.min() >= 1 and sizes.max() <= most
    assert e[-1] == stages
