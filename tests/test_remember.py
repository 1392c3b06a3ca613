"""The table that keeps the answers about launches, without a GPU (csrc/s2_remember.h compiled by itself)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sketch_compressed_sparse_gb300", "csrc")

SOURCE = """
#include "s2_remember.h"
namespace {
struct Key {
    uint64_t a;
    bool operator==(const Key& o) const { return a == o.a; }
    uint64_t hash() const { return s2::spread(a); }
};
s2::Remembered<Key, int, 512> table;
}
// Asks for each key in turn, as a launch does; how many had to be looked up. -1: a wrong answer.
extern "C" int64_t ask(const uint64_t* keys, int64_t n) {
    int64_t misses = 0;
    for (int64_t i = 0; i < n; ++i) {
        int v = 0;
        if (!table.find(Key{keys[i]}, &v)) {
            v = (int)(keys[i] * 7 + 3);
            table.put(Key{keys[i]}, v);
            ++misses;
        }
        if (v != (int)(keys[i] * 7 + 3) || !table.find(Key{keys[i]}, &v)) return -1;
    }
    return misses;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("remember")
    src, lib = str(d / "r.cpp"), str(d / "r.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib], check=True)
    so = ctypes.CDLL(lib)
    so.ask.restype = ctypes.c_int64

    def f(keys):
        k = np.ascontiguousarray(keys, dtype=np.uint64)
        n = so.ask(k.ctypes.data_as(ctypes.c_void_p), ctypes.c_int64(len(k)))
        assert n >= 0
        return n

    return f


def test_a_long_history_leaves_room(ask):
    """Keys of every kind of step are answered rightly, each is there after it was asked for, and after hundreds of
    thousands of others a new working set is looked up once and then kept."""
    rng = np.random.default_rng(1)
    for step in (1, 16, 2048, 1 << 20, 1 << 32):
        keys = np.arange(1, 100001, dtype=np.uint64) * np.uint64(step)
        ask(keys)
        # 300 keys (thirty shapes of ten candidates): more than eight in one of 512 sets in one run of 10^5
        few = rng.choice(keys[:50000], 300, replace=False)
        ask(few)
        assert ask(np.tile(few, 5)) == 0


def test_a_working_set_of_thousands_stays_mostly(ask):
    """2000 keys, four a set on average: the sets with more than eight are few."""
    keys = np.arange(2000, dtype=np.uint64) * np.uint64(2048) + np.uint64(1 << 40)
    ask(keys)
    ask(keys)
    assert ask(keys) < 400
