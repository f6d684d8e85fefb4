"""The walk over a request's (token, head) pairs of the 4-bit write, on the host: where each
pair lies, and that no table entry past the request's last position is read."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

HARNESS = """
#include "kv_fp4.cuh"
// out: per pair, the walk's (block, slot, head, token, next block's entry)
extern "C" void walk(const int32_t* table, uint32_t heads, uint32_t bs, uint32_t mb, uint32_t pos0, uint32_t end,
                     uint64_t first, int n, int64_t* out) {
  pkv::PairWalk at(table, heads, bs, mb, pos0, end, first);
  for (int k = 0; k < n; ++k, at.next()) {
    const int64_t v[5] = {at.blk, at.slot, at.h, at.i, at.blk_next};
    for (int j = 0; j < 5; ++j) out[5 * k + j] = v[j];
  }
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._build_module()
    d = tmp_path_factory.mktemp("walk")
    src, lib = os.path.join(d, "walk.cu"), os.path.join(d, "walk.so")
    with open(src, "w") as f:
        f.write(HARNESS)
    flags = [x for x in b.NVCC_FLAGS if x not in ("-Xcompiler", "-fvisibility=hidden", "-fPIC")]
    r = subprocess.run([b._nvcc(), *b.ARCH, *flags, "-Xcompiler", "-fPIC", "-shared", "-o", lib, src], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    fn = C.CDLL(lib).walk
    fn.argtypes = [C.c_void_p, C.c_uint32, C.c_uint32, C.c_uint32, C.c_uint32, C.c_uint32, C.c_uint64, C.c_int, C.c_void_p]

    def call(table, heads, bs, pos0, end, first, n):
        out = np.zeros((n, 5), dtype=np.int64)
        fn(table.ctypes.data, heads, bs, len(table), pos0, end, first, n, out.ctypes.data)
        return out
    return call


@pytest.mark.parametrize("bs", [8, 16, 24, 880])
@pytest.mark.parametrize("heads", [1, 4, 7])
def test_walk(walk, bs, heads):
    PAST = 12345  # an entry past the request's last
    for begin, end in ((0, 1), (0, bs), (0, bs + 1), (bs - 1, bs), (3, 2 * bs), (bs, 3 * bs), (5, 2 * bs + 3), (2 * bs - 1, 2 * bs + 1)):
        used = -(-end // bs)
        for columns in (used, used + 1, used + 3, max(1, used - 1)):
            table = np.where(np.arange(columns) < used, 100 + np.arange(columns), PAST).astype(np.int32)
            pairs = (end - begin) * heads
            for first in {0, pairs // 2, pairs - 1}:
                got = walk(table, heads, bs, begin, end, first, pairs - first)
                pair = np.arange(first, pairs)
                pos = begin + pair // heads
                blk = np.where(pos // bs < columns, 100 + pos // bs, -1)
                assert np.array_equal(got[:, :4], np.stack([blk, pos % bs, pair % heads, pair // heads], 1))
                assert not (got[:, 4] == PAST).any()


def test_walk_at_the_end_of_the_positions(walk):
    """Positions up to 2^31 - 1, in blocks of one and of many slots."""
    end = (1 << 31) - 1
    one = np.full(4, 9, dtype=np.int32)
    got = walk(one, 2, 1 << 30, end - 3, end, 0, 6)
    assert (got[:, 0] == 9).all() and got[:, 1].tolist() == [(end - 3 + k // 2) - (1 << 30) for k in range(6)] and (got[:, 4] == -1).all()
    got = walk(one, 1, 1, end - 3, end, 0, 3)
    assert (got[:, 0] == -1).all() and (got[:, 4] == -1).all()
