"""The 4-bit read-back where a warp holds four (position, head) pairs (large calls; max_tokens, an upper bound, makes
a small one large), and the last part of a long context."""
import numpy as np
import pytest

from test_gpu_fp4 import Batch, pkv, run_read  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
MANY = 100_000


@pytest.mark.parametrize("hkv,bs,layout", [(1, 8, "nbhd"), (4, 16, "nhbd"), (3, 24, "padded"), (8, 880, "nbhd"), (5, 8, "nhbd")])
def test_read_four_pairs_a_warp(pkv, hkv, bs, layout):
    b = Batch([37, 1, 0, 300, 130], hkv, bs, seed=8, layout=layout)
    run_read(pkv, b, [0, 0, 0, 17, 130], [37, 1, 0, 300, 130], 301, max_tokens=MANY)
    run_read(pkv, b, [5, 0, 0, 299, 3], [6, 1, 0, 300, 129], 300, max_tokens=MANY)


def test_read_four_pairs_of_bad_blocks_and_bounds(pkv):
    b = Batch([64, 64], 2, 16, seed=10)
    bt = b.bt.copy()
    bt[0, 2], bt[1, 0], bt[1, 1] = b.nb + 5, -1, -(1 << 31)
    bad = pkv.PKV_ERR_DEVICE_BOUNDS
    run_read(pkv, b, [0, 0], [64, 64], 64, expect_err=bad, bt=bt, max_tokens=MANY)
    run_read(pkv, b, [0, 0], [64, 64], 50, expect_err=bad, max_tokens=MANY)  # past the dense rows
    run_read(pkv, b, [0, 0], [64, 64], 64, expect_err=bad, bt=b.bt[:, :3].copy(), max_tokens=MANY)  # past the table


@pytest.mark.parametrize("bs", [16, 880])
def test_read_the_last_chunk_of_a_long_context(pkv, bs):
    """What a prompt that keeps its dense rows reads: only each chunk's new positions."""
    b = Batch([20000, 30011], 2, bs, seed=12)
    run_read(pkv, b, [19000, 29963], [20000, 30011], 30016)
    run_read(pkv, b, [19000, 29963], [20000, 30011], 30016, max_tokens=MANY)
