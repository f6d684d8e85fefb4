"""The 4-bit write's quotient (a product corrected by its remainder) where it decides and where it could leave fp32's
range: elements next to the codes' thresholds, tiny ones beside them, and scales at both ends of its range."""
import numpy as np
import pytest

import _fp4 as F
from test_gpu_fp4 import Batch, pkv, run_write  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
THRESHOLDS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


@pytest.mark.parametrize("scale", [2.0 ** -90, 1.3 * 2.0 ** -88, 2.0 ** -80, 1.7 * 2.0 ** -79, 1e-10, 0.0123, 1.0, 1.9 * 2.0 ** 60,
                                   2.0 ** 91, 1.1 * 2.0 ** 93, 2.0 ** 100])
def test_write_next_to_the_thresholds(pkv, scale):
    n = 128
    b = Batch([n], 2, 16, seed=13, fill=False, kg=scale, vg=np.float32(scale) * np.float32(0.7))
    rng = b.rng
    rows = {}
    for w, g in (("k", b.kg), ("v", b.vg)):
        # a group's largest element fixes its scale d; the others lie on a threshold of d, or a bf16 step or two beside
        # it, or far below: down to the smallest subnormal number
        groups = n * 2 * 16
        top = F.f32_to_bf16((np.float32(g) * 6 * 2.0 ** rng.uniform(-5, 8, groups)).astype(np.float32))
        x = np.zeros((groups, 16), np.uint16)
        x[:, 0] = top
        probe = np.zeros((groups, 256), np.uint16)
        probe[:, 0] = top
        sb = F.quantize(probe, g)[1][:, 0]
        d = F.E4M3[sb] * float(np.float32(g))
        near = F.f32_to_bf16((d[:, None] * THRESHOLDS[rng.integers(0, 7, (groups, 15))]).astype(np.float32)).astype(np.int32)
        near = np.minimum(near + rng.integers(-2, 3, near.shape), top[:, None])
        tiny = rng.integers(0, 512, near.shape) if scale < 1 else F.f32_to_bf16((d[:, None] * 2.0 ** rng.uniform(-60, -3, near.shape)).astype(np.float32))
        x[:, 1:] = np.where(rng.random(near.shape) < 0.3, np.minimum(tiny, top[:, None]), np.maximum(near, 0))
        x |= (rng.integers(0, 2, x.shape) << 15).astype(np.uint16)
        rows[w] = x.reshape(n, 2, 256)
    run_write(pkv, b, [n], rows)
