"""Attention over the 4-bit cache held to the sharp bound of tests/_fp4_bound.py."""
import numpy as np
import pytest
import torch

import _fp4 as F
import _fp4_bound as B
from _devsetup import DEV, u16_to_bf16
from test_gpu_fp4 import Batch, attend, check, pkv, rows_u16, ws  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def even_batch(lens, hkv, bs, seed, channel=None, **kw):
    """A Batch whose rows are alike in size: normal elements, K's times `channel`."""
    b = Batch(lens, hkv, bs, seed=seed, fill=False, **kw)
    for r, n in enumerate(lens):
        if not n:
            continue
        blk, slot = b.where(r, np.arange(n))
        for w, g in (("k", b.kg), ("v", b.vg)):
            x = rows_u16(b.rng, n, hkv, spread=False)
            if w == "k" and channel is not None:
                x = F.f32_to_bf16(F.bf16_to_f32(x) * channel)
            # rows of the tensor's size, whatever its scale
            b.codes[w][blk, slot], b.sb[w][blk, slot] = F.quantize(x, 0.013)
    return b


def reference(b, q, T, group, scale):
    parts = []
    for r, n in enumerate(b.lens):
        k, v = (b.value(w, r) if n else np.zeros((0, b.hkv, 256)) for w in ("k", "v"))
        parts.append(B.attention(q[r * T:(r + 1) * T], k, v, n, T, group, scale))
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])


def even_queries(rng, n, hq):
    return F.f32_to_bf16(rng.standard_normal((n, hq, 256)).astype(np.float32))


def outliers(rng, q_u16, big):
    """One element of each 16 `big` times the others, the same channels in every row, and K's factors."""
    at = rng.integers(0, 16, 16) + 16 * np.arange(16)
    f = F.bf16_to_f32(q_u16)
    f[..., at] *= big
    channel = np.ones(256, dtype=np.float32)
    channel[at] = 1 / big
    return F.f32_to_bf16(f), channel


@pytest.mark.parametrize("T,group", [(1, 4), (4, 4), (8, 4), (3, 7)])
@pytest.mark.parametrize("big", [1, 30, 100, 1000])
def test_attend_outlier_channels(pkv, ws, T, group, big):
    """A query row's small elements count beside large ones of the same 16 that meet small channels of K."""
    rng = np.random.default_rng(1000 * T + big)
    lens, hkv = [1500, 300], 2
    q, channel = outliers(rng, even_queries(rng, len(lens) * T, hkv * group), big)
    b = even_batch(lens, hkv, 16, seed=big, channel=channel, kg=0.013)
    check(attend(pkv, b, q, T, 0.25, ws), *reference(b, q, T, group, 0.25))


@pytest.mark.parametrize("vg", [2.0 ** -126, 2.0 ** -120, 3e-30, 1e30, 2.0 ** 110])
@pytest.mark.parametrize("lens,T", [([1000, 40], 1), ([5, 300], 4), ([70000], 1)])
def test_attend_value_scales(pkv, ws, vg, lens, T):
    """The tensor's scale of V anywhere in its range, in units that one CTA holds and in merged ones."""
    b = even_batch(lens, 2, 16, seed=T, vg=vg)
    q = even_queries(b.rng, len(lens) * T, 4)
    check(*(x / vg for x in (attend(pkv, b, q, T, 1 / 64, ws), *reference(b, q, T, 2, 1 / 64))))  # (check's own floor is 1e-30)


@pytest.mark.parametrize("qscale,kg,scale,size", [(2.0 ** -112, 2.0 ** 125, 2.0 ** -20, 1), (2.0 ** 124, 2.0 ** -126, 2.0 ** 11, 2.0 ** -14),
                                                  (2.0 ** 124, 2.0 ** -126, 2.0 ** -6, 1), (2.0 ** -120, 2.0 ** 120, 1 / 64, 1)])
def test_attend_scales_far_apart(pkv, ws, qscale, kg, scale, size):
    """Query rows, K's scale and softmax_scale whose product is ordinary and whose parts are not."""
    b = even_batch([900, 60], 2, 16, seed=5, kg=kg, channel=np.float32(size))
    q = F.f32_to_bf16(F.bf16_to_f32(even_queries(b.rng, 2 * 2, 4)) * np.float32(qscale))
    check(attend(pkv, b, q, 2, scale, ws), *reference(b, q, 2, 2, scale))


def test_attend_calls_that_follow_one_another(pkv, ws):
    """Calls of other shapes and lengths one after the other on a stream, one workspace, no wait between them: each
    merge reads what its own call left there, so each gives the bits that it gives alone."""
    b = even_batch([6000, 700, 3000, 50], 2, 16, seed=7)
    caches, scales, bt, _ = b.device()
    calls = []
    for T, group, lens in ((1, 4, [6000, 700, 3000, 50]), (8, 4, [130, 0, 2999, 8]), (1, 2, [6000, 1, 1, 1]), (3, 7, [257, 600, 5, 50]),
                           (2, 8, [0, 0, 2900, 0])):
        qd = u16_to_bf16(even_queries(b.rng, 4 * T, 2 * group)).to(DEV)
        calls.append((qd, torch.tensor(lens, dtype=torch.int32, device=DEV), T, torch.empty_like(qd)))

    def call(i, out):
        qd, sl, T, _ = calls[i]
        pkv.spec_verify_attn_fp4(qd, *caches, *scales, bt, sl, T, 1 / 64, out, ws)

    for i, c in enumerate(calls):
        call(i, c[3])
        torch.cuda.synchronize()
    order = np.random.default_rng(8).integers(0, len(calls), 300)
    outs = [torch.empty_like(calls[i][3]) for i in order]
    for i, out in zip(order, outs):
        call(i, out)
    torch.cuda.synchronize()
    for i, out in zip(order, outs):
        assert torch.equal(out.view(torch.int16), calls[i][3].view(torch.int16))
