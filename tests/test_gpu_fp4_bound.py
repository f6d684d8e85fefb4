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


def run_even(pkv, ws, lens, T, hkv, group, bs, seed=1, scale=1 / 64, **kw):
    """Rows of equal norms under a small scale: every key carries weight, and the bound is a fraction of what a
    key tile, a merged piece or the newest key adds (tests/test_fp4_bound_host.py)."""
    b = even_batch(lens, hkv, bs, seed, **kw)
    q = even_queries(b.rng, len(lens) * T, hkv * group)
    check(attend(pkv, b, q, T, scale, ws), *reference(b, q, T, group, scale))


@pytest.mark.parametrize("T,hkv,group", [(1, 4, 4), (1, 1, 1), (1, 2, 32), (1, 3, 7), (2, 8, 1), (3, 2, 7), (8, 4, 4), (8, 4, 6),
                                         (5, 1, 16), (17, 1, 3), (40, 2, 1), (1, 5, 12), (64, 4, 32)])
def test_attend_even_geometries(pkv, ws, T, hkv, group):
    run_even(pkv, ws, [130, 700, 64], T, hkv, group, 16, seed=T + hkv)


@pytest.mark.parametrize("n", [1, 2, 16, 17, 127, 128, 129, 256, 257, 640, 1025, 4000])
@pytest.mark.parametrize("T", [1, 8])
def test_attend_even_lengths(pkv, ws, n, T):
    run_even(pkv, ws, [n], T, 2, 4, 32, seed=n)


@pytest.mark.parametrize("bs", [8, 16, 24, 48, 64, 120, 128, 136, 256, 880])
@pytest.mark.parametrize("layout", ["nbhd", "nhbd", "padded"])
def test_attend_even_pages(pkv, ws, bs, layout):
    run_even(pkv, ws, [901, 129], 4, 2, 2, bs, seed=bs, layout=layout)


@pytest.mark.parametrize("T", [1, 8])
def test_attend_even_ragged_batch(pkv, ws, T):
    rng = np.random.default_rng(77)
    lens = [int(x) for x in np.exp(rng.uniform(np.log(20), np.log(4000), 37))]
    run_even(pkv, ws, lens + [9000, 0, 1], T, 4, 4, 16, seed=7)


@pytest.mark.parametrize("lens,T,hkv,group", [([40000, 3], 1, 2, 2), ([20008], 8, 4, 6), ([100000], 1, 1, 4), ([9000, 9000], 8, 2, 4)])
def test_attend_even_long_contexts(pkv, ws, lens, T, hkv, group):
    """Units that many CTAs share: each one's piece counts once."""
    run_even(pkv, ws, lens, T, hkv, group, 880, seed=41)


@pytest.mark.parametrize("ctas", [1, 2, 7, 31, 100])
def test_attend_even_small_workspace(pkv, ctas):
    small = torch.empty(pkv.spec_verify_fp4_workspace_bytes(ctas), dtype=torch.uint8, device=DEV)
    run_even(pkv, small, [700, 20, 1300, 0, 5000], 3, 2, 4, 16, seed=ctas)


@pytest.mark.parametrize("T,hkv,group", [(1, 2, 4), (4, 2, 4)])
def test_attend_even_growing_scores(pkv, ws, T, hkv, group):
    """Scores that rise along the keys by 40 and fall again, so that the maximum moves and O is rescaled in most tiles;
    the keys near the top share the weight."""
    n = 5000
    b = even_batch([n], hkv, 16, seed=52)
    blk, slot = b.where(0, np.arange(n))
    f = F.bf16_to_f32(rows_u16(b.rng, n, hkv, spread=False))
    f[..., 0] = (3 * np.sin(np.linspace(-1.5, 5.0, n, dtype=np.float32)))[:, None]
    b.codes["k"][blk, slot], b.sb["k"][blk, slot] = F.quantize(F.f32_to_bf16(f), 0.013)
    q = F.bf16_to_f32(even_queries(b.rng, T, hkv * group))
    q[..., 0] = 60.0
    q = F.f32_to_bf16(q)
    check(attend(pkv, b, q, T, 1 / 8, ws), *reference(b, q, T, group, 1 / 8))


def test_attend_nan_value_scale_under_many_tokens(pkv, ws):
    """A NaN V scale among many tokens of a request reaches the tokens from its key on, and costs a look at the few
    keys that a CTA's columns differ in: with a look at all that follow, 5 ms a unit, the waits of 2 ms ran out."""
    T, hkv, key = 6000, 4, 2999
    b = even_batch([T], hkv, 16, seed=53)
    blk, slot = b.where(0, np.array([key]))
    b.sb["v"][blk, slot, 1, 3] = 0x7F
    q = even_queries(b.rng, T, hkv)
    pkv.lib.pkv_testing_set_wait_limit_ns(2_000_000)
    got = attend(pkv, b, q, T, 1 / 64, ws)
    nan = np.isnan(got)
    assert nan[key:, 1, 48:64].all()
    nan[key:, 1, 48:64] = False
    assert not nan.any()
    b.sb["v"][blk, slot, 1, 3] = 0
    k, v = b.value("k", 0), b.value("v", 0)
    for t in (0, 1, 31, 32, 127, 128, key - 1, key, key + 1, key + 31, 4095, T - 1):
        for h in range(hkv):
            want, tol = B._rows(F.bf16_to_f32(q[t:t + 1, h]).astype(np.float64), k[:t + 1, h], v[:t + 1, h], 1 / 64)
            keep = np.r_[0:48, 64:256] if h == 1 else np.arange(256)
            check(got[t:t + 1, h][:, keep], want[:, keep], tol[:, keep])
