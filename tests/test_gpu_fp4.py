"""The 4-bit cache on the GPU: the write and the read-back bit for bit, the attention within the bound
its roundings give, against plain numpy (64 bits for the attention)."""
import math

import numpy as np
import pytest
import torch

import _fp4 as F
from _devsetup import DEV, bf16_to_u16, dev_err, u16_to_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_int64_gb300 as m
    assert torch.cuda.is_available()
    return m


@pytest.fixture(scope="module")
def ws(pkv):
    return torch.full((pkv.spec_verify_fp4_workspace_bytes(),), 0xFF, dtype=torch.uint8, device=DEV)


def rows_u16(rng, n, hkv, spread=True):
    x = rng.standard_normal((n, hkv, 256)).astype(np.float32)
    if spread:
        x *= np.exp(rng.standard_normal((n, hkv, 1))).astype(np.float32)
    return F.f32_to_bf16(x)


def same(got, want):
    bad = np.argwhere(got != want)
    assert not len(bad), (len(bad), bad[:3].tolist(), got[tuple(bad[0])], want[tuple(bad[0])])


class Batch:
    """Requests of given lengths in a shuffled pool; codes and scales quantized from normal rows (or
    given), slots that no request owns poisoned with NaN scales."""

    def __init__(self, lens, hkv, bs, seed=0, fill=True, layout="nbhd", kg=0.013, vg=0.4, big_stride=0):
        rng = np.random.default_rng(seed)
        self.lens, self.hkv, self.bs, self.kg, self.vg = list(lens), hkv, bs, kg, vg
        pages = [-(-n // bs) for n in lens]
        self.nb = sum(pages) + 2
        perm = rng.permutation(self.nb)
        self.bt = np.full((len(lens), max(1, max(pages)) + 1), -1, dtype=np.int32)
        at = 0
        for r, n in enumerate(pages):
            self.bt[r, :n] = perm[at:at + n]
            at += n
        self.codes, self.sb, self.tok = {}, {}, {}
        for w in ("k", "v"):
            self.codes[w] = np.full((self.nb, bs, hkv, 128), 0x5A, dtype=np.uint8)
            self.sb[w] = np.full((self.nb, bs, hkv, 16), 0x7F, dtype=np.uint8)
            for r, n in enumerate(lens):
                if not (fill and n):
                    continue
                c, s = F.quantize(rows_u16(rng, n, hkv), {"k": kg, "v": vg}[w])
                blk, slot = self.where(r, np.arange(n))
                self.codes[w][blk, slot], self.sb[w][blk, slot] = c, s
        self.rng, self.layout, self.big_stride = rng, layout, big_stride

    def where(self, r, pos):
        return self.bt[r, pos // self.bs], pos % self.bs

    def value(self, w, r):
        blk, slot = self.where(r, np.arange(self.lens[r]))
        return F.values(self.codes[w][blk, slot], self.sb[w][blk, slot]) * float(np.float32({"k": self.kg, "v": self.vg}[w]))

    def device(self):
        """(k_fp4, v_fp4, k_bscale, v_bscale), (k_scale, v_scale), block table, lengths. layout "nhbd": a
        block holds its heads one after the other; big_stride: a block stride of that many bytes."""
        def put(a):
            t = torch.from_numpy(a).to(DEV)
            if self.layout == "nhbd":
                return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
            if self.layout == "padded":  # slack after each head, token and block
                wide = torch.full((a.shape[0], a.shape[1] + 3, a.shape[2] + 1, a.shape[3] + 16), 0x7F, dtype=torch.uint8, device=DEV)
                view = wide[:, :a.shape[1], :a.shape[2], :a.shape[3]]
                view.copy_(t)
                return view
            if self.big_stride and a.shape[3] == 128:
                flat = torch.zeros(a.shape[0] * self.big_stride, dtype=torch.uint8, device=DEV)
                view = flat.as_strided(a.shape, (self.big_stride, a.shape[2] * 128, 128, 1))
                view.copy_(t)
                return view
            return t
        caches = tuple(put(x[w]) for x in (self.codes, self.sb) for w in ("k", "v"))
        scales = tuple(torch.tensor([g], dtype=torch.float32, device=DEV) for g in (self.kg, self.vg))
        return caches, scales, torch.from_numpy(self.bt).to(DEV), torch.tensor(self.lens, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------------
# write and read back
# ------------------------------------------------------------------------------------------------

def run_write(pkv, b, q_lens, rows, expect_err=0, bt=None, pad=0, tail=0):
    """Writes rows (dict k, v: bf16 bits [total][hkv][256]) and compares the whole pool, written slot or not."""
    caches, scales, bt_d, sl = b.device()
    if bt is not None:
        bt_d = torch.from_numpy(bt).to(DEV)
    else:
        bt = b.bt
    qsl = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    dev = {}
    for w in ("k", "v"):
        t = u16_to_bf16(np.concatenate([rows[w], np.full((tail, b.hkv, 256), 0x7FC0, np.uint16)])).to(DEV)
        if pad:
            wide = torch.full((t.shape[0], b.hkv * 256 + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
            wide[:, :b.hkv * 256] = t.reshape(t.shape[0], -1)
            t = wide[:, :b.hkv * 256].view(t.shape[0], b.hkv, 256)
        dev[w] = t
    err = dev_err()
    pkv.kv_cache_write_fp4(dev["k"], dev["v"], bt_d, sl, torch.from_numpy(qsl).to(DEV), max(q_lens), *caches, *scales, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == expect_err
    for i, w in enumerate(("k", "v")):
        codes, sb = b.codes[w].copy(), b.sb[w].copy()
        for r, n in enumerate(q_lens):
            if n > b.lens[r]:
                continue
            for j in range(n):
                pos = b.lens[r] - n + j
                blk = bt[r, pos // b.bs] if pos // b.bs < bt.shape[1] else -1
                if not 0 <= blk < b.nb:
                    continue
                c, s = F.quantize(rows[w][qsl[r] + j], {"k": b.kg, "v": b.vg}[w])
                codes[blk, pos % b.bs], sb[blk, pos % b.bs] = c, s
        same(caches[2 + i].cpu().numpy(), sb)
        same(caches[i].cpu().numpy(), codes)
    return caches


@pytest.mark.parametrize("hkv,bs,layout,pad", [(1, 8, "nbhd", 0), (4, 16, "nhbd", 48), (3, 24, "padded", 16), (8, 880, "nbhd", 0)])
def test_write_whole_pool(pkv, hkv, bs, layout, pad):
    b = Batch([37, 1, 0, 300, 16], hkv, bs, seed=3, layout=layout)
    q_lens = [5, 1, 0, 219, 16]
    rows = {w: rows_u16(b.rng, sum(q_lens), hkv) for w in ("k", "v")}
    run_write(pkv, b, q_lens, rows, pad=pad, tail=4)


def special_groups(rng, n):
    """Groups of 16 bf16 patterns: zeros, one tiny or subnormal element, ties of the scale and of the
    codes, infinities, NaN, the whole exponent range, raw random bits."""
    g = rng.integers(0, 1 << 16, (n, 16)).astype(np.uint16)          # raw bits: NaN, inf, everything
    k = n // 8
    exp = rng.integers(1, 255, (k, 1))
    g[:k] = (rng.integers(0, 2, (k, 16)) << 15 | np.clip(exp - rng.integers(0, 4, (k, 16)), 0, 254) << 7 | rng.integers(0, 128, (k, 16))).astype(np.uint16)
    small = rng.integers(0, 29, (k, 16)) * 0.25                       # multiples of a quarter: ties of e2m1
    g[k:2 * k] = F.f32_to_bf16((small * 2.0 ** rng.integers(-8, 9, (k, 1))).astype(np.float32))
    g[2 * k:3 * k] = F.f32_to_bf16((rng.integers(1, 64, (k, 1)) * 0.375 * np.where(np.arange(16) == 5, 1, 0.3)).astype(np.float32))
    g[3 * k:4 * k] = rng.integers(0, 8, (k, 16)).astype(np.uint16)    # subnormals and zeros
    g[4 * k:5 * k] = 0x8000
    return g


@pytest.mark.parametrize("scale", [1.0, 0.5, 3.0, 0.0123, 1e-6, 1e-37, 2.0 ** -126, 1e30, 3e38])
def test_write_special_values(pkv, scale):
    n = 512
    b = Batch([n], 2, 16, seed=11, fill=False, kg=scale, vg=scale * 0.75)
    rows = {w: special_groups(b.rng, n * 2 * 16).reshape(n, 2, 256)[b.rng.permutation(n)] for w in ("k", "v")}
    run_write(pkv, b, [n], rows)


def test_write_bad_blocks_and_long_chunks(pkv):
    b = Batch([40, 10, 64], 2, 16, seed=5)
    bt = b.bt.copy()
    bt[0, 1], bt[2, 3] = -7, b.nb  # both outside the pool
    rows = {w: rows_u16(b.rng, 40 + 11 + 20, 2) for w in ("k", "v")}
    run_write(pkv, b, [40, 11, 20], rows, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=bt)  # 11 new rows of a length of 10
    b = Batch([100], 1, 16, seed=6)
    rows = {w: rows_u16(b.rng, 100, 1) for w in ("k", "v")}
    run_write(pkv, b, [100], rows, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=b.bt[:, :4].copy())  # a table of 64 positions


def run_read(pkv, b, begin, end, max_ctx, expect_err=0, bt=None, max_tokens=None):
    caches, scales, bt_d, _ = b.device()
    if bt is not None:
        bt_d = torch.from_numpy(bt).to(DEV)
    else:
        bt = b.bt
    R = len(b.lens)
    dense = [torch.full((R, max_ctx, b.hkv, 256), 7.5, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    err = dev_err()
    pkv.kv_fp4_dequant_dense(*caches, bt_d, i32(begin), i32(end),
                             max(1, max(e - s for s, e in zip(begin, end))) if max_tokens is None else max_tokens, *scales,
                             *dense, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == expect_err
    for w, d in zip(("k", "v"), dense):
        want = np.full((R, max_ctx, b.hkv, 256), F.f32_to_bf16(np.float32(7.5)), dtype=np.uint16)
        for r in range(R):
            for pos in range(begin[r], min(end[r], max_ctx)):
                blk = bt[r, pos // b.bs] if pos // b.bs < bt.shape[1] else -1
                want[r, pos] = (F.dequantize_bf16(b.codes[w][blk, pos % b.bs], b.sb[w][blk, pos % b.bs], {"k": b.kg, "v": b.vg}[w])
                                if 0 <= blk < b.nb else 0)
        got = bf16_to_u16(d)
        nan = (want & 0x7FFF) > 0x7F80
        assert ((got[nan] & 0x7FFF) > 0x7F80).all()
        same(np.where(nan, 0, got), np.where(nan, 0, want))


@pytest.mark.parametrize("hkv,bs,layout", [(1, 8, "nbhd"), (4, 16, "nhbd"), (3, 24, "padded"), (8, 880, "nbhd")])
def test_read_ranges(pkv, hkv, bs, layout):
    b = Batch([37, 1, 0, 300, 130], hkv, bs, seed=8, layout=layout)
    run_read(pkv, b, [0, 0, 0, 17, 130], [37, 1, 0, 300, 130], 301)
    run_read(pkv, b, [5, 0, 0, 299, 3], [6, 1, 0, 300, 129], 300, max_tokens=1)  # the bound only sizes the grid


def test_read_every_code_and_scale(pkv):
    for scale in (1.0, 0.37, 1e-38, 1e36):
        b = Batch([256], 1, 16, seed=9, kg=scale, vg=-scale)
        for w in ("k", "v"):
            b.codes[w][:] = b.rng.integers(0, 256, b.codes[w].shape)
            blk, slot = b.where(0, np.arange(256))
            b.sb[w][blk, slot] = np.arange(256, dtype=np.uint8)[:, None, None]
        run_read(pkv, b, [0], [256], 256)


def test_read_bad_blocks_and_bounds(pkv):
    b = Batch([64, 64], 2, 16, seed=10)
    bt = b.bt.copy()
    bt[0, 2], bt[1, 0] = b.nb + 5, -1
    run_read(pkv, b, [0, 0], [64, 64], 64, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=bt)
    run_read(pkv, b, [0, 0], [64, 64], 50, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS)   # past the dense rows
    run_read(pkv, b, [0, 0], [64, 64], 64, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=b.bt[:, :3].copy())  # past the table


# ------------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------------

def queries(rng, n, hq, scale=1.0):
    return F.f32_to_bf16((rng.standard_normal((n, hq, 256)) * scale).astype(np.float32))


def reference(b, q, T, group, scale):
    parts = [F.attention(q[r * T:(r + 1) * T], b.value("k", r) if b.lens[r] else np.zeros((0, b.hkv, 256)),
                         b.value("v", r) if b.lens[r] else np.zeros((0, b.hkv, 256)), b.lens[r], T, group, scale)
             for r in range(len(b.lens))]
    return np.concatenate([p[0] for p in parts]), np.concatenate([p[1] for p in parts])


def attend(pkv, b, q, T, scale, ws, expect_err=0, bt=None):
    caches, scales, bt_d, sl = b.device()
    if bt is not None:
        bt_d = torch.from_numpy(bt).to(DEV)
    qd = u16_to_bf16(q).to(DEV)
    out = torch.full_like(qd, float("nan"))
    err = dev_err()
    pkv.spec_verify_attn_fp4(qd, *caches, *scales, bt_d, sl, T, scale, out, ws, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == expect_err
    return F.bf16_to_f32(bf16_to_u16(out)).astype(np.float64)


def check(got, want, tol):
    assert np.isfinite(got).all()
    ratio = np.abs(got - want) / (tol + 1e-30)  # zero where zero is exact
    i = np.unravel_index(int(np.argmax(ratio)), ratio.shape)
    assert ratio[i] <= 1, (i, got[i], want[i], tol[i], ratio[i])


def run_attend(pkv, ws, lens, T, hkv, group, bs, seed=1, layout="nbhd", qscale=1.0, scale=1 / 16, **kw):
    b = Batch(lens, hkv, bs, seed=seed, layout=layout, **kw)
    q = queries(b.rng, len(lens) * T, hkv * group, qscale)
    check(attend(pkv, b, q, T, scale, ws), *reference(b, q, T, group, scale))


@pytest.mark.parametrize("T,hkv,group", [(1, 4, 4), (1, 1, 1), (1, 2, 32), (1, 3, 7), (2, 8, 1), (3, 2, 7), (8, 4, 4),
                                         (8, 4, 6), (5, 1, 16), (17, 1, 3), (40, 2, 1), (1, 5, 12), (9, 160, 1)])
def test_attend_geometries(pkv, ws, T, hkv, group):
    run_attend(pkv, ws, [130, 700, 64] if hkv < 100 else [70, 140], T, hkv, group, 16, seed=T + hkv)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 255, 256, 257, 383, 512, 1000, 1025])
def test_attend_every_length(pkv, ws, n):
    run_attend(pkv, ws, [n], 1, 2, 4, 32, seed=n)


@pytest.mark.parametrize("bs", [8, 16, 24, 48, 64, 120, 128, 136, 176, 256, 880, 1000])
@pytest.mark.parametrize("layout", ["nbhd", "nhbd", "padded"])
def test_attend_pages(pkv, ws, bs, layout):
    run_attend(pkv, ws, [901, 129], 4, 2, 2, bs, seed=bs, layout=layout)


@pytest.mark.parametrize("T", [1, 8])
def test_attend_ragged_batch(pkv, ws, T):
    rng = np.random.default_rng(77)
    lens = [int(x) for x in np.exp(rng.uniform(np.log(20), np.log(4000), 37))]
    run_attend(pkv, ws, lens + [9000], T, 4, 4, 16, seed=7)


def test_attend_rows_without_a_key(pkv, ws):
    """Empty requests, requests shorter than T: the tokens before position 0 give zeros."""
    b = Batch([0, 1, 5, 3, 0, 200, 2], 2, 16, seed=21)
    q = queries(b.rng, 7 * 4, 6)
    got = attend(pkv, b, q, 4, 1 / 16, ws)
    check(got, *reference(b, q, 4, 3, 1 / 16))
    assert (got[:4] == 0).all() and (got[4:7] == 0).all() and (got[4 * 3] == 0).all()
    b = Batch([0, 0, 0], 4, 16, seed=22)
    assert (attend(pkv, b, queries(b.rng, 3, 16), 1, 1 / 16, ws) == 0).all()


def test_attend_many_requests(pkv, ws):
    rng = np.random.default_rng(5)
    run_attend(pkv, ws, [int(x) for x in rng.integers(0, 60, 1500)], 1, 1, 2, 8, seed=31)


def test_attend_long_contexts(pkv, ws):
    run_attend(pkv, ws, [40000, 3], 1, 2, 2, 880, seed=41)
    run_attend(pkv, ws, [20008], 8, 4, 6, 880, seed=42)


def test_attend_growing_scores(pkv, ws):
    """Scores that rise along the keys, so that the running maximum moves in every tile, and fall."""
    for sign in (1, -1):
        b = Batch([1500, 640], 1, 16, seed=51)
        for r, n in enumerate(b.lens):
            blk, slot = b.where(r, np.arange(n))
            x = rows_u16(b.rng, n, 1, spread=False)
            f = F.bf16_to_f32(x) * 0.05
            f[..., 0] = sign * np.linspace(-1, 1, n, dtype=np.float32)[:, None] * 30
            b.codes["k"][blk, slot], b.sb["k"][blk, slot] = F.quantize(F.f32_to_bf16(f), b.kg)
        q = queries(b.rng, 2 * 3, 2)
        q[:, :, 0] = F.f32_to_bf16(np.float32([[40.0, -35.0]]))
        check(attend(pkv, b, q, 3, 1 / 16, ws), *reference(b, q, 3, 2, 1 / 16))


@pytest.mark.parametrize("qscale,kg,scale", [(3e5, 0.013, 1e-6), (1e-6, 0.5, 3000.0), (1e30, 1e-20, 1e-10), (1e-30, 1e10, 1e18)])
def test_attend_query_range(pkv, ws, qscale, kg, scale):
    """Queries past fp16's range, both ways."""
    run_attend(pkv, ws, [300, 40], 2, 2, 3, 16, seed=61, qscale=qscale, kg=kg, scale=scale)


def test_attend_mixed_query_rows(pkv, ws):
    b = Batch([200], 1, 16, seed=62)
    q = queries(b.rng, 2, 8)
    f = F.bf16_to_f32(q) * (10.0 ** np.arange(-9, 7, 2)).astype(np.float32)[None, :, None]
    q = F.f32_to_bf16(f)
    check(attend(pkv, b, q, 2, 1e-4, ws), *reference(b, q, 2, 8, 1e-4))


def test_attend_nan_stays_where_it_is_seen(pkv, ws):
    """A NaN scale in the last tokens' K or V rows reaches only the queries that see the key; a NaN in the
    prefix reaches all of them; a NaN query row only itself."""
    T, n = 4, 150
    for w in ("k", "v"):
        b = Batch([n, 90], 1, 16, seed=71)
        blk, slot = b.where(0, np.array([n - 2]))  # the third of the four tokens
        b.sb[w][blk, slot, 0, 5] = 0x7F
        q = queries(b.rng, 2 * T, 2)
        got = attend(pkv, b, q, T, 1 / 16, ws)
        clean = Batch([n, 90], 1, 16, seed=71)
        want, tol = reference(clean, q, T, 2, 1 / 16)
        keep = [0, 1, 4, 5, 6, 7]
        check(got[keep], want[keep], tol[keep])
        if w == "k":
            assert np.isnan(got[2:4]).all()
        else:  # the elements of the NaN's group
            assert np.isnan(got[2:4, :, 80:96]).all()
            rest = np.r_[0:80, 96:256]
            assert np.isfinite(got[2:4][..., rest]).all()
        b.sb[w][b.where(0, np.array([7]))[0], 7, 0, 0] = 0x7F
        got = attend(pkv, b, q, T, 1 / 16, ws)
        assert np.isnan(got[:4, :, :16]).all() and np.isfinite(got[4:]).all()
    b = Batch([n], 1, 16, seed=72)
    q = queries(b.rng, T, 2)
    q[1, 1, 3] = 0x7FC0
    got = attend(pkv, b, q, T, 1 / 16, ws)
    assert np.isnan(got[1, 1]).all()
    got[1, 1] = 0
    assert np.isfinite(got).all()


def test_attend_bad_blocks_read_as_zero(pkv, ws):
    """A key in a bad block has a score of 0 and a value of 0."""
    T, group = 2, 2
    for bs, n in ((16, 300), (8, 131), (256, 700)):
        b = Batch([n, 50], 2, bs, seed=81)
        bad = b.bt.copy()
        bad[0, 1] = -5 if bs != 8 else b.nb
        zero = Batch([n, 50], 2, bs, seed=81)
        blk = zero.bt[0, 1]
        for w in ("k", "v"):
            zero.codes[w][blk] = 0
            zero.sb[w][blk] = 0
        q = queries(b.rng, 2 * T, 4)
        got = attend(pkv, b, q, T, 1 / 16, ws, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=bad)
        check(got, *reference(zero, q, T, group, 1 / 16))
    # a table that ends before the request does
    b = Batch([300], 1, 16, seed=82)
    zero = Batch([300], 1, 16, seed=82)
    for j in range(15, 19):
        for w in ("k", "v"):
            zero.codes[w][zero.bt[0, j]] = 0
            zero.sb[w][zero.bt[0, j]] = 0
    q = queries(b.rng, 1, 2)
    got = attend(pkv, b, q, 1, 1 / 16, ws, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=b.bt[:, :15].copy())
    check(got, *reference(zero, q, 1, 2, 1 / 16))


def test_attend_offsets_past_32_bits(pkv, ws):
    b = Batch([200, 100], 1, 16, seed=91, big_stride=400 << 20)
    assert b.nb * b.big_stride > 1 << 33
    q = queries(b.rng, 2, 4)
    check(attend(pkv, b, q, 1, 1 / 16, ws), *reference(b, q, 1, 4, 1 / 16))
    run_read(pkv, b, [0, 0], [200, 100], 200)
    rows = {w: rows_u16(b.rng, 40, 1) for w in ("k", "v")}
    run_write(pkv, b, [30, 10], rows)


def test_attend_same_bits_again_and_for_other_blocks(pkv, ws):
    """Bit for bit the same for the same call, whatever the workspace held, and for the same rows in other
    blocks."""
    lens = [3001, 17, 800, 5000]
    a, c = Batch(lens, 2, 16, seed=95), Batch(lens, 2, 16, seed=95)
    move = np.random.default_rng(1).permutation(c.nb)
    for w in ("k", "v"):
        for x in (c.codes, c.sb):
            moved = np.empty_like(x[w])
            moved[move] = x[w]
            x[w] = moved
    c.bt = np.where(c.bt >= 0, move[np.maximum(c.bt, 0)], -1).astype(np.int32)
    q = queries(a.rng, 4 * 3, 4)
    first = attend(pkv, a, q, 3, 1 / 16, ws)
    ws.fill_(0x7F)
    assert np.array_equal(first, attend(pkv, a, q, 3, 1 / 16, ws))
    assert np.array_equal(first, attend(pkv, c, q, 3, 1 / 16, ws))


@pytest.mark.parametrize("entry", [-1, -2, -(1 << 31), (1 << 31) - 1])
def test_attend_every_bad_table_entry(pkv, ws, entry):
    """Also -1, which tables are padded with: below seq_len it is a bad block like any other, read as zero."""
    b, zero = Batch([900, 300], 2, 16, seed=83), Batch([900, 300], 2, 16, seed=83)
    bad = b.bt.copy()
    for r, j in ((0, 0), (0, 20), (0, 56), (1, 18)):
        bad[r, j] = entry
        for w in ("k", "v"):
            zero.codes[w][zero.bt[r, j]] = 0
            zero.sb[w][zero.bt[r, j]] = 0
    q = queries(b.rng, 2 * 2, 8)
    got = attend(pkv, b, q, 2, 1 / 16, ws, expect_err=pkv.PKV_ERR_DEVICE_BOUNDS, bt=bad)
    check(got, *reference(zero, q, 2, 4, 1 / 16))


@pytest.mark.parametrize("T,hkv,group", [(1, 100, 2), (64, 4, 32), (33, 3, 5)])
def test_attend_more_rows_than_ctas(pkv, ws, T, hkv, group):
    """Column groups that do not fill the SMs evenly, and more of them than SMs: one line of all of them."""
    run_attend(pkv, ws, [150, 70], T, hkv, group, 16, seed=hkv)


def test_attend_every_code_and_scale(pkv, ws):
    """Keys and values of random codes under every scale that is not negative or NaN, subnormal ones and
    zero among them."""
    b = Batch([508], 1, 16, seed=97)
    blk, slot = b.where(0, np.arange(508))
    for w in ("k", "v"):
        b.codes[w][blk, slot] = b.rng.integers(0, 256, (508, 1, 128))
        b.sb[w][blk, slot] = ((np.arange(508)[:, None, None] + 8 * np.arange(16)) % 127).astype(np.uint8)
    for T, scale in ((1, 1e-3), (8, 1e-3), (8, 0.2)):
        q = queries(b.rng, T, 4)
        check(attend(pkv, b, q, T, scale, ws), *reference(b, q, T, 4, scale))


def test_attend_query_rows_of_zero_and_infinity(pkv, ws):
    """A zero row weighs its keys alike; a row with an infinity is NaN and leaves the others as they are."""
    b = Batch([500], 2, 16, seed=98)
    q = queries(b.rng, 3, 8)
    q[1, 2], q[2, 5] = 0, 0x8000
    q[0, 1], q[0, 6] = 1, 0x0080  # the smallest subnormal, the smallest normal number
    want = attend(pkv, b, q, 3, 1 / 16, ws)
    check(want, *reference(b, q, 3, 4, 1 / 16))
    bad = q.copy()
    bad[1, 0, 17], bad[2, 7, 255] = 0x7F80, 0xFF80
    got = attend(pkv, b, bad, 3, 1 / 16, ws)
    assert np.isnan(got[1, 0]).all() and np.isnan(got[2, 7]).all()
    got[1, 0], got[2, 7] = want[1, 0], want[2, 7]
    check(got, *reference(b, q, 3, 4, 1 / 16))


def test_attend_requests_that_share_blocks(pkv, ws):
    """The same blocks in two requests' tables, and twice in one."""
    b = Batch([300, 300, 300], 2, 16, seed=99)
    b.bt[1, :10] = b.bt[0, :10]
    b.bt[2, 1:12] = b.bt[2, 0]
    q = queries(b.rng, 3 * 2, 8)
    check(attend(pkv, b, q, 2, 1 / 16, ws), *reference(b, q, 2, 4, 1 / 16))


def test_attend_graphs_that_take_turns_with_a_workspace(pkv, ws):
    """Two graphs over the same workspace and tables, one after the other on a stream, with an eager call of
    another shape between them; the lengths change between the rounds."""
    b = Batch([900, 2000, 40], 2, 16, seed=103)
    caches, scales, bt, sl = b.device()
    calls = []
    for T, group in ((1, 4), (8, 4), (3, 2)):
        q = queries(b.rng, 3 * T, 2 * group)
        calls.append((T, group, q, u16_to_bf16(q).to(DEV)))
    outs = [torch.empty_like(c[3]) for c in calls]

    def call(i):
        T, _, _, qd = calls[i]
        pkv.spec_verify_attn_fp4(qd, *caches, *scales, bt, sl, T, 1 / 16, outs[i], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in range(3):
            call(i)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i)
    for lens in ([900, 2000, 40], [1, 1500, 39], [0, 8, 0]):
        sl.copy_(torch.tensor(lens, dtype=torch.int32))
        for o in outs:
            o.fill_(float("nan"))
        graphs[0].replay()
        call(2)
        graphs[1].replay()
        torch.cuda.synchronize()
        b.lens = lens
        for (T, group, q, _), o in zip(calls, outs):
            check(F.bf16_to_f32(bf16_to_u16(o)).astype(np.float64), *reference(b, q, T, group, 1 / 16))


def test_refuses_strided_index_tensors(pkv, ws):
    b = Batch([40, 40], 1, 16, seed=104)
    caches, scales, bt, sl = b.device()
    q = torch.zeros(2, 4, 256, dtype=torch.bfloat16, device=DEV)
    dense = [torch.zeros(2, 64, 1, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    new = [torch.zeros(2, 1, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    qsl = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    wide = sl.repeat_interleave(2)[::2]
    for table, lens in ((bt.t().contiguous().t(), sl), (bt, wide), (bt, sl.long())):
        with pytest.raises(AssertionError):
            pkv.spec_verify_attn_fp4(q, *caches, *scales, table, lens, 1, 1 / 16, torch.empty_like(q), ws)
        with pytest.raises(AssertionError):
            pkv.kv_fp4_dequant_dense(*caches, table, lens, lens, 40, *scales, *dense)
        with pytest.raises(AssertionError):
            pkv.kv_cache_write_fp4(*new, table, lens, qsl, 1, *caches, *scales)
    torch.cuda.synchronize()


@pytest.mark.parametrize("ctas", [1, 2, 7, 100])
def test_attend_small_workspace(pkv, ctas):
    small = torch.empty(pkv.spec_verify_fp4_workspace_bytes(ctas), dtype=torch.uint8, device=DEV)
    run_attend(pkv, small, [700, 20, 1300], 3, 2, 4, 16, seed=ctas)


def test_attend_on_two_streams(pkv):
    """Two calls at once, each with its own workspace and stream."""
    b = Batch([2500, 900, 33], 4, 16, seed=101)
    q = queries(b.rng, 3 * 2, 16)
    caches, scales, bt, sl = b.device()
    qd = u16_to_bf16(q).to(DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [torch.empty(pkv.spec_verify_fp4_workspace_bytes(), dtype=torch.uint8, device=DEV) for _ in streams]
    outs = [torch.full_like(qd, float("nan")) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, o in zip(streams, wss, outs):
            pkv.spec_verify_attn_fp4(qd, *caches, *scales, bt, sl, 2, 1 / 16, o, w, stream=s)
    torch.cuda.synchronize()
    want, tol = reference(b, q, 2, 4, 1 / 16)
    for o in outs:
        check(F.bf16_to_f32(bf16_to_u16(o)).astype(np.float64), want, tol)


@pytest.mark.parametrize("T,lens", [(8, [3000, 900, 64]), (1, [20000, 0, 5]), (4, [90] * 40)])
def test_attend_gives_up_reports_timeout_and_recovers(pkv, ws, T, lens):
    """With a bound of one nanosecond the CTAs give up at their first wait that is not already satisfied,
    with their copies in flight: the call reports the timeout, and the next one is as before."""
    b = Batch(lens, 2, 16, seed=T)
    q = queries(b.rng, len(lens) * T, 8)
    ref = attend(pkv, b, q, T, 1 / 16, ws)
    caches, scales, bt, sl = b.device()
    qd = u16_to_bf16(q).to(DEV)
    err, out = dev_err(), torch.zeros_like(qd)
    pkv.lib.pkv_testing_set_wait_limit_ns(1)
    pkv.spec_verify_attn_fp4(qd, *caches, *scales, bt, sl, T, 1 / 16, out, ws, dev_err=err)
    torch.cuda.synchronize()
    assert err.item() == pkv.PKV_ERR_TIMEOUT
    assert np.array_equal(ref, attend(pkv, b, q, T, 1 / 16, ws))


# ------------------------------------------------------------------------------------------------
# together
# ------------------------------------------------------------------------------------------------

def test_decode_loop_in_a_graph(pkv, ws):
    """Captured once, replayed for every step: append T new rows a request, attend; the lengths grow on the
    device."""
    T, hkv, group, bs, steps = 2, 2, 4, 16, 6
    start = [30, 127, 250]
    b = Batch([n + T * steps for n in start], hkv, bs, seed=111, fill=False)
    rng = b.rng
    for r, n in enumerate(start):
        blk, slot = b.where(r, np.arange(n))
        for w, g in (("k", b.kg), ("v", b.vg)):
            b.codes[w][blk, slot], b.sb[w][blk, slot] = F.quantize(rows_u16(rng, n, hkv), g)
    caches, scales, bt, _ = b.device()
    lens = torch.tensor(start, dtype=torch.int32, device=DEV)
    qsl = torch.arange(0, T * 3 + 1, T, dtype=torch.int32, device=DEV)
    new = {w: torch.zeros(3 * T, hkv, 256, dtype=torch.bfloat16, device=DEV) for w in ("k", "v")}
    q = torch.zeros(3 * T, hkv * group, 256, dtype=torch.bfloat16, device=DEV)
    out, err = torch.empty_like(q), dev_err()

    def step():
        lens.add_(T)
        pkv.kv_cache_write_fp4(new["k"], new["v"], bt, lens, qsl, T, *caches, *scales, dev_err=err)
        pkv.spec_verify_attn_fp4(q, *caches, *scales, bt, lens, T, 1 / 16, out, ws, dev_err=err)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    lens.copy_(torch.tensor(start, dtype=torch.int32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        rows = {w: rows_u16(rng, 3 * T, hkv) for w in ("k", "v")}
        qh = queries(rng, 3 * T, hkv * group)
        for w, g in (("k", b.kg), ("v", b.vg)):
            new[w].copy_(u16_to_bf16(rows[w]))
            for r, n in enumerate(start):
                blk, slot = b.where(r, n + i * T + np.arange(T))
                b.codes[w][blk, slot], b.sb[w][blk, slot] = F.quantize(rows[w][r * T:(r + 1) * T], g)
        q.copy_(u16_to_bf16(qh))
        graph.replay()
        torch.cuda.synchronize()
        b.lens = [n + (i + 1) * T for n in start]
        check(F.bf16_to_f32(bf16_to_u16(out)).astype(np.float64), *reference(b, qh, T, group, 1 / 16))
    assert err.item() == 0


def test_prefill_chunks_from_the_cache(pkv):
    """A prompt in two chunks: write a chunk, read its rows back into the kept dense rows, run the bf16
    prefill on those."""
    hkv, group, bs, n, cut = 2, 4, 48, 300, 170
    b = Batch([n], hkv, bs, seed=121, fill=False)
    rows = {w: rows_u16(b.rng, n, hkv) for w in ("k", "v")}
    q = queries(b.rng, n, hkv * group)
    caches, scales, bt, _ = b.device()
    # the dense rows as one block a request, its length a multiple of 8 as the prefill wants it
    dense = [torch.zeros(1, 304, hkv, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    identity = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    err = dev_err()
    got = []
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    for lo, hi in ((0, cut), (cut, n)):
        new = [u16_to_bf16(rows[w][lo:hi]).to(DEV) for w in ("k", "v")]
        qd = u16_to_bf16(q[lo:hi]).to(DEV)
        out = torch.empty_like(qd)
        sl, qsl = i32(hi), i32(0, hi - lo)
        pkv.kv_cache_write_fp4(*new, bt, sl, qsl, hi - lo, *caches, *scales, dev_err=err)
        pkv.kv_fp4_dequant_dense(*caches, bt, i32(lo), sl, hi - lo, *scales, *dense, dev_err=err)
        pkv.paged_prefill_attn(qd, *dense, identity, sl, qsl, hi - lo, 1 / 16, out, dev_err=err)
        got.append(out)
    torch.cuda.synchronize()
    assert err.item() == 0
    got = F.bf16_to_f32(bf16_to_u16(torch.cat(got))).astype(np.float64)
    val = {}
    for w, g in (("k", b.kg), ("v", b.vg)):
        val[w] = F.bf16_to_f32(F.dequantize_bf16(*F.quantize(rows[w], g), g)).astype(np.float64)
    want, _ = F.attention(q, val["k"], val["v"], n, n, group, 1 / 16)
    # the prefill's own bar: 2e-3 beyond the rounding of its bf16 output, for values of order one
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2e-3 * max(1.0, np.abs(val["v"]).max())).all()
