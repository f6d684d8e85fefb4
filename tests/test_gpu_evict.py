"""Attention weights of the cached keys, the choice of those that stay, and the move of their rows, against plain numpy."""
import numpy as np
import pytest
import torch

import _step as S
from _devsetup import DEV, dev_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_int64_gb300 as m
    return m


class Cache:
    """Requests of given lengths in a shuffled pool; slots that no request owns are poisoned."""

    def __init__(self, fmt, lens, hkv, bs, seed=0, pad=0, spare=2, extra_cols=1):
        rng = np.random.default_rng(seed)
        self.fmt, self.lens, self.hkv, self.bs = fmt, list(lens), hkv, bs
        pages = [-(-n // bs) for n in lens]
        self.nb = sum(pages) + spare
        perm, at = rng.permutation(self.nb), 0
        self.bt = np.full((len(lens), max(1, max(pages)) + extra_cols), -1, dtype=np.int32)
        for r, n in enumerate(pages):
            self.bt[r, :n] = perm[at:at + n]
            at += n
        self.free = perm[at:]
        shape = (self.nb, bs, hkv + pad, 256)
        self.scale = None
        self.rows = []  # per request: the stored values in 64 bits
        if fmt == "bf16":
            pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        elif fmt == "int8":
            pool = torch.full(shape, 127, dtype=torch.int8)
            self.scale = torch.full((self.nb, bs, hkv + pad), float("nan"))
        else:
            pool = torch.full(shape, 0x7F, dtype=torch.uint8)
            self.scale = torch.tensor([0.037])
        for r, n in enumerate(lens):
            x = torch.from_numpy(rng.standard_normal((n, hkv, 256)) * np.exp(0.5 * rng.standard_normal((hkv, 256)))).float()
            pos = np.arange(n)
            blk, slot = torch.from_numpy(self.bt[r, pos // bs].astype(np.int64)), torch.from_numpy(pos % bs)
            if fmt == "bf16":
                v = x.to(torch.bfloat16)
                pool[blk, slot, :hkv] = v
                self.rows.append(v.double().numpy())
            elif fmt == "int8":
                a = x.abs().amax(-1)
                c = torch.round(x * (127.0 / a)[..., None]).to(torch.int8)
                pool[blk, slot, :hkv] = c
                self.scale[blk, slot, :hkv] = a / 127.0
                self.rows.append(c.double().numpy() * (a / 127.0).double().numpy()[..., None])
            else:
                c = (x / 0.037).clamp(-448, 448).to(torch.float8_e4m3fn)
                pool[blk, slot, :hkv] = c.view(torch.uint8)
                self.rows.append(c.double().numpy() * float(np.float32(0.037)))
        self.pool = pool.to(DEV)[:, :, :hkv]
        if self.scale is not None:
            self.scale = self.scale.to(DEV)
            if fmt == "int8":
                self.scale = self.scale[:, :, :hkv]
        self.table = torch.from_numpy(self.bt).to(DEV)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device=DEV)


KV = {"bf16": 0, "int8": 1, "fp8": 2}


def weigh(pkv, c, q, T, scale, weights, **kw):
    err = dev_err()
    ws = torch.full((pkv.kv_attn_weights_workspace_bytes(q.shape[0], q.shape[1], kw.pop("ctas", None)),), 0xFF, dtype=torch.uint8, device=DEV)
    kw = {k: v if v is None or not isinstance(v, list) else torch.tensor(v, dtype=torch.int32, device=DEV) for k, v in kw.items()}
    pkv.kv_attn_weights(q, c.pool, c.table, c.seq, T, scale, weights, ws, kv_dtype=KV[c.fmt], k_scale=c.scale, dev_err=err, **kw)
    torch.cuda.synchronize()
    return err.item()


def queries(R, T, hq, seed):
    return torch.randn(R * T, hq, 256, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def expect(c, q, T, scale, valid=None, lse=None):
    qd = q.double().numpy()
    out = []
    for r, n in enumerate(c.lens):
        out.append(S.weights(qd[r * T:(r + 1) * T], c.rows[r], n, T, scale, T if valid is None else max(0, min(valid[r], T)),
                             None if lse is None else lse[r * T:(r + 1) * T], rounded=c.fmt != "bf16"))
    return out


def verify_weights(got, want, lens, base=None, tail=None):
    got = got.double().cpu().numpy()
    for r, n in enumerate(lens):
        w, bound = want[r]
        if base is not None:
            w = w + base[r]
            bound = bound + 2.0 ** -23 * np.abs(w)
        e = np.abs(got[r, :, :n] - w)
        ok = bool((e <= bound + 1e-37).all())  # false for NaN too
        assert ok, (r, float((e / (bound + 1e-37)).max()), float(e.max()))
        if tail is not None:
            assert (got[r, :, n:] == tail).all(), "positions behind the last key"


GEOMETRIES = [  # lens, T, hkv, group, block
    ([1], 1, 1, 1, 8),
    ([7], 1, 4, 4, 16),
    ([128, 129, 127], 1, 2, 4, 16),
    ([300, 0, 1, 555], 3, 2, 7, 48),
    ([1000, 131], 8, 4, 4, 880),
    ([513, 700], 8, 2, 6, 24),
    ([640], 16, 1, 8, 64),
    ([900, 40], 32, 2, 4, 176),
    ([260], 20, 1, 16, 8),
    ([333], 5, 2, 32, 16),
    ([200], 2, 1, 128, 128),
    ([2500, 90, 1700], 1, 4, 4, 256),
]


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("lens,T,hkv,g,bs", GEOMETRIES)
def test_weights(pkv, fmt, lens, T, hkv, g, bs):
    c = Cache(fmt, lens, hkv, bs, seed=len(lens) + T)
    q = queries(len(lens), T, hkv * g, seed=T)
    w = torch.full((len(lens), hkv, max(lens) + 5), -7.0, device=DEV)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w) == 0
    verify_weights(w, expect(c, q, T, 1 / 16), lens, tail=-7.0)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("in_place", [True, False])
def test_weights_on_top_of_earlier_ones(pkv, fmt, in_place):
    lens, T, hkv, g = [500, 260, 0, 77], 4, 2, 5
    c = Cache(fmt, lens, hkv, 32, seed=9)
    q = queries(4, T, hkv * g, seed=3)
    prev = torch.rand(4, hkv, 512, generator=torch.Generator().manual_seed(1)).to(DEV)
    prev_lens, valid = [496, 100, 0, 99], [4, 0, 2, 1]
    before = prev.clone()
    w = prev if in_place else torch.zeros_like(prev)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, prev=prev, prev_lens=prev_lens, q_valid=valid) == 0
    base = []
    for r, n in enumerate(lens):
        b = before[r, :, :n].double().cpu().numpy()
        b[:, prev_lens[r]:] = 0.0
        base.append(b)
    verify_weights(w, expect(c, q, T, 1 / 16, valid), lens, base, None)
    if in_place:
        for r, n in enumerate(lens):
            assert torch.equal(w[r, :, n:], before[r, :, n:])
    # prev_lens left out: everything takes from prev
    w2 = torch.zeros_like(prev)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w2, prev=before, q_valid=valid) == 0
    verify_weights(w2, expect(c, q, T, 1 / 16, valid), lens, [before[r, :, :n].double().cpu().numpy() for r, n in enumerate(lens)])


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("T,hkv,g", [(20, 1, 16), (5, 2, 32), (3, 1, 100)])
def test_weights_of_more_columns_than_a_pass_takes(pkv, fmt, T, hkv, g):
    """Tokens in several passes, each on top of the one before: earlier weights and rejected tokens count once."""
    lens = [400, 150, 2]
    c = Cache(fmt, lens, hkv, 48, seed=T)
    q = queries(3, T, hkv * g, seed=T)
    w = torch.rand(3, hkv, 400, generator=torch.Generator().manual_seed(2)).to(DEV)
    before = w.clone()
    valid, prev_lens = [T - 1, T, 1], [400, 100, 1]
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, prev=w, prev_lens=prev_lens, q_valid=valid) == 0
    base = []
    for r, n in enumerate(lens):
        b = before[r, :, :n].double().cpu().numpy()
        b[:, prev_lens[r]:] = 0.0
        base.append(b)
    verify_weights(w, expect(c, q, T, 1 / 16, valid), lens, base)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("given", [False, True])
def test_weights_wait_that_runs_out(pkv, fmt, given):
    """Waits of 1 ns: the call gives up and says so; the one after it is whole."""
    lens, T, hkv, g = [3000, 2000], 2, 2, 4
    c = Cache(fmt, lens, hkv, 16, seed=41)
    q = queries(2, T, hkv * g, seed=41)
    kw = dict(part_lse=torch.full((1, 2 * T, hkv * g), 5.0, device=DEV), split_tokens=4096) if given else {}
    w = torch.zeros(2, hkv, 3000, device=DEV)
    pkv.lib.pkv_testing_set_wait_limit_ns(1)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, **kw) == pkv.PKV_ERR_TIMEOUT
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, **kw) == 0
    verify_weights(w, expect(c, q, T, 1 / 16, lse=np.full((2 * T, hkv * g), 5.0) if given else None), lens)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T,split", [(1, 128), (8, 512)])
def test_weights_from_the_verify_calls_partials(pkv, fmt, T, split):
    """The chain a step runs: verify attention, then the weights from its partials' log-sum-exps. What comes out is within
    the bound of the given log-sum-exps, and its sum over the keys within their error of the number of query rows."""
    lens, hkv, g = [1300, 400, 130], 2, 4
    c = Cache(fmt, lens, hkv, 80, seed=4)
    q = queries(3, T, hkv * g, seed=5)
    splits = pkv.splits_needed(max(lens), split)
    po = torch.full((splits, 3 * T, hkv * g, 256), float("nan"), device=DEV)
    pl = torch.full((splits, 3 * T, hkv * g), float("nan"), device=DEV)
    call = pkv.spec_verify_attn_partial if fmt == "int8" else pkv.spec_verify_attn_partial_fp8
    call(q.to(DEV), c.pool, c.pool, c.scale, c.scale, c.table, c.seq, T, 1 / 16, split, po, pl)
    w = torch.zeros(3, hkv, max(lens), device=DEV)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, part_lse=pl, split_tokens=split) == 0
    part = pl.double().cpu().numpy()
    lse = np.stack([np.logaddexp.reduce(part[:-(-lens[r] // split), r * T + t], 0) for r in range(3) for t in range(T)])
    verify_weights(w, expect(c, q, T, 1 / 16, lse=lse), lens)
    # the verify kernel's scores are of fp16 queries: 2^-12 of each product at most
    assert np.allclose(w.double().sum((1, 2)).cpu().numpy(), T * hkv * g, rtol=0.02)


def test_weights_many_requests_and_few_ctas(pkv):
    """Keys divided over the CTAs in the middle of requests and heads: the same numbers however many there are."""
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 700, 40)]
    c = Cache("int8", lens, 3, 16, seed=1)
    q = queries(40, 2, 9, seed=2)
    want = expect(c, q, 2, 1 / 16)
    for ctas in (1, 5, None):
        w = torch.zeros(40, 3, 704, device=DEV)
        assert weigh(pkv, c, q.to(DEV), 2, 1 / 16, w, ctas=ctas) == 0
        verify_weights(w, want, lens, tail=0.0)


def test_weights_of_far_apart_scores(pkv):
    """Scores that reach from -3,000 to 3,000: the maximum moves along the keys, weights vanish or are one."""
    c = Cache("bf16", [700], 1, 16, seed=6)
    q = queries(1, 2, 4, seed=6) * 100
    w = torch.zeros(1, 1, 700, device=DEV)
    assert weigh(pkv, c, q.to(DEV), 2, 1.0, w) == 0
    verify_weights(w, expect(c, q, 2, 1.0), [700])
    # keys in ascending and descending order of their scores for the first query
    s = c.rows[0][:, 0] @ q[0, 0].double().numpy()
    for order in (np.argsort(s), np.argsort(-s)):
        rows = c.rows[0][order]
        pos = np.arange(700)
        c.pool[torch.from_numpy(c.bt[0, pos // 16].astype(np.int64)).to(DEV), torch.from_numpy(pos % 16).to(DEV)] = \
            torch.from_numpy(rows).to(DEV, torch.bfloat16)
        d = Cache.__new__(Cache)
        d.__dict__.update(c.__dict__, rows=[rows])
        assert weigh(pkv, d, q.to(DEV), 2, 1.0, w) == 0
        verify_weights(w, expect(d, q, 2, 1.0), [700])


@pytest.mark.parametrize("x,y", [(1.0, 1.0), (175 / 128, 147 / 128)])  # of the second's scores every factor rounds
@pytest.mark.parametrize("T,g", [(1, 4), (4, 8), (8, 8), (8, 16)])
def test_weights_of_very_low_scores(pkv, T, g, x, y):
    """Every score far below -1e30 and no two of them near: each query's weight is its largest key's, the first."""
    lens = [300, 5, 1]
    c = Cache("bf16", lens, 1, 16)
    for r, n in enumerate(lens):
        for pos in range(n):
            c.pool[int(c.bt[r, pos // 16]), pos % 16, 0] = y * 2.0 ** 60 * (1.0 if pos == 0 else 2.0)
    q = torch.full((len(lens) * T, g, 256), -x * 2.0 ** 50, dtype=torch.bfloat16, device=DEV)  # scores of about -2^114, -2^115
    w = torch.full((len(lens), 1, 320), 7.0, device=DEV)
    assert weigh(pkv, c, q, T, 1.0 / 16, w) == 0
    for r, n in enumerate(lens):
        seeing = sum(n - T + t >= 0 for t in range(T))
        assert w[r, 0, 0].item() == seeing * g
        assert (w[r, 0, 1:n] == 0).all() and (w[r, 0, n:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_weights_of_queries_of_unlike_sizes(pkv, fmt):
    """Query heads and elements from 2^-60 to 2^9 side by side, rows of zeros, requests whose queries are all tiny, and the
    largest that bf16 holds beside keys of zeros."""
    lens, T, hkv, g = [300, 200, 140, 130], 3, 2, 4
    c = Cache(fmt, lens, hkv, 16, seed=31)
    gen = torch.Generator().manual_seed(31)
    q = torch.randn(4 * T, hkv * g, 256, generator=gen) * torch.exp2(torch.randint(-60, 4, (4 * T, hkv * g, 1), generator=gen).float())
    q[:T] *= torch.exp2(torch.randint(-20, 3, (T, hkv * g, 256), generator=gen).float())
    q[0, 3] = 0.0
    q[T:2 * T] *= 2.0 ** -40
    q[2 * T:3 * T] *= 2.0 ** -80
    q[3 * T:, :, 8:] = 0.0
    q[3 * T:, :, :8] = 3e38
    pos = np.arange(130)
    c.pool[torch.from_numpy(c.bt[3, pos // 16].astype(np.int64)).to(DEV), torch.from_numpy(pos % 16).to(DEV), :, :8] = 0
    c.rows[3][:, :, :8] = 0.0
    q = q.to(torch.bfloat16)
    w = torch.zeros(4, hkv, 300, device=DEV)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w) == 0
    verify_weights(w, expect(c, q, T, 1 / 16), lens)


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_weights_bad_blocks_and_lengths(pkv, fmt):
    lens, T, hkv, g, bs = [300, 200], 2, 2, 3, 16
    c = Cache(fmt, lens, hkv, bs, seed=7)
    q = queries(2, T, hkv * g, seed=8)
    c.table[0, 3], c.table[1, 5] = -1, c.nb
    c.rows[0][48:64] = 0.0  # a bad block's keys read as zero
    c.rows[1][80:96] = 0.0
    w = torch.full((2, hkv, 320), -7.0, device=DEV)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w) == pkv.PKV_ERR_DEVICE_BOUNDS
    verify_weights(w, expect(c, q, T, 1 / 16), lens, tail=-7.0)
    # a buffer that is too short for one request: the rest is written all the same
    w = torch.full((2, hkv, 400), -7.0, device=DEV)[:, :, :250]
    c.table.copy_(torch.from_numpy(c.bt))
    c = Cache(fmt, lens, hkv, bs, seed=7)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w) == pkv.PKV_ERR_DEVICE_BOUNDS
    want = expect(c, q, T, 1 / 16)
    verify_weights(w, [(x[:, :250], b[:, :250]) for x, b in want], [250, 200], tail=-7.0)
    assert (w._base[:, :, 250:] == -7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_weights_nan_keys_stay_their_own(pkv, fmt):
    """A NaN in one key's row: that key's weight, and with it the log-sum-exp of every query that sees it, is NaN; the other
    requests and heads are not touched. Values behind the last key are not read at all (the pool is poisoned)."""
    c = Cache(fmt, [200, 200], 2, 16, seed=3)
    q = queries(2, 1, 4, seed=3)
    blk, slot = int(c.bt[0, 100 // 16]), 100 % 16
    if fmt == "int8":
        c.scale[blk, slot, 1] = float("nan")
    else:
        c.pool[blk, slot, 1, 255] = float("nan") if fmt == "bf16" else 0xFF
    want = expect(c, q, 1, 1 / 16)
    w = torch.zeros(2, 2, 200, device=DEV)
    assert weigh(pkv, c, q.to(DEV), 1, 1 / 16, w) == 0
    got = w.cpu().numpy()
    assert np.isnan(got[0, 1]).all()
    for r, h in ((0, 0), (1, 0), (1, 1)):
        assert (np.abs(got[r, h] - want[r][0][h]) <= want[r][1][h] + 1e-37).all()
    # with the log-sum-exp given, the other keys keep theirs
    lse = torch.full((1, 2, 4), 3.0, device=DEV)
    assert weigh(pkv, c, q.to(DEV), 1, 1 / 16, w, part_lse=lse, split_tokens=256) == 0
    got = w.cpu().numpy()
    assert np.isnan(got[0, 1, 100]) and np.isnan(got).sum() == 1
    # -inf: a row without a visible key; it adds nothing
    assert weigh(pkv, c, q.to(DEV), 1, 1 / 16, w, part_lse=torch.full((1, 2, 4), -np.inf, device=DEV), split_tokens=256) == 0
    got = w.cpu().numpy()
    assert (got[1] == 0).all() and (got[0, 0] == 0).all()


def test_weights_strided_cache_graph_and_stream(pkv):
    """Heads inside a wider pool, weights inside a wider buffer; captured, replayed as the lengths grow, beside a call on
    another stream with a workspace of its own."""
    lens, T, hkv, g = [600, 450], 2, 2, 4
    c = Cache("bf16", lens, hkv, 64, seed=11, pad=2)
    q = queries(2, T, hkv * g, seed=11)
    qd, buf = q.to(DEV), torch.zeros(2, 5, 700, device=DEV)
    w = buf[:, 1:4:2, 13:]
    ws = [torch.zeros(pkv.kv_attn_weights_workspace_bytes(2 * T, hkv * g), dtype=torch.uint8, device=DEV) for _ in range(2)]
    other = torch.zeros(2, hkv, 687, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_attn_weights(qd, c.pool, c.table, c.seq, T, 1 / 16, w, ws[0])
    side = torch.cuda.Stream()
    for cut in (400, 100, 0):
        now = [n - cut for n in lens]
        c.seq.copy_(torch.tensor(now, dtype=torch.int32))
        buf.zero_()
        torch.cuda.synchronize()
        graph.replay()
        pkv.kv_attn_weights(qd, c.pool, c.table, c.seq, T, 1 / 16, other, ws[1], stream=side)
        torch.cuda.synchronize()
        d = Cache.__new__(Cache)
        d.__dict__.update(c.__dict__, lens=now, rows=[x[:n] for x, n in zip(c.rows, now)])
        want = expect(d, q, T, 1 / 16)
        verify_weights(w, want, now, tail=0.0)
        verify_weights(other, want, now)
        assert torch.equal(buf[:, 0], torch.zeros_like(buf[:, 0])) and torch.equal(buf[:, :, :13], torch.zeros_like(buf[:, :, :13]))


# ------------------------------------------------------------------------------------------------
# selection
# ------------------------------------------------------------------------------------------------

def pick(pkv, scores, lens, sinks, recent, budget, stream=None):
    R, hkv, _ = scores.shape
    keep = torch.full((R, hkv, budget), -5, dtype=torch.int32, device=DEV)
    new, err = torch.full((R,), -5, dtype=torch.int32, device=DEV), dev_err()
    pkv.kv_evict_select(scores.to(DEV) if not scores.is_cuda else scores, torch.tensor(lens, dtype=torch.int32, device=DEV), sinks, recent, budget, keep,
                        new, dev_err=err, stream=stream)
    torch.cuda.synchronize()
    return keep.cpu().numpy(), new.cpu().numpy(), err.item()


def check_pick(pkv, scores, lens, sinks, recent, budget, status=0):
    keep, new, err = pick(pkv, scores, lens, sinks, recent, budget)
    assert err == status
    sc = scores.cpu().numpy()
    for r, n in enumerate(lens):
        n = max(0, min(n, sc.shape[2]))
        assert new[r] == min(n, budget)
        for h in range(sc.shape[1]):
            want = S.select(sc[r, h], n, sinks, recent, budget)
            assert np.array_equal(keep[r, h, :new[r]], want), (r, h)
            assert (keep[r, h, new[r]:] == -5).all()


@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([1], 1, 0, 0), ([2, 0, 1], 1, 0, 1), ([9], 8, 4, 4), ([33, 300, 64], 32, 1, 3), ([1000], 999, 0, 0), ([1000, 5000, 777], 500, 4, 64),
    ([5000], 5000, 10, 10), ([40960, 12345], 8192, 4, 256), ([262144], 16384, 0, 1024), ([70001], 1, 0, 0), ([4096], 4095, 4, 4090),
])
@pytest.mark.parametrize("hkv", [1, 3])
def test_select(pkv, lens, budget, sinks, recent, hkv):
    g = torch.Generator().manual_seed(sum(lens))
    sc = torch.exp(2 * torch.randn(len(lens), hkv, max(lens) + 3, generator=g) - 6)
    for r, n in enumerate(lens):
        sc[r, :, n:] = float("inf")  # behind the last position: never chosen
    check_pick(pkv, sc, lens, sinks, recent, budget)


@pytest.mark.parametrize("kind", ["equal", "few", "signed", "odd", "close", "wide", "outlier"])
def test_select_ties_and_odd_scores(pkv, kind):
    g = torch.Generator().manual_seed(4)
    sc = torch.rand(2, 2, 3001, generator=g)
    if kind == "equal":
        sc.fill_(0.25)
    elif kind == "few":
        sc = torch.randint(0, 3, sc.shape, generator=g).float()
    elif kind == "signed":
        sc = torch.randn(sc.shape, generator=g)
        sc[0, 0, ::3] = 0.0
        sc[0, 0, 1::3] = -0.0
    elif kind == "odd":
        x = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 3.4e38, -3.4e38])
        sc = x[torch.randint(0, 10, sc.shape, generator=g)]
    elif kind == "wide":  # over the whole exponent range
        sc = torch.exp2(200 * torch.rand(sc.shape, generator=g) - 100)
    elif kind == "outlier":  # a few far above all others
        sc = torch.rand(sc.shape, generator=g) * 1e-20
        sc[:, :, ::1000] = 1e30
    else:  # neighbours in the last digit
        sc = (torch.randint(0, 1500, sc.shape, generator=g) + 0x3F800000).int().view(torch.float32)
    for budget in (1, 700, 1500, 2990):
        check_pick(pkv, sc, [3001, 2999], 0 if budget == 1 else 2, 1, budget)
        check_pick(pkv, sc, [3001, 2999], 0, 0, budget)


def test_select_longer_than_shared_memory(pkv):
    """A slice that shared memory does not hold is read again."""
    n = 16 * 49152 + 16 * 700 + 3
    sc = torch.rand(1, 1, n, generator=torch.Generator().manual_seed(1))
    check_pick(pkv, sc, [n], 4, 100, 60001)


def test_select_many_requests_of_a_long_buffer(pkv):
    """More (request, KV head) pairs than the device holds clusters for, in a buffer whose slices shared memory does not hold
    whole."""
    lens = [60000] + [500] * 90 + [59999, 0, 300, 47105]
    sc = torch.rand(len(lens), 2, 60000, generator=torch.Generator().manual_seed(3))
    check_pick(pkv, sc, lens, 4, 32, 400)


def test_select_strides_bad_lengths_graph(pkv):
    g = torch.Generator().manual_seed(9)
    wide = torch.rand(3, 6, 900, generator=g).to(DEV)
    sc = wide[:, 1:5:3, 7:807]
    check_pick(pkv, sc, [800, 500, 100], 2, 10, 128)
    check_pick(pkv, sc, [801, -3, 100], 2, 10, 128, status=pkv.PKV_ERR_DEVICE_BOUNDS)
    lens = torch.tensor([800, 500, 100], dtype=torch.int32, device=DEV)
    keep, new = torch.zeros(3, 2, 128, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_evict_select(sc, lens, 2, 10, 128, keep, new)
    for _ in range(2):
        wide.copy_(torch.rand(wide.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = pick(pkv, sc, [800, 500, 100], 2, 10, 128)
        for r in range(3):
            assert np.array_equal(keep.cpu().numpy()[r, :, :want[1][r]], want[0][r, :, :want[1][r]])


# ------------------------------------------------------------------------------------------------
# the move
# ------------------------------------------------------------------------------------------------

FORMATS = {"bf16": (torch.bfloat16, 256, None), "int8": (torch.int8, 256, torch.float32), "fp8": (torch.uint8, 256, None),
           "fp4": (torch.uint8, 128, torch.uint8)}


def random_bytes(shape, dtype, g):
    size = torch.empty((), dtype=dtype).element_size()
    return torch.randint(0, 256, (*shape[:-1], shape[-1] * size), generator=g, dtype=torch.uint8).view(dtype)


class Rows:
    """K, V, scales and weights of random bits, a shuffled table, and kept positions."""

    def __init__(self, fmt, lens, hkv, bs, budget, seed, pad=0, apart=False, dense=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt, row, sdt = FORMATS[fmt]
        pages = [-(-n // bs) for n in lens]
        new = [min(n, budget) for n in lens]
        more = [-(-n // bs) for n in new] if apart else [0] * len(lens)
        self.nb = sum(pages) + sum(more) + 1
        perm, at = rng.permutation(self.nb), 0
        self.src = np.full((len(lens), max(1, max(pages))), -1, dtype=np.int32)
        for r, n in enumerate(pages):
            self.src[r, :n] = perm[at:at + n]
            at += n
        self.dst = self.src
        if apart:
            self.dst = np.full((len(lens), max(1, max(more)) + 1), -1, dtype=np.int32)
            for r, n in enumerate(more):
                self.dst[r, :n] = perm[at:at + n]
                at += n
        self.pools = [random_bytes((self.nb, bs, hkv + pad, row), dt, g).to(DEV)[:, :, pad:] for _ in range(2)]
        if sdt is None:
            self.scales = [None, None]
        elif fmt == "int8":
            self.scales = [torch.rand(self.nb, bs, hkv + pad, generator=g).to(DEV)[:, :, pad:] for _ in range(2)]
        else:
            self.scales = [random_bytes((self.nb, bs, hkv + pad, 16), sdt, g).to(DEV)[:, :, pad:] for _ in range(2)]
        self.weights = torch.rand(len(lens), hkv, max(lens) + 2, generator=g).to(DEV)
        self.keep = np.full((len(lens), hkv, budget), -9, dtype=np.int32)
        for r, n in enumerate(lens):
            for h in range(hkv):
                k = np.sort(rng.permutation(n)[:new[r]])
                if dense == "front" and n > budget:  # one gap early: every row moves by a little, through its neighbours
                    k = np.concatenate(([0], np.arange(1 + n - budget, n))) if h % 2 == 0 else np.arange(budget) + 1
                self.keep[r, h, :new[r]] = k
        self.fmt, self.lens, self.new, self.bs, self.hkv, self.budget = fmt, lens, new, bs, hkv, budget

    def run(self, pkv, weights=True, keep=None, new=None, stream=None):
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
        err = dev_err()
        src = i32(self.src)
        ws = torch.full((pkv.kv_cache_compact_workspace_bytes(len(self.lens), self.hkv, self.budget),), 0xFF, dtype=torch.uint8, device=DEV)
        pkv.kv_cache_compact(*self.pools, src, src if self.dst is self.src else i32(self.dst), i32(self.keep if keep is None else keep),
                             i32(self.new if new is None else new), ws, kv_dtype={"bf16": 0, "int8": 1, "fp8": 2, "fp4": 3}[self.fmt],
                             k_scale=self.scales[0], v_scale=self.scales[1], weights=self.weights if weights else None, dev_err=err,
                             stream=stream)
        torch.cuda.synchronize()
        return err.item()

    def state(self):
        bits = lambda t: t.contiguous().view(torch.uint8).cpu().numpy().copy()  # noqa: E731
        return [bits(t) for t in (*self.pools, *self.scales) if t is not None], self.weights.cpu().numpy().copy()

    def expect(self, weights=True, keep=None, skip=lambda r, h, j: False):
        pools, w = self.state()
        out, ow = [p.copy() for p in pools], w.copy()
        keep = self.keep if keep is None else keep
        for r, n in enumerate(self.new):
            for h in range(self.hkv):
                for j in range(n):
                    if skip(r, h, j):
                        continue
                    k = int(keep[r, h, j])
                    a, b = int(self.src[r, k // self.bs]), int(self.dst[r, j // self.bs])
                    for p, o in zip(pools, out):
                        if p.ndim == 3:  # fp32 scales seen as bytes
                            o[b, j % self.bs, 4 * h:4 * h + 4] = p[a, k % self.bs, 4 * h:4 * h + 4]
                        else:
                            o[b, j % self.bs, h] = p[a, k % self.bs, h]
                    if weights:
                        ow[r, h, j] = w[r, h, k]
        return out, ow

    def same(self, want):
        got, w = self.state()
        assert all(np.array_equal(a, b) for a, b in zip(got, want[0])) and np.array_equal(w, want[1])


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("lens,hkv,bs,budget", [([1], 1, 8, 1), ([2], 1, 8, 1), ([65, 0, 64], 2, 16, 64), ([700, 90, 300], 3, 24, 130),
                                                ([2000], 2, 176, 1500), ([5000, 4097], 1, 64, 1000)])
@pytest.mark.parametrize("apart", [False, True])
def test_compact(pkv, fmt, lens, hkv, bs, budget, apart):
    x = Rows(fmt, lens, hkv, bs, budget, seed=budget, apart=apart)
    want = x.expect()
    assert x.run(pkv) == 0
    x.same(want)


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("n,budget", [(4000, 3999), (4000, 3936), (4000, 3900), (6000, 3000)])
def test_compact_in_place_through_neighbours(pkv, fmt, n, budget):
    """Every row moves onto rows that are themselves still to be read, by one place, by a chunk, by more."""
    x = Rows(fmt, [n, n - 1, n // 2], 2, 16, budget, seed=n, dense="front")
    want = x.expect()
    assert x.run(pkv) == 0
    x.same(want)


def test_compact_strides_and_no_weights(pkv):
    for fmt in FORMATS:
        x = Rows(fmt, [300, 250], 2, 16, 100, seed=3, pad=1)
        want = x.expect(weights=False)
        assert x.run(pkv, weights=False) == 0
        x.same(want)


def test_compact_bad_entries(pkv):
    """Entries of keep below their index, behind the table, behind the weights, rows in bad blocks: not moved, reported; the
    rest is moved."""
    x = Rows("bf16", [400, 400], 1, 16, 100, seed=5)
    keep = np.stack([np.arange(100) + 200, np.arange(100) + 250])[:, None].astype(np.int32)
    keep[0, 0, 0], keep[0, 0, 99] = -1, 25 * 16
    keep[1, 0, 99] = 2 ** 31 - 1
    x.src[1, 17] = -1  # positions 272..287
    bad = {(0, 0, 0), (0, 0, 99), (1, 0, 99)} | {(1, 0, j) for j in range(100) if 272 <= keep[1, 0, j] < 288}
    want = x.expect(keep=keep, skip=lambda r, h, j: (r, h, j) in bad)
    assert x.run(pkv, keep=keep) == pkv.PKV_ERR_DEVICE_BOUNDS
    x.same(want)
    y = Rows("int8", [50, 60], 1, 16, 40, seed=6)
    want = y.expect()
    assert y.run(pkv, new=[41, 40]) == pkv.PKV_ERR_DEVICE_BOUNDS  # clamped to the budget
    y.same(want)
    z = Rows("int8", [50, 60], 1, 16, 40, seed=6)
    z.new = [0, 40]
    want = z.expect()
    assert z.run(pkv, new=[-1, 40]) == pkv.PKV_ERR_DEVICE_BOUNDS
    z.same(want)


def test_compact_in_a_pool_past_32_bits(pkv):
    """Blocks whose element offsets pass 2^32."""
    bs, hkv = 880, 4
    nb = 2 ** 32 // (bs * hkv * 256) + 8  # 4,774 blocks, 8.6 GB a tensor
    x = Rows("bf16", [1700], hkv, bs, 900, seed=8)
    big = [torch.empty(nb, bs, hkv, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    place = np.array([nb - 1, nb - 3, 5][:x.nb])
    for a, b in zip(x.pools, big):
        b[torch.from_numpy(place).to(DEV)] = a
    want = x.expect()
    small, x.pools, x.src = x.pools, big, place[x.src].astype(np.int32)
    x.dst = x.src
    assert x.run(pkv) == 0
    x.pools = [b[torch.from_numpy(place).to(DEV)] for b in big]
    x.same(want)
    del small


def test_compact_wait_that_runs_out(pkv):
    """Waits of 1 ns: a chunk that gives up leaves its rows where they are and says so; the next call is whole."""
    x = Rows("bf16", [6000, 5999], 2, 16, 5990, seed=15, dense="front")
    pkv.lib.pkv_testing_set_wait_limit_ns(1)
    assert x.run(pkv) in (0, pkv.PKV_ERR_TIMEOUT)
    want = x.expect()
    assert x.run(pkv) == 0
    x.same(want)


def test_compact_graph(pkv):
    x = Rows("int8", [3000, 2500], 2, 16, 700, seed=14)
    first = [t.clone() for t in (*x.pools, *x.scales)]
    w0 = x.weights.clone()
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    src, keep, new = i32(x.src), i32(x.keep), i32(x.new)
    ws = torch.zeros(pkv.kv_cache_compact_workspace_bytes(2, 2, 700), dtype=torch.uint8, device=DEV)
    want = x.expect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_cache_compact(*x.pools, src, src, keep, new, ws, kv_dtype=pkv.PKV_KV_INT8, k_scale=x.scales[0], v_scale=x.scales[1], weights=x.weights)
    for _ in range(3):
        for t, f in zip((*x.pools, *x.scales), first):
            t.copy_(f)
        x.weights.copy_(w0)
        ws.random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        x.same(want)


# ------------------------------------------------------------------------------------------------
# a step
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_step_over_a_bounded_cache(pkv, fmt):
    """Verify attention, accept, weights of the accepted tokens, select, compact, and attention over what stayed: the output
    equals attention over the kept rows computed apart, and the weights follow their keys."""
    lens, T, hkv, g, budget = [700, 333, 150], 4, 2, 4, 256
    c = Cache(fmt, lens, hkv, 80, seed=21, extra_cols=0)
    R = len(lens)
    q = queries(R, T, hkv * g, seed=22).to(DEV)
    split = 256
    S_ = pkv.splits_needed(max(lens), split)
    po, pl = torch.zeros(S_, R * T, hkv * g, 256, device=DEV), torch.zeros(S_, R * T, hkv * g, device=DEV)
    call = pkv.spec_verify_attn_partial if fmt == "int8" else pkv.spec_verify_attn_partial_fp8
    call(q, c.pool, c.pool, c.scale, c.scale, c.table, c.seq, T, 1 / 16, split, po, pl)
    gen = torch.Generator().manual_seed(23)
    P = torch.softmax(2 * torch.randn(R, T, 997, generator=gen), -1).to(DEV)
    Q = torch.softmax(2 * torch.randn(R, T - 1, 997, generator=gen), -1).to(DEV)
    ids = torch.randint(0, 997, (R, T - 1), generator=gen, dtype=torch.int32).to(DEV)
    tokens, num = torch.zeros(R, T, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    pkv.spec_verify_accept(P, Q, ids, torch.rand(R, T - 1, generator=gen).to(DEV) * 0.2, torch.rand(R, generator=gen).to(DEV), tokens, num)
    assert ((num >= 1) & (num <= T)).all()
    w = torch.rand(R, hkv, max(lens), generator=gen).to(DEV)
    prev = w.clone()
    before = c.seq - T
    assert weigh(pkv, c, q, T, 1 / 16, w, prev=w, prev_lens=before.tolist(), q_valid=num.tolist(), part_lse=pl, split_tokens=split) == 0
    valid = num.cpu().numpy()
    part = pl.double().cpu().numpy()
    lse = np.stack([np.logaddexp.reduce(part[:-(-lens[r] // split), r * T + t], 0) for r in range(R) for t in range(T)])
    base = []
    for r, n in enumerate(lens):
        b = prev[r, :, :n].double().cpu().numpy()
        b[:, n - T:] = 0.0
        base.append(b)
    verify_weights(w, expect(c, q.cpu(), T, 1 / 16, valid, lse), lens, base)
    length = (c.seq - T + num).int()
    keep, new = torch.zeros(R, hkv, budget, dtype=torch.int32, device=DEV), torch.zeros(R, dtype=torch.int32, device=DEV)
    pkv.kv_evict_select(w, length, 4, 32, budget, keep, new)
    ws = torch.zeros(pkv.kv_cache_compact_workspace_bytes(R, hkv, budget), dtype=torch.uint8, device=DEV)
    v = c.pool.clone()
    kw = dict(k_scale=c.scale, v_scale=c.scale.clone()) if fmt == "int8" else {}
    w_before = w.clone()
    pkv.kv_cache_compact(c.pool, v, c.table, c.table, keep, new, ws, kv_dtype=KV[fmt], weights=w, **kw)
    out = torch.empty(R, hkv * g, 256, dtype=torch.bfloat16, device=DEV)
    q1 = queries(R, 1, hkv * g, seed=24)
    po, pl = torch.zeros(1, R, hkv * g, 256, device=DEV), torch.zeros(1, R, hkv * g, device=DEV)
    vs = kw.get("v_scale", c.scale)
    call(q1.to(DEV), c.pool, v, c.scale, vs, c.table, new, 1, 1 / 16, 256, po, pl)
    pkv.spec_verify_combine(po, pl, new, 1, 256, out)
    torch.cuda.synchronize()
    kept = keep.cpu().numpy()
    for r in range(R):
        n = int(new[r])
        assert n == min(int(length[r]), budget)
        for h in range(hkv):
            idx = kept[r, h, :n]
            assert np.array_equal(idx, S.select(w_before[r, h].cpu().numpy(), int(length[r]), 4, 32, budget))
            assert torch.equal(w[r, h, :n], w_before[r, h, torch.from_numpy(idx.astype(np.int64)).to(DEV)])
            rows = c.rows[r][idx, h]
            for a in range(g):
                s = rows @ q1[r, h * g + a].double().numpy() / 16
                p = np.exp(s - s.max())
                ref = p @ rows / p.sum()
                got = out[r, h * g + a].double().cpu().numpy()
                # the verify calls' bar, beyond the rounding of a bf16 output
                assert (np.abs(got - ref) <= 2e-3 + 2.0 ** -8 * np.abs(ref)).all()
