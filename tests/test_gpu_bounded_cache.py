"""The calls after the verify attention at the borders of what they take: uniform numbers out of
range, log-sum-exps that do not reach, kept lists out of order, waits that run out, offsets past 32
bits, sums that no rounding has touched."""
import numpy as np
import pytest
import torch

import _step as S
from _devsetup import DEV
from test_gpu_accept import run as accept
from test_gpu_evict import FORMATS, Cache, Rows, expect, queries, verify_weights, weigh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_int64_gb300 as m
    return m


# ------------------------------------------------------------------------------------------------
# accept
# ------------------------------------------------------------------------------------------------

def clamped(u):
    """To [0, 1 - 2^-24], NaN to 0."""
    return np.clip(np.nan_to_num(u.astype(np.float64), nan=0.0, posinf=2.0, neginf=-2.0), 0.0, 1.0 - 2.0 ** -24).astype(np.float32)


ODD_U = [-1.0, -1e-30, -0.0, 0.0, 1.0 - 2.0 ** -24, 1.0, 1.5, float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("drafted", [True, False])
def test_accept_takes_u_to_its_range(pkv, dtype, drafted):
    """Each odd u against a draft of p = 0, p = q and p = q / 2: below 0 is 0, 1 and above the largest below 1, NaN 0."""
    V, ratios = 64, (0.0, 1.0, 0.5)
    R = len(ODD_U) * len(ratios)
    P, Q = torch.full((R, 2, V), 2.0 ** -7), torch.full((R, 1, V), 2.0 ** -6)
    ids = (torch.arange(R, dtype=torch.int32) % V)[:, None]
    q = 2.0 ** -6 if drafted else 1.0
    for i in range(R):
        P[i, 0, ids[i, 0]] = ratios[i % 3] * q
    ua = torch.tensor(ODD_U).repeat_interleave(3)[:, None]
    us = (torch.arange(R) + 0.5) / R
    got = accept(pkv, P.to(dtype), Q.to(dtype) if drafted else None, ids, ua, us, None)
    want = S.accept(P.numpy(), Q.numpy() if drafted else None, ids.numpy(), clamped(ua.numpy()), us.numpy(), [1] * R)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0
    for i in range(R):  # by hand: u q < p
        u = float(clamped(ua.numpy())[i, 0])
        assert got[1][i] == 1 + (u < ratios[i % 3])


@pytest.mark.parametrize("bad", [-1, 4, 2 ** 31 - 1, -2 ** 31])
def test_accept_ids_out_of_range(pkv, bad):
    """By hand: the draft goes; with draft probabilities the token comes from max(p - q, 0), without from all of p."""
    P = torch.tensor([[[0.125, 0.5, 0.25, 0.125], [1.0, 0.0, 0.0, 0.0]]]).expand(4, 2, 4).contiguous()
    Q = torch.tensor([[[0.5, 0.25, 0.25, 0.0]]]).expand(4, 1, 4).contiguous()  # what is left: 0, 1/4, 0, 1/8
    ids, us = torch.full((4, 1), bad, dtype=torch.int64).int(), torch.tensor([0.0, 0.6, 0.7, 0.9])
    for q, tokens in ((Q, [1, 1, 3, 3]), (None, [0, 1, 2, 3])):
        got = accept(pkv, P, q, ids, torch.zeros(4, 1), us, None)
        assert got[0].tolist() == [[x, -1] for x in tokens] and got[1].tolist() == [1] * 4
        assert got[2] == pkv.PKV_ERR_DEVICE_BOUNDS


def test_accept_counts_in_place(pkv):
    """num_out over num_drafts, many requests: each count is read before its own is written."""
    R, T, V = 700, 4, 300
    g = torch.Generator().manual_seed(4)
    P, Q = torch.softmax(torch.randn(R, T, V, generator=g), -1).to(DEV), torch.softmax(torch.randn(R, T - 1, V, generator=g), -1).to(DEV)
    ids = torch.randint(0, V, (R, T - 1), generator=g, dtype=torch.int32).to(DEV)
    ua, us = torch.rand(R, T - 1, generator=g).to(DEV), torch.rand(R, generator=g).to(DEV)
    nd = torch.randint(0, T, (R,), generator=g, dtype=torch.int32).to(DEV)
    want = accept(pkv, P, Q, ids, ua, us, nd)
    out = torch.zeros(R, T, dtype=torch.int32, device=DEV)
    pkv.spec_verify_accept(P, Q, ids, ua, us, out, nd, num_drafts=nd)
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(nd.cpu().numpy(), want[1])


def exact(x):
    """fp32 values as integers in 2^-149."""
    return [int(v) for v in np.ldexp(x.astype(np.float64), 149)]


@pytest.mark.parametrize("sharp,near", [(2.0, 0.7), (12.0, 0.7), (12.0, 0.01), (2.0, 0.001)])
def test_tokens_beside_unrounded_probabilities(pkv, sharp, near):
    """The drawn token against sums that no rounding has touched. A value is taken to a multiple of 2^-46, so off by 2^-47
    at most, a difference of two by 2^-46, a sum of V of them by V 2^-46; u times the total by as much, and by the one
    unit that its floor takes: the token's own range of the exact sums, widened by (2 V + 1) 2^-46, holds u times the
    exact total. More than a fifth of the sharp rows' values lie below 2^-47 and are taken to 0."""
    R, V = 24, 4001
    g = torch.Generator().manual_seed(int(sharp * 100 + near * 10))
    base = sharp * torch.randn(R, 2, V, generator=g)
    P = torch.softmax(base, -1)
    Q = torch.softmax(base[:, :1] + near * torch.randn(R, 1, V, generator=g), -1)
    ids = torch.randint(0, V, (R, 1), generator=g, dtype=torch.int32)
    P[: R // 2, 0, 7], ids[: R // 2, 0] = 0.0, 7  # half of the drafts go
    if sharp > 10:
        assert (P < 2.0 ** -47).float().mean() > 0.2
    us = torch.rand(R, generator=g)
    tokens, num, status = accept(pkv, P, Q, ids, torch.zeros(R, 1), us, None)
    assert status == 0
    slack = (2 * V + 1) << (149 - 46)
    for r in range(R):
        goes = r < R // 2 or P[r, 0, ids[r, 0]].item() == 0.0
        assert num[r] == (1 if goes else 2)
        p = exact(P[r, 0 if goes else 1].numpy())
        w = [max(a - b, 0) for a, b in zip(p, exact(Q[r, 0].numpy()))] if goes else p
        total, i = sum(w), int(tokens[r, num[r] - 1])
        assert total > 4 * slack
        num_u, den_u = float(us[r]).as_integer_ratio()
        before = sum(w[:i])
        assert (before - slack) * den_u <= num_u * total < (before + w[i] + slack) * den_u


# ------------------------------------------------------------------------------------------------
# attention weights
# ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("lens,split,splits", [([700, 100, 512], 256, 2), ([129, 128, 1], 128, 1), ([300, 0, 5], 100, 2)])
def test_weights_report_log_sum_exps_that_do_not_reach(pkv, fmt, lens, split, splits):
    """A request longer than the given splits reach is reported, as by the verify call that made them; the others are
    whole, and its own come from the splits that there are."""
    T, hkv, g = 2, 2, 3
    c = Cache(fmt, lens, hkv, 16, seed=2)
    q = queries(3, T, hkv * g, seed=2)
    gen = torch.Generator().manual_seed(3)
    for s, status in ((splits, pkv.PKV_ERR_DEVICE_BOUNDS), (-(-max(lens) // split), 0)):
        part = 4.0 + torch.rand(s, 3 * T, hkv * g, generator=gen)
        lse = np.stack([np.logaddexp.reduce(part.double().numpy()[:max(1, min(s, -(-lens[r] // split))), r * T + t], 0)
                        for r in range(3) for t in range(T)])
        w = torch.full((3, hkv, max(lens) + 1), -7.0, device=DEV)
        assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w, part_lse=part.to(DEV), split_tokens=split) == status
        verify_weights(w, expect(c, q, T, 1 / 16, lse=lse), lens, tail=-7.0)


# ------------------------------------------------------------------------------------------------
# the move
# ------------------------------------------------------------------------------------------------

def not_ascending(kind, budget, rng):
    """Entries for a request of 2 * budget + 40 positions."""
    j = np.arange(budget)
    if kind == "below":  # the part of the search that the entry ends is taken for one without a reader
        k = j + 34
        k[31::64] = -1
    elif kind == "high":  # the window of readers begins at the entry
        k = j + 1
        k[20::97] = budget + 20 + np.arange(len(k[20::97]))
    elif kind == "repeated":
        k = j + 40
        k[5::40] = k[4::40][:len(k[5::40])]
    elif kind == "stairs":  # ascending for a while, then again from further down, never below the row itself
        k = j + 1 + (j % 113) * (1 + j % 113 > 50) // 2
    elif kind == "late":  # one entry, in the list's last part
        k = j + 33
        k[budget - 70] = 2 * budget
    else:
        k = j + rng.integers(0, 70, budget)
    return k.astype(np.int32)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("kind", ["below", "high", "repeated", "stairs", "late", "random"])
@pytest.mark.parametrize("budget", [700, 9000])
def test_compact_in_place_with_a_list_out_of_order(pkv, fmt, kind, budget):
    """Lists that do not ascend, in place, every row's destination another row's source: an entry below its index or not above
    the one before it moves nothing, every other row arrives whole; requests in order beside it too."""
    n, hkv = 2 * budget + 40, 2
    x = Rows(fmt, [n, n, 300], hkv, 16, budget, seed=budget, dense="front")
    for h in range(hkv):
        x.keep[1, h] = not_ascending(kind, budget, np.random.default_rng(h))
    k = x.keep[1]
    bad = (k < np.arange(budget)) | np.concatenate((np.zeros((hkv, 1), bool), k[:, 1:] <= k[:, :-1]), 1)
    assert bad.any(1).all()
    assert (k[:, 1:] < k[:, :-1]).any() or kind == "repeated"
    want = x.expect(skip=lambda r, h, j: r == 1 and bad[h, j])
    assert x.run(pkv) == pkv.PKV_ERR_DEVICE_BOUNDS
    x.same(want)


def test_compact_in_place_with_a_long_list_out_of_order(pkv):
    """More parts of a list than a warp has lanes: one entry, in the last of them."""
    budget = 32 * 4096 + 9000
    x = Rows("fp4", [2 * budget + 40, 300], 1, 16, budget, seed=1, dense="front")
    x.keep[0, 0] = not_ascending("late", budget, None)
    want = x.expect(skip=lambda r, h, j: r == 0 and j == budget - 69)
    assert x.run(pkv) == pkv.PKV_ERR_DEVICE_BOUNDS
    x.same(want)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("lens,budget", [([700, 30, 650], 600), ([9000, 32, 8000], 7000)])
def test_compact_waits_that_run_out(pkv, fmt, lens, budget):
    """A bound below 20 us counts as run out at once. It is reported; chunks that wait for nothing (the first 32 rows of a
    request and KV head) are moved, the others write nothing; the next call is whole."""
    x = Rows(fmt, lens, 2, 16, budget, seed=budget, dense="front")
    x.keep[1, :, :x.new[1]] = np.arange(x.new[1])
    x.keep[1, 0, 5:x.new[1] - 1] += 1  # rows of the short request move by one
    x.new[1] -= 1
    first = [t.clone() for t in (*x.pools, *x.scales, x.weights) if t is not None]
    partly, whole = x.expect(skip=lambda r, h, j: j >= 32), x.expect()
    for limit in (1, 19999):
        pkv.lib.pkv_testing_set_wait_limit_ns(limit)
        assert x.run(pkv) == pkv.PKV_ERR_TIMEOUT
        x.same(partly)
        for t, f in zip([t for t in (*x.pools, *x.scales, x.weights) if t is not None], first):
            t.copy_(f)
    assert x.run(pkv) == 0
    x.same(whole)


# ------------------------------------------------------------------------------------------------
# offsets past 32 bits
# ------------------------------------------------------------------------------------------------

def test_accept_over_rows_past_32_bits(pkv):
    """Requests, then tokens, 2^32 elements apart."""
    V = 1021
    big = torch.empty(2 ** 32 + 3 * V, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(1)
    for R, T in ((2, 3), (1, 2)):
        P = torch.softmax(2 * torch.randn(R, T, V, generator=g), -1).to(torch.bfloat16)
        Q = torch.softmax(2 * torch.randn(R, T - 1, V, generator=g), -1).to(torch.bfloat16)
        ids = torch.randint(0, V, (R, T - 1), generator=g, dtype=torch.int32)
        ua, us = torch.zeros(R, T - 1), torch.rand(R, generator=g)  # every draft stays: the last row is read
        strides = (2 ** 32, V, 1) if R == 2 else (0, 2 ** 32, 1)
        far = big.as_strided((R, T, V), strides)
        far.copy_(P)
        want = accept(pkv, P, Q, ids, ua, us, None)
        got = accept(pkv, far, Q, ids, ua, us, None)
        assert (want[1] == T).all() and np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
        if R == 2:  # the draft's rows there, and every draft goes
            gone = P.clone()
            gone.scatter_(2, torch.nn.functional.pad(ids, (0, 1))[..., None].long(), 0.0)
            far_q = big.as_strided((R, T - 1, V), strides)
            far_q.copy_(Q)
            want, got = accept(pkv, gone, Q, ids, ua, us, None), accept(pkv, gone, far_q, ids, ua, us, None)
            assert (want[1] == 1).all() and np.array_equal(got[0], want[0])


@pytest.mark.parametrize("fmt", ["bf16", "int8", "fp8"])
def test_weights_in_a_pool_and_an_array_past_32_bits(pkv, fmt):
    """Blocks, and requests of the weights, whose element offsets pass 2^32."""
    bs, hkv, lens, T, g = 880, 4, [1700, 300], 2, 2
    nb = 2 ** 32 // (bs * hkv * 256) + 8
    c = Cache(fmt, lens, hkv, bs, seed=8, spare=0, extra_cols=0)
    q = queries(2, T, hkv * g, seed=9)
    place = torch.from_numpy(np.array([nb - 1, 5, nb - 3][:c.nb])).to(DEV)
    pool = torch.empty(nb, bs, hkv, 256, dtype=c.pool.dtype, device=DEV)
    pool[place] = c.pool
    if fmt == "int8":
        scale = torch.empty(nb, bs, hkv, device=DEV)
        scale[place] = c.scale
        c.scale = scale
    c.pool, c.table = pool, place[c.table.clamp(min=0).long()].int()
    buffer = torch.empty(2 ** 32 + hkv * 1800, device=DEV)
    w = buffer.as_strided((2, hkv, 1800), (2 ** 32, 1800, 1))
    w.fill_(-7.0)
    assert weigh(pkv, c, q.to(DEV), T, 1 / 16, w) == 0
    verify_weights(w, expect(c, q, T, 1 / 16), lens, tail=-7.0)
