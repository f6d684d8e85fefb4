"""Plain forms of what follows the verify attention, for the tests: numpy, in exact integers (accept, select, the
move) or 64 bits (attention weights, with a bound on a kernel's error)."""
from __future__ import annotations

from fractions import Fraction

import numpy as np


def accept(P, Q, ids, u_accept, u_sample, num_drafts):
    """P [R][T][V] and Q [R][T-1][V] or None: the values as fp32. -> tokens [R][T], num_out [R]."""
    R, T, V = P.shape
    tokens, count = np.full((R, T), -1, dtype=np.int32), np.zeros(R, dtype=np.int32)
    def fixed(x):  # the nearest multiple of 2^-46, of x taken to [0, 1]
        return np.rint(np.clip(np.nan_to_num(x.astype(np.float64), nan=0.0), 0.0, 1.0) * 2.0 ** 46).astype(np.uint64)

    for r in range(R):
        nd = int(np.clip(num_drafts[r], 0, T - 1))
        t = 0
        while t < nd:
            x = ids[r, t]
            if not 0 <= x < V:
                break
            q = 1.0 if Q is None else float(Q[r, t, x])
            if not float(u_accept[r, t]) * q < float(P[r, t, x]):
                break
            tokens[r, t] = x
            t += 1
        p = w = fixed(P[r, t])
        if t < nd:
            if Q is not None:
                q = fixed(Q[r, t])
                w = np.where(p > q, p - np.minimum(p, q), np.uint64(0))
            elif 0 <= ids[r, t] < V:
                w = p.copy()
                w[ids[r, t]] = 0
            if not w.any():
                w = p
        cdf = np.cumsum(w, dtype=np.uint64)
        u = float(u_sample[r])
        u = 0.0 if not u > 0.0 else min(u, 1.0 - 2.0 ** -24)
        target = int(Fraction(u) * int(cdf[-1]))
        tokens[r, t] = int(np.searchsorted(cdf, np.uint64(target), side="right")) if cdf[-1] else 0
        count[r] = t + 1
    return tokens, count


def select(scores, n, sinks, recent, budget):
    """scores fp32 [max_ctx] of one (request, head) of n positions -> the kept positions."""
    if n <= budget:
        return np.arange(n, dtype=np.int32)
    x = scores[:n].astype(np.float64)
    nan = np.isnan(x)
    first = np.arange(sinks, n - recent)
    order = first[np.lexsort((first, -np.where(nan, 0.0, x)[first], nan[first]))]
    kept = np.concatenate((np.arange(sinks), order[:budget - sinks - recent], np.arange(n - recent, n)))
    return np.sort(kept).astype(np.int32)


def weights(q, k, n, T, scale, valid, lse=None, rounded=False):
    """One request: q [T][Hq][256], k [n][Hkv][256] in 64 bits, n keys; lse [T][Hq] or None.
    -> w [Hkv][n] and a bound on the error of an fp32 kernel of it (u = 2^-24 the rounding of one operation).

    A score sums 256 exact products: a matrix instruction adds 16 at a time, so a product passes at most 16 running
    sums and 16 places of its own step, each within 2u (truncation) of the sum of magnitudes m = scale sum |q k|:
    64 u m. Scale, log2(e) and the subtraction: 4 u (|s| + |lse|). exp2 in hardware: 2^-22 = 4 u relative. Where the
    kernel computes lse itself, it has the largest of the scores' errors, a sum of n positive terms kept in at
    most n + 128 additions (their running sums never pass the total): (n + 128) u, and a logarithm, 4 u |lse|. Adding up
    the columns: one rounding each of the running sum. rounded: the queries are taken to 2^-39 of the largest of the
    request's and KV head's."""
    u = 2.0 ** -24
    hq, hkv = q.shape[1], k.shape[1]
    g = hq // hkv
    w, bound = np.zeros((hkv, n)), np.zeros((hkv, n))
    q_max = np.abs(q).reshape(q.shape[0], hkv, -1).max((0, 2))
    for t in range(min(T, valid)):
        m = n - T + t + 1
        if m <= 0:
            continue
        for h in range(hq):
            key = k[:m, h // g]
            s = scale * (key @ q[t, h])
            mag = scale * (np.abs(key) @ np.abs(q[t, h]))
            off = scale * 2.0 ** -39 * q_max[h // g] * np.abs(key).sum(1) if rounded else np.zeros(m)
            L = lse[t, h] if lse is not None else s.max() + np.log(np.exp(s - s.max()).sum())
            if L == -np.inf:
                continue
            p = np.exp(s - L)
            rel = off + 64 * u * mag + 4 * u * (np.abs(s) + abs(L)) + 4 * u
            if lse is None:
                rel = rel + off.max() + 64 * u * mag.max() + 4 * u * (np.abs(s).max() + abs(L)) + (m + 128) * u + 4 * u
            else:
                rel = rel + 16 * u * (1.0 + abs(L))  # the splits' log-sum-exps put together
            w[h // g, :m] += p
            bound[h // g, :m] += p * rel * (1.0 + rel)
    bound += (T * g + 1) * u * w
    return w, bound
