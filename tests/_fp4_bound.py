"""A sharp bound on the error of attention over the 4-bit cache: what its own roundings can do to each
output, key by key, where `_fp4.allowed` takes the worst key for all of them.

With p the probabilities, an output element is o = sum_j p_j v_j, and what moves it is
  - each weight's rounding to fp16, at most 2^-11 of it (the sum takes the fp32 weights): p_j v_j 2^-11, or half a
    quantum, 2^-25 against a row sum of at least 2^8, below fp16's normal range;
  - an error ds_j of a score, which moves numerator and denominator: p_j ds_j (v_j - o);
  - fp32 accumulation of O: a step takes 8 keys and may lose 2^-22 of the partial sum;
  - the row sum: each thread adds n / 128 weights, then a tree; and the output's rounding to bf16, 2^-8 of it or half a step
    of its subnormal numbers, 2^-134.
The first two are sums over the keys of terms whose signs are independent (a rounding's sign; the sign of v_j -
o for rows of random values, whatever made ds_j), so by Hoeffding's inequality seven times the root of the sum of
their squares is passed with probability 2 exp(-49 / 2) = 5e-11 an element, where the worst case would
grow with the number of keys and hide a lost tile.
"""
from __future__ import annotations

import numpy as np

import _fp4 as F

TERMS = 6  # of a query row


def _power(x):
    """The power of two of x > 0 (2^E <= x < 2^(E+1)); 0 for 0."""
    return np.where(x > 0, 2.0 ** np.floor(np.log2(np.where(x > 0, x, 1.0))), 0.0)


def q_unit(q):
    """The step in which a query row's elements are kept: those that are multiples of it exactly, the others
    within half of it. The first of six base-8 digits counts in halves of the power of two of the
    block of 16's largest magnitude, the last in 2^-16 of it; a digit's scale is at least 2^-9 in a row brought to
    [2^8, 2^9), where a step is 2^-18 of the row's power of two (2^-136 in rows that cannot be brought there).
    (_fp4.q_error allows more: what four digits would leave.)"""
    a = np.abs(q)
    block = np.repeat(a.reshape(*a.shape[:-1], F.D // F.G, F.G).max(-1), F.G, axis=-1)
    return np.maximum(2.0 ** -16 * _power(block), np.maximum(2.0 ** -18 * _power(a.max(-1, keepdims=True)), 2.0 ** -136))


def q_lost(q):
    u = q_unit(q)
    with np.errstate(over="ignore"):
        return np.where(np.mod(np.abs(q), u) == 0, 0.0, u / 2)


def q_terms(q, terms=TERMS):
    """A query row as the kernel holds it: the sum of its first `terms` digits."""
    a = np.abs(q)
    row = np.maximum(_power(a.max(-1, keepdims=True)), 2.0 ** -118)
    up = 256.0 / row
    x = (q * up).reshape(*q.shape[:-1], F.D // F.G, F.G)
    e = np.maximum(_power(np.abs(x).max(-1, keepdims=True)), 2.0 ** -9)
    acc, y = np.zeros_like(x), x / e
    for _ in range(terms):
        digit = np.round(2 * y) / 2  # half to even, as e2m1 rounds up to 2
        acc += digit * e
        down = np.minimum(8.0, e * 512)
        y = (y - digit) * down
        e = e / down
    return acc.reshape(q.shape) / up


def attention(q_u16, k, v, seq_len, T, group, softmax_scale):
    """One request, as _fp4.attention: the output in 64 bits and the bound."""
    q = F.bf16_to_f32(q_u16).astype(np.float64)
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(T):
        n = seq_len - T + t + 1
        if n <= 0:
            continue
        for h in range(k.shape[1]):
            rows = slice(h * group, (h + 1) * group)
            out[t, rows], tol[t, rows] = _rows(q[t, rows], k[:n, h], v[:n, h], softmax_scale)
    return out, tol


def probabilities(q, k, scale):
    s = scale * (q @ k.T)
    p = np.exp(s - s.max(-1, keepdims=True))
    return s, p / p.sum(-1, keepdims=True)


def _rows(q, k, v, scale):
    n = len(k)
    s, p = probabilities(q, k, scale)
    o = p @ v
    ak, v2 = np.abs(k), v * v
    # 8 accumulating products and the additions of their columns, 2^-23 of the sum of magnitudes each; the exponent's
    # rounding (of s and the maximum, in bits) and the exponential's own error
    ds = scale * (q_lost(q) @ ak.T) + 11 * 2.0 ** -23 * scale * (np.abs(q) @ ak.T) + \
        2.0 ** -22 * (2 + np.abs(s) + np.abs(s).max(-1, keepdims=True))
    w = (p * ds) ** 2
    var = (2.0 ** -11 * p) ** 2 @ v2 + np.maximum(w @ v2 - 2 * o * (w @ v) + o * o * w.sum(-1, keepdims=True), 0.0) + \
        n * (2.0 ** -33 * np.abs(v).max()) ** 2
    tiles = np.arange(0, n, 128)
    partial = np.cumsum(np.stack([p[:, a:a + 128] @ v[a:a + 128] for a in tiles]), 0)
    acc = 16 * 2.0 ** -22 * (2 * np.abs(partial).sum(0) + p @ np.abs(v)) + 10 * 2.0 ** -22 * np.abs(partial).max(0)
    return o, (2.0 ** -8 + (n / 128 + 40) * 2.0 ** -24) * np.abs(o) + 7 * np.sqrt(var) + acc + 2.0 ** -134
