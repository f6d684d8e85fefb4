"""Plain numpy statements of the 4-bit cache: its formats, its quantizer (fp32 steps, each rounded once)
and decode / verify attention over it in 64 bits."""
from __future__ import annotations

import numpy as np

D, G = 256, 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1_ALL = np.concatenate([E2M1, -E2M1])


def _e4m3_table():
    t = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = np.nan if (e == 15 and m == 7) else ((8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9)
        t[b] = -v if b & 128 else v
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]  # increasing finite magnitudes, codes 0..126


def _nearest_even(x, table):
    """Index of the entry of `table` (increasing, index parity = mantissa parity) nearest to x >= 0, ties
    to the even index, the last entry for larger x. Exact: midpoints of these tables fit in float64."""
    x = np.asarray(x, dtype=np.float64)
    mid = (table[:-1] + table[1:]) / 2
    i = np.searchsorted(mid, x, side="left")          # mid[i-1] < x <= mid[i]
    tie = (i < len(mid)) & (x == mid[np.minimum(i, len(mid) - 1)])
    return i + (tie & (i % 2 == 1))


def bf16_to_f32(u):
    return (np.asarray(u, dtype=np.uint16).astype(np.uint32) << 16).view(np.float32)


def f32_to_bf16(x):
    """Round to nearest even; finite values and infinities."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def quantize(x_u16, scale):
    """bf16 bits [..., 256] -> (codes uint8 [..., 128], scale bytes uint8 [..., 16])."""
    x = bf16_to_f32(x_u16).reshape(*x_u16.shape[:-1], D // G, G)
    g = np.float32(scale)
    with np.errstate(all="ignore"):
        a = np.abs(x).max(-1)
        nan = np.isnan(x).any(-1)
        r = a / np.float32(np.float32(6) * g)
        sb = np.where(np.isnan(r), 0x7F, _nearest_even(np.where(np.isnan(r), 0, r), _POS)).astype(np.uint8)
        d = (E4M3[sb].astype(np.float32) * g)[..., None]
        ok = (d >= np.float32(2.0 ** -126)) & np.isfinite(d)
        q = np.abs(np.where(ok, x / np.where(ok, d, np.float32(1)), np.float32(0)))
        code = _nearest_even(np.where(np.isnan(q), 0, q), E2M1).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 3)
    code = np.where(nan[..., None], 0, code).astype(np.uint8)
    sb = np.where(nan, 0x7F, sb).astype(np.uint8)
    code = code.reshape(*x_u16.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), sb


def values(codes, sb):
    """float64 e2m1 * e4m3 [..., 256] (without the tensor's scale)."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], D)
    v = E2M1_ALL[c].reshape(*codes.shape[:-1], D // G, G) * E4M3[sb][..., None]
    return v.reshape(*codes.shape[:-1], D)


def dequantize_bf16(codes, sb, scale):
    with np.errstate(all="ignore"):
        f = values(codes, sb).astype(np.float32) * np.float32(scale)
    nan = np.isnan(f)
    return np.where(nan, 0x7FC0, f32_to_bf16(np.where(nan, 0, f))).astype(np.uint16)


def attention(q_u16, k, v, seq_len, T, group, softmax_scale):
    """One request in float64: q bf16 bits [T][Hq][256], k / v float64 [seq_len][hkv][256]. Returns the
    output [T][Hq][256] and the error a bf16 result may have (see allowed)."""
    q = bf16_to_f32(q_u16).astype(np.float64)
    Hq = q.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(T):
        n = seq_len - T + t + 1
        if n <= 0:
            continue
        for h in range(Hq):
            kk, vv = k[:n, h // group], v[:n, h // group]
            s = softmax_scale * (kk @ q[t, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[t, h] = p @ vv
            size = softmax_scale * (np.abs(kk) @ np.abs(q[t, h])).max()
            lost = softmax_scale * (np.abs(kk) @ q_error(q[t, h])).max()
            tol[t, h] = allowed(out[t, h], p @ np.abs(vv), np.abs(vv).max(), n, size, lost)
    return out, tol


def q_error(q):
    """What the four-term form of a query row may leave of each element: 2^-11 of the largest magnitude of
    its block of 16 (the last of four base-8 digits, the first of which counts in halves of the block's
    power of two, is off by at most half a unit: 2^(E - 1 - 1 - 9) for a block in [2^E, 2^(E+1))), and no
    less than 2^-19 of the row's (a digit's scale is at least 2^-9 in a row brought to [2^8, 2^9))."""
    a = np.abs(q)
    block = np.repeat(a.reshape(D // G, G).max(-1), G)
    return np.maximum(2.0 ** -11 * block, 2.0 ** -19 * a.max())


def allowed(out, mag, vmax, n, size, lost):
    """Allowed |error| of one bf16 output row: half a step of the output (2^-8 of its value); half a step
    of the fp16 probabilities (2^-11 of each, so of mag = sum_j p_j |v_j|); for probabilities below
    fp16's normal range half a quantum, 2^-25, against a row sum of at least 2^8 (n of them, times
    the largest |v|); scores of 256 products summed in fp32 (256 * 2^-24 of size = max_j scale * sum_d
    |q_d k_jd|) from a query row that is off by at most q_error (lost = max_j scale * sum_d q_error_d
    |k_jd|), which move numerator and denominator; fp32 sums over n keys in steps of 16 (2^-23 each)."""
    return (2.0 ** -8 * np.abs(out) +
            (2.0 ** -11 + 2 * (256 * 2.0 ** -24 * size + lost) + (n / 16 + 16) * 2.0 ** -23) * mag +
            n * 2.0 ** -33 * vmax + 1e-30)
