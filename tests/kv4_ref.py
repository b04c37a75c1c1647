"""Plain FP64 forms of the 4-bit KV cache and of the attention over it, for
the tests: numpy only, no code of the library.

BF16 arrays travel as uint16 bit patterns (see workloads.synth)."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_to_f64(bits):
    with np.errstate(invalid="ignore"):  # signalling NaN
        return (np.ascontiguousarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _e4m3_table():
    t = np.empty(128)
    for c in range(128):
        e, m = c >> 3, c & 7
        t[c] = (m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
    t[127] = np.nan
    return t


E4M3 = _e4m3_table()  # codes of non-negative scales


def _nearest(x, values):
    """Index of the nearest entry of an ascending table, ties to the even
    index, saturating (x >= 0, finite)."""
    i = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo, hi = values[i - 1], values[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return np.where(x >= values[-1], len(values) - 1, np.where(up, i, i - 1))


def quantise(bits, g):
    """[..., d] BF16 bits -> (codes [..., d/2], scales [..., d/16]) uint8.
    Every step is exact but the two roundings: the values have 8 significant
    bits, so FP64 holds all quotients next to a rounding border apart."""
    x = bf16_to_f64(bits)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16) / g
    broken = ~np.isfinite(b).all(-1)
    b = np.where(broken[..., None], 0.0, b)
    scale = _nearest(np.abs(b).max(-1) / 6.0, E4M3[:127]).astype(np.uint8)
    s = E4M3[scale][..., None]
    code = _nearest(np.divide(np.abs(b), s, out=np.zeros_like(b), where=s > 0), E2M1).astype(np.uint8)
    neg = np.signbit(x.reshape(b.shape)) & (s > 0) & ~broken[..., None]
    code = (code + 8 * neg).astype(np.uint8)
    scale[broken] = 0x7F
    code = code.reshape(x.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), scale


def values(codes, scales, g):
    """The values codes and scales stand for, FP64."""
    n = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    return v * np.repeat(E4M3[scales], 16, -1) * g


def attend(q, k, v, scale):
    """One row: q [h_q][d], k and v [n][h_kv][d], FP64.  Returns out, lse, and
    for the tolerances a = sum_j w_j |v_j| [h_q][d], the largest
    scale * sum_d |q_d k_jd| and scale * max|q| * sum_d |k_jd| per head."""
    h_q, d = q.shape
    g = h_q // k.shape[1]
    out, a = np.zeros((h_q, d)), np.zeros((h_q, d))
    lse, big, spread = np.full(h_q, -np.inf), np.zeros(h_q), np.zeros(h_q)
    if k.shape[0] == 0:
        return out, lse, a, big, spread
    for h in range(h_q):
        kk, vv = k[:, h // g], v[:, h // g]
        x = scale * (kk @ q[h])
        m = x.max()
        w = np.exp(x - m)
        lse[h] = m + math.log(w.sum())
        w = w / w.sum()
        out[h], a[h] = w @ vv, w @ np.abs(vv)
        big[h] = abs(scale) * (np.abs(kk) @ np.abs(q[h])).max()
        spread[h] = abs(scale) * np.abs(q[h]).max() * np.abs(kk).sum(-1).max()
    return out, lse, a, big, spread


def tolerance(d, n, ref, a, big, spread, weight_eps, out_eps, q16, vmax):
    """Bounds of |out - ref| [h_q][d] and of |lse - ref| [h_q].

    A logit is accumulated in FP32 from exact products, 16 of them a step;
    each step may be off by 2^-22 of sum|q k| (an adder that truncates), and
    the factor and the subtraction of the maximum by another step each:
    (d/16 + 2) 2^-22 big.  With q held in FP16 (q16) each component is off by
    at most 2^-25 of the head's largest: 2^-25 spread.  A weight adds the
    error of exp2 (2^-22) and of its own storage (weight_eps relative; held in
    FP16 as 2^10 w with the largest w = 1, it is a multiple of the smallest
    subnormal 2^-24, so off by up to 2^-25 / 2^10 = 2^-35 as well, which
    counts where a tiny weight meets the only non-zero value of a column:
    n 2^-35 max|v|, taken as n 2^-35 vmax); sums over n
    entries of 16 a step, and the merges of up to 64 partial sums, add
    (n/16 + 64) 2^-22.  The relative error r of a weight enters the weighted
    sum as r a and the normaliser as r |out| <= r a.  The output is rounded
    once (out_eps relative)."""
    logit = (d / 16 + 2) * 2.0 ** -22 * big + (2.0 ** -25 * spread if q16 else 0.0)
    r = logit + 2.0 ** -22 + weight_eps + (n / 16 + 64) * 2.0 ** -22
    floor = n * 2.0 ** -35 * vmax if q16 else 0.0
    return 2 * r[:, None] * a + floor + out_eps * (np.abs(ref) + 2 * r[:, None] * a) + 1e-30, \
        logit + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -22


def window_positions(length, window, n_sink):
    """Positions that a row seeing `length` tokens attends to."""
    p = np.arange(length)
    return p[(p >= length - window) | (p < n_sink)]


def slots_of(pt_row, pos, page_size):
    return pt_row[pos // page_size].astype(np.int64) * page_size + pos % page_size
