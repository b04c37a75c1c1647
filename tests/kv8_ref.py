"""Plain FP64 forms of the 8-bit KV cache, of the attention over it and of the
paging calls, for the tests: numpy only, no code of the library.

BF16 arrays travel as uint16 bit patterns (see workloads.synth)."""
import numpy as np

from kv4_ref import E4M3, attend, bf16_to_f64, slots_of  # noqa: F401

MIN_EXP, MAX_EXP = -64, 63


def encode(x):
    """e4m3 codes of FP64 numbers (a NaN for what is not finite): nearest, ties
    to the even code, saturating at 448."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    i = np.clip(np.searchsorted(E4M3[:127], a), 1, 126)
    lo, hi = E4M3[i - 1], E4M3[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    c = np.where(a >= 448.0, 126, np.where(up, i, i - 1))
    c = np.where(np.isfinite(x), c, 127)
    return (c + 128 * (np.signbit(x) & np.isfinite(x))).astype(np.uint8)


def decode(c):
    return E4M3[c & 127] * np.where(c & 128, -1.0, 1.0)


def values(codes, scales, block):
    """codes [n_slots][h][d], scales [n_slots / block][h] -> FP64."""
    return decode(codes) * np.exp2(np.repeat(scales, block, 0).astype(np.float64) - 127)[..., None]


def exponent(top):
    """Smallest e in [-64, 63] with top <= 448 2^e."""
    for e in range(MIN_EXP, MAX_EXP):
        if top <= 448.0 * 2.0 ** e:
            return e
    return MAX_EXP


def append(codes, scales, bits, slots, block, first):
    """Rows `bits` [n][h][d] of one request at its slots [n] (of positions first,
    first + 1, ...; a negative slot: skipped) into one tensor's arrays, in place."""
    x = bf16_to_f64(bits)
    at = 0
    while at < len(slots):
        n = min(block - (first + at) % block, len(slots) - at)
        rows = x[at:at + n]
        s0, s = slots[at], slots[at:at + n]
        at += n
        if s0 < 0:
            continue
        b, kept = s0 // block, s0 % block
        for h in range(codes.shape[1]):
            r = rows[:, h]
            fin = np.where(np.isfinite(r), np.abs(r), 0.0)
            e = exponent(fin.max())
            if kept:
                old = int(scales[b, h]) - 127
                e = max(e, old)
                if e > old:
                    o = slice(b * block, b * block + kept)
                    codes[o, h] = encode(decode(codes[o, h]) * 2.0 ** (old - e))
            codes[s, h] = encode(r / 2.0 ** e)
            scales[b, h] = e + 127


def tolerance(d, n, ref, a, big, spread, out_eps, ev, p_top, parts):
    """Bounds of |out - ref| [h_q][d] and of |lse - ref| [h_q].

    A logit is accumulated in FP32 from exact products, 16 or more of them a
    step; each step may be off by 2^-22 of sum|q k| (an adder that truncates),
    and the factor and the subtraction of the maximum by another step each:
    (d/16 + 2) 2^-22 big.  q is held in two e4m3 numbers, the second for the
    remainder times 32, with the largest component in [2^7, 2^8): every
    component is off by half of the second's smallest step at most, 2^-10 / 32
    = 2^-15, 2^-22 of the largest: 2^-22 spread.  The exponent of a weight also
    holds that of the largest V scale (ev bounds both exponents' magnitude),
    so its subtraction is off by 2^-22 ev more.

    A weight adds exp2's 2^-22, the sums' (n/16 + 64) 2^-22, and its storage in
    e4m3 parts: each leaves at most 2^-4 of what it takes, so 2^(-4 parts) of
    the weight is left, or half of the last part's smallest step: 2^-10 /
    32^(parts - 1), where the row's largest product of weight and V scale,
    p_top [h_q], is held as 2^3 at least; so 2^-13 / 32^(parts - 1) p_top, and
    meets a code of up to 448."""
    logit = (d / 16 + 2) * 2.0 ** -22 * big + 2.0 ** -22 * spread + 2.0 ** -22 * ev
    r = logit + 2.0 ** -22 + 2.0 ** (-4 * parts) + (n / 16 + 64) * 2.0 ** -22
    floor = n * 2.0 ** -13 / 32.0 ** (parts - 1) * 448.0 * p_top[:, None]
    return 2 * r[:, None] * a + floor + out_eps * (np.abs(ref) + 2 * r[:, None] * a) + 1e-30, \
        logit + 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -22


def top_products(q, k, ev, scale, lse):
    """max_j w_j 2^ev_j per query head: k [n][h_kv][d], ev [n][h_kv]."""
    g = q.shape[0] // k.shape[1]
    out = np.zeros(q.shape[0])
    for h in range(q.shape[0]):
        if k.shape[0]:
            out[h] = (np.exp(scale * (k[:, h // g] @ q[h]) - lse[h]) * np.exp2(ev[:, h // g])).max()
    return out


def plan(ctx, new, table, page, free, n_free, n_tok):
    """plan_step on host arrays, request by request: (start, new_len, row_len,
    row_req, slots, table, n_free, fault bits)."""
    table = table.copy()
    bits = 0
    if not 0 <= n_free <= len(free):
        bits, n_free = bits | 8, 0
    grant, jobs = [], []
    need_sum = tok_sum = 0
    for c, n in zip(ctx, new):
        c, n = int(c), int(n)
        ok, pages = True, 0
        if c < 0 or n < 0:
            ok, bits = False, bits | 8
        n = max(n, 0)
        held = -(-c // page)
        if ok and n:
            end = -(-(c + n) // page)
            if end > table.shape[1] or c + n > 2 ** 31 - 1:
                ok, bits = False, bits | 1
            else:
                pages = end - held
        tok_sum += n
        need_sum += pages
        if tok_sum > n_tok or need_sum > n_free:
            bits |= 16
        ok = ok and tok_sum <= n_tok and (pages == 0 or need_sum <= n_free)
        grant.append(ok)
        jobs.append((c, n, held, pages))
    taken = sum(p for (_, _, _, p), ok in zip(jobs, grant) if ok)
    at = n_free - taken
    start = [0]
    row_len, row_req, slots = np.zeros(n_tok, np.int32), np.full(n_tok, -1, np.int32), np.full(n_tok, -1, np.int32)
    new_len = []
    for r, ((c, n, held, pages), ok) in enumerate(zip(jobs, grant)):
        if ok:
            table[r, held:held + pages] = free[at:at + pages]
            at += pages
        for i in range(n):
            t = start[-1] + i
            if t >= n_tok:
                break
            row_req[t] = r
            if ok:
                pg = int(table[r, (c + i) // page])
                if pg < 0:
                    bits |= 1
                else:
                    slots[t] = pg * page + (c + i) % page
                row_len[t] = c + i + 1
        start.append(min(start[-1] + n, n_tok))
        new_len.append(c + n if ok else c)
    return (np.array(start, np.int32), np.array(new_len, np.int32), row_len, row_req, slots, table, n_free - taken, bits)


def release(table, lo, hi, free, n_free):
    """release_pages on host arrays: (table, free, n_free, fault bits)."""
    table, free = table.copy(), free.copy()
    bits, room = 0, len(free)
    if not 0 <= n_free <= room:
        return table, free, n_free, 8 | (16 if any(table[r, a] >= 0 for r, (f, t) in enumerate(zip(lo, hi))
                                                   if 0 <= f < t <= table.shape[1] for a in range(f, t)) else 0)
    for r, (f, t) in enumerate(zip(lo, hi)):
        if f >= t:
            continue
        if f < 0 or t > table.shape[1]:
            bits |= 1
            continue
        for a in range(f, t):
            if table[r, a] < 0:
                continue
            if n_free == room:
                bits |= 16
                continue
            free[n_free] = table[r, a]
            table[r, a] = -1
            n_free += 1
    return table, free, n_free, bits
