"""Weights of the attention over the 8-bit cache where their storage, and the
distance of the scales, show: rows that share a tile against FP64, the same
bounds as for rows alone (four parts to a weight, see kv8_ref.tolerance)."""
import numpy as np
import pytest

import kv8_ref as ref
from gpu_util import bf16_dev, to_dev
from test_gpu_kv8 import BF16_HALF_STEP, bits_to_f64, host, one_row, page_table, random_cache, same
from workloads.synth import bf16_bits, normal_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import torch
    assert torch.cuda.is_available()
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.lib()
    qsa.device_status(clear=True)
    return qsa


@pytest.fixture(autouse=True)
def no_fault_left(qsa):
    yield
    assert qsa.device_status(clear=True) == 0


# (row, head) pairs to a tile: 8, 16, 32, 48
SHARED = [(1, 8), (2, 8), (4, 8), (6, 8), (3, 16)]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("rows,group", SHARED)
@pytest.mark.parametrize("at,n_req", [(0, 152), (1500, 152), (0, 1), (2999, 40)])
def test_many_small_weights_behind_a_large_one(qsa, rows, group, d, at, n_req):
    """One token holds nearly all of the weight and has V = 0, the others are
    at 2^-24 of it: the output is theirs alone.  152 requests (of the same
    pages): a CTA for each, with one reference for all of its entries.

    Every weight of theirs is held as at least 2^3 2^-24 = 2^-21 (the largest
    product of weight and V scale as 2^3 at least), and is off by half of the
    last part's smallest step, 2^-10 / 32^3 = 2^-25, or by 2^-16 of itself:
    2^-4 of itself at most.  The logits are sums of one product each, in base 2,
    times log2(e) ln(2): off by 2^-22 of 24 and the factor.  The output is
    rounded once (2^-8)."""
    n = 3000
    codes = np.zeros((n // 8 * 8 + 8, 1, d), np.uint8)
    kx = np.zeros(codes.shape)
    rng = np.random.default_rng(d + rows)
    kx[:, 0, 0] = rng.choice([-2.0, -1.0, -0.5, 0.0], codes.shape[0])
    kx[at, 0, 0] = 22.0
    vx = rng.choice([0.5, 1.0, 1.5], codes.shape)
    vx[at] = 0.0
    scales = np.full((codes.shape[0] // 8, 1), 127, np.uint8)
    cache = [ref.encode(kx), scales, ref.encode(vx), scales.copy()]
    pt = np.broadcast_to(np.arange(codes.shape[0] // 8, dtype=np.int32), (n_req, codes.shape[0] // 8)).copy()
    qf = np.zeros((n_req * rows, group, d), np.float32)
    qf[:, :, 0] = 1.0
    out, lse = qsa.window_attn_fp8(bf16_dev(bf16_bits(qf)), *map(to_dev, cache),
                                   to_dev((np.arange(n_req + 1) * rows).astype(np.int32)),
                                   to_dev(np.full(n_req * rows, n, np.int32)), to_dev(pt), 8, n, n,
                                   scale=float(np.log(2.0)), max_rows_per_req=rows)
    w = np.exp2(kx[:n, 0, 0] - 22.0)
    want = (w @ vx[:n, 0]) / w.sum()
    got = bits_to_f64(out)
    assert (np.abs(got - want) <= (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -14) * want).all(), np.abs(got / want - 1).max()
    assert np.abs(host(lse) - (22.0 * np.log(2.0) + np.log(w.sum()))).max() <= 2.0 ** -16


@pytest.mark.parametrize("h_q,h_kv,d,rows", [(16, 2, 256, 2), (16, 2, 256, 4), (16, 2, 256, 6), (16, 1, 256, 3),
                                             (16, 2, 128, 6), (8, 1, 128, 4), (7, 1, 256, 13)])
@pytest.mark.parametrize("ctx,window,n_sink", [(1500, 5000, 0), (900, 130, 5)])
def test_shared_tiles_hold_weights_as_rows_alone(qsa, h_q, h_kv, d, rows, ctx, window, n_sink):
    rng = np.random.default_rng(ctx + rows + h_q + d)
    page, block = 32, 16
    pt, n_slots = page_table(rng, [ctx], page)
    cache = [*random_cache(rng, n_slots, h_kv, d, block), *random_cache(rng, n_slots, h_kv, d, block)]
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    bits = normal_bf16(rng, (rows, h_q, d))
    out, lse = qsa.window_attn_fp8(bf16_dev(bits), *map(to_dev, cache), to_dev(np.array([0, rows], np.int32)), to_dev(lens),
                                   to_dev(pt), page, ctx, window, n_sink, max_rows_per_req=rows)
    kf, vf, ev = ref.values(*cache[:2], block), ref.values(*cache[2:], block), cache[3].astype(np.float64) - 127
    o, l, qf = bits_to_f64(out), host(lse).astype(np.float64), ref.bf16_to_f64(bits)
    for t in range(rows):
        p = np.arange(lens[t])
        s = ref.slots_of(pt[0], p[(p >= lens[t] - window) | (p < n_sink)], page)
        ro, rl, tol, tol_l = one_row(qf[t], kf[s], vf[s], ev[s // block], d ** -0.5, BF16_HALF_STEP, 4)
        same(o[t], ro, tol, t)
        same(l[t], rl, tol_l, t)


# ------------------------------------------------------------ the same bits
@pytest.mark.parametrize("n_req,rows,h_q,h_kv,d,ctx,window", [(32, 6, 16, 2, 256, 3000, 1024), (8, 2, 16, 4, 128, 9000, 9000),
                                                              (1, 6, 16, 2, 256, 20011, 20011), (5, 4, 8, 1, 128, 700, 90),
                                                              (32, 1, 16, 2, 256, 5000, 4096)])
def test_same_window_call_gives_the_same_bits(qsa, n_req, rows, h_q, h_kv, d, ctx, window):
    """Alone, one after the other and behind other work: how the CTAs run
    beside each other changes nothing."""
    import torch
    rng = np.random.default_rng(n_req + rows)
    page = 16
    ctxs = rng.integers(ctx // 2, ctx + 1, n_req)
    pt, n_slots = page_table(rng, ctxs, page)
    base = [*random_cache(rng, 4096, h_kv, d, page), *random_cache(rng, 4096, h_kv, d, page)]
    pick = rng.integers(0, 4096 // page, n_slots // page)
    cache = [to_dev(a.reshape(256, -1, *a.shape[1:])[pick].reshape(-1, *a.shape[1:])) for a in base]
    lens = np.concatenate([np.arange(c - rows + 1, c + 1) for c in ctxs]).astype(np.int32)
    start = to_dev((np.arange(n_req + 1) * rows).astype(np.int32))
    q, lens, pt = bf16_dev(normal_bf16(rng, (n_req * rows, h_q, d))), to_dev(lens), to_dev(pt)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def call():
        return qsa.window_attn_fp8(q, *cache, start, lens, pt, page, int(ctxs.max()), window, 4, max_rows_per_req=rows)

    want = call()
    torch.cuda.synchronize()
    for i in range(40):
        if i % 4 == 0:
            flush.fill_(i)
        got = [call() for _ in range(i % 3 + 1)]
        if i % 2:
            torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want)), i


# -------------------------------------------------------- scales far apart
def far_apart(n, h_kv, d, block, first, lo, hi):
    """Codes 1 in K and V, V scales 2^lo in the first entries and 2^hi behind them."""
    codes = np.full((n, h_kv, d), ref.encode(np.array([1.0]))[0], np.uint8)
    ks = np.full((n // block, h_kv), 127, np.uint8)
    vs = np.full((n // block, h_kv), 127 + hi, np.uint8)
    vs[:first // block] = 127 + lo
    return [codes, ks, codes.copy(), vs]


@pytest.mark.parametrize("lo,hi", [(-64, 63), (63, -64), (-63, 63), (-40, 60)])
@pytest.mark.parametrize("d,h_q", [(256, 8), (128, 8), (128, 16)])
@pytest.mark.parametrize("n,first,rows", [(1024, 512, 300), (1024, 512, 2), (20480, 10240, 1), (512, 256, 400)])
def test_sparse_attn_fp8_normaliser_with_v_scales_far_apart(qsa, lo, hi, d, h_q, n, first, rows):
    """All logits 0: the log-sum-exp is log n, whatever the V scales are, in a
    CTA alone, in a cluster and in shares; the output the mean of the values."""
    cache = far_apart(n, 1, d, 64, first, lo, hi)
    q = np.zeros((rows, h_q, d), np.uint16)
    slots = np.broadcast_to(np.arange(n, dtype=np.int32), (rows, n)).copy()
    out, lse = qsa.sparse_attn_fp8(bf16_dev(q), *map(to_dev, cache), to_dev(slots))
    assert np.abs(host(lse) - np.log(n)).max() <= 2.0 ** -20 + (n / 16 + 64) * 2.0 ** -22 + 2.0 ** -20 * 2
    want = (first * 2.0 ** lo + (n - first) * 2.0 ** hi) / n
    assert np.abs(host(out) / want - 1).max() <= 2.0 ** -15 + (n / 16 + 64) * 2.0 ** -21


@pytest.mark.parametrize("lo,hi", [(-64, 63), (63, -64), (-63, 62)])
@pytest.mark.parametrize("d,rows", [(256, 1), (256, 6), (128, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("n_req,n", [(1, 1024), (150, 1024), (1, 20480)])
def test_window_attn_fp8_normaliser_with_v_scales_far_apart(qsa, lo, hi, d, rows, n_req, n):
    cache = far_apart(n, 1, d, 64, n // 2, lo, hi)
    q = np.zeros((n_req * rows, 8, d), np.uint16)
    pt = np.broadcast_to(np.arange(n // 64, dtype=np.int32), (n_req, n // 64)).copy()
    lens = np.full(n_req * rows, n, np.int32)
    out, lse = qsa.window_attn_fp8(bf16_dev(q), *map(to_dev, cache), to_dev((np.arange(n_req + 1) * rows).astype(np.int32)),
                                   to_dev(lens), to_dev(pt), 64, n, n, max_rows_per_req=rows)
    assert np.abs(host(lse) - np.log(n)).max() <= 2.0 ** -20 * 3 + (n / 16 + 64) * 2.0 ** -22
    want = (2.0 ** lo + 2.0 ** hi) / 2
    assert np.abs(bits_to_f64(out) / want - 1).max() <= 2.0 ** -8 + 2.0 ** -14 + (n / 16 + 64) * 2.0 ** -21
