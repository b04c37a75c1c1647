"""The 4-bit KV cache and the window attention on the GPU, against plain FP64
forms (kv4_ref) at the sizes, masks, strides and layouts where they can go
wrong.  The cache's codes, scales and values are compared to the bit; the
attention within the bounds of kv4_ref.tolerance."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import bf16_dev, to_dev
from workloads import decode_workload
from workloads.synth import normal_bf16

pytestmark = pytest.mark.gpu

# How the weights are held where the softmax meets V: FP16 high part and
# remainder (11 + 11 bits, clear of the subnormals by the 2^10 offset), BF16
# high part and remainder (8 + 8 bits), or one BF16.
W_F16X2, W_BF16X2, W_BF16 = 2.0 ** -22, 2.0 ** -16, 2.0 ** -8
BF16_HALF_STEP = 2.0 ** -8


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


def host(t):
    import torch
    t = t.detach().contiguous()
    return t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy()


def bits_to_f64(t):
    return ref.bf16_to_f64(host(t))


def page_table(rng, ctx, page, spare=2):
    """Page table of requests with ctx tokens: a random permutation of the
    pool; entries past a request's pages are -1."""
    n = [-(-int(c) // page) for c in ctx]
    perm = rng.permutation(sum(n) + spare).astype(np.int32)
    pt = np.full((len(n), max(1, max(n))), -1, np.int32)
    off = 0
    for r, m in enumerate(n):
        pt[r, :m] = perm[off:off + m]
        off += m
    return pt, (sum(n) + spare) * page


def random_cache4(rng, n_slots, h_kv, d, g=1.0, gain=1.0):
    """Codes and scales of quantised normal rows, host arrays."""
    bits = normal_bf16(rng, (n_slots, h_kv, d))
    if gain != 1.0:
        import torch
        x = torch.from_numpy(ref.bf16_to_f64(bits) * gain).to(torch.bfloat16)
        bits = x.view(torch.int16).numpy().view(np.uint16)
    return ref.quantise(bits, g)


# ------------------------------------------------------------------- writing
@pytest.mark.parametrize("h_kv,d,page,fused", [(2, 256, 64, True), (1, 128, 4, False), (3, 128, 12, True),
                                               (8, 128, 16, False), (1, 256, 20, True)])
def test_append_matches_the_format_to_the_bit(qsa, h_kv, d, page, fused):
    """Ragged requests (one empty, one of a single token), rows behind the
    last request, K and V as columns of one projection; other slots keep
    their bytes."""
    import torch
    rng = np.random.default_rng(d + h_kv)
    n = np.array([5, 0, 1, 70, 33])
    first = np.array([3, 9, 0, 61, 1000])
    behind = 7
    pt, n_slots = page_table(rng, first + n, page)
    total = int(n.sum()) + behind
    if fused:  # [q | k | v] columns, a token's row wider than what is read
        qkv = bf16_dev(normal_bf16(rng, (total, 4 + 2 * h_kv, d)))
        k_new, v_new = qkv[:, 4:4 + h_kv], qkv[:, 4 + h_kv:]
    else:
        k_new, v_new = bf16_dev(normal_bf16(rng, (total, h_kv, d))), bf16_dev(normal_bf16(rng, (total, h_kv, d)))
    gk, gv = 2.0 ** -4, 4.0
    cache = [to_dev(rng.integers(0, 256, (n_slots, h_kv, w)).astype(np.uint8)) for w in (d // 2, d // 16) * 2]
    want = [host(c).copy() for c in cache]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    got = qsa.append_kv_fp4(k_new, v_new, to_dev(start), to_dev(first.astype(np.int32)), *cache, to_dev(pt), page, gk, gv)
    for r in range(len(n)):
        at = ref.slots_of(pt[r], first[r] + np.arange(n[r]), page)
        rows = slice(start[r], start[r + 1])
        want[0][at], want[1][at] = ref.quantise(host(k_new)[rows], gk)
        want[2][at], want[3][at] = ref.quantise(host(v_new)[rows], gv)
    for g, w, name in zip(got, want, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert np.array_equal(host(g), w), name
    assert all(a is b for a, b in zip(got, cache))
    torch.cuda.synchronize()


def test_append_block_edges(qsa):
    """Zeros, scales that round to zero or saturate, ties in code and scale,
    signed zeros, infinities and NaN, each in its own block."""
    d = 128
    x = np.zeros((12, d), np.float32)
    x[0, 3] = 1e-5
    x[1, :3] = [3e38, -3e38, 1.0]
    x[2, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x[2, 8:16] = -x[2, :8]
    x[3, 0] = 6 * 1.0625                      # scale half way between 1 and 1.125
    x[4, 0] = 6 * 1.1875                      # and between 1.125 and 1.25
    x[5, 16] = np.inf
    x[6, 33] = -np.inf
    x[8, :16] = -0.0
    x[9, :16] = np.linspace(-6 * 448, 6 * 448, 16)
    x[10, 0] = 6 * 2.0 ** -10                 # half the smallest scale: to zero
    x[11, 0] = 6 * 1.5 * 2.0 ** -9            # between one and two smallest: to two
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    bits[7, 127] = 0x7FC1                     # NaN
    bits[7, 0] = 0xFF81
    rows = bits[:, None, :]
    n_slots = 16
    pt = np.array([[3, 1, 0, 2]], np.int32)
    import torch
    cache = [torch.zeros((n_slots, 1, w), dtype=torch.uint8, device="cuda") for w in (64, 8) * 2]
    for g in (1.0, 2.0 ** -20, 2.0 ** 30):
        qsa.append_kv_fp4(bf16_dev(rows), bf16_dev(rows[::-1].copy()), to_dev(np.array([0, 12], np.int32)),
                          to_dev(np.array([2], np.int32)), *cache, to_dev(pt), 4, g, g)
        at = ref.slots_of(pt[0], 2 + np.arange(12), 4)
        for got, want in zip(cache, (*ref.quantise(rows, g), *ref.quantise(rows[::-1], g))):
            assert np.array_equal(host(got)[at], want), g


def test_append_out_of_range_is_skipped_and_flagged(qsa):
    import torch
    rng = np.random.default_rng(3)
    cache = [torch.full((64, 2, w), 9, dtype=torch.uint8, device="cuda") for w in (64, 8) * 2]
    k = bf16_dev(normal_bf16(rng, (6, 2, 128)))
    pt = np.array([[1, 4], [-1, 2], [0, 3]], np.int32)  # 16-token pages, 4 in the cache: page 4 and -1 are bad
    start = np.array([0, 2, 4, 6], np.int32)
    first = np.array([15, 14, 31], np.int32)            # 15, 16 (page 4); 14, 15 (page -1); 31, 32 (no entry)
    qsa.append_kv_fp4(k, k, to_dev(start), to_dev(first), *cache, to_dev(pt), 16)
    assert qsa.device_status(clear=True) == 1
    want = ref.quantise(host(k), 1.0)
    for got, w in zip(cache, (*want, *want)):
        got = host(got)
        assert np.array_equal(got[31], w[0]) and np.array_equal(got[63], w[4])
        keep = np.ones(64, bool)
        keep[[31, 63]] = False
        assert (got[keep] == 9).all()
    # a negative first position
    qsa.append_kv_fp4(k[:1], k[:1], to_dev(np.array([0, 1, 1, 1], np.int32)), to_dev(np.array([-1, 0, 0], np.int32)),
                      *cache, to_dev(pt), 16)
    assert qsa.device_status(clear=True) == 1 and (host(cache[0])[0] == 9).all()


def test_append_many_requests(qsa):
    """More requests than one round of the request search, most empty."""
    import torch
    rng = np.random.default_rng(4)
    n = (rng.random(1500) < 0.1) * rng.integers(1, 4, 1500)
    first = rng.integers(0, 9, 1500)
    pt, n_slots = page_table(rng, np.maximum(first + n, 1), 4)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    k = bf16_dev(normal_bf16(rng, (int(start[-1]), 1, 128)))
    cache = [torch.zeros((n_slots, 1, w), dtype=torch.uint8, device="cuda") for w in (64, 8) * 2]
    qsa.append_kv_fp4(k, k, to_dev(start), to_dev(first.astype(np.int32)), *cache, to_dev(pt), 4)
    want = [np.zeros((n_slots, 1, w), np.uint8) for w in (64, 8)]
    codes, scales = ref.quantise(host(k), 1.0)
    for r in np.flatnonzero(n):
        at = ref.slots_of(pt[r], first[r] + np.arange(n[r]), 4)
        want[0][at], want[1][at] = codes[start[r]:start[r + 1]], scales[start[r]:start[r + 1]]
    assert np.array_equal(host(cache[0]), want[0]) and np.array_equal(host(cache[3]), want[1])


# ------------------------------------------------------------------- reading
@pytest.mark.parametrize("h_kv,d", [(2, 256), (1, 128), (5, 128)])
def test_gather_matches_the_format_to_the_bit(qsa, h_kv, d):
    """Every code and scale byte, slots in any order, twice and negative."""
    rng = np.random.default_rng(h_kv)
    n_slots = 700
    arrays = [rng.integers(0, 256, (n_slots, h_kv, w)).astype(np.uint8) for w in (d // 2, d // 16) * 2]
    for s in arrays[1::2]:
        s &= 0x7F  # scales are never negative
    slots = rng.integers(-1, n_slots, (3, 211)).astype(np.int32)
    slots[1, 5] = slots[1, 6] = -2**31
    slots[2, :2] = [0, n_slots - 1]
    gk, gv = 2.0 ** -7, 2.0 ** 9
    k, v = qsa.gather_kv_fp4(*map(to_dev, arrays), to_dev(slots), gk, gv)
    assert tuple(k.shape) == (3, 211, h_kv, d)
    for got, (c, s), g in ((k, arrays[:2], gk), (v, arrays[2:], gv)):
        want = ref.values(c[np.maximum(slots, 0)], s[np.maximum(slots, 0)], g)
        want[slots < 0] = 0.0
        got = bits_to_f64(got)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.nan_to_num(got), np.nan_to_num(want))


def test_gather_past_the_cache_is_flagged(qsa):
    rng = np.random.default_rng(8)
    c, s = random_cache4(rng, 10, 1, 128)
    k, v = qsa.gather_kv_fp4(*map(to_dev, (c, s, c, s)), to_dev(np.array([9, 10, 2**31 - 1], np.int32)))
    assert qsa.device_status(clear=True) == 1
    assert np.array_equal(bits_to_f64(k)[0], ref.values(c, s, 1.0)[9]) and (bits_to_f64(v)[1:] == 0).all()


# --------------------------------------------------- attention over a selection
def sparse_check(qsa, q, arrays, slots, scale, gk, gv, faults=0, **kw):
    q_bits = host(q)
    out, lse = qsa.sparse_attn_fp4(q, *map(to_dev, arrays), to_dev(slots), scale, gk, gv, **kw)
    assert qsa.device_status(clear=True) == faults
    k, v = ref.values(*arrays[:2], gk), ref.values(*arrays[2:], gv)
    o, l = host(out).astype(np.float64), host(lse).astype(np.float64)
    n_idx = kw.get("n_idx") or slots.shape[1]
    for t in range(q_bits.shape[0]):
        sl = slots[t, :n_idx]
        sl = sl[(sl >= 0) & (sl < k.shape[0])]
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q_bits[t]), k[sl], v[sl], scale)
        tol, tol_l = ref.tolerance(q.shape[2], sl.size, ro, a, big, spread, W_F16X2, 2.0 ** -24, True,
                                   np.abs(v[sl]).max(initial=0.0))
        assert (np.abs(o[t] - ro) <= tol).all(), (t, float((np.abs(o[t] - ro) / tol).max()))
        if sl.size == 0:
            assert (o[t] == 0).all() and np.isneginf(l[t]).all()
        else:
            assert (np.abs(l[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all(), t
    return out, lse


@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (5, 1, 256), (1, 1, 256), (8, 8, 128), (12, 1, 128), (16, 1, 128),
                                        (6, 2, 128), (9, 1, 128)])
def test_sparse_attn_fp4_shapes(qsa, h_q, h_kv, d):
    """Any group size; masked entries anywhere, a masked row, a row with one
    entry, duplicates; q with a row pitch."""
    rng = np.random.default_rng(h_q * 100 + h_kv * 10 + d)
    n_slots, w = 3000, 2051
    gk, gv = 2.0 ** -3, 2.0 ** -9
    arrays = (*random_cache4(rng, n_slots, h_kv, d, gk), *random_cache4(rng, n_slots, h_kv, d, gv, 0.05))
    q = bf16_dev(normal_bf16(rng, (5, h_q + 2, d)))[:, :h_q]
    slots = rng.integers(0, n_slots, (5, w)).astype(np.int32)
    slots[0, rng.random(w) < 0.3] = -1
    slots[1, -300:] = -1
    slots[2] = -1
    slots[3] = -1
    slots[3, 1234] = 77
    slots[4, 100:200] = slots[4, 0]
    sparse_check(qsa, q, arrays, slots, d ** -0.5, gk, gv)


@pytest.mark.parametrize("w", [0, 1, 15, 16, 17, 63, 65, 257, 700])
@pytest.mark.parametrize("h_kv,d", [(2, 256), (1, 128)])
def test_sparse_attn_fp4_widths(qsa, w, h_kv, d):
    rng = np.random.default_rng(w)
    arrays = (*random_cache4(rng, 900, h_kv, d), *random_cache4(rng, 900, h_kv, d))
    q = bf16_dev(normal_bf16(rng, (3, 8, d)))
    slots = rng.integers(-1, 900, (3, w)).astype(np.int32)
    sparse_check(qsa, q, arrays, slots, 0.1, 1.0, 1.0)


def test_sparse_attn_fp4_first_entries_of_wider_rows(qsa):
    rng = np.random.default_rng(2)
    arrays = (*random_cache4(rng, 500, 1, 128), *random_cache4(rng, 500, 1, 128))
    slots = rng.integers(0, 500, (2, 400)).astype(np.int32)
    slots[:, 333:] = 10 ** 6  # never looked at
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, 4, 128))), arrays, slots, 0.1, 1.0, 1.0, n_idx=333)


def test_sparse_attn_fp4_slot_past_the_cache_is_flagged(qsa):
    rng = np.random.default_rng(5)
    arrays = (*random_cache4(rng, 100, 1, 256), *random_cache4(rng, 100, 1, 256))
    slots = rng.integers(0, 100, (2, 300)).astype(np.int32)
    slots[1, 7] = 100
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, 8, 256))), arrays, slots, 0.0625, 1.0, 1.0, faults=1)


@pytest.mark.parametrize("w,h_kv,d", [(8192, 1, 128), (20000, 2, 256), (70001, 1, 256)])
def test_sparse_attn_fp4_long_rows_join_several_clusters(qsa, w, h_kv, d):
    rng = np.random.default_rng(w)
    arrays = (*random_cache4(rng, 4000, h_kv, d), *random_cache4(rng, 4000, h_kv, d))
    assert qsa.lib().qsa_sparse_attn_fp4_workspace_size(2, 4 * h_kv, h_kv, d, w) > 0
    slots = rng.integers(0, 4000, (2, w)).astype(np.int32)
    slots[1, 100:] = -1  # whole clusters without an entry
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, 4 * h_kv, d))), arrays, slots, 0.05, 1.0, 1.0)


@pytest.mark.parametrize("mag", [1e-30, 1e-4, 300.0, 1e30])
def test_sparse_attn_fp4_query_magnitudes(qsa, mag):
    """Queries far outside FP16's range, with a softmax scale that takes the
    magnitude back; a zero head; components far below the largest."""
    import torch
    rng = np.random.default_rng(6)
    arrays = (*random_cache4(rng, 300, 1, 128), *random_cache4(rng, 300, 1, 128))
    x = rng.standard_normal((2, 4, 128)) * mag
    x[0, 1] = 0
    x[1, 2, 1:] *= 2.0 ** -13
    q = torch.from_numpy(x).to(torch.bfloat16).cuda()
    sparse_check(qsa, q, arrays, rng.integers(0, 300, (2, 200)).astype(np.int32), 0.09 / mag, 1.0, 1.0)


def test_sparse_attn_fp4_large_logits(qsa):
    """Weights that concentrate on one entry, wherever it lies."""
    rng = np.random.default_rng(7)
    arrays = (*random_cache4(rng, 400, 1, 128), *random_cache4(rng, 400, 1, 128))
    slots = np.stack([rng.permutation(400) for _ in range(6)]).astype(np.int32)
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (6, 8, 128))), arrays, slots, 4.0, 1.0, 1.0)


def test_sparse_attn_fp4_broken_rows_show_only_where_they_are_read(qsa):
    rng = np.random.default_rng(9)
    arrays = [*random_cache4(rng, 200, 1, 128), *random_cache4(rng, 200, 1, 128)]
    arrays[1][150:, 0, 3] = 0x7F  # NaN scales in K from slot 150
    slots = rng.integers(0, 150, (2, 100)).astype(np.int32)
    q = bf16_dev(normal_bf16(rng, (2, 8, 128)))
    sparse_check(qsa, q, arrays, slots, 0.1, 1.0, 1.0)
    slots[1, 60] = 170
    out, lse = qsa.sparse_attn_fp4(q, *map(to_dev, arrays), to_dev(slots), 0.1)
    assert np.isfinite(host(out)[0]).all() and np.isnan(host(out)[1]).all() and np.isnan(host(lse)[1]).all()
    slots[1] = 170
    out, lse = qsa.sparse_attn_fp4(q, *map(to_dev, arrays), to_dev(slots), 0.1)
    assert np.isnan(host(out)[1]).all() and np.isnan(host(lse)[1]).all()


def test_sparse_attn_fp4_without_lse_and_into_given_buffers(qsa):
    import torch
    rng = np.random.default_rng(10)
    arrays = list(map(to_dev, (*random_cache4(rng, 200, 2, 128), *random_cache4(rng, 200, 2, 128))))
    q, slots = bf16_dev(normal_bf16(rng, (3, 8, 128))), to_dev(rng.integers(0, 200, (3, 150)).astype(np.int32))
    want, _ = qsa.sparse_attn_fp4(q, *arrays, slots)
    out = torch.empty_like(want)
    got, lse = qsa.sparse_attn_fp4(q, *arrays, slots, out=out, want_lse=False)
    assert got is out and lse is None and torch.equal(out, want)


# ------------------------------------------------------------ window attention
def window_case(rng, lens, page, h_kv, d, fp4, spare_rows=0):
    """lens[r]: the row lengths of request r.  Returns the call's arguments."""
    ctx = [max(rows, default=0) for rows in lens]
    pt, n_slots = page_table(rng, np.maximum(ctx, 1), page)
    start = np.concatenate([[0], np.cumsum([len(r) for r in lens])]).astype(np.int32)
    row_len = np.array([x for rows in lens for x in rows] + [5] * spare_rows, np.int32)
    if fp4:
        cache = [*random_cache4(rng, n_slots, h_kv, d, 2.0 ** -3), *random_cache4(rng, n_slots, h_kv, d, 2.0 ** -5, 0.1)]
    else:
        cache = [normal_bf16(rng, (n_slots, h_kv, d)) for _ in range(2)]
    return pt, start, row_len, cache, max(ctx)


def window_check(qsa, rng, lens, page, h_q, h_kv, d, window, n_sink, fp4, spare_rows=0, scale=None, weight_eps=None,
                 cache=None, max_rows=None):
    import torch
    pt, start, row_len, made, max_len = window_case(rng, lens, page, h_kv, d, fp4, spare_rows)
    cache = cache(pt, made) if cache else made
    scale = d ** -0.5 if scale is None else scale
    n_rows = row_len.size
    q = bf16_dev(normal_bf16(rng, (n_rows, h_q + 3, d)))[:, 1:1 + h_q]  # rows of a wider projection
    out = torch.full((n_rows, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n_rows, h_q), 7.0, device="cuda")
    rest = (to_dev(start), to_dev(row_len), to_dev(pt), page, max_len, window, n_sink, scale)
    if max_rows is None:
        max_rows = max(len(r) for r in lens)
    if fp4:
        got = qsa.window_attn_fp4(q, *map(to_dev, cache), *rest, 2.0 ** -3, 2.0 ** -5, max_rows_per_req=max_rows, out=out,
                                  lse=lse)
        k, v = ref.values(*cache[:2], 2.0 ** -3), ref.values(*cache[2:], 2.0 ** -5)
    else:
        got = qsa.window_attn(q, *map(bf16_dev, cache), *rest, max_rows_per_req=max_rows, out=out, lse=lse)
        k, v = map(ref.bf16_to_f64, cache)
    assert got[0] is out and got[1] is lse
    o, l, qh = bits_to_f64(out), host(lse).astype(np.float64), bits_to_f64(q)
    if weight_eps is None:
        weight_eps = W_F16X2 if fp4 else W_BF16
    worst = 0.0
    for r in range(len(lens)):
        for t in range(start[r], start[r + 1]):
            pos = ref.window_positions(row_len[t], window, n_sink)
            sl = ref.slots_of(pt[r], pos, page)
            ro, rl, a, big, spread = ref.attend(qh[t], k[sl], v[sl], scale)
            tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, weight_eps, BF16_HALF_STEP, fp4,
                                       np.abs(v[sl]).max(initial=0.0))
            err = np.abs(o[t] - ro) / tol
            assert (err <= 1).all(), (r, t, int(row_len[t]), float(err.max()))
            worst = max(worst, float(err.max()))
            if pos.size == 0:
                assert (o[t] == 0).all() and np.isneginf(l[t]).all()
            else:
                assert (np.abs(l[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all(), (r, t)
    tail = start[-1]
    assert (o[tail:] == 7.0).all() and (l[tail:] == 7.0).all()  # rows behind the last request
    return out, lse


EDGE_LENS = [[1], [0], [40, 41, 42, 43, 44, 45], [63, 64, 65], [], [100, 101], [500], [33]]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("h_q,h_kv,d,page", [(16, 2, 256, 64), (5, 1, 256, 4), (8, 4, 128, 16), (16, 1, 128, 12),
                                             (12, 1, 128, 128), (3, 3, 128, 20)])
@pytest.mark.parametrize("window,n_sink", [(40, 4), (1, 0), (1, 1), (64, 0), (1000, 4), (33, 70)])
def test_window_attn_edges(qsa, fp4, h_q, h_kv, d, page, window, n_sink):
    """Rows of 0 and 1 tokens, shorter and longer than the window, sinks in
    and beside the window, an empty request, rows behind the last request."""
    rng = np.random.default_rng(window * 7 + d + page)
    window_check(qsa, rng, EDGE_LENS, page, h_q, h_kv, d, window, n_sink, fp4, spare_rows=3)


@pytest.mark.parametrize("h_q,h_kv,d,page", [(16, 2, 256, 64), (16, 4, 128, 16), (8, 8, 128, 64), (10, 2, 256, 12),
                                             (7, 1, 128, 4), (16, 1, 128, 256)])
@pytest.mark.parametrize("window,n_sink", [(100, 4), (500, 0), (37, 130), (5000, 0)])
def test_window_attn_prompts(qsa, h_q, h_kv, d, page, window, n_sink):
    """Whole prompts and chunks of a longer context, ragged, in one call."""
    rng = np.random.default_rng(window + h_q + page)
    lens = [list(range(1, 131)), list(range(1, 2)), list(range(700, 777)), [], list(range(250, 267)),
            list(range(1, 18)), list(range(1200, 1264))]
    window_check(qsa, rng, lens, page, h_q, h_kv, d, window, n_sink, False, spare_rows=2)


def test_window_attn_rows_in_any_order(qsa):
    """Rows of a request need not be consecutive positions."""
    rng = np.random.default_rng(21)
    lens = [[300, 7, 0, 150, 299, 300, 12, 64, 65, 1, 128, 129, 77, 300, 5, 6, 191, 192, 193, 2] * 3]
    window_check(qsa, rng, lens, 64, 8, 2, 128, 50, 3, False)
    window_check(qsa, rng, lens, 64, 8, 2, 128, 50, 3, True)


@pytest.mark.parametrize("fp4", [False, True])
def test_window_attn_long_rows_join_several_clusters(qsa, fp4):
    rng = np.random.default_rng(22)
    assert qsa.lib().qsa_window_attn_workspace_size(3, 4, 1, 128, 30001, 30000, 4) > 0
    window_check(qsa, rng, [[30001], [100, 20000]], 64, 4, 1, 128, 30000, 4, fp4, spare_rows=1, scale=0.02)


@pytest.mark.parametrize("rows", [1, 40])
def test_window_attn_masked_positions_have_no_effect(qsa, rows):
    """Infinities and NaN everywhere outside the window and the sinks, and in
    the pages' unused tail, change nothing."""
    rng = np.random.default_rng(23 + rows)
    window, n_sink, ctx, page = 50, 3, 400, 64

    def poison(pt, cache):
        seen = set()
        for length in range(ctx - rows + 1, ctx + 1):
            seen |= set(ref.slots_of(pt[0], ref.window_positions(length, window, n_sink), page).tolist())
        hide = np.array([s for s in range(cache[0].shape[0]) if s not in seen])
        for c in cache:
            c[hide[0::3]], c[hide[1::3]], c[hide[2::3]] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
        return cache

    window_check(qsa, rng, [list(range(ctx - rows + 1, ctx + 1))], page, 8, 1, 128, window, n_sink, False, cache=poison)
    window_check(qsa, rng, [list(range(ctx - rows + 1, ctx + 1))], page, 8, 1, 256, window, n_sink, False, cache=poison)


@pytest.mark.parametrize("rows", [1, 64])
@pytest.mark.parametrize("d", [128, 256])
def test_window_attn_bad_pages_are_skipped_and_flagged(qsa, rows, d):
    rng = np.random.default_rng(24 + rows)
    page, ctx, window, n_sink = 16, 330, 200, 20
    pt, n_slots = page_table(rng, [ctx], page)
    k, v = normal_bf16(rng, (n_slots, 2, d)), normal_bf16(rng, (n_slots, 2, d))
    q = normal_bf16(rng, (rows, 4, d))
    bad = pt.copy()
    bad[0, 1], bad[0, 12], bad[0, 15] = -1, n_slots // page, 2**31 - 1
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, rows], np.int32)), to_dev(lens),
                               to_dev(bad), page, ctx, window, n_sink)
    assert qsa.device_status(clear=True) == 1
    kf, vf = ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    for t in range(rows):
        pos = ref.window_positions(lens[t], window, n_sink)
        pos = pos[~np.isin(pos // page, [1, 12, 15])]
        sl = ref.slots_of(pt[0], pos, page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(bits_to_f64(out)[t] - ro) <= tol).all(), t
        assert (np.abs(host(lse)[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all()


@pytest.mark.parametrize("rows", [1, 40])
def test_window_attn_bad_row_lengths_count_as_zero(qsa, rows):
    rng = np.random.default_rng(25)
    pt, n_slots = page_table(rng, [200], 64)
    k = bf16_dev(normal_bf16(rng, (n_slots, 1, 128)))
    lens = np.full(rows + 2, 200, np.int32)
    lens[0], lens[-1] = 201, -5
    q = bf16_dev(normal_bf16(rng, (rows + 2, 8, 128)))
    out, lse = qsa.window_attn(q, k, k, to_dev(np.array([0, rows + 2], np.int32)), to_dev(lens), to_dev(pt), 64, 200, 64)
    assert qsa.device_status(clear=True) == 8
    o = host(out)
    assert (o[0] == 0).all() and (o[-1] == 0).all() and (o[1:-1] != 0).any()
    assert np.isneginf(host(lse)[[0, -1]]).all() and np.isfinite(host(lse)[1:-1]).all()


@pytest.mark.parametrize("rows", [1, 40])
def test_window_attn_offsets_past_32_bits(qsa, rows):
    """Pages at the far end of a cache of more than 2^32 bytes."""
    import torch
    rng = np.random.default_rng(26)
    h_kv, d, page = 2, 256, 64
    n_pages = 70_000  # 4.6 GB each of K and V
    k = torch.zeros((n_pages * page, h_kv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    pt = np.array([[n_pages - 1, n_pages - 3, 3, n_pages - 2]], np.int32)
    small = [normal_bf16(rng, (4 * page, h_kv, d)) for _ in range(2)]
    for i, p in enumerate(pt[0]):
        k[p * page:(p + 1) * page] = bf16_dev(small[0][i * page:(i + 1) * page])
        v[p * page:(p + 1) * page] = bf16_dev(small[1][i * page:(i + 1) * page])
    q = bf16_dev(normal_bf16(rng, (rows, 16, d)))
    lens = to_dev(np.arange(250 - rows + 1, 251).astype(np.int32))
    start = to_dev(np.array([0, rows], np.int32))
    out, lse = qsa.window_attn(q, k, v, start, lens, to_dev(pt), page, 250, 100, 4)
    near = np.arange(4, dtype=np.int32)[None]
    want, want_l = qsa.window_attn(q, *map(bf16_dev, small), start, lens, to_dev(near), page, 250, 100, 4)
    assert torch.equal(out, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("h_q,h_kv,d,page", [(16, 2, 256, 64), (16, 4, 128, 16), (5, 1, 256, 24), (16, 16, 128, 64)])
@pytest.mark.parametrize("window,n_sink", [(1024, 4), (4000, 0), (700, 200)])
def test_window_attn_shared_tiles(qsa, h_q, h_kv, d, page, window, n_sink):
    """A few requests of a few rows: the CTAs of a cluster share each tile,
    also those of rows too short to give all of them a part, and of no tokens."""
    rng = np.random.default_rng(window + h_q + d)
    window_check(qsa, rng, [list(range(4495, 4501))], page, h_q, h_kv, d, window, n_sink, False, spare_rows=2)
    window_check(qsa, rng, [[7, 0, 8], [0, 0, 0], [], list(range(2995, 3001)), [1], [129, 130]], page, h_q, h_kv, d,
                 window, n_sink, False, spare_rows=2)
    window_check(qsa, rng, [[900 + 37 * r, 0, 901 + 37 * r] for r in range(20)], page, h_q, h_kv, d, window, n_sink, False)


def test_window_attn_shared_tiles_of_poisoned_and_missing_pages(qsa):
    """As test_window_attn_masked_positions_have_no_effect and
    test_window_attn_bad_pages_are_skipped_and_flagged, in shared tiles."""
    rng = np.random.default_rng(40)
    window, n_sink, ctx, page, d = 1000, 70, 1800, 64, 256

    def poison(pt, cache):
        seen = set()
        for length in range(ctx - 5, ctx + 1):
            seen |= set(ref.slots_of(pt[0], ref.window_positions(length, window, n_sink), page).tolist())
        hide = np.array([s for s in range(cache[0].shape[0]) if s not in seen])
        for c in cache:
            c[hide[0::3]], c[hide[1::3]], c[hide[2::3]] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
        return cache

    window_check(qsa, rng, [list(range(ctx - 5, ctx + 1))], page, 8, 1, d, window, n_sink, False, cache=poison)
    pt, n_slots = page_table(rng, [ctx], page)
    k, v, q = (normal_bf16(rng, s) for s in ((n_slots, 1, d), (n_slots, 1, d), (6, 8, d)))
    bad = pt.copy()
    bad[0, 1], bad[0, 20], bad[0, 28] = n_slots // page, -7, 2**31 - 1
    lens = np.arange(ctx - 5, ctx + 1).astype(np.int32)
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, 6], np.int32)), to_dev(lens), to_dev(bad),
                               page, ctx, window, n_sink)
    assert qsa.device_status(clear=True) == 1
    kf, vf = ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    for t in range(6):
        pos = ref.window_positions(lens[t], window, n_sink)
        pos = pos[~np.isin(pos // page, [1, 20, 28])]
        sl = ref.slots_of(pt[0], pos, page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(bits_to_f64(out)[t] - ro) <= tol).all(), t
        assert (np.abs(host(lse)[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all()


@pytest.mark.parametrize("n_req", [33, 1024, 1025, 1400])
def test_window_attn_many_requests(qsa, n_req):
    """Requests of 0 to 3 rows; the tiles are found by counting up to 1,024
    requests, by a search from there on."""
    rng = np.random.default_rng(n_req)
    lens = [rng.integers(0, 60, rng.integers(0, 4)).tolist() for _ in range(n_req)]
    lens[n_req // 2] = list(range(20, 60))
    window_check(qsa, rng, lens, 16, 4, 1, 128, 20, 2, False, spare_rows=1)


@pytest.mark.parametrize("n_req", [300, 1100])
def test_window_attn_many_tiles_of_no_tokens(qsa, n_req):
    """Tiles without a block of entries between tiles with some."""
    rng = np.random.default_rng(n_req + 1)
    lens = [[0] * 5 if r % 50 else [3, 0, 200, 201] for r in range(n_req)]
    window_check(qsa, rng, lens, 64, 8, 4, 128, 64, 1, False)


@pytest.mark.parametrize("h_q,h_kv,d,page", [(16, 2, 256, 64), (5, 1, 256, 8), (8, 4, 128, 16), (16, 1, 128, 24),
                                             (12, 1, 128, 128), (3, 3, 128, 40)])
@pytest.mark.parametrize("window,n_sink", [(40, 4), (1, 0), (1, 1), (64, 0), (1000, 4), (33, 70)])
def test_window_attn_edges_of_tiles(qsa, h_q, h_kv, d, page, window, n_sink):
    """test_window_attn_edges in the form for requests of many rows."""
    rng = np.random.default_rng(window * 7 + d + page + 1)
    window_check(qsa, rng, EDGE_LENS, page, h_q, h_kv, d, window, n_sink, False, spare_rows=3, max_rows=17)


@pytest.mark.parametrize("h_q,h_kv,d,page", [(16, 2, 256, 64), (16, 4, 128, 16), (5, 1, 256, 24), (16, 16, 128, 64)])
@pytest.mark.parametrize("window,n_sink", [(1024, 4), (4000, 0), (700, 200)])
def test_window_attn_shared_tiles_of_short_requests(qsa, h_q, h_kv, d, page, window, n_sink):
    """test_window_attn_shared_tiles in the form for requests of many rows."""
    rng = np.random.default_rng(window + h_q + d + 1)
    window_check(qsa, rng, [list(range(4495, 4501))], page, h_q, h_kv, d, window, n_sink, False, 2, max_rows=17)
    window_check(qsa, rng, [[7, 0, 8], [0, 0, 0], [], list(range(2995, 3001)), [1], [129, 130]], page, h_q, h_kv, d,
                 window, n_sink, False, 2, max_rows=17)
    window_check(qsa, rng, [[900 + 37 * r, 0, 901 + 37 * r] for r in range(20)], page, h_q, h_kv, d, window, n_sink,
                 False, max_rows=17)


@pytest.mark.parametrize("rows", [17, 24])
def test_window_attn_shared_tiles_beside_poisoned_and_missing_pages(qsa, rows):
    """test_window_attn_shared_tiles_of_poisoned_and_missing_pages at row
    counts that the form for many rows serves."""
    rng = np.random.default_rng(44 + rows)
    window, n_sink, ctx, page, d = 1000, 70, 1800, 64, 256

    def poison(pt, cache):
        seen = set()
        for length in range(ctx - rows + 1, ctx + 1):
            seen |= set(ref.slots_of(pt[0], ref.window_positions(length, window, n_sink), page).tolist())
        hide = np.array([s for s in range(cache[0].shape[0]) if s not in seen])
        for c in cache:
            c[hide[0::3]], c[hide[1::3]], c[hide[2::3]] = 0x7F80, 0xFF80, 0x7FC0  # inf, -inf, NaN
        return cache

    window_check(qsa, rng, [list(range(ctx - rows + 1, ctx + 1))], page, 8, 1, d, window, n_sink, False, cache=poison)
    pt, n_slots = page_table(rng, [ctx], page)
    k, v, q = (normal_bf16(rng, s) for s in ((n_slots, 1, d), (n_slots, 1, d), (rows, 8, d)))
    bad = pt.copy()
    bad[0, 1], bad[0, 20], bad[0, 28] = n_slots // page, -7, 2**31 - 1
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, rows], np.int32)), to_dev(lens),
                               to_dev(bad), page, ctx, window, n_sink)
    assert qsa.device_status(clear=True) == 1
    kf, vf = ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    for t in range(rows):
        pos = ref.window_positions(lens[t], window, n_sink)
        pos = pos[~np.isin(pos // page, [1, 20, 28])]
        sl = ref.slots_of(pt[0], pos, page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(bits_to_f64(out)[t] - ro) <= tol).all(), t
        assert (np.abs(host(lse)[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all()


@pytest.mark.parametrize("n_req", [33, 1025])
def test_window_attn_many_requests_of_few_rows_in_tiles(qsa, n_req):
    rng = np.random.default_rng(n_req + 2)
    lens = [rng.integers(0, 60, rng.integers(0, 4)).tolist() for _ in range(n_req)]
    window_check(qsa, rng, lens, 16, 4, 1, 128, 20, 2, False, spare_rows=1, max_rows=17)


@pytest.mark.parametrize("n_req", [300, 1100])
def test_window_attn_tiles_of_no_tokens(qsa, n_req):
    rng = np.random.default_rng(n_req + 3)
    lens = [[0] * 5 if r % 50 else [3, 0, 200, 201] for r in range(n_req)]
    window_check(qsa, rng, lens, 64, 8, 4, 128, 64, 1, False, max_rows=17)

@pytest.mark.parametrize("h_q,h_kv,d,rows", [(8, 1, 256, 48), (16, 2, 128, 48), (4, 4, 128, 200), (8, 1, 256, 20)])
@pytest.mark.parametrize("window,n_sink", [(5000, 0), (60, 3), (700, 0)])
def test_window_attn_broken_values_reach_only_the_rows_that_see_them(qsa, h_q, h_kv, d, rows, window, n_sink):
    """Infinities and NaN at positions that some rows of a request see and
    others, in the same tile, do not: in the others they have no effect."""
    rng = np.random.default_rng(45 + rows + d)
    page, ctx = 32, 1500
    pt, n_slots = page_table(rng, [ctx], page)
    k, v, q = (normal_bf16(rng, s) for s in ((n_slots, h_kv, d), (n_slots, h_kv, d), (rows, h_q, d)))
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    # seen by the last rows, by the second half, and by the first quarter (where its windows begin)
    at = [ctx - 3, ctx - rows // 2, lens[0] + rows // 4 - window]
    at = [p for p in at if p >= 0]
    for i, p in enumerate(at):
        sl = ref.slots_of(pt[0], np.array([p]), page)[0]
        k[sl, :, 5] = (0x7F80, 0x7FC0, 0xFF80)[i]
        v[sl, :, 7 + i:d:16] = (0x7FC0, 0x7F80, 0xFF80)[i]
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, rows], np.int32)), to_dev(lens), to_dev(pt),
                               page, ctx, window, n_sink, max_rows_per_req=max(rows, 17))
    o, l, kf, vf = bits_to_f64(out), host(lse).astype(np.float64), ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    clean = 0
    for t in range(rows):
        pos = ref.window_positions(lens[t], window, n_sink)
        if np.isin(at, pos).any():
            continue
        clean += 1
        sl = ref.slots_of(pt[0], pos, page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(o[t] - ro) <= tol).all(), t
        assert (np.abs(l[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all()
    assert clean >= rows // 4 - 2


@pytest.mark.parametrize("rows", [20, 60])
def test_window_attn_broken_values_seen_show_as_they_are(qsa, rows):
    """An infinity of V that every row sees makes that column infinite, and
    leaves the other columns alone."""
    rng = np.random.default_rng(46)
    pt, n_slots = page_table(rng, [300], 64)
    k, v, q = (normal_bf16(rng, s) for s in ((n_slots, 1, 128), (n_slots, 1, 128), (rows, 8, 128)))
    v[ref.slots_of(pt[0], np.array([200]), 64)[0], 0, 9] = 0x7F80
    lens = np.arange(300 - rows + 1, 301).astype(np.int32)
    out, _ = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, rows], np.int32)), to_dev(lens), to_dev(pt), 64,
                             300, 250, max_rows_per_req=rows)
    o, kf, vf = bits_to_f64(out), ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    assert np.isposinf(o[:, :, 9]).all()
    vf[:, 0, 9] = 0
    for t in range(rows):
        pos = ref.window_positions(lens[t], 250, 0)
        sl = ref.slots_of(pt[0], pos, 64)
        ro, _, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], 128 ** -0.5)
        tol, _ = ref.tolerance(128, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        keep = np.arange(128) != 9
        assert (np.abs(o[t] - ro) <= tol)[:, keep].all()

@pytest.mark.parametrize("scale", [-0.07, 0.0, -30.0, 1e-20])
@pytest.mark.parametrize("rows", [1, 6, 40])
@pytest.mark.parametrize("fp4", [False, True])
def test_window_attn_scales(qsa, fp4, rows, scale):
    rng = np.random.default_rng(41 + rows)
    lens = [list(range(300 - rows, 300))]
    window_check(qsa, rng, lens, 32, 8, 2, 128, 150, 3, fp4, scale=scale)


@pytest.mark.parametrize("d,h_kv", [(256, 2), (128, 4)])
def test_window_attn_single_rows_keep_both_parts_of_the_weights(qsa, d, h_kv):
    """One row a request: the weights are held as a BF16 and its remainder."""
    rng = np.random.default_rng(42)
    window_check(qsa, rng, [[700], [33], [1], [0], [2000]], 16, 16, h_kv, d, 900, 4, False, weight_eps=W_BF16X2)


def test_graphs_sharing_a_workspace(qsa):
    """Two captured graphs that split long rows over the same workspace, in
    turn on one stream."""
    import torch
    rng = np.random.default_rng(43)
    arrays = list(map(to_dev, (*random_cache4(rng, 4000, 1, 128), *random_cache4(rng, 4000, 1, 128))))
    q = [bf16_dev(normal_bf16(rng, (2, 8, 128))) for _ in range(2)]
    slots = [to_dev(rng.integers(0, 4000, (2, n)).astype(np.int32)) for n in (20000, 12000)]
    need = max(qsa.lib().qsa_sparse_attn_fp4_workspace_size(2, 8, 1, 128, s.shape[1]) for s in slots)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = [[t.clone() for t in qsa.sparse_attn_fp4(q[i], *arrays, slots[i])] for i in range(2)]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(qsa.sparse_attn_fp4(q[i], *arrays, slots[i], workspace=ws))
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for got, exp in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, exp))

def test_window_attn_of_an_empty_context_in_tiles(qsa):
    import torch
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    start = torch.tensor([0, 40, 40], dtype=i32, device="cuda")
    out, lse = qsa.window_attn(z(40, 8, 128) + 1, z(64, 2, 128), z(64, 2, 128), start, z(40, dt=i32), z(2, 4, dt=i32), 16, 0, 8)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_window_attn_largest_window_and_sinks(qsa):
    """window and n_sink at the type's limit: plain causal attention."""
    rng = np.random.default_rng(47)
    for lens in ([[300]], [list(range(1, 60))]):
        for window, n_sink in ((2**31 - 1, 0), (2**31 - 1, 2**31 - 1), (1, 2**31 - 1)):
            window_check(qsa, rng, lens, 16, 8, 2, 128, window, n_sink, False)


def test_first_calls_inside_a_capture():
    """A fresh process whose first use of the calls is a stream capture.  A
    block of ones is held as 6 * 11/64: e4m3 has 10/64 and 11/64 around 1/6,
    and 64/11 is nearer to 6 than to 4."""
    import pathlib
    import subprocess
    import sys
    code = """
import torch, sparse_attention_indexer_index_gb300 as qsa
qsa.lib()
z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device='cuda')
i32, u8 = torch.int32, torch.uint8
q1, q2, k = z(2, 8, 128), z(40, 8, 128), z(64, 2, 128) + 1
c = [z(64, 2, 64, dt=u8), z(64, 2, 8, dt=u8), z(64, 2, 64, dt=u8), z(64, 2, 8, dt=u8)]
s1, s2 = (torch.tensor([0, n], dtype=i32, device='cuda') for n in (2, 40))
l1, l2 = (torch.full((n,), 50, dtype=i32, device='cuda') for n in (2, 40))
pt, slots, first = torch.arange(4, dtype=i32, device='cuda')[None], z(2, 30, dt=i32), z(1, dt=i32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    qsa.append_kv_fp4(k[:40], k[:40], s2, first, *c, pt, 16)
    a = qsa.sparse_attn_fp4(q1, *c, slots)
    b = qsa.window_attn(q1, k, k, s1, l1, pt, 16, 64, 20)
    d = qsa.window_attn(q2, k, k, s2, l2, pt, 16, 64, 20)
    e = qsa.window_attn_fp4(q1, *c, s1, l1, pt, 16, 64, 20)
g.replay()
torch.cuda.synchronize()
assert qsa.device_status() == 0
assert ((a[0] - 66 / 64).abs() < 1e-6).all() and (b[0] == 1).all() and (d[0] == 1).all() and torch.isfinite(e[0]).all()
print('fine')
"""
    root = pathlib.Path(__file__).resolve().parents[1]
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]

def test_cache4_offsets_past_32_bits(qsa):
    """Append, read back and attend at the far end of a 4-bit cache whose
    codes take more than 2^32 bytes."""
    import torch
    rng = np.random.default_rng(27)
    h_kv, d, page, n_pages = 8, 256, 64, 70_000  # 1 KB of codes a slot: 4.6 GB each
    cache = [torch.zeros((n_pages * page, h_kv, w), dtype=torch.uint8, device="cuda") for w in (d // 2, d // 16) * 2]
    small = [torch.zeros((2 * page, h_kv, w), dtype=torch.uint8, device="cuda") for w in (d // 2, d // 16) * 2]
    k, v = bf16_dev(normal_bf16(rng, (100, h_kv, d))), bf16_dev(normal_bf16(rng, (100, h_kv, d)))
    start, first, lens = (to_dev(np.array(x, np.int32)) for x in ([0, 100], [0], [100]))
    one = to_dev(np.array([0, 1], np.int32))
    q = bf16_dev(normal_bf16(rng, (1, 16, d)))
    got = []
    for c, pt in ((cache, [[n_pages - 1, n_pages - 2]]), (small, [[0, 1]])):
        pt = np.array(pt, np.int32)
        qsa.append_kv_fp4(k, v, start, first, *c, to_dev(pt), page)
        slots = to_dev(ref.slots_of(pt[0], np.arange(100), page).astype(np.int32)[None])
        got.append([*qsa.gather_kv_fp4(*c, slots), *qsa.sparse_attn_fp4(q, *c, slots),
                    *qsa.window_attn_fp4(q, *c, one, lens, to_dev(pt), page, 100, 60, 4)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------- together, streams and graphs
def test_cache4_in_the_decode_path(qsa):
    """The path a user runs: append the context's K and V in chunks, select
    with the indexer, attend over the selection and over a window.  The same
    calls on the BF16 values read back agree within both sides' bounds."""
    import torch
    w = decode_workload(91, [[5003], [700], [2999, 3000]], page_size=64, k_blk=128)
    rng = np.random.default_rng(92)
    h_q, h_kv, d, page = 16, 2, 256, w.page_size
    n_slots = w.n_pages * page
    gk, gv = 2.0 ** -5, 2.0 ** -6
    cache = [torch.zeros((n_slots, h_kv, x), dtype=torch.uint8, device="cuda") for x in (d // 2, d // 16) * 2]
    ctx = np.array([5003, 700, 3000])
    done = np.zeros(3, np.int64)
    pt = to_dev(w.page_table)
    for step in (np.array([5000, 1, 0]), np.array([3, 699, 3000])):  # two calls, ragged
        start = np.concatenate([[0], np.cumsum(step)]).astype(np.int32)
        qkv = bf16_dev(normal_bf16(rng, (int(start[-1]), 2 * h_kv, d)))
        qsa.append_kv_fp4(qkv[:, :h_kv], qkv[:, h_kv:], to_dev(start), to_dev(done.astype(np.int32)), *cache, pt, page,
                          gk, gv)
        done += step
    assert (done == ctx).all()
    # index keys are the caller's; here random ones stand in the pool
    pool = bf16_dev(normal_bf16(rng, (w.pool_rows, 128)))
    sel = qsa.indexer_select(bf16_dev(w.q), pool, to_dev(w.req_row_start), to_dev(w.row_len), pt, page, w.max_len,
                             w.max_rows_per_req, k_blk=w.k_blk)
    q = bf16_dev(normal_bf16(rng, (w.n_rows, h_q, d)))
    out, lse = qsa.sparse_attn_fp4(q, *cache, sel["slots"], None, gk, gv)
    every = torch.arange(n_slots, dtype=torch.int32, device="cuda")
    k, v = qsa.gather_kv_fp4(*cache, every, gk, gv)
    want, want_l = qsa.sparse_attn(q, k, v, sel["slots"])
    assert (out - want).abs().max().item() <= 4e-5 * v.abs().max().item()
    assert (lse - want_l).abs().max().item() <= 1e-4
    rest = (to_dev(w.req_row_start), to_dev(w.row_len), pt, page, w.max_len, 600, 4)
    wo, wl = qsa.window_attn_fp4(q, *cache, *rest, None, gk, gv)
    bo, bl = qsa.window_attn(q, k, v, *rest)
    assert (wl - bl).abs().max().item() <= 1e-4
    assert (wo.float() - bo.float()).abs().max().item() <= 2.0 ** -7 * v.abs().max().item()


def calls_on_one_state(qsa, rng, rows):
    """The five calls over one small state: a function running them, and their
    outputs."""
    import torch
    h_q, h_kv, d, page, ctx = 8, 2, 128, 16, 300
    pt, n_slots = page_table(rng, [ctx, ctx], page)
    cache = [torch.zeros((n_slots, h_kv, x), dtype=torch.uint8, device="cuda") for x in (d // 2, d // 16) * 2]
    k, v = bf16_dev(normal_bf16(rng, (2 * ctx, h_kv, d))), bf16_dev(normal_bf16(rng, (2 * ctx, h_kv, d)))
    kb, vb = bf16_dev(normal_bf16(rng, (n_slots, h_kv, d))), bf16_dev(normal_bf16(rng, (n_slots, h_kv, d)))
    q = bf16_dev(normal_bf16(rng, (2 * rows, h_q, d)))
    ts, fp = to_dev(np.array([0, ctx, 2 * ctx], np.int32)), to_dev(np.array([0, 0], np.int32))
    rs = to_dev(np.array([0, rows, 2 * rows], np.int32))
    rl = to_dev(np.concatenate([np.arange(ctx - rows + 1, ctx + 1)] * 2).astype(np.int32))
    slots = to_dev(rng.integers(0, n_slots, (2 * rows, 12000 if rows == 1 else 200)).astype(np.int32))
    some = slots[:, :50].contiguous()
    pt = to_dev(pt)

    def run(ws):
        qsa.append_kv_fp4(k, v, ts, fp, *cache, pt, page)
        return [*qsa.gather_kv_fp4(*cache, some),
                *qsa.sparse_attn_fp4(q, *cache, slots, workspace=ws),
                *qsa.window_attn(q, kb, vb, rs, rl, pt, page, ctx, 100, 4, max_rows_per_req=rows, workspace=ws),
                *qsa.window_attn_fp4(q, *cache, rs, rl, pt, page, ctx, 100, 4, max_rows_per_req=rows, workspace=ws)]

    need = qsa.lib().qsa_sparse_attn_fp4_workspace_size(2 * rows, h_q, h_kv, d, slots.shape[1])
    return run, max(need, 16), (k, v, kb, vb, q)


@pytest.mark.parametrize("rows", [1, 20])
def test_calls_captured_and_replayed_on_new_inputs(qsa, rows):
    import torch
    rng = np.random.default_rng(30)
    run, need, inputs = calls_on_one_state(qsa, rng, rows)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    run(ws)  # set-up outside the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(ws)
    for _ in range(2):
        for t in inputs:
            t.copy_(bf16_dev(normal_bf16(rng, tuple(t.shape))))
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, run(ws)):
            assert torch.equal(a, b)


def test_calls_on_two_streams_at_once(qsa):
    """Calls on different streams, each with its own workspace, do not touch
    one another; the current stream is the one used."""
    import torch
    rng = np.random.default_rng(31)
    states = [calls_on_one_state(qsa, rng, 1) for _ in range(2)]
    want = [run(torch.empty(need, dtype=torch.uint8, device="cuda")) for run, need, _ in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    work = [torch.empty(need, dtype=torch.uint8, device="cuda") for _, need, _ in states]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, (run, _, _) in enumerate(states):
            with torch.cuda.stream(streams[i]):
                got[i] = run(work[i])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


def test_buffers_of_a_call_on_another_stream_are_that_stream_s(qsa, monkeypatch):
    """What a call allocates for a stream that is not the current one is not
    handed out to the current one while the call may still run."""
    import torch
    rng = np.random.default_rng(48)
    arrays = list(map(to_dev, (*random_cache4(rng, 4000, 1, 128), *random_cache4(rng, 4000, 1, 128))))
    q, slots = bf16_dev(normal_bf16(rng, (2, 8, 128))), to_dev(rng.integers(0, 4000, (2, 20000)).astype(np.int32))
    need = qsa.lib().qsa_sparse_attn_fp4_workspace_size(2, 8, 1, 128, 20000)
    assert need > 0
    want, want_l = qsa.sparse_attn_fp4(q, *arrays, slots)
    torch.cuda.synchronize()
    seen, call = [], qsa._call
    monkeypatch.setattr(qsa, "_call", lambda fn, *a: (seen.append(a), call(fn, *a))[1])
    side = torch.cuda.Stream()
    torch.cuda._sleep(1)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # the call's turn comes later
    out, lse = qsa.sparse_attn_fp4(q, *arrays, slots, stream=side)
    used = {a[-3] for a in seen if a[-2:-1] == (need,)} | {out.data_ptr(), lse.data_ptr()}
    assert len(used) == 3
    mine = [torch.full((n,), 77, dtype=torch.uint8, device="cuda") for n in (need, need, out.nbytes, lse.nbytes)]
    assert not used & {t.data_ptr() for t in mine}
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_l)

def test_same_call_twice_gives_the_same_bits(qsa):
    import torch
    rng = np.random.default_rng(32)
    run, need, _ = calls_on_one_state(qsa, rng, 20)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a, b = run(ws), run(ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------- refusals
def test_binding_refusals(qsa):
    import torch
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    bf, i32 = torch.bfloat16, torch.int32
    cache = [z(64, 2, 64), z(64, 2, 8), z(64, 2, 64), z(64, 2, 8)]
    k, pt, st, fp = z(3, 2, 128, dt=bf), z(1, 4, dt=i32), z(2, dt=i32), z(1, dt=i32)
    q, slots, rl = z(1, 4, 128, dt=bf), z(1, 9, dt=i32), z(1, dt=i32)
    for exc, call in [
        (TypeError, lambda: qsa.append_kv_fp4(k.float(), k, st, fp, *cache, pt, 16)),
        (TypeError, lambda: qsa.append_kv_fp4(k.cpu(), k, st, fp, *cache, pt, 16)),
        (ValueError, lambda: qsa.append_kv_fp4(k.transpose(1, 2).contiguous().transpose(1, 2), k, st, fp, *cache, pt, 16)),
        (ValueError, lambda: qsa.append_kv_fp4(k[:2], k, st, fp, *cache, pt, 16)),
        (ValueError, lambda: qsa.append_kv_fp4(k[:, :1], k[:, :1], st, fp, *cache, pt, 16)),
        (ValueError, lambda: qsa.append_kv_fp4(k, k, st[:1], fp, *cache, pt, 16)),
        (ValueError, lambda: qsa.append_kv_fp4(k, k, st, fp, cache[0], z(64, 2, 4), *cache[2:], pt, 16)),
        (qsa.QSAError, lambda: qsa.append_kv_fp4(k, k, st, fp, *cache, pt, 16, k_scale=0.3)),
        (qsa.QSAError, lambda: qsa.append_kv_fp4(k, k, st, fp, *cache, pt, 18)),
        (TypeError, lambda: qsa.gather_kv_fp4(*cache, slots.long())),
        (ValueError, lambda: qsa.gather_kv_fp4(*cache, slots, k_out=z(9, 2, 128, dt=bf))),
        (ValueError, lambda: qsa.gather_kv_fp4(*cache, z(9, 2, dt=i32).t())),
        (ValueError, lambda: qsa.sparse_attn_fp4(z(1, 4, 256, dt=bf), *cache, slots)),
        (ValueError, lambda: qsa.sparse_attn_fp4(z(2, 4, 128, dt=bf), *cache, slots)),
        (ValueError, lambda: qsa.sparse_attn_fp4(q, *cache, slots, out=z(1, 4, 64, dt=torch.float32))),
        (TypeError, lambda: qsa.sparse_attn_fp4(q, *cache, slots, out=z(1, 4, 128, dt=bf))),
        (qsa.QSAError, lambda: qsa.sparse_attn_fp4(z(1, 3, 128, dt=bf), *cache, slots)),
        (qsa.QSAError, lambda: qsa.sparse_attn_fp4(q, *cache, slots, n_idx=10)),
        (TypeError, lambda: qsa.window_attn(q, cache[0], cache[0], st, rl, pt, 16, 64, 8)),
        (ValueError, lambda: qsa.window_attn(q, k, k[:2], st, rl, pt, 16, 64, 8)),
        (ValueError, lambda: qsa.window_attn(q, k, k, st[:1], rl, pt, 16, 64, 8)),
        (ValueError, lambda: qsa.window_attn(q, k, k, st, z(2, dt=i32), pt, 16, 64, 8)),
        (qsa.QSAError, lambda: qsa.window_attn(q, k, k, st, rl, pt, 16, 64, 0)),
        (qsa.QSAError, lambda: qsa.window_attn(q, k, k, st, rl, pt, 16, 65, 8)),
        (qsa.QSAError, lambda: qsa.window_attn_fp4(q, *cache, st, rl, pt, 16, 64, 8, v_scale=3.0)),
        (TypeError, lambda: qsa.window_attn_fp4(q, *cache, st, rl, pt, 16, 64, 8, out=z(1, 4, 128, dt=torch.float32))),
    ]:
        with pytest.raises(exc):
            call()


def test_empty_calls(qsa):
    import torch
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    bf, i32 = torch.bfloat16, torch.int32
    cache = [z(64, 2, 64), z(64, 2, 8), z(64, 2, 64), z(64, 2, 8)]
    qsa.append_kv_fp4(z(0, 2, 128, dt=bf), z(0, 2, 128, dt=bf), z(2, dt=i32), z(1, dt=i32), *cache, z(1, 4, dt=i32), 16)
    k, v = qsa.gather_kv_fp4(*cache, z(0, dt=i32))
    assert tuple(k.shape) == (0, 2, 128)
    out, lse = qsa.sparse_attn_fp4(z(0, 4, 128, dt=bf), *cache, z(0, 5, dt=i32))
    assert tuple(out.shape) == (0, 4, 128) and tuple(lse.shape) == (0, 4)
    out, lse = qsa.window_attn(z(0, 4, 128, dt=bf), z(64, 2, 128, dt=bf), z(64, 2, 128, dt=bf), z(2, dt=i32),
                               z(0, dt=i32), z(1, 4, dt=i32), 16, 64, 8)
    assert tuple(out.shape) == (0, 4, 128)
    # a context of no tokens: nothing to attend to
    out, lse = qsa.window_attn(z(1, 4, 128, dt=bf), z(64, 2, 128, dt=bf), z(64, 2, 128, dt=bf),
                               torch.tensor([0, 1], dtype=i32, device="cuda"), z(1, dt=i32), z(1, 4, dt=i32), 16, 0, 8)
    assert (out == 0).all() and torch.isneginf(lse).all()
