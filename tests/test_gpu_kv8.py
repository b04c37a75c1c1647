"""The 8-bit KV cache and the attention over it on the GPU, against plain FP64
forms (kv8_ref) at the sizes, masks, strides and layouts where they can go
wrong.  Codes, scales and values are compared to the bit; the attention within
the bounds of kv8_ref.tolerance."""
import numpy as np
import pytest

import kv8_ref as ref
from gpu_util import bf16_dev, to_dev
from kv4_ref import window_positions
from workloads.synth import bf16_bits, normal_bf16

pytestmark = pytest.mark.gpu

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


def random_cache(rng, n_slots, h_kv, d, block, lo=-10, hi=-4):
    """Codes of all kinds but NaN (subnormal and large ones rarer), scales of
    exponents lo .. hi."""
    codes = ref.encode(rng.standard_normal((n_slots, h_kv, d)) * 2.0 ** rng.integers(-3, 7, (n_slots, h_kv, 1)))
    return codes, rng.integers(127 + lo, 128 + hi, (n_slots // block, h_kv)).astype(np.uint8)


def normal_bits(rng, shape, gains):
    """Normal rows times a power of two per row (and head)."""
    x = rng.standard_normal(shape) * gains
    return bf16_bits(x.astype(np.float32))


# ------------------------------------------------------------------- writing
def append_check(qsa, rng, h_kv, d, page, block, n, first, behind=0, fused=False, bits=None, faults=0, drop=None):
    """Appends to a random cache and compares every byte."""
    n, first = np.asarray(n), np.asarray(first)
    pt, n_slots = page_table(rng, first + n, page)
    if drop is not None:
        pt[drop] = rng.choice([-3, n_slots // page, 2 ** 31 - 1])
    total = int(n.sum()) + behind
    if bits is None:
        bits = [normal_bits(rng, (total, h_kv, d), 2.0 ** rng.integers(-6, 7, (total, h_kv, 1))) for _ in range(2)]
    if fused:  # [q | k | v] columns, a token's row wider than what is read
        import torch
        qkv = torch.cat([bf16_dev(normal_bf16(rng, (total, 3, d))), *map(bf16_dev, bits)], 1)
        k_new, v_new = qkv[:, 3:3 + h_kv], qkv[:, 3 + h_kv:]
    else:
        k_new, v_new = map(bf16_dev, bits)
    arrays = [*random_cache(rng, n_slots, h_kv, d, block, -12, 2), *random_cache(rng, n_slots, h_kv, d, block, -12, 2)]
    want = [a.copy() for a in arrays]
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    dev = list(map(to_dev, arrays))
    got = qsa.append_kv_fp8(k_new, v_new, to_dev(start), to_dev(first.astype(np.int32)), *dev, to_dev(pt), page)
    assert qsa.device_status(clear=True) == faults
    for r in range(len(n)):
        pos = first[r] + np.arange(n[r])
        pg = pt[r, np.clip(pos // page, 0, pt.shape[1] - 1)].astype(np.int64)
        slots = np.where((pg >= 0) & ((pg + 1) * page <= n_slots), pg * page + pos % page, -1)
        for i in (0, 1):
            ref.append(want[2 * i], want[2 * i + 1], bits[i][start[r]:start[r + 1]], slots, block, first[r])
    # what a block holds behind the request's last position has no meaning: its codes are left as they were
    for g, w, name in zip(got, want, ("k_codes", "k_scales", "v_codes", "v_scales")):
        assert np.array_equal(host(g), w), name
    assert all(a is b for a, b in zip(got, dev))


@pytest.mark.parametrize("h_kv,d,page,block,fused", [(2, 256, 64, 64, True), (1, 128, 4, 4, False), (3, 128, 48, 16, True),
                                                     (8, 128, 16, 8, False), (1, 256, 128, 128, True), (2, 128, 128, 32, False)])
def test_append_matches_the_format_to_the_bit(qsa, h_kv, d, page, block, fused):
    """Ragged requests (one empty, one of a single token, starts and ends
    inside a block), rows behind the last request; other blocks keep theirs."""
    rng = np.random.default_rng(d + h_kv + block)
    append_check(qsa, rng, h_kv, d, page, block, [5, 0, 1, 170, 33, 2], [3, 9, 0, 61, 1000, 2 * block - 1], behind=7,
                 fused=fused)


@pytest.mark.parametrize("n_req,most", [(40, 1), (300, 6), (1500, 1), (3, 5000), (64, 300)])
def test_append_many_requests_and_many_tokens(qsa, n_req, most):
    """CTAs of one token, of some, of a block."""
    rng = np.random.default_rng(n_req)
    n = np.full(n_req, 1) if most == 1 else rng.integers(0, most + 1, n_req)
    append_check(qsa, rng, 2, 128, 64, 64, n, rng.integers(0, 300, n_req))


def test_append_value_by_value(qsa):
    """A request built up token by token holds what the reference says at every
    step, scales that grow among them."""
    rng = np.random.default_rng(4)
    pt, n_slots = page_table(rng, [40], 16)
    arrays = [*random_cache(rng, n_slots, 1, 128, 16), *random_cache(rng, n_slots, 1, 128, 16)]
    dev, want = list(map(to_dev, arrays)), [a.copy() for a in arrays]
    p = 0
    while p < 40:
        n = int(rng.integers(1, 4))
        n = min(n, 40 - p)
        bits = [normal_bits(rng, (n, 1, 128), 2.0 ** rng.integers(-9, 10, (n, 1, 1))) for _ in range(2)]
        qsa.append_kv_fp8(*map(bf16_dev, bits), to_dev(np.array([0, n], np.int32)), to_dev(np.array([p], np.int32)), *dev,
                          to_dev(pt), 16)
        slots = ref.slots_of(pt[0], np.arange(p, p + n), 16)
        for i in (0, 1):
            ref.append(want[2 * i], want[2 * i + 1], bits[i], slots, 16, p)
        for g, w in zip(dev, want):
            assert np.array_equal(host(g), w), p
        p += n


def test_append_block_edges(qsa):
    """Zeros, the borders of the scale and of codes, signed zeros, magnitudes
    past both ends of the scales, infinities and NaN."""
    x = np.zeros((10, 1, 128), np.float32)
    x[0, 0, 5] = 448.0
    x[1, 0, 5] = 450.0
    x[2, 0, :8] = [448.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 2.5 * 2.0 ** -9, 17.0, 19.0, -0.0]
    x[3, 0, :2] = [3e38, 1.0]
    x[4, 0, :2] = [1e-30, -1e-38]
    x[5, 0, :3] = [np.inf, 1.0, -2.0]
    x[6, 0, :3] = [-np.inf, np.nan, 400.0]
    x[7, 0, :2] = [np.nan, 1e-3]
    x[8, 0, :] = -0.0
    bits = bf16_bits(x)
    bits[np.isnan(x)] = 0x7FC1
    bits[6, 0, 7] = 0xFFFF
    for block, first in ((4, [0]), (4, [1]), (16, [0]), (16, [9])):
        append_check(qsa, np.random.default_rng(block), 1, 128, 16, block, [10], first, bits=[bits, bits[::-1].copy()])


def test_append_out_of_range_is_skipped_and_flagged(qsa):
    rng = np.random.default_rng(5)
    for drop in ((0, 1), (1, 0), (0, 3)):
        append_check(qsa, rng, 2, 128, 16, 8, [50, 20], [3, 9], drop=drop, faults=1)
    # positions outside the table, before its start, past 2^31
    pt, n_slots = page_table(rng, [64, 64, 64, 64], 16)
    arrays = [*random_cache(rng, n_slots, 1, 128, 16), *random_cache(rng, n_slots, 1, 128, 16)]
    dev = list(map(to_dev, arrays))
    new = bf16_dev(normal_bf16(rng, (8, 1, 128)))
    first = np.array([62, -1, 2 ** 31 - 1, 2 ** 31 - 2], np.int32)
    qsa.append_kv_fp8(new, new, to_dev(np.array([0, 2, 4, 6, 8], np.int32)), to_dev(first), *dev, to_dev(pt), 16)
    assert qsa.device_status(clear=True) == 1
    bits = host(new)
    for i in (0, 1):
        ref.append(arrays[2 * i], arrays[2 * i + 1], bits[:2], ref.slots_of(pt[0], np.array([62, 63]), 16), 16, 62)
        ref.append(arrays[2 * i], arrays[2 * i + 1], bits[3:4], ref.slots_of(pt[1], np.array([0]), 16), 16, 0)  # is in range
    for g, w in zip(dev, arrays):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("n", [30, 4000])
def test_append_from_a_negative_position_on(qsa, n):
    """Positions from 0 on are written whatever comes before them, with CTAs of
    one token and of several."""
    rng = np.random.default_rng(n)
    pt, n_slots = page_table(rng, [n], 16)
    arrays = [*random_cache(rng, n_slots, 1, 128, 16), *random_cache(rng, n_slots, 1, 128, 16)]
    dev = list(map(to_dev, arrays))
    bits = normal_bf16(rng, (n, 1, 128))
    qsa.append_kv_fp8(bf16_dev(bits), bf16_dev(bits), to_dev(np.array([0, n], np.int32)), to_dev(np.array([-5], np.int32)),
                      *dev, to_dev(pt), 16)
    assert qsa.device_status(clear=True) == 1
    for i in (0, 1):
        ref.append(arrays[2 * i], arrays[2 * i + 1], bits[5:], ref.slots_of(pt[0], np.arange(n - 5), 16), 16, 0)
    for g, w in zip(dev, arrays):
        assert np.array_equal(host(g), w)


@pytest.mark.parametrize("h_kv,d,block", [(2, 256, 64), (1, 128, 4), (5, 128, 32)])
def test_gather_matches_the_format_to_the_bit(qsa, h_kv, d, block):
    rng = np.random.default_rng(h_kv)
    n_slots = 5 * block * 16
    arrays = [*random_cache(rng, n_slots, h_kv, d, block, -64, 63), *random_cache(rng, n_slots, h_kv, d, block, -64, 63)]
    slots = rng.integers(-2, n_slots, (3, 217)).astype(np.int32)
    k, v = qsa.gather_kv_fp8(*map(to_dev, arrays), to_dev(slots))
    for got, c, s in ((k, *arrays[:2]), (v, *arrays[2:])):
        want = ref.values(c, s, block)[np.maximum(slots, 0)] * (slots >= 0)[..., None, None]
        assert np.array_equal(bits_to_f64(got), want)


def test_gather_past_the_cache_is_flagged(qsa):
    rng = np.random.default_rng(1)
    arrays = [*random_cache(rng, 64, 2, 128, 16), *random_cache(rng, 64, 2, 128, 16)]
    arrays[0][5, 1, 7] = 0x7F
    k, v = qsa.gather_kv_fp8(*map(to_dev, arrays), to_dev(np.array([5, 64, -1], np.int32)))
    assert qsa.device_status(clear=True) == 1
    k, v = bits_to_f64(k), bits_to_f64(v)
    assert np.isnan(k[0, 1, 7]) and np.isnan(k).sum() == 1 and (k[1:] == 0).all() and (v[1:] == 0).all()


# ---------------------------------------------------------------- selections
def one_row(q, kf, vf, ev, scale, out_eps, parts=4):
    """Reference and bounds of one row: q [h_q][d], kf, vf [n][h_kv][d], ev
    [n][h_kv].  parts: e4m3 parts of a weight, 3 in windows of more than 8
    (row, head) pairs to a tile."""
    o, lse, a, big, spread = ref.attend(q, kf, vf, scale)
    top = ref.top_products(q, kf, ev, scale, lse)
    tol, tol_l = ref.tolerance(q.shape[1], kf.shape[0], o, a, big, spread, out_eps, np.abs(ev).max(initial=0), top, parts)
    return o, lse, tol, tol_l + 2.0 ** -23 * np.where(np.isfinite(lse), np.abs(lse), 0.0)


def same(got, want, tol, what):
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin], want[~fin]), what
    err = np.abs(got[fin] - want[fin])
    assert (err <= tol[fin]).all(), (what, (err / tol[fin]).max())


def sparse_check(qsa, q, arrays, block, slots, scale, n_idx=None, faults=0):
    n_slots, h_kv, _ = arrays[0].shape
    out, lse = qsa.sparse_attn_fp8(q, *map(to_dev, arrays), to_dev(slots), scale, n_idx=n_idx)
    assert qsa.device_status(clear=True) == faults
    kf, vf = ref.values(*arrays[:2], block), ref.values(*arrays[2:], block)
    ev = arrays[3].astype(np.float64) - 127
    qf, o, l = bits_to_f64(q), host(out).astype(np.float64), host(lse).astype(np.float64)
    for t in range(q.shape[0]):
        s = slots[t, :n_idx]
        s = s[(s >= 0) & (s < n_slots)]
        ro, rl, tol, tol_l = one_row(qf[t], kf[s], vf[s], ev[s // block], scale, 2.0 ** -24)
        same(o[t], ro, tol, t)
        same(l[t], rl, tol_l, t)


@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (5, 1, 256), (1, 1, 256), (8, 8, 128), (12, 1, 128), (16, 1, 256),
                                        (32, 2, 128), (9, 1, 256)])
def test_sparse_attn_fp8_shapes(qsa, h_q, h_kv, d):
    """Head layouts, q as columns of a wider tensor, rows of all, some and no
    entries."""
    rng = np.random.default_rng(h_q * 10 + h_kv)
    arrays = (*random_cache(rng, 640, h_kv, d, 32), *random_cache(rng, 640, h_kv, d, 32))
    q = bf16_dev(normal_bf16(rng, (5, h_q + 3, d)))[:, :h_q]
    slots = rng.integers(0, 640, (5, 333)).astype(np.int32)
    slots[1, 5:] = -1
    slots[2] = -1
    slots[3, ::2] = -1
    slots[4] = 17  # one entry over and over
    sparse_check(qsa, q, arrays, 32, slots, 0.05)


@pytest.mark.parametrize("w", [0, 1, 15, 16, 17, 33, 63, 65, 257, 700])
@pytest.mark.parametrize("h_kv,d", [(2, 256), (1, 128)])
def test_sparse_attn_fp8_widths(qsa, w, h_kv, d):
    rng = np.random.default_rng(w)
    arrays = (*random_cache(rng, 960, h_kv, d, 4), *random_cache(rng, 960, h_kv, d, 4))
    q = bf16_dev(normal_bf16(rng, (3, 8, d)))
    sparse_check(qsa, q, arrays, 4, rng.integers(-1, 960, (3, w)).astype(np.int32), 0.04)


def test_sparse_attn_fp8_first_entries_of_wider_rows(qsa):
    rng = np.random.default_rng(2)
    arrays = (*random_cache(rng, 512, 1, 128, 64), *random_cache(rng, 512, 1, 128, 64))
    slots = rng.integers(0, 512, (2, 400)).astype(np.int32)
    slots[:, 333:] = 10 ** 6  # never looked at
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, 4, 128))), arrays, 64, slots, 0.1, n_idx=333)


def test_sparse_attn_fp8_slot_past_the_cache_is_flagged(qsa):
    rng = np.random.default_rng(5)
    arrays = (*random_cache(rng, 128, 1, 256, 16), *random_cache(rng, 128, 1, 256, 16))
    slots = rng.integers(0, 128, (2, 300)).astype(np.int32)
    slots[1, 7] = 128
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, 8, 256))), arrays, 16, slots, 0.0625, faults=1)


# clusters of 8 CTAs, then shares
@pytest.mark.parametrize("w,g,h_kv,d,shares", [(5000, 4, 1, 128, False), (3000, 8, 2, 256, False), (2500, 11, 1, 128, False),
                                               (20000, 8, 2, 256, True), (30001, 5, 1, 128, True), (70001, 12, 1, 256, True)])
def test_sparse_attn_fp8_long_rows_join_several_ctas(qsa, w, g, h_kv, d, shares):
    rng = np.random.default_rng(w)
    arrays = (*random_cache(rng, 4096, h_kv, d, 64), *random_cache(rng, 4096, h_kv, d, 64))
    assert (qsa.lib().qsa_sparse_attn_fp8_workspace_size(2, g * h_kv, h_kv, d, w) > 0) == shares
    slots = rng.integers(0, 4096, (2, w)).astype(np.int32)
    slots[1, 100:] = -1  # whole CTAs without an entry
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (2, g * h_kv, d))), arrays, 64, slots, 0.05)


@pytest.mark.parametrize("mag", [1e-30, 1e-4, 300.0, 1e30])
def test_sparse_attn_fp8_query_magnitudes(qsa, mag):
    """Queries far outside FP16's range, with a softmax scale that takes the
    magnitude back; a zero head; components far below the largest."""
    import torch
    rng = np.random.default_rng(6)
    arrays = (*random_cache(rng, 320, 1, 128, 16), *random_cache(rng, 320, 1, 128, 16))
    x = rng.standard_normal((2, 12, 128)) * mag
    x[0, 1] = 0
    x[1, 2, 1:] *= 2.0 ** -13
    q = torch.from_numpy(x).to(torch.bfloat16).cuda()
    for h in (12, 4):
        sparse_check(qsa, q[:, :h], arrays, 16, rng.integers(0, 320, (2, 200)).astype(np.int32), 0.09 / mag)


@pytest.mark.parametrize("lo,hi,scale", [(-64, -50, 0.1), (40, 63, 0.1), (-64, 63, 0.1), (-30, 10, 3.0), (-64, 63, -8.0)])
def test_sparse_attn_fp8_v_scales_of_any_size(qsa, lo, hi, scale):
    """V scales far apart and at the ends of their range: the normaliser and
    the weighted sum keep their own magnitudes."""
    rng = np.random.default_rng(hi + 100)
    arrays = (*random_cache(rng, 640, 1, 128, 4), *random_cache(rng, 640, 1, 128, 4, lo, hi))
    slots = np.stack([rng.permutation(640)[:500] for _ in range(4)]).astype(np.int32)
    sparse_check(qsa, bf16_dev(normal_bf16(rng, (4, 8, 128))), arrays, 4, slots, scale)


def test_sparse_attn_fp8_broken_rows_show_only_where_they_are_read(qsa):
    rng = np.random.default_rng(9)
    arrays = [*random_cache(rng, 192, 1, 128, 16), *random_cache(rng, 192, 1, 128, 16)]
    arrays[0][150:, 0, 3] = 0xFF   # NaN in K from slot 150 on
    arrays[2][149, 0, 5] = 0x7F    # and in V of slot 149
    slots = rng.integers(0, 149, (3, 100)).astype(np.int32)
    q = bf16_dev(normal_bf16(rng, (3, 8, 128)))
    sparse_check(qsa, q, arrays, 16, slots, 0.1)
    slots[1, 60], slots[2, 7] = 170, 149
    out, lse = map(host, qsa.sparse_attn_fp8(q, *map(to_dev, arrays), to_dev(slots), 0.1))
    assert np.isfinite(out[0]).all() and np.isnan(out[1]).all() and np.isnan(lse[1]).all()
    assert np.isnan(out[2, :, 5]).all() and np.isnan(out[2]).sum() == 8 and np.isfinite(lse[2]).all()
    slots[1] = 170
    out, lse = map(host, qsa.sparse_attn_fp8(q, *map(to_dev, arrays), to_dev(slots), 0.1))
    assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()


# ------------------------------------------------------------------- windows
def window_check(qsa, rng, lens, page, block, h_q, h_kv, d, window, n_sink, spare_rows=0, max_rows=None, scale=None,
                 arrays=None, ld=0, sample=None):
    """lens: row lengths per request.  Rows behind the last request keep what
    they held."""
    import torch
    ctx = [max([0, *r]) for r in lens]
    n = [len(r) for r in lens]
    rows = sum(n)
    pt, n_slots = page_table(rng, ctx, page)
    cache = [*random_cache(rng, n_slots, h_kv, d, block), *random_cache(rng, n_slots, h_kv, d, block)]
    if arrays is not None:
        arrays(pt, cache)
    flat = np.array([x for r in lens for x in r] + [5] * spare_rows, np.int32)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = bf16_dev(normal_bf16(rng, (rows + spare_rows, h_q + ld, d)))[:, :h_q]
    out = torch.full((rows + spare_rows, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows + spare_rows, h_q), 7.0, device="cuda")
    sc = d ** -0.5 if scale is None else scale
    qsa.window_attn_fp8(q, *map(to_dev, cache), to_dev(start), to_dev(flat), to_dev(pt), page, max([1, *ctx]), window, n_sink,
                        scale, max_rows_per_req=max([1, *n]) if max_rows is None else max_rows, out=out, lse=lse)
    assert qsa.device_status(clear=True) == 0
    kf, vf = ref.values(*cache[:2], block), ref.values(*cache[2:], block)
    ev = cache[3].astype(np.float64) - 127
    qf, o, l = bits_to_f64(q), bits_to_f64(out), host(lse).astype(np.float64)
    parts = 4 if (max([1, *n]) if max_rows is None else max_rows) * (h_q // h_kv) <= 8 else 3
    which = range(rows) if sample is None or rows <= sample else sorted(rng.choice(rows, sample, replace=False))
    for t in which:
        r = int(np.searchsorted(start[1:], t, side="right"))
        s = ref.slots_of(pt[r], window_positions(int(flat[t]), window, n_sink), page)
        ro, rl, tol, tol_l = one_row(qf[t], kf[s], vf[s], ev[s // block], sc, BF16_HALF_STEP, parts)
        same(o[t], ro, tol, (t, flat[t]))
        same(l[t], rl, tol_l, (t, flat[t]))
    assert (o[rows:] == 7.0).all() and (l[rows:] == 7.0).all()


EDGE_LENS = [[0], [1], [2], [], [39], [40], [41], [63, 64, 65], [0, 0, 100], [300, 299], [257]]


@pytest.mark.parametrize("h_q,h_kv,d,page,block", [(16, 2, 256, 64, 64), (5, 1, 256, 4, 4), (8, 4, 128, 16, 8),
                                                   (16, 1, 128, 48, 16), (12, 1, 256, 128, 128), (3, 3, 128, 40, 8)])
@pytest.mark.parametrize("window,n_sink", [(40, 4), (1, 0), (1, 1), (64, 0), (1000, 4), (33, 70)])
@pytest.mark.parametrize("max_rows", [1, 3])
def test_window_attn_fp8_edges(qsa, h_q, h_kv, d, page, block, window, n_sink, max_rows):
    """Row by row, and in tiles of the rows of a request."""
    rng = np.random.default_rng(window * 7 + d + page)
    window_check(qsa, rng, EDGE_LENS, page, block, h_q, h_kv, d, window, n_sink, spare_rows=3, max_rows=max_rows, ld=1)


# 8, 16, 32 and 48 pairs a tile, one request's rows in several tiles, heads that do not divide 16
@pytest.mark.parametrize("h_q,h_kv,d,rows", [(16, 2, 256, 2), (16, 2, 256, 4), (16, 2, 256, 6), (16, 2, 256, 8),
                                             (16, 2, 256, 21), (8, 8, 128, 70), (16, 4, 128, 6), (5, 1, 128, 9),
                                             (16, 1, 256, 3), (7, 1, 256, 30), (16, 2, 128, 2), (16, 2, 128, 4)])
@pytest.mark.parametrize("window,n_sink", [(100, 4), (5000, 0), (37, 130)])
def test_window_attn_fp8_shared_tiles(qsa, h_q, h_kv, d, rows, window, n_sink):
    rng = np.random.default_rng(window + h_q + d + rows)
    lens = [list(range(c - rows + 1, c + 1)) for c in (rows, 331, 1200)] + [[77], [], [0] * rows]
    window_check(qsa, rng, lens, 32, 16, h_q, h_kv, d, window, n_sink, 2, sample=60)


@pytest.mark.parametrize("lens", [[1, 1, 30], [30, 1, 1], [1, 40, 0, 0, 1, 9], [60] + [1] * 9])
@pytest.mark.parametrize("h_q,h_kv,d", [(16, 2, 256), (8, 2, 128)])
def test_window_attn_fp8_more_tiles_than_even_requests_have(qsa, lens, h_q, h_kv, d):
    """Requests of very different numbers of rows: tiles past those that as
    many requests of equal length would have."""
    rng = np.random.default_rng(sum(lens) + d)
    window_check(qsa, rng, [list(range(200, 200 + n)) for n in lens], 32, 32, h_q, h_kv, d, 90, 2, 3, sample=50)


@pytest.mark.parametrize("n_req,h_kv", [(20, 8), (32, 5), (40, 4), (150, 1), (33, 16)])
@pytest.mark.parametrize("d,rows", [(256, 1), (128, 1), (256, 3), (128, 4)])
def test_window_attn_fp8_shares_of_uneven_requests(qsa, n_req, h_kv, d, rows):
    """More units than SMs, cut into equal shares of their blocks: lengths of
    nothing, of one entry, of a block and around it, and long ones."""
    rng = np.random.default_rng(n_req + d + rows)
    some = [0, 1, 127, 128, 129, 256, 257, 600, 3001]
    lens = []
    for i in range(n_req):
        c = some[i % len(some)]
        lens.append([max(0, c - rows + 1 + j) for j in range(1 if i % 7 == 3 else rows)])
    window_check(qsa, rng, lens, 16, 16, 4 * h_kv, h_kv, d, 100000, 0, 2, max_rows=rows, sample=60)


def test_window_attn_fp8_rows_in_any_order(qsa):
    rng = np.random.default_rng(11)
    window_check(qsa, rng, [rng.integers(0, 700, 13).tolist(), [5, 600, 1]], 16, 16, 8, 2, 128, 60, 5)
    window_check(qsa, rng, [rng.integers(0, 700, 13).tolist(), [5, 600, 1]], 16, 16, 16, 2, 256, 60, 5)


@pytest.mark.parametrize("rows,h_q,d", [(1, 8, 256), (1, 16, 128), (6, 8, 256), (3, 4, 128)])
def test_window_attn_fp8_long_rows_join_several_ctas(qsa, rows, h_q, d):
    rng = np.random.default_rng(12 + rows)
    n = 30011
    assert qsa.lib().qsa_window_attn_fp8_workspace_size(rows, 1, rows, h_q, 1, d, n, n, 0) > 0
    window_check(qsa, rng, [list(range(n - rows + 1, n + 1))], 64, 64, h_q, 1, d, n, 0)
    window_check(qsa, rng, [[3] * (rows - 1) + [n]], 64, 64, h_q, 1, d, n, 0)


@pytest.mark.parametrize("scale", [-0.07, 0.0, -30.0, 1e-20])
@pytest.mark.parametrize("rows", [1, 6])
def test_window_attn_fp8_scales(qsa, rows, scale):
    rng = np.random.default_rng(41 + rows)
    window_check(qsa, rng, [list(range(300 - rows, 300))], 32, 32, 8, 2, 128, 150, 3, scale=scale)


@pytest.mark.parametrize("n_req", [33, 1024, 1025, 1400])
def test_window_attn_fp8_many_requests(qsa, n_req):
    """Requests of 0 to 3 rows; tiles are counted up to 1,024 requests and
    found by a search from there on."""
    rng = np.random.default_rng(n_req)
    lens = [rng.integers(0, 60, rng.integers(0, 4)).tolist() for _ in range(n_req)]
    lens[n_req // 2] = list(range(20, 60))
    window_check(qsa, rng, lens, 16, 16, 4, 1, 128, 20, 2, spare_rows=1, max_rows=3, sample=300)


def test_window_attn_fp8_largest_window_and_sinks(qsa):
    rng = np.random.default_rng(47)
    big = 2 ** 31 - 1
    for lens in ([[300]], [list(range(1, 60))]):
        window_check(qsa, rng, lens, 16, 16, 8, 2, 128, big, 0)
        window_check(qsa, rng, lens, 16, 16, 8, 2, 128, big, big)
        window_check(qsa, rng, lens, 16, 16, 8, 2, 128, 1, big)


@pytest.mark.parametrize("rows", [1, 6])
def test_window_attn_fp8_masked_positions_have_no_effect(qsa, rows):
    """NaN in K and V everywhere outside the windows."""
    rng = np.random.default_rng(13)
    ctx, window, n_sink, page = 700, 150, 20, 32

    def poison(pt, cache):
        seen = set()
        for length in range(ctx - rows + 1, ctx + 1):
            seen |= set(ref.slots_of(pt[0], window_positions(length, window, n_sink), page).tolist())
        hide = np.array([s for s in range(cache[0].shape[0]) if s not in seen])
        cache[0][hide[0::2]], cache[2][hide] = 0x7F, 0xFF

    window_check(qsa, rng, [list(range(ctx - rows + 1, ctx + 1))], page, 16, 8, 1, 256, window, n_sink, arrays=poison)
    window_check(qsa, rng, [list(range(ctx - rows + 1, ctx + 1))], page, 16, 8, 2, 128, window, n_sink, arrays=poison)


@pytest.mark.parametrize("h_q,h_kv,d,rows", [(8, 1, 256, 6), (16, 2, 128, 8), (4, 4, 128, 20), (16, 1, 256, 4)])
@pytest.mark.parametrize("window,n_sink", [(5000, 0), (60, 3), (700, 0)])
def test_window_attn_fp8_broken_values_reach_only_the_rows_that_see_them(qsa, h_q, h_kv, d, rows, window, n_sink):
    rng = np.random.default_rng(45 + rows + d)
    page, block, ctx = 32, 32, 1500
    pt, n_slots = page_table(rng, [ctx], page)
    cache = [*random_cache(rng, n_slots, h_kv, d, block), *random_cache(rng, n_slots, h_kv, d, block)]
    q = normal_bf16(rng, (rows, h_q, d))
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    # seen by the last rows, by the second half, and by the first quarter (where its windows begin)
    at_k, at_v = ctx - 1, [p for p in (ctx - 2, ctx - rows // 2, lens[0] + rows // 4 - window) if p >= 0]
    cache[0][ref.slots_of(pt[0], np.array([at_k]), page)[0], :, 5] = 0x7F
    cols = []
    for i, p in enumerate(at_v):
        cols.append(np.arange(7 + i, d, 16))
        cache[2][ref.slots_of(pt[0], np.array([p]), page)[0], :, 7 + i::16] = 0xFF
    out, lse = qsa.window_attn_fp8(bf16_dev(q), *map(to_dev, cache), to_dev(np.array([0, rows], np.int32)), to_dev(lens),
                                   to_dev(pt), page, ctx, window, n_sink, max_rows_per_req=rows)
    o, l = bits_to_f64(out), host(lse).astype(np.float64)
    clean = [c.copy() for c in cache]
    clean[2][clean[2] == 0xFF] = 0
    kf, vf = ref.values(*clean[:2], block), ref.values(*clean[2:], block)
    ev = cache[3].astype(np.float64) - 127
    for t in range(rows):
        pos = window_positions(lens[t], window, n_sink)
        if at_k in pos:
            assert np.isnan(o[t]).all() and np.isnan(l[t]).all()
            continue
        s = ref.slots_of(pt[0], pos, page)
        ro, rl, tol, tol_l = one_row(ref.bf16_to_f64(q[t]), kf[s], vf[s], ev[s // block], d ** -0.5, BF16_HALF_STEP, 3)
        for p, c in zip(at_v, cols):
            if p in pos:
                ro[:, c] = np.nan
        assert np.array_equal(np.isnan(o[t]), np.isnan(ro)), t
        fin = ~np.isnan(ro)
        assert (np.abs(o[t] - ro)[fin] <= tol[fin]).all()
        same(l[t], rl, tol_l, t)


@pytest.mark.parametrize("rows", [1, 6])
@pytest.mark.parametrize("d", [128, 256])
def test_window_attn_fp8_bad_pages_are_skipped_and_flagged(qsa, rows, d):
    """Pages outside the cache: those that a row attends to fault and are left
    out, the others may hold anything."""
    rng = np.random.default_rng(14 + rows)
    ctx, page, window, n_sink = 900, 64, 300, 10
    pt, n_slots = page_table(rng, [ctx], page)
    cache = [*random_cache(rng, n_slots, 1, d, 64), *random_cache(rng, n_slots, 1, d, 64)]
    q = normal_bf16(rng, (rows, 8, d))
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    args = (to_dev(np.array([0, rows], np.int32)), to_dev(lens))
    kf, vf = ref.values(*cache[:2], 64), ref.values(*cache[2:], 64)
    ev = cache[3].astype(np.float64) - 127
    for gone, faults in (([3, 5], 0), ([3, 11], 1), ([0], 1), ([14, 9], 1)):
        bad = pt.copy()
        bad[0, gone] = rng.choice([n_slots // page, -7, 2 ** 31 - 1], len(gone))
        out, lse = qsa.window_attn_fp8(bf16_dev(q), *map(to_dev, cache), *args, to_dev(bad), page, ctx, window, n_sink,
                                       max_rows_per_req=rows)
        assert qsa.device_status(clear=True) == faults
        for t in range(rows):
            pos = window_positions(lens[t], window, n_sink)
            s = ref.slots_of(pt[0], pos[~np.isin(pos // page, gone)], page)
            ro, rl, tol, tol_l = one_row(ref.bf16_to_f64(q[t]), kf[s], vf[s], ev[s // 64], d ** -0.5, BF16_HALF_STEP, 4 if rows == 1 else 3)
            same(bits_to_f64(out)[t], ro, tol, t)
            same(host(lse)[t].astype(np.float64), rl, tol_l, t)


@pytest.mark.parametrize("rows", [1, 5])
def test_window_attn_fp8_bad_row_lengths_count_as_zero(qsa, rows):
    rng = np.random.default_rng(15)
    pt, n_slots = page_table(rng, [100], 16)
    cache = [*random_cache(rng, n_slots, 2, 128, 16), *random_cache(rng, n_slots, 2, 128, 16)]
    q = bf16_dev(normal_bf16(rng, (rows, 8, 128)))
    lens = np.full(rows, 100, np.int32)
    lens[0] = 101
    lens[-1] = -4
    out, lse = qsa.window_attn_fp8(q, *map(to_dev, cache), to_dev(np.array([0, rows], np.int32)), to_dev(lens), to_dev(pt), 16,
                                   100, 50, max_rows_per_req=rows)
    assert qsa.device_status(clear=True) == 8
    o, l = bits_to_f64(out), host(lse)
    for t in (0, rows - 1):
        assert (o[t] == 0).all() and np.isneginf(l[t]).all()
    assert rows == 1 or (np.isfinite(l[1:-1]).all() and (o[1:-1] != 0).any())


@pytest.mark.parametrize("rows", [1, 6])
def test_offsets_past_32_bits(qsa, rows):
    """A cache of more than 4 GB: blocks near its end written, read back and
    attended to."""
    import torch
    rng = np.random.default_rng(16)
    h_kv, d, page, n_slots = 8, 256, 64, 2_200_000 // 64 * 64
    cache = [torch.zeros((n_slots, h_kv, d), dtype=torch.uint8, device="cuda"),
             torch.full((n_slots // 64, h_kv), 127, dtype=torch.uint8, device="cuda")]
    cache += [t.clone() for t in cache]
    assert cache[0].numel() > 2 ** 32
    n, last = 130, n_slots // page
    pt = np.array([[last - 1, 5, last - 2]], np.int32)
    bits = [normal_bf16(rng, (n, h_kv, d)) for _ in range(2)]
    qsa.append_kv_fp8(*map(bf16_dev, bits), to_dev(np.array([0, n], np.int32)), to_dev(np.array([0], np.int32)), *cache,
                      to_dev(pt), page)
    slots = ref.slots_of(pt[0], np.arange(n), page)
    small = [np.zeros((192, h_kv, d), np.uint8), np.full((3, h_kv), 127, np.uint8)]
    small += [a.copy() for a in small]
    for i in (0, 1):
        ref.append(small[2 * i], small[2 * i + 1], bits[i], np.arange(n), 64, 0)
    k, v = qsa.gather_kv_fp8(*cache, to_dev(slots.astype(np.int32)))
    kf, vf = ref.values(*small[:2], 64)[:n], ref.values(*small[2:], 64)[:n]
    assert np.array_equal(bits_to_f64(k), kf) and np.array_equal(bits_to_f64(v), vf)
    q = normal_bf16(rng, (rows, 8, d))
    out, _ = qsa.window_attn_fp8(bf16_dev(q), *cache, to_dev(np.array([0, rows], np.int32)),
                                 to_dev(np.full(rows, n, np.int32)), to_dev(pt), page, n, n, max_rows_per_req=rows)
    lst = np.broadcast_to(slots.astype(np.int32), (rows, n)).copy()
    out2, _ = qsa.sparse_attn_fp8(bf16_dev(q), *cache, to_dev(lst))
    ev = np.repeat(small[3], 64, 0)[:n].astype(np.float64) - 127
    for t in range(rows):
        ro, _, tol, _ = one_row(ref.bf16_to_f64(q[t]), kf, vf, ev, d ** -0.5, BF16_HALF_STEP, 4)
        same(bits_to_f64(out)[t], ro, tol, t)
        same(host(out2)[t].astype(np.float64), ro, tol, t)


# ------------------------------------------------------- as they are used together
@pytest.mark.parametrize("captured", [False, True])
def test_decode_steps_from_plan_to_attention(qsa, captured):
    """Steps of a few requests, as a server makes them: rows, slots and pages
    planned on the device, K and V appended, a window layer and a selection
    read from the 8-bit cache, and the step's pages given back at the end."""
    import torch
    rng = np.random.default_rng(17)
    page, block, h_q, h_kv, d, window, n_sink = 16, 16, 8, 2, 128, 50, 4
    n_req, n_tok, n_pages = 3, 40, 40
    n_slots = n_pages * page
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((n_req, 12), -1, dtype=torch.int32, device="cuda")
    free = to_dev(rng.permutation(n_pages).astype(np.int32))
    n_free, ctx, new = to_dev(np.array([n_pages], np.int32)), i32(n_req), i32(n_req)
    cache = [torch.zeros((n_slots, h_kv, d), dtype=torch.uint8, device="cuda"),
             torch.full((n_pages, h_kv), 63, dtype=torch.uint8, device="cuda")]
    cache += [t.clone() for t in cache]
    k_new, v_new = (torch.zeros((n_tok, h_kv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((n_tok, h_q, d), dtype=torch.bfloat16, device="cuda")
    sel = torch.full((n_tok, 30), -1, dtype=torch.int32, device="cuda")

    def step():
        start, new_len, row_len, row_req, slots = qsa.plan_step(ctx, new, table, page, free, n_free, n_tok)
        qsa.append_kv_fp8(k_new, v_new, start, ctx, *cache, table, page)
        w = qsa.window_attn_fp8(q, *cache, start, row_len, table, page, 12 * page, window, n_sink, max_rows_per_req=8)
        s = qsa.sparse_attn_fp8(q, *cache, sel)
        back = qsa.gather_kv_fp8(*cache, slots)
        ctx.copy_(new_len)
        return start, row_len, slots, *w, *s, *back

    if captured:
        step()  # not inside the capture: first calls of a process look devices up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
    small = [c.cpu().numpy().copy() for c in cache]
    h_table, h_free, h_n, h_ctx = table.cpu().numpy().copy(), free.cpu().numpy(), n_pages, np.zeros(n_req, np.int64)
    for it, counts in enumerate(([30, 0, 7], [1, 9, 1], [2, 3, 0], [6, 1, 6], [1, 1, 1])):
        counts = np.array(counts)
        start_h, len_h, rl_h, _, sl_h, h_table, h_n, bits = ref.plan(h_ctx, counts, h_table, page, h_free, h_n, n_tok)
        assert bits == 0
        kb, vb = (normal_bits(rng, (n_tok, h_kv, d), 2.0 ** rng.integers(-2, 3, (n_tok, 1, 1))) for _ in range(2))
        qb = normal_bf16(rng, (n_tok, h_q, d))
        seen = np.full((n_tok, 30), -1, np.int32)
        for r in range(n_req):
            for t in range(start_h[r], start_h[r + 1]):
                pos = np.sort(rng.permutation(int(rl_h[t]))[:25])
                seen[t, :len(pos)] = ref.slots_of(h_table[r], pos, page)
        for dst, src in ((k_new, kb), (v_new, vb), (q, qb)):
            dst.copy_(bf16_dev(src))
        new.copy_(to_dev(counts.astype(np.int32)))
        sel.copy_(to_dev(seen))
        if captured:
            g.replay()
        else:
            outs = step()
        start, row_len, slots, wo, wl, so, sl, bk, bv = map(host, outs)
        assert np.array_equal(start, start_h) and np.array_equal(row_len, rl_h) and np.array_equal(slots, sl_h)
        assert np.array_equal(table.cpu().numpy(), h_table) and int(n_free) == h_n
        for r in range(n_req):
            rows = slice(start_h[r], start_h[r + 1])
            for i, b in ((0, kb), (1, vb)):
                ref.append(small[2 * i], small[2 * i + 1], b[rows], sl_h[rows], block, int(h_ctx[r]))
        kf, vf, ev = ref.values(*small[:2], block), ref.values(*small[2:], block), small[3].astype(np.float64) - 127
        total = start_h[-1]
        assert np.array_equal(ref.bf16_to_f64(bk)[:total], kf[sl_h[:total]]) and (bk[total:] == 0).all()
        assert np.array_equal(ref.bf16_to_f64(bv)[:total], vf[sl_h[:total]])
        for r in range(n_req):
            for t in range(start_h[r], start_h[r + 1]):
                qt = ref.bf16_to_f64(qb[t])
                for got, gl, at, eps in (
                        (ref.bf16_to_f64(wo[t]), wl[t], ref.slots_of(h_table[r], window_positions(int(rl_h[t]), window, n_sink),
                                                                     page), BF16_HALF_STEP),
                        (so[t].astype(np.float64), sl[t], seen[t][seen[t] >= 0], 2.0 ** -24)):
                    ro, rl, tol, tol_l = one_row(qt, kf[at], vf[at], ev[at // block], d ** -0.5, eps, 3 if eps == BF16_HALF_STEP else 4)
                    same(got, ro, tol, (it, t))
                    same(gl.astype(np.float64), rl, tol_l, (it, t))
        h_ctx = len_h.astype(np.int64)
    end = to_dev((-(-h_ctx // page)).astype(np.int32))
    qsa.release_pages(table, i32(n_req), end, free, n_free)
    assert int(n_free) == n_pages and (table == -1).all() and sorted(free.tolist()) == list(range(n_pages))


def test_first_calls_inside_a_capture():
    """In a fresh process, the first call of each kind is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch, sparse_attention_indexer_index_gb300 as qsa
z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
u8, bf = torch.uint8, torch.bfloat16
c = [z(64, 1, 128, dt=u8), z(4, 1, dt=u8) + 120] * 2
c = [t.clone() for t in c]
pt, start, ctx, new = z(1, 4), z(2), z(1), z(1) + 5
free, n = torch.arange(4, dtype=torch.int32, device="cuda"), z(1) + 4
x, q = z(5, 1, 128, dt=bf) + 1, z(5, 4, 128, dt=bf) + 1
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    start, new_len, row_len, _, slots = qsa.plan_step(ctx, new, pt, 16, free, n, 5)
    qsa.append_kv_fp8(x, x, start, ctx, *c, pt, 16)
    out, _ = qsa.window_attn_fp8(q, *c, start, row_len, pt, 16, 64, 64)
    out2, _ = qsa.sparse_attn_fp8(q, *c, slots.view(5, 1))
    k, v = qsa.gather_kv_fp8(*c, slots)
g.replay()
torch.cuda.synchronize()
assert qsa.device_status() == 0
assert all((t == 1).all() for t in (out, out2, k, v)) and int(n) == 3 and slots.tolist() == [48, 49, 50, 51, 52]
print("ok")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr[-2000:]


def test_graphs_sharing_a_workspace(qsa):
    """Two captured graphs that split long rows over the same workspace, in
    turn on one stream."""
    import torch
    rng = np.random.default_rng(43)
    arrays = list(map(to_dev, (*random_cache(rng, 4096, 1, 128, 64), *random_cache(rng, 4096, 1, 128, 64))))
    q = [bf16_dev(normal_bf16(rng, (2, 8, 128))) for _ in range(2)]
    slots = [to_dev(rng.integers(0, 4096, (2, n)).astype(np.int32)) for n in (20000, 12000)]
    need = max(qsa.lib().qsa_sparse_attn_fp8_workspace_size(2, 8, 1, 128, s.shape[1]) for s in slots)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = [[t.clone() for t in qsa.sparse_attn_fp8(q[i], *arrays, slots[i])] for i in range(2)]
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(qsa.sparse_attn_fp8(q[i], *arrays, slots[i], workspace=ws))
    for i in (0, 1, 1, 0, 1, 0):
        graphs[i].replay()
    torch.cuda.synchronize()
    for got, exp in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, exp))


def test_calls_on_two_streams_at_once(qsa):
    import torch
    rng = np.random.default_rng(21)
    arrays = list(map(to_dev, (*random_cache(rng, 4096, 2, 256, 64), *random_cache(rng, 4096, 2, 256, 64))))
    q = [bf16_dev(normal_bf16(rng, (4, 16, 256))) for _ in range(2)]
    slots = [to_dev(rng.integers(0, 4096, (4, 9000)).astype(np.int32)) for _ in range(2)]
    want = [qsa.sparse_attn_fp8(q[i], *arrays, slots[i])[0].clone() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for i, s in enumerate(streams):
            got.append((i, qsa.sparse_attn_fp8(q[i], *arrays, slots[i], stream=s)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)


def test_same_call_twice_gives_the_same_bits(qsa):
    import torch
    rng = np.random.default_rng(22)
    arrays = list(map(to_dev, (*random_cache(rng, 4096, 2, 128, 32), *random_cache(rng, 4096, 2, 128, 32))))
    q = bf16_dev(normal_bf16(rng, (6, 8, 128)))
    slots = to_dev(rng.integers(-1, 4096, (6, 2051)).astype(np.int32))
    runs = [qsa.sparse_attn_fp8(q, *arrays, slots) for _ in range(5)]
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_binding_refusals(qsa):
    import torch
    z = lambda *s, dt=torch.uint8, dev="cuda": torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    cache = dict(k_codes=z(64, 2, 128), k_scales=z(4, 2), v_codes=z(64, 2, 128), v_scales=z(4, 2))
    broken = [("k_codes", z(64, 2, 64)), ("k_scales", z(3, 2)), ("v_scales", z(4, 1)), ("v_codes", z(64, 2, 128, dt=torch.int8)),
              ("v_codes", z(64, 2, 128, dev="cpu")), ("k_scales", z(8))]
    app = dict(k_new=z(3, 2, 128, dt=bf), v_new=z(3, 2, 128, dt=bf), req_tok_start=z(2, dt=i32), req_first_pos=z(1, dt=i32),
               page_table=z(1, 4, dt=i32), page_size=16)
    gat = dict(slots=z(5, dt=i32))
    spa = dict(q=z(3, 4, 128, dt=bf), slots=z(3, 7, dt=i32))
    win = dict(q=z(3, 4, 128, dt=bf), req_row_start=z(2, dt=i32), row_len=z(3, dt=i32), page_table=z(1, 4, dt=i32),
               page_size=16, max_len=64, window=9)
    for fn, args, bad in (
            (qsa.append_kv_fp8, app, [("k_new", z(3, 2, 128, dt=f32)), ("v_new", z(2, 2, 128, dt=bf)),
                                      ("req_first_pos", z(2, dt=i32)), ("page_table", z(1, 4, dt=torch.int64))]),
            (qsa.gather_kv_fp8, gat, [("slots", z(5, dt=torch.int64)), ("k_out", z(5, 2, 64, dt=bf)),
                                      ("v_out", z(5, 2, 128, dt=f32))]),
            (qsa.sparse_attn_fp8, spa, [("q", z(3, 4, 64, dt=bf)), ("slots", z(2, 7, dt=i32)), ("out", z(3, 4, 128, dt=bf)),
                                        ("lse", z(3, 4, dt=bf)), ("workspace", z(64, dev="cpu"))]),
            (qsa.window_attn_fp8, win, [("q", z(3, 4, 256, dt=bf)), ("row_len", z(4, dt=i32)), ("out", z(3, 4, 128, dt=f32)),
                                        ("req_row_start", z(3, dt=i32))])):
        fn(**args, **cache)
        for k, v in bad:
            with pytest.raises((TypeError, ValueError)):
                fn(**{**args, **cache, k: v})
        for k, v in broken:
            with pytest.raises((TypeError, ValueError)):
                fn(**{**args, **cache, k: v})
        # 64 slots in 3 or 32 blocks: sizes that are no block
        with pytest.raises((ValueError, qsa.QSAError)):
            fn(**args, **{**cache, "k_scales": z(32, 2), "v_scales": z(32, 2)})
    with pytest.raises(qsa.QSAError):
        qsa.window_attn_fp8(**{**win, "page_size": 8}, **cache)  # a block longer than the page


def test_empty_calls(qsa):
    import torch
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    i32, bf = torch.int32, torch.bfloat16
    cache = [z(64, 2, 128), z(4, 2), z(64, 2, 128), z(4, 2)]
    qsa.append_kv_fp8(z(0, 2, 128, dt=bf), z(0, 2, 128, dt=bf), z(2, dt=i32), z(1, dt=i32), *cache, z(1, 4, dt=i32), 16)
    k, _ = qsa.gather_kv_fp8(*cache, z(0, dt=i32))
    assert k.shape == (0, 2, 128)
    out, lse = qsa.sparse_attn_fp8(z(0, 4, 128, dt=bf), *cache, z(0, 7, dt=i32))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    out, lse = qsa.sparse_attn_fp8(z(2, 4, 128, dt=bf), *cache, z(2, 0, dt=i32))
    assert (out == 0).all() and torch.isneginf(lse).all()
    out, _ = qsa.window_attn_fp8(z(0, 4, 128, dt=bf), *cache, z(2, dt=i32), z(0, dt=i32), z(1, 4, dt=i32), 16, 64, 9)
    assert out.shape == (0, 4, 128)
