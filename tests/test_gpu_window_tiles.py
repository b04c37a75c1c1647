"""window_attn in its tensor-core form, where roles of a CTA and the CTAs of a
cluster have to keep out of each other's way."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import bf16_dev, to_dev
from test_gpu_kv4 import (BF16_HALF_STEP, W_BF16, bits_to_f64, host, no_fault_left, page_table,  # noqa: F401
                          qsa, window_check)
from workloads.synth import normal_bf16

pytestmark = pytest.mark.gpu


def check_clean_rows(qsa, q, k, v, pt, lens, page, max_len, window, n_sink, broken, rows=None):  # noqa: F811
    """One request of len(lens) rows in tiles; positions `broken` hold infinities
    or NaN: rows that see none of them get the formula's values.  Returns how many."""
    d = q.shape[-1]
    n = len(lens)
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(np.array([0, n], np.int32)), to_dev(lens), to_dev(pt),
                               page, max_len, window, n_sink, max_rows_per_req=max(n, 17))
    o, l, kf, vf = bits_to_f64(out), host(lse).astype(np.float64), ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    clean = 0
    for t in range(n) if rows is None else rows:
        pos = ref.window_positions(lens[t], window, n_sink)
        if np.isin(broken, pos).any():
            continue
        clean += 1
        sl = ref.slots_of(pt[0], pos, page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, pos.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(o[t] - ro) <= tol).all(), t
        assert (np.abs(l[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all(), t
    return clean


@pytest.mark.parametrize("h_q,d,rows", [(3, 256, 42), (3, 256, 40), (7, 128, 17), (3, 128, 37), (1, 256, 90)])
@pytest.mark.parametrize("window", [300, 500, 1200])
def test_broken_values_in_a_shared_tile_of_odd_size(qsa, h_q, d, rows, window):  # noqa: F811
    """Tiles whose pairs do not fill whole passes of the join's threads."""
    rng = np.random.default_rng(50 + rows + window)
    page, ctx = 32, 1500
    pt, n_slots = page_table(rng, [ctx], page)
    k, v, q = (normal_bf16(rng, s) for s in ((n_slots, 1, d), (n_slots, 1, d), (rows, h_q, d)))
    lens = np.arange(ctx - rows + 1, ctx + 1).astype(np.int32)
    lens = lens[rng.permutation(rows)]
    lens[-1] = ctx - rows + 1  # the tile's last row sees none of them
    broken = [ctx - 1, ctx - 2, ctx - rows // 2]
    for i, p in enumerate(broken):
        v[ref.slots_of(pt[0], np.array([p]), page)[0], 0, i::2] = (0x7FC0, 0x7F80, 0xFF80)[i]
    assert check_clean_rows(qsa, q, k, v, pt, lens, page, ctx, window, 2, broken) >= rows // 4


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("ctx", [65_601, 262_209])
def test_broken_values_in_a_long_window_hold_up_the_next_tile(qsa, ctx, d):  # noqa: F811
    """A tile of 16 heads and 8 rows over a long window, the last row's own V
    broken: the other rows are summed once more, entry by entry, for longer than
    the limit of a wait, while the CTA's other roles wait with the next tile."""
    rng = np.random.default_rng(51 + d)
    page, h_q, n_req, own = 64, 128 * 16 // d, 170, 40
    rows = 128 // h_q
    n_pages = -(-ctx // page)
    pt = np.full((n_req, n_pages), -1, np.int32)
    pt[0] = rng.integers(0, own, n_pages)  # positions share pages: they are only read
    pt[0, -1] = own                        # but for the last, which holds the broken one
    pt[1:, :2] = rng.integers(0, own, (n_req - 1, 2))
    k, v = (normal_bf16(rng, ((own + 1) * page, 1, d)) for _ in range(2))
    v[ref.slots_of(pt[0], np.array([ctx - 1]), page)[0], 0, ::3] = 0x7FC0
    lens = np.concatenate([np.arange(ctx - rows + 1, ctx + 1)] + [np.arange(91, 91 + rows)] * (n_req - 1)).astype(np.int32)
    q = normal_bf16(rng, (rows * n_req, h_q, d))
    start = (np.arange(n_req + 1) * rows).astype(np.int32)
    out, lse = qsa.window_attn(*map(bf16_dev, (q, k, v)), to_dev(start), to_dev(lens), to_dev(pt), page, ctx, ctx,
                               max_rows_per_req=17)
    assert qsa.device_status() == 0
    o, l, kf, vf = bits_to_f64(out), host(lse).astype(np.float64), ref.bf16_to_f64(k), ref.bf16_to_f64(v)
    assert np.isnan(o[rows - 1][:, ::3]).all()
    for t in [0, rows - 2, *range(rows, rows * n_req, 97)]:
        r = t // rows
        sl = ref.slots_of(pt[r], np.arange(lens[t]), page)
        ro, rl, a, big, spread = ref.attend(ref.bf16_to_f64(q[t]), kf[sl], vf[sl], d ** -0.5)
        tol, tol_l = ref.tolerance(d, sl.size, ro, a, big, spread, W_BF16, BF16_HALF_STEP, False, 0.0)
        assert (np.abs(o[t] - ro) <= tol).all(), t
        assert (np.abs(l[t] - rl) <= tol_l + 2.0 ** -23 * np.abs(rl)).all(), t


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("d,page", [(128, 64), (256, 16)])
@pytest.mark.parametrize("rows,max_rows", [(2, 1), (2, 17), (20, 20)])
@pytest.mark.parametrize("n_sink", [0, 3])
def test_pages_that_no_row_attends_to_may_be_gone(qsa, rows, max_rows, d, page, fp4, n_sink):  # noqa: F811
    """Rows of a request whose windows lie apart: the pages between them, which
    were given back, are no fault; a page that a row attends to is one."""
    rng = np.random.default_rng(52)
    window, near, far = 64, 200, 2000

    def gone(pt, cache):
        for r in range(2):
            lens = [near] + [far - i for i in range(rows - 1)]
            seen = np.unique(np.concatenate([ref.window_positions(x, window, n_sink) for x in lens]) // page)
            keep = np.isin(np.arange(pt.shape[1]), seen)
            pt[r, ~keep] = np.where(np.arange((~keep).sum()) % 2, -1, 2**31 - 1)
        return cache

    lens = [[near] + [far - i for i in range(rows - 1)]] * 2
    window_check(qsa, rng, lens, page, 8, 1, d, window, n_sink, fp4, cache=gone, max_rows=max_rows)
    assert qsa.device_status() == 0

    def one_more(pt, cache):
        gone(pt, cache)
        pt[1, (near - 1) // page] = -1
        return cache

    pt, n_slots = page_table(rng, [far, far], page)
    k, v = (bf16_dev(normal_bf16(rng, (n_slots, 1, d))) for _ in range(2))
    one_more(pt, None)
    q = bf16_dev(normal_bf16(rng, (2 * rows, 8, d)))
    qsa.window_attn(q, k, v, to_dev(np.array([0, rows, 2 * rows], np.int32)), to_dev(np.array(sum(lens, []), np.int32)),
                    to_dev(pt), page, far, window, n_sink, max_rows_per_req=max_rows)
    assert qsa.device_status(clear=True) == 1
