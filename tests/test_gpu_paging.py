"""plan_step and release_pages on the GPU against host loops (kv8_ref), to the
bit: ragged and empty requests, lists that run out, rows that do not fit,
broken lengths, captured graphs."""
import numpy as np
import pytest

import kv8_ref as ref
from gpu_util import to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import torch
    assert torch.cuda.is_available()
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.lib()
    qsa.device_status(clear=True)
    return qsa


def state(rng, ctx, new, page, spare=5, width=None, gaps=True):
    """A table that holds the pages of ctx, and a list of free ones."""
    held, end = -(-ctx // page), -(-(ctx + np.maximum(new, 0)) // page)
    total = int(np.maximum(held, 0).sum()) + int(np.maximum(end - held, 0).sum()) + spare
    perm = rng.permutation(total).astype(np.int32)
    table = np.full((len(ctx), width or int(end.max(initial=0)) + 2), -1, np.int32)
    off = 0
    for r, h in enumerate(held):
        h = min(max(int(h), 0), table.shape[1])
        table[r, :h] = perm[off:off + h]
        off += h
    n_free = total - off
    free = np.concatenate([perm[off:], rng.integers(-9, 9, 7 if gaps else 0).astype(np.int32)])
    return table, free, n_free


def check(qsa, ctx, new, table, page, free, n_free, n_tok, want_faults=0):
    want = ref.plan(ctx, new, table, page, free, n_free, n_tok)
    assert want[7] == want_faults
    d_table, d_free, d_n = to_dev(table), to_dev(free), to_dev(np.array([n_free], np.int32))
    got = qsa.plan_step(to_dev(np.asarray(ctx, np.int32)), to_dev(np.asarray(new, np.int32)), d_table, page, d_free, d_n, n_tok)
    for g, w, name in zip((*got, d_table), want, ("start", "new_len", "row_len", "row_req", "slots", "table")):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert qsa.device_status(clear=True) == want[7]
    assert np.array_equal(d_free.cpu().numpy(), free)
    if want[6] != n_free or 0 <= n_free <= len(free):
        assert int(d_n) == want[6]
    return want


# requests in one group of 32, one round of groups and more; rows in the kernel's own CTA and beside it
@pytest.mark.parametrize("n_req,most,page", [(1, 1, 4), (1, 9000, 64), (7, 40, 16), (32, 1, 64), (33, 6, 12), (100, 0, 64),
                                             (1000, 7, 16), (1024, 4, 4), (1025, 3, 64), (3000, 9, 16), (40, 700, 128)])
@pytest.mark.parametrize("pad", [0, 77])
def test_plan_step(qsa, n_req, most, page, pad):
    rng = np.random.default_rng(n_req + most)
    ctx = rng.integers(0, 300, n_req)
    ctx[::3] -= ctx[::3] % page  # full pages
    new = rng.integers(0, most + 1, n_req) if most > 1 else np.full(n_req, most)
    table, free, n_free = state(rng, ctx, new, page)
    check(qsa, ctx, new, table, page, free, n_free, int(new.sum()) + pad)


@pytest.mark.parametrize("n_req", [20, 65, 2000])
def test_plan_step_requests_without_rows_between(qsa, n_req):
    rng = np.random.default_rng(n_req)
    new = np.zeros(n_req, np.int64)
    new[rng.integers(0, n_req, 5)] = rng.integers(1, 90, 5)
    new[-1] = 3
    ctx = rng.integers(0, 99, n_req)
    table, free, n_free = state(rng, ctx, new, 8)
    check(qsa, ctx, new, table, 8, free, n_free, int(new.sum()) + 40)


@pytest.mark.parametrize("n_req", [9, 1500])
@pytest.mark.parametrize("short", [1, 7, 10 ** 6])
def test_plan_step_refuses_when_the_list_runs_out(qsa, n_req, short):
    rng = np.random.default_rng(n_req + short)
    ctx, new = rng.integers(0, 60, n_req), rng.integers(0, 30, n_req)
    new[n_req // 2:] = np.minimum(new[n_req // 2:], 16 - ctx[n_req // 2:] % 16) * (ctx[n_req // 2:] % 16 > 0)  # need no page
    table, free, n_free = state(rng, ctx, new, 16, spare=0)
    out = check(qsa, ctx, new, table, 16, free, max(n_free - short, 0), int(new.sum()), 16)
    assert (out[1][n_req // 2:] == ctx[n_req // 2:] + new[n_req // 2:]).all()  # those are served


@pytest.mark.parametrize("n_req", [9, 1500])
@pytest.mark.parametrize("cut", [1, 25, 10 ** 6])
def test_plan_step_refuses_rows_past_the_outputs(qsa, n_req, cut):
    rng = np.random.default_rng(n_req + cut)
    ctx, new = rng.integers(0, 60, n_req), rng.integers(1, 30, n_req)
    table, free, n_free = state(rng, ctx, new, 16)
    check(qsa, ctx, new, table, 16, free, n_free, max(int(new.sum()) - cut, 0), 16)


def test_plan_step_broken_lengths(qsa):
    """Negative lengths, a request past its row of the table or past 2^31, a
    page that is missing: each is refused, the others served."""
    rng = np.random.default_rng(3)
    ctx = np.array([5, -1, 7, 20, 2 ** 31 - 2, 30, 0, 2 ** 31 - 1])
    new = np.array([3, 2, -4, 50, 5, 4, 6, 2 ** 31 - 1])
    small = np.where(np.arange(8) == 3, 20, np.clip(ctx, 0, 40))
    table, free, n_free = state(rng, small, np.clip(new, 0, 6), 8, width=6)
    table[5, 3] = -1
    table[4] = 0
    check(qsa, ctx, new, table, 8, free, n_free, 90, 1 | 8 | 16)
    check(qsa, ctx[:7], new[:7], table[:7], 8, free, n_free, 90, 1 | 8)


def test_plan_step_huge_counts_do_not_wrap(qsa):
    """Sums of rows and of pages far past 32 bits."""
    n_req = 3000
    ctx, new = np.zeros(n_req, np.int64), np.full(n_req, 2 ** 31 - 1)
    new[:3] = [5, 4, 0]
    table = np.full((n_req, 4), -1, np.int32)
    free = np.arange(8, dtype=np.int32)
    check(qsa, ctx, new, table, 4, free, 8, 20, 1 | 16)
    # rows longer than any context: pages past 32 bits too
    import torch
    wide = torch.full((8, 1 << 26), -1, dtype=torch.int32, device="cuda")
    i32 = lambda a: to_dev(np.array(a, np.int32))  # noqa: E731
    n = i32([8])
    new = [3, 200000000, 200000000, 200000000, 200000000, 200000000, 200000000, 1]
    got = qsa.plan_step(i32([0] * 8), i32(new), wide, 4, i32(list(range(8))), n, 2 ** 30 // 64)
    assert qsa.device_status(clear=True) == 16
    assert got[0].tolist() == [0, 3] + [2 ** 30 // 64] * 7 and got[1].tolist() == [3] + [0] * 7 and int(n) == 7
    assert int((wide >= 0).sum()) == 1


@pytest.mark.parametrize("n_free", [-1, 9])
def test_plan_step_list_length_out_of_range(qsa, n_free):
    table = np.full((2, 3), -1, np.int32)
    table[0, 0] = 2
    free = np.arange(8, dtype=np.int32)
    n = to_dev(np.array([n_free], np.int32))
    got = qsa.plan_step(to_dev(np.array([1, 0], np.int32)), to_dev(np.array([2, 2], np.int32)), to_dev(table), 4, to_dev(free),
                        n, 5)
    assert qsa.device_status(clear=True) == 8 | 16
    assert got[1].tolist() == [3, 0] and got[4].tolist() == [9, 10, -1, -1, -1] and int(n) == n_free


def test_plan_step_of_nothing(qsa):
    import torch
    e = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    n = to_dev(np.array([0], np.int32))
    got = qsa.plan_step(e(0), e(0), e(0, 4), 16, e(0), n, 3)
    assert [g.tolist() for g in got] == [[0], [], [0, 0, 0], [-1] * 3, [-1] * 3]
    got = qsa.plan_step(e(2).fill_(5), e(2).zero_(), e(2, 4), 16, e(0), n, 0)
    assert got[0].tolist() == [0, 0, 0] and got[1].tolist() == [5, 5] and qsa.device_status(clear=True) == 0


def check_release(qsa, table, lo, hi, free, n_free, want_faults=0):
    want = ref.release(table, lo, hi, free, n_free)
    assert want[3] == want_faults
    d = [to_dev(np.asarray(a, np.int32)) for a in (table, lo, hi, free, [n_free])]
    got = qsa.release_pages(*d)
    assert got[0] is d[0] and got[1] is d[3] and got[2] is d[4]
    assert np.array_equal(d[0].cpu().numpy(), want[0]) and np.array_equal(d[3].cpu().numpy(), want[1])
    assert int(d[4]) == want[2] and qsa.device_status(clear=True) == want[3]


@pytest.mark.parametrize("n_req,most", [(1, 1), (1, 3000), (31, 4), (33, 9), (1024, 6), (1025, 5), (2500, 70)])
def test_release_pages(qsa, n_req, most):
    rng = np.random.default_rng(n_req + most)
    width = most + 3
    table = rng.integers(-1, 10 ** 6, (n_req, width)).astype(np.int32)
    table[rng.random(table.shape) < 0.2] = -7
    lo = rng.integers(0, 4, n_req)
    hi = np.minimum(lo + rng.integers(-1, most + 1, n_req), width)
    pool = table.size + 9
    free = rng.integers(0, 99, pool).astype(np.int32)
    check_release(qsa, table, lo, hi, free, 9)


@pytest.mark.parametrize("n_req", [40, 1100])
@pytest.mark.parametrize("room", [0, 1, 13])
def test_release_pages_past_the_list(qsa, n_req, room):
    rng = np.random.default_rng(n_req + room)
    table = rng.integers(0, 10 ** 6, (n_req, 40)).astype(np.int32)
    lo, hi = np.full(n_req, 1), rng.integers(1, 40, n_req)
    check_release(qsa, table, lo, hi, np.zeros(room + 5, np.int32), 5, 16)


def test_release_pages_ranges_out_of_the_row(qsa):
    table = np.arange(30, dtype=np.int32).reshape(5, 6)
    check_release(qsa, table, [-1, 0, 4, 5, 2], [3, 7, 4, 6, 5], np.zeros(30, np.int32), 0, 1)
    check_release(qsa, table, [0, 0, 0, 0, 0], [1, 1, 1, 1, 1], np.zeros(30, np.int32), -3, 8 | 16)


def test_a_step_taken_back_leaves_list_and_table(qsa):
    rng = np.random.default_rng(5)
    ctx, new = rng.integers(0, 500, 77), rng.integers(0, 40, 77)
    table, free, n_free = state(rng, ctx, new, 16)
    d_t, d_f, d_n = to_dev(table), to_dev(free), to_dev(np.array([n_free], np.int32))
    qsa.plan_step(to_dev(ctx.astype(np.int32)), to_dev(new.astype(np.int32)), d_t, 16, d_f, d_n, 4000)
    qsa.release_pages(d_t, to_dev((-(-ctx // 16)).astype(np.int32)), to_dev((-(-(ctx + new) // 16)).astype(np.int32)), d_f, d_n)
    assert np.array_equal(d_t.cpu().numpy(), table) and np.array_equal(d_f.cpu().numpy(), free) and int(d_n) == n_free


@pytest.mark.parametrize("n_tok", [64, 5000])
def test_steps_in_a_captured_graph(qsa, n_tok):
    """A graph of one step, replayed: every replay plans from the lengths that
    the one before left."""
    import torch
    rng = np.random.default_rng(6)
    ctx, new = rng.integers(0, 50, 9), rng.integers(0, 5, 9)
    table = np.full((9, 40), -1, np.int32)
    off = 0
    for r, c in enumerate(ctx):
        h = -(-int(c) // 4)
        table[r, :h] = np.arange(off, off + h)
        off += h
    free = rng.permutation(np.arange(off, off + 90)).astype(np.int32)
    d = [to_dev(a.astype(np.int32)) for a in (ctx, new)]
    d_t, d_f, d_n = to_dev(table), to_dev(free), to_dev(np.array([90], np.int32))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = qsa.plan_step(*d, d_t, 4, d_f, d_n, n_tok)
        d[0].copy_(out[1])
    n_free = 90
    for _ in range(4):
        want = ref.plan(ctx, new, table, 4, free, n_free, n_tok)
        g.replay()
        for a, b in zip((*out, d_t), want):
            assert np.array_equal(a.cpu().numpy(), b)
        ctx, table, n_free = want[1], want[5], want[6]
        assert int(d_n) == n_free and qsa.device_status(clear=True) == 0


def test_on_another_stream_and_into_given_buffers(qsa):
    import torch
    rng = np.random.default_rng(8)
    ctx, new = rng.integers(0, 50, 40), rng.integers(0, 5, 40)
    table, free, n_free = state(rng, ctx, new, 8)
    want = ref.plan(ctx, new, table, 8, free, n_free, 200)
    d = [to_dev(a.astype(np.int32)) for a in (ctx, new)]
    d_t, d_f, d_n = to_dev(table), to_dev(free), to_dev(np.array([n_free], np.int32))
    row_len = torch.empty(200, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = qsa.plan_step(*d, d_t, 8, d_f, d_n, 200, row_len=row_len, stream=s)
    assert out[2] is row_len
    s.synchronize()
    for a, b in zip((*out, d_t), want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_binding_refusals(qsa):
    import torch
    z = lambda *s, dt=torch.int32, dev="cuda": torch.zeros(s, dtype=dt, device=dev)  # noqa: E731
    ok = dict(ctx_len=z(3), n_new=z(3), page_table=z(3, 4), page_size=16, free_pages=z(5), n_free=z(1), n_tok=6)
    qsa.plan_step(**ok)
    for k, v in [("ctx_len", z(4)), ("n_new", z(3, dt=torch.int64)), ("page_table", z(12)), ("page_table", z(4, 3).t()),
                 ("free_pages", z(5, 1)), ("n_free", z(2)), ("n_free", z(1, dev="cpu")), ("ctx_len", z(3, dev="cpu"))]:
        with pytest.raises((TypeError, ValueError)):
            qsa.plan_step(**{**ok, k: v})
    for k, v in [("slots", z(5)), ("new_len", z(4)), ("row_len", z(6, dt=torch.int64)), ("req_row_start", z(3)),
                 ("row_req", z(12)[::2])]:
        with pytest.raises((TypeError, ValueError)):
            qsa.plan_step(**ok, **{k: v})
    with pytest.raises(qsa.QSAError):
        qsa.plan_step(**{**ok, "page_size": 10})
    with pytest.raises(qsa.QSAError):
        qsa.plan_step(**ok, new_len=ok["ctx_len"])
    ok = dict(page_table=z(3, 4), from_page=z(3), to_page=z(3), free_pages=z(5), n_free=z(1))
    qsa.release_pages(**ok)
    for k, v in [("from_page", z(4)), ("to_page", z(3, dt=torch.int64)), ("page_table", z(12)), ("n_free", z(0)),
                 ("free_pages", z(5, 1))]:
        with pytest.raises((TypeError, ValueError)):
            qsa.release_pages(**{**ok, k: v})
    assert qsa.device_status(clear=True) == 0
