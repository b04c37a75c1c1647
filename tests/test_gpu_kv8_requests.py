"""window_attn_fp8 on batches of more than 1,024 requests: every row is
written, whatever the requests' numbers of rows, the heads and
max_rows_per_req, and holds what FP64 says."""
import numpy as np
import pytest

import kv8_ref as ref
from gpu_util import bf16_dev, to_dev
from test_gpu_kv8 import BF16_HALF_STEP, bits_to_f64, host, page_table, random_cache, same
from workloads.synth import normal_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    import torch
    assert torch.cuda.is_available()
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.lib()
    qsa.device_status(clear=True)
    return qsa


def check(qsa, seed, counts, h_q, h_kv, d, max_rows, spare=1, compare=None):
    import torch
    rng = np.random.default_rng(seed)
    page, block, window, n_sink, n_req = 16, 16, 20, 2, len(counts)
    lens = [rng.integers(0, 48, c) for c in counts]
    pt, n_slots = page_table(rng, [max([0, *x]) for x in lens], page)
    pt = np.pad(pt, ((0, 0), (0, 3 - pt.shape[1])), constant_values=-1)
    cache = [*random_cache(rng, n_slots, h_kv, d, block), *random_cache(rng, n_slots, h_kv, d, block)]
    rows = int(np.sum(counts))
    flat = np.concatenate([*lens, np.full(spare, 5)]).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    bits = normal_bf16(rng, (rows + spare, h_q, d))
    out = torch.full((rows + spare, h_q, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows + spare, h_q), 7.0, device="cuda")
    kw = {} if max_rows is None else dict(max_rows_per_req=max_rows)
    qsa.window_attn_fp8(bf16_dev(bits), *map(to_dev, cache), to_dev(start), to_dev(flat), to_dev(pt), page, 48, window,
                        n_sink, out=out, lse=lse, **kw)
    assert qsa.device_status(clear=True) == 0
    o, l = bits_to_f64(out), host(lse).astype(np.float64)
    assert (l[:rows] != 7.0).all(), f"{int((l[:rows] == 7.0).any(1).sum())} of {rows} rows unwritten"
    assert (o[rows:] == 7.0).all() and (l[rows:] == 7.0).all()
    # FP64, all rows at once: each with room for the 22 entries that it may have
    kf, vf, ev = ref.values(*cache[:2], block), ref.values(*cache[2:], block), cache[3].astype(np.float64) - 127
    req, which = np.repeat(np.arange(n_req), counts), np.arange(rows)
    if compare is not None and rows > compare:
        which = np.sort(rng.choice(rows, compare, replace=False))
    L, width = flat[which].astype(np.int64)[:, None], window + n_sink
    first = np.maximum(L - window, 0)
    sinks = np.minimum(first, n_sink)
    e = np.arange(width)[None]
    pos = np.where(e < sinks, e, first + e - sinks)
    there = pos < L
    pos = np.where(there, pos, 0)
    s = np.where(there, pt[req[which][:, None], pos // page].astype(np.int64) * page + pos % page, 0)
    group = h_q // h_kv
    qf = ref.bf16_to_f64(bits[which]).reshape(-1, h_kv, group, d)
    k, v = kf[s], vf[s]                                         # [rows][22][h_kv][d]
    x = np.einsum("thgd,tjhd->thgj", qf, k) * d ** -0.5
    x = np.where(there[:, None, None], x, -np.inf)
    m = x.max(-1, initial=-1e300, keepdims=True)
    w = np.exp(x - m)
    z = w.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        rl = np.where(z > 0, m + np.log(z), -np.inf).reshape(-1)
    w = np.where(z > 0, w / np.where(z > 0, z, 1.0), 0.0)
    flatten = lambda a: a.reshape(len(which) * h_q, *a.shape[3:])  # noqa: E731
    ro, a = flatten(np.einsum("thgj,tjhd->thgd", w, v)), flatten(np.einsum("thgj,tjhd->thgd", w, np.abs(v)))
    far = there[:, None, None]
    big = flatten((np.einsum("thgd,tjhd->thgj", np.abs(qf), np.abs(k)) * far).max(-1, initial=0.0)) * d ** -0.5
    spread = flatten(np.abs(qf).max(-1) * (np.abs(k).sum(-1) * there[..., None]).max(1, initial=0.0)[:, :, None]) * d ** -0.5
    top = flatten((w * np.exp2(ev[s // block]).transpose(0, 2, 1)[:, :, None]).max(-1, initial=0.0))
    tol, tol_l = ref.tolerance(d, width, ro, a, big, spread, BF16_HALF_STEP, np.abs(ev).max(), top, 4)
    same(o[which].reshape(-1, d), ro, tol, "out")
    same(l[which].reshape(-1), rl, tol_l + 2.0 ** -23 * np.where(np.isfinite(rl), np.abs(rl), 0.0), "lse")


@pytest.mark.parametrize("n_req", [1025, 1100, 2000])
@pytest.mark.parametrize("h_q,h_kv,d", [(8, 1, 256), (16, 1, 128)])
@pytest.mark.parametrize("max_rows", [1, 2, 6, None])
def test_one_row_a_request(qsa, n_req, h_q, h_kv, d, max_rows):
    check(qsa, n_req + h_q, np.ones(n_req, np.int64), h_q, h_kv, d, max_rows)


@pytest.mark.parametrize("n_req", [1025, 2000])
@pytest.mark.parametrize("h_q,h_kv", [(8, 1), (16, 1), (8, 2)])
@pytest.mark.parametrize("max_rows", [1, 2, 6, None])
def test_requests_of_no_or_one_row(qsa, n_req, h_q, h_kv, max_rows):
    check(qsa, n_req, np.random.default_rng(n_req).integers(0, 2, n_req), h_q, h_kv, 128, max_rows)


@pytest.mark.parametrize("n_req,some", [(1025, 3), (3000, 1), (3000, 40), (1100, 0)])
@pytest.mark.parametrize("h_q,max_rows", [(8, 6), (16, 1), (4, 3)])
def test_few_rows_among_many_requests(qsa, n_req, some, h_q, max_rows):
    rng = np.random.default_rng(some)
    counts = np.zeros(n_req, np.int64)
    counts[rng.choice(n_req, some, replace=False)] = rng.integers(1, max_rows + 3, some)
    if some == 0:
        counts[[0, -1]] = 1
    check(qsa, some, counts, h_q, 1, 128, max_rows)


@pytest.mark.parametrize("n_req", [1025, 1500])
@pytest.mark.parametrize("most", [2, 3, 9])
@pytest.mark.parametrize("h_q", [4, 16])
def test_requests_of_some_rows(qsa, n_req, most, h_q):
    counts = np.random.default_rng(most).integers(0, most + 1, n_req)
    counts[n_req // 2] = 40
    check(qsa, most, counts, h_q, 1, 128, most, compare=4000)


def test_as_many_requests_as_there_may_be(qsa):
    counts = (np.random.default_rng(1).random(65535) < 0.04).astype(np.int64)
    counts[-1] = 1
    check(qsa, 1, counts, 8, 1, 128, 2)
