"""The tiles of window_attn_fp8's requests, without a GPU: how many slots the
host gives them, and which tile the kernel finds in each.  Both rules are read
from the sources and replayed: every row belongs to exactly one tile."""
import os
import re

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc")
KERNEL = open(os.path.join(CSRC, "kv8_tc.cuh")).read()
HOST = open(os.path.join(CSRC, "kv8_api.cu")).read()
FIND = KERNEL[KERNEL.index("int k8_find("):KERNEL.index("kv8_tc_kernel(const")]
FORM = HOST[HOST.index("K8Form window_form("):HOST.index("constexpr size_t kJobBytes")]
EXACT = int(re.search(r"constexpr int kK8Exact = (\d+);", KERNEL).group(1))


def tile_rows(max_rows, group):
    """Rows to a tile, as window_form has it."""
    assert "const int kind = pairs <= 8 ? kTile8 : pairs <= 16 ? kTile16 : pairs <= 32 ? kTile32 : kTile48;" in FORM
    pairs = max(max_rows, 1) * group
    return next(n for n in (8, 16, 32, 48) if pairs <= n or n == 48) // group


def tile_slots(n_rows, n_req, rows):
    """The host's slots: the lesser of the rows and the requests' room."""
    if "k8_tile_slots(n_rows, n_req, rows)" in FORM:
        f = KERNEL[KERNEL.index("k8_tile_slots("):]
        assert "n_rows / R + n_req" in f and "return n_rows < by_request ? n_rows : by_request;" in f
    else:
        assert "std::min<int64_t>(n_rows, n_rows / rows + (int64_t)n_req)" in FORM
    return min(n_rows, n_rows // rows + n_req)


def find(start, s, rows, slots):
    """k8_find: (request, tile of it) in slot s, None where there is none."""
    n_req, n_rows = len(start) - 1, int(start[-1])
    tiles = -(-np.diff(start) // rows)
    if n_req <= EXACT:
        assert "if (a.n_req <= kK8Exact) {" in FIND
        ends = np.cumsum(tiles)
        r = int(np.searchsorted(ends, s, side="right"))
        return (r, s - int(ends[r] - tiles[r])) if r < n_req else None
    if "if (a.tile_slots == a.n_rows) {" in FIND and slots == n_rows:  # by their first rows
        r = int(np.searchsorted(start, s, side="right")) - 1
        if r >= n_req:
            return None
        assert "in == rank * a.rows" in FIND
        rank, rest = divmod(s - int(start[r]), rows)
        return (r, rank) if rest == 0 and rank < tiles[r] else None
    assert "/ a.rows + lo + i <= s" in FIND and "rank = s - (ld_in(a.req_row_start + lo) / a.rows + lo);" in FIND
    at = start // rows + np.arange(n_req + 1)
    lo = int(np.searchsorted(at, s, side="right")) - 1
    if lo >= n_req:
        return None
    rank = s - int(at[lo])
    return (lo, rank) if 0 <= rank < tiles[lo] else None


def check(counts, group, max_rows):
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
    n_rows, n_req, rows = int(start[-1]), len(counts), tile_rows(max_rows, group)
    slots = tile_slots(n_rows, n_req, rows)
    seen = np.zeros(n_rows, np.int64)
    for s in range(slots):
        f = find(start, s, rows, slots)
        if f is not None:
            t0 = int(start[f[0]]) + f[1] * rows
            seen[t0:min(t0 + rows, int(start[f[0] + 1]))] += 1
    assert (seen == 1).all(), f"{int((seen != 1).sum())} of {n_rows} rows ({n_req} requests, {rows} rows a tile)"


@pytest.mark.parametrize("n_req", [1, 33, 1024, 1025, 1100, 2000])
@pytest.mark.parametrize("group", [1, 5, 8, 16])
@pytest.mark.parametrize("max_rows", [1, 2, 6, 10 ** 6])
def test_one_row_a_request(n_req, group, max_rows):
    check(np.ones(n_req, np.int64), group, max_rows)


@pytest.mark.parametrize("seed", range(60))
def test_every_row_is_in_one_tile(seed):
    rng = np.random.default_rng(seed)
    n_req = int(rng.choice([3, 700, 1024, 1025, 1300, 3000]))
    most = int(rng.choice([1, 1, 2, 3, 9, 40]))
    counts = rng.integers(0, most + 1, n_req) * (rng.random(n_req) < rng.choice([1.0, 0.5, 0.01]))
    counts[rng.integers(n_req)] += 1
    check(counts, int(rng.choice([1, 2, 4, 5, 8, 12, 16])), int(rng.choice([1, 2, 3, 6, 30])))
