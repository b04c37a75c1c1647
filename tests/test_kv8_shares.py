"""Shares of the blocks of all units (8-bit cache attention), without a GPU:
the kernel numbers the blocks in 32 bits, so a call whose blocks may be more,
whatever its rows' lengths are, is dealt in another way.  Whether shares are
taken shows in the workspace that a call wants."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def L():
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.build()
    return qsa.lib()


def most_blocks(slots, h_kv, span, block):
    """All blocks that the kernel may number: two more to every (tile, KV head)."""
    return slots * h_kv * (max(1, -(-span // block)) + 2)


def test_rows_far_apart_in_a_long_context(L):
    """A tile's rows may lie in any order, and its window then spans all of the
    context: 100 requests of 6 rows in windows of 16,384."""
    w = L.qsa_window_attn_fp8_workspace_size
    assert w(600, 100, 6, 32, 4, 256, 131072, 16384, 0) > 0
    assert most_blocks(200, 4, 2 ** 30, 128) > 2 ** 31
    assert w(600, 100, 6, 32, 4, 256, 2 ** 30, 16384, 0) == 0


@pytest.mark.parametrize("seed", range(20))
def test_blocks_are_counted_in_32_bits(L, seed):
    rng = np.random.default_rng(seed)
    shared = 0
    for _ in range(400):
        d, h_kv, group = int(rng.choice([128, 256])), int(rng.choice([1, 2, 4, 8, 16])), int(rng.choice([1, 3, 4, 8, 12, 16]))
        n_req = int(2 ** rng.uniform(0, 11))
        n_rows = int(n_req * 2 ** rng.uniform(0, 4))
        max_len, window = int(2 ** rng.uniform(10, 30.01)), int(2 ** rng.uniform(10, 31)) - 1
        max_rows = int(rng.choice([1, 2, 4, 6, 30]))
        max_len = min(max_len, 2 ** 30)
        pairs = max_rows * group
        single = max_rows == 1 and group <= 8
        rows = 1 if single else next(n for n in (8, 16, 32, 48) if pairs <= n or n == 48) // group
        block = 256 if d == 128 and (single or pairs <= 16) else 128
        if L.qsa_window_attn_fp8_workspace_size(n_rows, n_req, max_rows, group * h_kv, h_kv, d, max_len, window, 4) > 0:
            shared += 1
            slots = n_rows if single else min(n_rows, n_rows // rows + n_req)
            span = min(max_len, window + 4) if rows == 1 else max_len
            assert most_blocks(slots, h_kv, span, block) < 2 ** 31
        n_idx = max_len
        if L.qsa_sparse_attn_fp8_workspace_size(n_rows, group * h_kv, h_kv, d, n_idx) > 0:
            assert most_blocks(n_rows, h_kv, n_idx, 256 if d == 128 else 128) < 2 ** 31
    assert shared > 20
