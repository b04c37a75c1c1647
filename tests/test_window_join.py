"""The join of a tile that a cluster shares (tensor-core form of window_attn),
without a GPU: who writes which 8 columns of which pair.

A vector that holds a sum spoilt by a neighbour's infinity is written, and then
summed and written once more by its warp.  So no thread of another warp may
write it: nothing orders the two."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc", "window_tc.cuh")).read()
JOIN = SRC[SRC.index("void wt_join("):SRC.index("window_tc_kernel(")]


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("cluster", [2, 4, 8])
def test_every_vector_is_written_by_one_thread(d, cluster):
    guard = r"if \(own\) \*reinterpret_cast<uint4\*>\(a\.out"
    assert "for (int i0 = 0; i0 < n; i0 += 256)" in JOIN
    assert len(re.findall(r"\*reinterpret_cast<uint4\*>\(a\.out", JOIN)) == 1
    only_own = re.search(guard, JOIN) is not None and "const bool own = i0 + (int)threadIdx.x < n;" in JOIN
    vecs = d // cluster // 8
    for pairs in range(1, 129):
        n = pairs * vecs
        writers = [0] * n
        for i0 in range(0, n, 256):
            for tid in range(256):
                if i0 + tid < n or not only_own:
                    writers[min(i0 + tid, n - 1)] += 1
        assert writers == [1] * n, (pairs, writers[-1])
