"""append_kv_fp4 with n_tok beyond the last request's rows, over buffers that
end with those rows."""
import numpy as np
import pytest

import kv4_ref as ref
from gpu_util import bf16_dev, to_dev
from test_gpu_kv4 import host, no_fault_left, qsa  # noqa: F401
from workloads.synth import normal_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("h_kv,d", [(1, 128), (2, 256), (3, 128)])
@pytest.mark.parametrize("counts", [[5], [0], [3, 0, 4], [1] * 40, [0, 7, 0]])
@pytest.mark.parametrize("n_tok", [8, 40, 3001])
def test_rows_behind_the_last_request_need_not_exist(qsa, h_kv, d, counts, n_tok):  # noqa: F811
    import torch
    rng = np.random.default_rng(70 + h_kv + n_tok)
    n, page = sum(counts), 16
    n_tok = max(n_tok, n)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    first = rng.integers(0, 20, len(counts)).astype(np.int32)
    pt = rng.permutation(4 * len(counts)).astype(np.int32).reshape(len(counts), 4)
    n_slots = pt.size * page
    k, v = (normal_bf16(rng, (max(n, 1), h_kv, d)) for _ in range(2))
    kd, vd = bf16_dev(k), bf16_dev(v)
    cache = [torch.full((n_slots, h_kv, w), 0x55, dtype=torch.uint8, device="cuda") for w in (d // 2, d // 16) * 2]
    row = h_kv * d
    sd, fd, ptd = map(to_dev, (start, first, pt))
    st = qsa.lib().qsa_append_kv_fp4(kd.data_ptr(), vd.data_ptr(), row, row, n_tok, h_kv, d, sd.data_ptr(), fd.data_ptr(),
                                     len(counts), ptd.data_ptr(), 4, page, 1.0, 0.5, *(c.data_ptr() for c in cache), n_slots,
                                     torch.cuda.current_stream().cuda_stream)
    assert st == 0
    want = [np.full(c.shape, 0x55, np.uint8) for c in cache]
    for r, m in enumerate(counts):
        for i in range(m):
            s = ref.slots_of(pt[r], np.array([first[r] + i]), page)[0]
            for j, (x, g) in enumerate(((k, 1.0), (v, 0.5))):
                want[2 * j][s], want[2 * j + 1][s] = ref.quantise(x[start[r] + i], g)
    for got, exp in zip(cache, want):
        assert np.array_equal(host(got), exp)
