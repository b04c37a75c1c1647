"""Calls whose inputs the kernel before them is still writing: it lets its
dependents in first, waits a while and only then writes.  What the calls read
must be what it wrote."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from gpu_util import bf16_dev, to_dev
from test_gpu_kv4 import no_fault_left, page_table, qsa, random_cache4  # noqa: F401
from workloads.synth import normal_bf16

pytestmark = pytest.mark.gpu

# A copy that lets dependent launches in before it writes.  The wait is bounded
# by the clock; 8 CTAs leave room for the dependents beside it.
LATE_COPY = r"""
#include <cuda_runtime.h>
__global__ void late_copy_kernel(const uint4* src, uint4* dst, long long n, long long clocks) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t0 = clock64();
  while (clock64() - t0 < clocks) {
  }
  for (long long i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) dst[i] = src[i];
}
extern "C" int late_copy(const void* src, void* dst, long long bytes, long long clocks, void* stream) {
  late_copy_kernel<<<8, 256, 0, (cudaStream_t)stream>>>((const uint4*)src, (uint4*)dst, bytes / 16, clocks);
  return (int)cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def late_copy(tmp_path_factory):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    d = tmp_path_factory.mktemp("late")
    src, lib = d / "late.cu", d / "late.so"
    src.write_text(LATE_COPY)
    subprocess.run([nvcc, "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-Xcompiler", "-fPIC", "-o",
                    str(lib), str(src)], check=True, capture_output=True)
    fn = ctypes.CDLL(str(lib)).late_copy
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_void_p]
    return fn


class Arena:
    """Inputs in one buffer, so that one copy replaces them all."""

    def __init__(self, first, second):
        import torch
        offs, size = [], 0
        for t in first:
            offs.append(size)
            size += -(-t.numel() * t.element_size() // 256) * 256
        self.bufs = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(3)]  # live, first, second
        for buf, ts in zip(self.bufs[1:], (first, second)):
            for o, t in zip(offs, ts):
                n = t.numel() * t.element_size()
                buf[o:o + n] = t.contiguous().view(torch.uint8).reshape(-1)
        self.views = [self.bufs[0][o:o + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
                      for o, t in zip(offs, first)]

    def set(self, which):
        import torch
        self.bufs[0].copy_(self.bufs[which])
        torch.cuda.synchronize()

    def set_late(self, late_copy, which, clocks=200_000):  # 100 us
        import torch
        assert late_copy(self.bufs[which].data_ptr(), self.bufs[0].data_ptr(), self.bufs[0].numel(), clocks,
                         torch.cuda.current_stream().cuda_stream) == 0


def check_late(late_copy, first, second, call, clear=lambda: None):
    """call(views) -> tensors, on inputs that arrive late; it launches nothing
    but the library's kernels.  clear() resets what it updates in place."""
    import torch
    arena = Arena(first, second)
    arena.set(2)
    clear()
    want = [t.clone() for t in call(arena.views)]
    arena.set(1)
    clear()
    assert not all(torch.equal(a, b) for a, b in zip(call(arena.views), want))  # the inputs matter
    for _ in range(4):
        clear()
        arena.set(1)
        arena.set_late(late_copy, 2)
        got = call(arena.views)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("n_tok", [3, 700])
def test_append_reads_rows_that_arrive_late(qsa, late_copy, n_tok):  # noqa: F811
    import torch
    rng = np.random.default_rng(60)
    h_kv, d, page, n_slots = 2, 256, 64, 2048

    def inputs():
        cut = int(rng.integers(1, n_tok))
        pt = rng.permutation(n_slots // page).astype(np.int32).reshape(2, -1)
        return [bf16_dev(normal_bf16(rng, (n_tok, h_kv, d))), bf16_dev(normal_bf16(rng, (n_tok, h_kv, d))),
                to_dev(np.array([0, cut, n_tok], np.int32)), to_dev(rng.integers(0, 60, 2).astype(np.int32)), to_dev(pt)]

    cache = [torch.zeros((n_slots, h_kv, w), dtype=torch.uint8, device="cuda") for w in (128, 16, 128, 16)]
    check_late(late_copy, inputs(), inputs(), lambda x: qsa.append_kv_fp4(*x[:4], *cache, x[4], page),
               lambda: [c.zero_() for c in cache])


@pytest.mark.parametrize("n", [5, 6000])
def test_gather_reads_slots_and_rows_that_arrive_late(qsa, late_copy, n):  # noqa: F811
    rng = np.random.default_rng(61)

    def inputs():
        return [*map(to_dev, (*random_cache4(rng, 512, 2, 128), *random_cache4(rng, 512, 2, 128))),
                to_dev(rng.integers(-1, 512, n).astype(np.int32))]

    check_late(late_copy, inputs(), inputs(), lambda x: qsa.gather_kv_fp4(*x))


@pytest.mark.parametrize("rows,w,h_q,h_kv,d", [(1, 2051, 16, 2, 256), (7, 300, 16, 1, 128), (1, 20000, 8, 1, 128)])
def test_sparse_attn_fp4_reads_inputs_that_arrive_late(qsa, late_copy, rows, w, h_q, h_kv, d):  # noqa: F811
    rng = np.random.default_rng(62)

    def inputs():
        return [bf16_dev(normal_bf16(rng, (rows, h_q, d))),
                *map(to_dev, (*random_cache4(rng, 512, h_kv, d), *random_cache4(rng, 512, h_kv, d))),
                to_dev(rng.integers(-1, 512, (rows, w)).astype(np.int32))]

    check_late(late_copy, inputs(), inputs(), lambda x: qsa.sparse_attn_fp4(*x))


@pytest.mark.parametrize("rows,max_rows,ctx", [(1, 1, 700), (3, 1, 700), (24, 24, 700), (2, 17, 90), (1, 1, 20000)])
@pytest.mark.parametrize("fp4", [False, True])
def test_window_attn_reads_inputs_that_arrive_late(qsa, late_copy, rows, max_rows, ctx, fp4):  # noqa: F811
    rng = np.random.default_rng(63)
    page, h_q, h_kv, d = 64, 8, 2, 128

    def inputs():
        lens = np.sort(rng.integers(ctx // 2, ctx + 1, 2 * rows)).astype(np.int32)
        cut = int(rng.integers(1, 2 * rows))
        pt = rng.integers(0, 40, (2, -(-ctx // page))).astype(np.int32)
        if fp4:
            cache = [*map(to_dev, (*random_cache4(rng, 40 * page, h_kv, d), *random_cache4(rng, 40 * page, h_kv, d)))]
        else:
            cache = [bf16_dev(normal_bf16(rng, (40 * page, h_kv, d))) for _ in range(2)]
        return [bf16_dev(normal_bf16(rng, (2 * rows, h_q, d))), *cache, to_dev(np.array([0, cut, 2 * rows], np.int32)),
                to_dev(lens), to_dev(pt)]

    fn = qsa.window_attn_fp4 if fp4 else qsa.window_attn
    window = ctx if ctx > 1000 else 100
    check_late(late_copy, inputs(), inputs(), lambda x: fn(*x, page, ctx, window, 3, max_rows_per_req=max_rows))


@pytest.mark.parametrize("lens,page", [([[4099, 4100, 4101], [1030]], 64), ([[800], [900], [33]], 8),
                                       ([list(range(3000, 3064))], 64)])
def test_indexer_reads_inputs_that_arrive_late(qsa, late_copy, lens, page):  # noqa: F811
    """Scores and selection: a verify step, single rows on small pages, a chunk."""
    import torch
    from workloads import decode_workload

    def inputs(seed):
        w = decode_workload(seed, lens, page_size=page, k_blk=512)
        pool = normal_bf16(np.random.default_rng(seed), (w.pool_rows, 128))
        return w, [bf16_dev(w.q), bf16_dev(pool), *map(to_dev, (w.req_row_start, w.row_len, w.page_table))]

    (w, first), (_, second) = inputs(64), inputs(65)
    assert all(a.shape == b.shape for a, b in zip(first, second))
    scores = torch.zeros((w.n_rows, -(-w.max_len // 4)), device="cuda")

    def call(x):
        out = qsa.indexer_select(*x, page, w.max_len, w.max_rows_per_req, k_blk=512, want_blocks=True, scores_out=scores)
        return out["blocks"], out["slots"]

    check_late(late_copy, first, second, call)
    # scores past a row's length are not written
    check_late(late_copy, first, second,
               lambda x: [qsa.index_scores(*x, page, w.max_len, w.max_rows_per_req, scores=scores)], scores.zero_)
