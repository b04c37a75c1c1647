"""The 8-bit KV cache and the paging calls without a GPU: the test reference
against closed forms, and the C ABI's refusals (no call here reaches a CUDA
launch)."""
import ctypes
import os

import numpy as np
import pytest

import kv8_ref as ref
from workloads.synth import bf16_bits


@pytest.fixture(scope="module")
def L():
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.build()
    return qsa.lib()


FAKE = ctypes.c_void_p(0x1000)
OTHER = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1010)  # 16-byte but not 32-byte aligned
BAD = ctypes.c_void_p(0x1002)
F = ctypes.c_float


# ------------------------------------------------------------ the reference
def test_codes_match_torch():
    import torch
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 60, np.arange(-460, 460) / 2.0 ** 9, [0.0, -0.0, 448.0, -448.0]])
    want = torch.from_numpy(x.clip(-448, 448)).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref.encode(x.astype(np.float32).astype(np.float64))
    assert np.array_equal(got, want)
    assert np.array_equal(ref.decode(got), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_exponents():
    assert ref.exponent(448.0) == 0 and ref.exponent(448.5) == 1 and ref.exponent(224.0) == -1
    assert ref.exponent(0.0) == -64 and ref.exponent(3e38) == 63


def test_append_keeps_and_grows_the_scale():
    codes, scales = np.zeros((8, 1, 16), np.uint8), np.zeros((2, 1), np.uint8)
    x = np.zeros((3, 1, 16), np.float32)
    x[0, 0, :3] = [448.0, 0.0146484375, -1.0]  # 7.5 * 2^-9: between two subnormal codes, to the even one
    x[1, 0, 0] = 100.0
    x[2, 0, 0] = 900.0                           # two binades and a bit more: 2^2
    ref.append(codes, scales, bf16_bits(x[:1]), np.array([4]), 4, 0)
    assert scales[1, 0] == 127 and ref.values(codes, scales, 4)[4, 0, :3].tolist() == [448.0, 2.0 ** -6, -1.0]
    ref.append(codes, scales, bf16_bits(x[1:2]), np.array([5]), 4, 1)
    assert scales[1, 0] == 127 and ref.values(codes, scales, 4)[5, 0, 0] == 96.0  # a tie between 96 and 104
    ref.append(codes, scales, bf16_bits(x[2:]), np.array([6]), 4, 2)
    v = ref.values(codes, scales, 4)
    assert scales[1, 0] == 129 and v[4, 0, :3].tolist() == [448.0, 2.0 ** -6, -1.0] and v[6, 0, 0] == 896.0
    assert (codes[:4] == 0).all() and scales[0, 0] == 0


def test_plan_reference_closed_form():
    table = np.full((2, 4), -1, np.int32)
    table[0, 0] = 9
    out = ref.plan([3, 0], [2, 5], table, 4, np.array([7, 5, 6, 8, 4], np.int32), 4, 8)
    start, new_len, row_len, row_req, slots, t, n_free, bits = out
    assert bits == 0 and n_free == 1 and t.tolist() == [[9, 5, -1, -1], [6, 8, -1, -1]]
    assert start.tolist() == [0, 2, 7] and new_len.tolist() == [5, 5]
    assert row_len.tolist() == [4, 5, 1, 2, 3, 4, 5, 0] and row_req.tolist() == [0, 0, 1, 1, 1, 1, 1, -1]
    assert slots.tolist() == [39, 20, 24, 25, 26, 27, 32, -1]


# --------------------------------------------------------------- refusals
def append(L, k=FAKE, v=FAKE, ld_k=512, ld_v=512, n_tok=3, h_kv=2, d=256, start=FAKE, first=FAKE, n_req=1, pt=FAKE,
           ld_pt=4, page=64, block=64, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_slots=256):
    return L.qsa_append_kv_fp8(k, v, ld_k, ld_v, n_tok, h_kv, d, start, first, n_req, pt, ld_pt, page, block, kc, ks, vc,
                               vs, n_slots, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=64), -2), (dict(d=192), -2), (dict(page=6), -2), (dict(n_req=70000), -2), (dict(n_tok=(1 << 30) + 1), -2),
    (dict(block=2), -2), (dict(block=48), -2), (dict(block=128), -2), (dict(block=256, page=256), -2), (dict(block=0), -2),
    (dict(block=-4), -2), (dict(n_slots=200), -1), (dict(page=0), -1), (dict(page=-64), -1),
    (dict(k=None), -1), (dict(start=None), -1), (dict(first=None), -1), (dict(pt=None), -1),
    (dict(k=BAD), -1), (dict(v=BAD), -1), (dict(ld_k=511), -1), (dict(ld_k=516), -1), (dict(ld_v=256), -1),
    (dict(kc=None), -1), (dict(vs=None), -1), (dict(vc=BAD), -1), (dict(n_slots=-64), -1), (dict(n_tok=-1), -1),
    (dict(h_kv=0), -1), (dict(n_slots=1 << 31), -1), (dict(n_req=-1), -1), (dict(h_kv=65536), -2),
    (dict(n_tok=0, k=None), 0), (dict(n_req=0, start=None), 0)])
def test_append_refusals(L, change, status):
    assert append(L, **change) == status


def gather(L, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_slots=256, h_kv=2, d=256, block=16, slots=FAKE, n=3, ko=FAKE,
           vo=FAKE):
    return L.qsa_gather_kv_fp8(kc, ks, vc, vs, n_slots, h_kv, d, block, slots, n, ko, vo, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=96), -2), (dict(block=3), -2), (dict(n_slots=250), -1), (dict(slots=None), -1), (dict(slots=BAD), -1),
    (dict(ko=None), -1), (dict(vo=ODD), -1), (dict(kc=BAD), -1), (dict(ks=None), -1), (dict(n=-1), -1),
    (dict(n=1 << 50), -2), (dict(h_kv=0), -1), (dict(n=0, slots=None, ko=None), 0)])
def test_gather_refusals(L, change, status):
    assert gather(L, **change) == status


def sparse(L, q=FAKE, ld_q=4096, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_slots=256, block=64, n_rows=1, h_q=16, h_kv=2,
           d=256, slots=FAKE, ld_slots=2051, n_idx=2051, scale=0.1, out=FAKE, lse=None, ws=None, ws_bytes=0):
    return L.qsa_sparse_attn_fp8(q, ld_q, kc, ks, vc, vs, n_slots, block, n_rows, h_q, h_kv, d, slots, ld_slots, n_idx,
                                 F(scale), out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=64), -2), (dict(h_q=34), -2), (dict(h_q=15), -2), (dict(h_q=17, h_kv=1, d=128), -2), (dict(block=1), -2),
    (dict(h_kv=0), -2), (dict(ld_slots=2050), -1), (dict(n_idx=-1), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(n_slots=100), -1),
    (dict(q=None), -1), (dict(q=BAD), -1), (dict(out=None), -1), (dict(slots=None), -1), (dict(lse=BAD), -1),
    (dict(ld_q=4095), -1), (dict(ld_q=4100), -1), (dict(vc=None), -1), (dict(n_slots=1 << 31), -1),
    (dict(n_idx=9000, ld_slots=9000), -3), (dict(n_idx=9000, ld_slots=9000, ws=FAKE, ws_bytes=16), -3),
    (dict(n_idx=9000, ld_slots=9000, ws=BAD, ws_bytes=1 << 30), -1), (dict(n_rows=0, q=None), 0)])
def test_sparse_attn_fp8_refusals(L, change, status):
    assert sparse(L, **change) == status


def window(L, q=FAKE, ld_q=4096, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n_slots=256, block=16, n_req=1, start=FAKE, n_rows=1,
           row_len=FAKE, max_len=200, max_rows=1, h_q=16, h_kv=2, d=256, pt=FAKE, ld_pt=4, page=64, window=50, n_sink=2,
           out=FAKE, lse=None, ws=None, ws_bytes=0, scale=0.1):
    return L.qsa_window_attn_fp8(q, ld_q, k, ks, v, vs, n_slots, block, n_req, start, n_rows, row_len, max_len, max_rows,
                                 h_q, h_kv, d, pt, ld_pt, page, window, n_sink, F(scale), out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(window=0), -1), (dict(n_sink=-1), -1), (dict(d=64), -2), (dict(h_q=34), -2), (dict(block=128), -2),
    (dict(block=24), -2), (dict(n_slots=264), -1), (dict(page=10), -2), (dict(page=0), -1), (dict(ld_pt=3), -1),
    (dict(max_len=-1), -1), (dict(max_rows=-1), -1), (dict(n_req=0), -1), (dict(start=None), -1),
    (dict(row_len=None), -1), (dict(pt=None), -1), (dict(q=BAD), -1), (dict(out=None), -1), (dict(out=ODD), -1),
    (dict(lse=BAD), -1), (dict(ld_q=4000), -1), (dict(ld_q=4099), -1), (dict(k=None), -1), (dict(v=BAD), -1),
    (dict(n_slots=-16), -1), (dict(n_req=70000), -2), (dict(scale=float("nan")), -1), (dict(scale=-float("inf")), -1),
    (dict(max_len=90000, ld_pt=2000, window=80000), -3),
    (dict(max_len=90000, ld_pt=2000, window=80000, max_rows=6, n_rows=6), -3), (dict(n_rows=0, q=None), 0)])
def test_window_attn_fp8_refusals(L, change, status):
    assert window(L, **change) == status


def test_workspace_sizes(L):
    """Room for two partial results of every CTA (152) where the blocks of long
    units are shared out; none where clusters or whole units take them."""
    f, w = L.qsa_sparse_attn_fp8_workspace_size, L.qsa_window_attn_fp8_workspace_size
    size = lambda pairs, d: 2560 + 2 * 152 * pairs * (d + 4) * 4  # noqa: E731
    assert f(32, 16, 2, 256, 2051) == 0 and f(1, 16, 2, 256, 2051) == 0 and f(1, 32, 2, 128, 0) == 0
    assert f(1, 16, 2, 256, 9000) == size(8, 256) and f(1, 32, 2, 128, 20000) == size(16, 128)
    assert f(607, 16, 2, 256, 2051) == size(8, 256) and f(608, 16, 2, 256, 2051) == 0
    assert w(1, 1, 1, 16, 2, 256, 80000, 1024, 4) == 0 and w(1, 1, 1, 16, 2, 256, 80000, 80000, 4) == size(8, 256)
    assert w(6, 1, 6, 16, 2, 256, 80000, 80000, 0) == size(48, 256) and w(6, 1, 6, 16, 2, 256, 500, 9, 4) == 0
    assert w(2, 1, 2, 8, 2, 128, 80000, 80000, 4) == size(8, 128) and w(3, 1, 3, 12, 1, 128, 80000, 80000, 4) == size(48, 128)
    assert w(1, 1, 1, 16, 1, 128, 80000, 80000, 4) == size(16, 128)
    assert w(9, 3, 4, 8, 1, 128, 80000, 80000, 4) == size(32, 128)
    assert w(1216, 1216, 1, 8, 1, 256, 80000, 1024, 4) == 0 and w(300, 700, 1, 8, 1, 256, 80000, 80000, 4) == 0
    assert f(0, 16, 2, 256, 9000) == 0 and f(1, 16, 3, 256, 9000) == 0 and w(1, 1, 1, 16, 2, 256, 80000, 0, 4) == 0


def plan(L, ctx=FAKE, new=OTHER, n_req=3, pt=FAKE, ld_pt=4, page=64, free=FAKE, n_pool=9, n_free=FAKE, n_tok=5,
         start=FAKE, new_len=OTHER, row_len=FAKE, row_req=None, slots=FAKE):
    return L.qsa_plan_step(ctx, new, n_req, pt, ld_pt, page, free, n_pool, n_free, n_tok, start, new_len, row_len,
                           row_req, slots, None)


@pytest.mark.parametrize("change,status", [
    (dict(n_req=-1), -1), (dict(n_req=65536), -2), (dict(n_tok=-1), -1), (dict(n_tok=(1 << 30) + 1), -2),
    (dict(n_pool=-1), -1), (dict(n_pool=2 ** 31 - 1), -2), (dict(ld_pt=-1), -1), (dict(page=0), -1), (dict(page=6), -2),
    (dict(ctx=None), -1), (dict(new=None), -1), (dict(pt=None), -1), (dict(free=None), -1), (dict(n_free=None), -1),
    (dict(start=None), -1), (dict(new_len=None), -1), (dict(row_len=None), -1), (dict(slots=None), -1),
    (dict(ctx=BAD), -1), (dict(row_req=BAD), -1), (dict(slots=BAD), -1), (dict(new_len=FAKE), -1)])
def test_plan_step_refusals(L, change, status):
    assert plan(L, **change) == status


def release(L, pt=FAKE, ld_pt=4, n_req=3, lo=FAKE, hi=FAKE, free=FAKE, n_pool=9, n_free=FAKE):
    return L.qsa_release_pages(pt, ld_pt, n_req, lo, hi, free, n_pool, n_free, None)


@pytest.mark.parametrize("change,status", [
    (dict(n_req=-1), -1), (dict(n_req=65536), -2), (dict(ld_pt=-1), -1), (dict(n_pool=-1), -1),
    (dict(n_pool=2 ** 31 - 1), -2), (dict(pt=None), -1), (dict(lo=None), -1), (dict(hi=BAD), -1), (dict(free=None), -1),
    (dict(n_free=None), -1), (dict(n_free=BAD), -1), (dict(n_req=0, pt=None), 0)])
def test_release_pages_refusals(L, change, status):
    assert release(L, **change) == status


def test_cpython_entry_points_match_ctypes(L):
    """The CPython entry points of these calls reach the same C functions: the
    host checks give the same statuses, argument by argument."""
    from sparse_attention_indexer_index_gb300 import _build
    if not os.path.exists(_build.fastcall_path()):
        pytest.skip("the CPython entry points were not built (no Python headers here)")
    from sparse_attention_indexer_index_gb300 import _fastcall as fc
    X, Y, B = 0x1000, 0x2000, 0x1002

    def same(name, args, positions, bad):
        for i in positions:
            a = list(args)
            a[i] = bad
            want = getattr(L, name)(*a)
            assert want < 0 and getattr(fc, name)(*a) == want, (name, i)
        with pytest.raises(TypeError):
            getattr(fc, name)(*args[:-1])

    # a bad pointer, a bad size, a missing pointer in every checked position
    a = [X, X, 512, 512, 3, 2, 256, X, X, 1, X, 4, 64, 16, X, X, X, X, 256, None]
    same("qsa_append_kv_fp8", a, [0, 1, 14, 16], B)
    same("qsa_append_kv_fp8", a, [2, 3, 4, 5, 6, 9, 12, 13, 18], -1)
    same("qsa_append_kv_fp8", a, [7, 8, 10, 15, 17], None)
    a = [X, X, X, X, 256, 2, 256, 16, X, 3, X, X, None]
    same("qsa_gather_kv_fp8", a, [0, 2, 8, 10, 11], B)
    same("qsa_gather_kv_fp8", a, [4, 5, 6, 7, 9], -1)
    same("qsa_gather_kv_fp8", a, [1, 3], None)
    a = [X, 4096, X, X, X, X, 256, 16, 1, 16, 2, 256, X, 9000, 9000, 0.1, X, X, X, 1, None]
    same("qsa_sparse_attn_fp8", a, [0, 2, 4, 12, 16, 17], B)
    same("qsa_sparse_attn_fp8", a, [1, 6, 7, 8, 9, 10, 11, 13, 14], -1)
    same("qsa_sparse_attn_fp8", a, [18, 19], 0)
    a = [X, 4096, X, X, X, X, 256, 16, 1, X, 1, X, 90000, 1, 16, 2, 256, X, 2000, 64, 80000, 2, 0.1, X, X, X, 1, None]
    same("qsa_window_attn_fp8", a, [0, 2, 4, 23, 24], B)
    same("qsa_window_attn_fp8", a, [1, 6, 7, 8, 10, 12, 13, 14, 15, 16, 18, 19, 20, 21], -1)
    same("qsa_window_attn_fp8", a, [9, 11, 17], None)
    same("qsa_window_attn_fp8", a, [25, 26], 0)
    a = [X, X, 3, X, 4, 64, X, 9, X, 5, X, Y, X, X, X, None]
    same("qsa_plan_step", a, [0, 1, 3, 6, 8, 10, 11, 12, 13, 14], B)
    same("qsa_plan_step", a, [2, 4, 5, 7, 9], -1)
    a = [X, 4, 3, X, X, X, 9, X, None]
    same("qsa_release_pages", a, [0, 3, 4, 5, 7], B)
    same("qsa_release_pages", a, [1, 2, 6], -1)
