"""The 4-bit KV cache and the window attention without a GPU: the test
reference against closed forms, and the C ABI's refusals (no call here
reaches a CUDA launch)."""
import ctypes

import numpy as np
import pytest

import kv4_ref as ref
from workloads.synth import bf16_bits, normal_bf16


@pytest.fixture(scope="module")
def L():
    import sparse_attention_indexer_index_gb300 as qsa
    qsa.build()
    return qsa.lib()


FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1010)  # 16-byte but not 32-byte aligned
BAD = ctypes.c_void_p(0x1002)
FAKE_16 = ctypes.c_void_p(0x1010)  # 16-byte aligned, not 32
F = ctypes.c_float


# ------------------------------------------------------------ the reference
def test_e4m3_table_matches_torch():
    import torch
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.E4M3[:127])


def test_quantise_closed_forms():
    x = np.zeros(16, np.float32)
    x[:8] = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    x[8:] = -x[:8]
    codes, scales = ref.quantise(bf16_bits(x), 1.0)
    assert scales.tolist() == [0x38]  # 1.0
    assert np.array_equal(np.abs(ref.values(codes, scales, 1.0)), np.abs(x))
    # ties go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x[:8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    codes, scales = ref.quantise(bf16_bits(x), 1.0)
    assert ref.values(codes, scales, 1.0)[:8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]
    # a tensor scale of 2^-3 holds the block / 8 exactly
    c8, s8 = ref.quantise(bf16_bits(x / 8), 0.125)
    assert np.array_equal(c8, codes) and np.array_equal(s8, scales)


def test_quantise_edges():
    x = np.zeros((5, 16), np.float32)
    x[1, 3] = 1e-5                      # scale rounds to zero
    x[2, :2] = [3.0e38, -1.0]           # saturates
    x[3, 0] = np.inf
    x[4, 15] = np.nan
    bits = bf16_bits(x)
    bits[4, 15] = 0x7FC0
    codes, scales = ref.quantise(bits, 1.0)
    v = ref.values(codes, scales, 1.0)
    assert (v[:2] == 0).all() and v[2, 0] == 2688.0 and v[2, 1] == 0
    assert np.isnan(v[3:]).all() and scales[3, 0] == scales[4, 0] == 0x7F


def test_quantise_error_is_at_most_half_a_step():
    """Within a block the error is at most half the e2m1 step at the value
    (a sixth of the block's largest) and the scale's own rounding, 2^-4."""
    rng = np.random.default_rng(0)
    bits = normal_bf16(rng, (400, 64))
    x = ref.bf16_to_f64(bits).reshape(400, 4, 16)
    v = ref.values(*ref.quantise(bits, 2.0 ** -5), 2.0 ** -5).reshape(x.shape)
    top = np.abs(x).max(-1, keepdims=True)
    assert (np.abs(v - x) <= top * (1 / 6 + 2.0 ** -4)).all()


def test_attend_closed_forms():
    q = np.zeros((2, 128))
    k, v = np.random.default_rng(1).standard_normal((2, 5, 1, 128))
    out, lse, *_ = ref.attend(q, k, v, 0.3)
    assert np.allclose(out, v[:, 0].mean(0)) and np.allclose(lse, np.log(5))
    out, lse, *_ = ref.attend(q, k[:0], v[:0], 0.3)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_window_positions():
    assert ref.window_positions(0, 4, 2).tolist() == []
    assert ref.window_positions(3, 4, 2).tolist() == [0, 1, 2]
    assert ref.window_positions(10, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert ref.window_positions(10, 1, 0).tolist() == [9]
    assert ref.window_positions(10, 9, 4).tolist() == list(range(10))


# --------------------------------------------------------------- refusals
def append(L, k=FAKE, v=FAKE, ld_k=512, ld_v=512, n_tok=3, h_kv=2, d=256, start=FAKE, first=FAKE, n_req=1, pt=FAKE,
           ld_pt=4, page=64, ks=1.0, vs=1.0, kc=FAKE, kss=FAKE, vc=FAKE, vss=FAKE, n_slots=256):
    return L.qsa_append_kv_fp4(k, v, ld_k, ld_v, n_tok, h_kv, d, start, first, n_req, pt, ld_pt, page, F(ks), F(vs), kc,
                               kss, vc, vss, n_slots, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=64), -2), (dict(d=192), -2), (dict(page=6), -2), (dict(n_req=70000), -2),
    (dict(ks=0.3), -1), (dict(vs=0.0), -1), (dict(ks=-1.0), -1), (dict(ks=float("nan")), -1),
    (dict(ks=float("inf")), -1), (dict(ks=2.0 ** -65), -1), (dict(vs=2.0 ** 64), -1),
    (dict(k=None), -1), (dict(start=None), -1), (dict(first=None), -1), (dict(pt=None), -1),
    (dict(k=ODD), -1), (dict(v=BAD), -1), (dict(ld_k=511), -1), (dict(ld_k=520), -1), (dict(ld_v=256), -1),
    (dict(kc=None), -1), (dict(vss=BAD), -1), (dict(n_slots=-1), -1), (dict(n_tok=-1), -1), (dict(h_kv=0), -1),
    (dict(n_tok=0, k=None), 0), (dict(n_req=0, start=None), 0)])
def test_append_refusals(L, change, status):
    assert append(L, **change) == status


def gather(L, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_slots=256, h_kv=2, d=256, slots=FAKE, n=3, gk=1.0, gv=1.0,
           ko=FAKE, vo=FAKE):
    return L.qsa_gather_kv_fp4(kc, ks, vc, vs, n_slots, h_kv, d, slots, n, F(gk), F(gv), ko, vo, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=96), -2), (dict(gk=3.0), -1), (dict(slots=None), -1), (dict(slots=BAD), -1), (dict(ko=None), -1),
    (dict(vo=ODD), -1), (dict(kc=BAD), -1), (dict(ks=None), -1), (dict(n=-1), -1), (dict(n=1 << 50), -2),
    (dict(n=0, slots=None, ko=None), 0)])
def test_gather_refusals(L, change, status):
    assert gather(L, **change) == status


def sparse(L, q=FAKE, ld_q=4096, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, n_slots=256, n_rows=1, h_q=16, h_kv=2, d=256,
           slots=FAKE, ld_slots=2051, n_idx=2051, gk=1.0, gv=1.0, out=FAKE, lse=None, ws=None, ws_bytes=0):
    return L.qsa_sparse_attn_fp4(q, ld_q, kc, ks, vc, vs, n_slots, n_rows, h_q, h_kv, d, slots, ld_slots, n_idx, F(0.1),
                                 F(gk), F(gv), out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(d=64), -2), (dict(h_q=18), -2), (dict(h_q=15), -2), (dict(h_q=17, h_kv=1, d=128), -2),
    (dict(h_kv=0), -2), (dict(ld_slots=2050), -1), (dict(n_idx=-1), -1), (dict(gk=0.7), -1), (dict(gv=-2.0), -1),
    (dict(q=None), -1), (dict(q=BAD), -1), (dict(out=None), -1), (dict(slots=None), -1), (dict(lse=BAD), -1),
    (dict(ld_q=4095), -1), (dict(ld_q=4100), -1), (dict(vc=None), -1), (dict(n_slots=1 << 31), -1),
    (dict(n_idx=9000, ld_slots=9000), -3), (dict(n_idx=9000, ld_slots=9000, ws=FAKE, ws_bytes=16), -3),
    (dict(n_idx=9000, ld_slots=9000, ws=BAD, ws_bytes=1 << 30), -1), (dict(n_rows=0, q=None), 0)])
def test_sparse_attn_fp4_refusals(L, change, status):
    assert sparse(L, **change) == status


def test_workspace_sizes(L):
    f, w = L.qsa_sparse_attn_fp4_workspace_size, L.qsa_window_attn_workspace_size
    assert f(32, 16, 2, 256, 2051) == 0 and f(1, 16, 2, 256, 2051) == 0
    assert f(1, 16, 2, 256, 9000) == 16 * 2 * 258 * 4
    assert w(1, 16, 2, 256, 80000, 1024, 4) == 0 and w(1, 16, 2, 256, 80000, 80000, 4) > 0
    assert w(1, 16, 2, 256, 500, 80000, 4) == 0  # the context bounds the window
    assert f(0, 16, 2, 256, 9000) == 0 and f(1, 16, 3, 256, 9000) == 0 and w(1, 16, 2, 256, 80000, 0, 4) == 0


def window(L, fp4=False, q=FAKE, ld_q=4096, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n_slots=256, n_req=1, start=FAKE,
           n_rows=1, row_len=FAKE, max_len=200, max_rows=1, h_q=16, h_kv=2, d=256, pt=FAKE, ld_pt=4, page=64, window=50,
           n_sink=2, gk=1.0, gv=1.0, out=FAKE, lse=None, ws=None, ws_bytes=0, scale=0.1):
    rest = (n_slots, n_req, start, n_rows, row_len, max_len, max_rows, h_q, h_kv, d, pt, ld_pt, page, window, n_sink,
            F(scale))
    if fp4:
        return L.qsa_window_attn_fp4(q, ld_q, k, ks, v, vs, *rest, F(gk), F(gv), out, lse, ws, ws_bytes, None)
    return L.qsa_window_attn(q, ld_q, k, v, *rest, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(window=0), -1), (dict(window=-3), -1), (dict(n_sink=-1), -1), (dict(d=64), -2), (dict(h_q=18), -2),
    (dict(page=10), -2), (dict(page=0), -1), (dict(ld_pt=3), -1), (dict(max_len=-1), -1), (dict(max_rows=-1), -1),
    (dict(n_req=0), -1), (dict(start=None), -1), (dict(row_len=None), -1), (dict(pt=None), -1), (dict(q=BAD), -1),
    (dict(out=None), -1), (dict(out=BAD), -1), (dict(lse=BAD), -1), (dict(ld_q=4000), -1), (dict(ld_q=4099), -1),
    (dict(k=None), -1), (dict(v=BAD), -1), (dict(n_slots=-1), -1), (dict(n_req=70000), -2),
    (dict(max_len=90000, ld_pt=2000, window=80000), -3), (dict(n_rows=0, q=None), 0)])
def test_window_attn_refusals(L, fp4, change, status):
    assert window(L, fp4, **change) == status


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_window_attn_refuses_a_scale_that_is_not_finite(L, fp4, scale):
    assert window(L, fp4, scale=scale) == -1


@pytest.mark.parametrize("fp4", [False, True])
def test_window_attn_refuses_outputs_off_a_32_byte_boundary(L, fp4):
    assert window(L, fp4, out=FAKE_16) == -1


def test_window_attn_fp4_refuses_other_scales(L):
    assert window(L, True, gk=0.3) == -1 and window(L, True, gv=0.0) == -1


def test_cpython_entry_points_match_ctypes(L):
    """The CPython entry points of these calls reach the same C functions: the
    host checks give the same statuses, argument by argument."""
    import os
    from sparse_attention_indexer_index_gb300 import _build
    if not os.path.exists(_build.fastcall_path()):
        pytest.skip("the CPython entry points were not built (no Python headers here)")
    from sparse_attention_indexer_index_gb300 import _fastcall as fc
    X, B = 0x1000, 0x1002

    def same(name, args, positions, bad):
        for i in positions:
            a = list(args)
            a[i] = bad
            want = getattr(L, name)(*a)
            assert want < 0 and getattr(fc, name)(*a) == want, (name, i)
        with pytest.raises(TypeError):
            getattr(fc, name)(*args[:-1])

    # a bad pointer, then a bad size, in every checked position
    a = [X, X, 512, 512, 3, 2, 256, X, X, 1, X, 4, 64, 1.0, 1.0, X, X, X, X, 256, None]
    same("qsa_append_kv_fp4", a, [0, 1, 15, 16, 17, 18], B)
    same("qsa_append_kv_fp4", a, [2, 3, 4, 5, 6, 9, 12, 13, 14, 19], -1)
    same("qsa_append_kv_fp4", a, [7, 8, 10], None)
    a = [X, X, X, X, 256, 2, 256, X, 3, 1.0, 1.0, X, X, None]
    same("qsa_gather_kv_fp4", a, [0, 1, 2, 3, 7, 11, 12], B)
    same("qsa_gather_kv_fp4", a, [4, 5, 6, 8, 9, 10], -1)
    a = [X, 4096, X, X, X, X, 256, 1, 16, 2, 256, X, 9000, 9000, 0.1, 1.0, 1.0, X, X, X, 1, None]
    same("qsa_sparse_attn_fp4", a, [0, 2, 3, 4, 5, 11, 17, 18], B)
    same("qsa_sparse_attn_fp4", a, [1, 6, 7, 8, 9, 10, 12, 13, 15, 16], -1)
    same("qsa_sparse_attn_fp4", a, [19, 20], 0)
    w = [256, 1, X, 1, X, 90000, 1, 16, 2, 256, X, 2000, 64, 80000, 2, 0.1]
    for name, a in [("qsa_window_attn", [X, 4096, X, X] + w + [X, X, X, 1, None]),
                    ("qsa_window_attn_fp4", [X, 4096, X, X, X, X] + w + [1.0, 1.0, X, X, X, 1, None])]:
        c = 2 if name.endswith("fp4") else 0
        same(name, a, [0, 2, 3, 20 + 2 * c, 21 + 2 * c], B)
        same(name, a, [1] + [4 + c + i for i in (0, 1, 3, 5, 6, 7, 8, 9, 11, 12, 13, 14)], -1)
        same(name, a, [6 + c, 8 + c, 14 + c], None)
        same(name, a, [22 + 2 * c, 23 + 2 * c], 0)
    assert fc.qsa_sparse_attn_fp4_workspace_size(1, 16, 2, 256, 9000) == 16 * 2 * 258 * 4
    assert fc.qsa_window_attn_workspace_size(1, 16, 2, 256, 80000, 80000, 4) == \
        L.qsa_window_attn_workspace_size(1, 16, 2, 256, 80000, 80000, 4)
