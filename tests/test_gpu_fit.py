"""The one-pass tensor checks of the 8-bit cache's and the paging's calls: the
compiled form and the Python form say the same, and what fits has the
addresses, sizes and strides that torch gives."""
import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_index_gb300 as qsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fits():
    try:
        from sparse_attention_indexer_index_gb300._tensors import fit
    except ImportError:
        pytest.skip("the compiled checks were not built (no torch headers here)")
    return fit, qsa._fit_py


def z(*shape, dtype=torch.int32, device="cuda"):
    return torch.zeros(shape, dtype=dtype, device=device)


def test_answers(fits):
    t, u = z(3, 5), z(4)
    q = torch.zeros(7, 4 * 128 + 64, dtype=torch.bfloat16, device="cuda")[:, 64:].unflatten(1, (4, 128))
    w = z(10, dtype=torch.float32)
    for fit in fits:
        assert fit("iAB iA+", t, u) == (0, 3, 5, t.data_ptr(), u.data_ptr())
        assert fit("iA+ iAB", u, t) == (0, 3, 5, u.data_ptr(), t.data_ptr())
        assert fit("iAB ?iC ?w", t, None, None) == (0, 3, 5, -1, t.data_ptr(), None, None, 0)
        assert fit("iAB ?w", t, w) == (0, 3, 5, t.data_ptr(), w.data_ptr(), 40)
        assert fit("qNHD", q) == (0, 7, 4, 128, q.data_ptr(), 4 * 128 + 64)
        assert fit("qNHD", q[:1]) == (0, 1, 4, 128, q.data_ptr(), 512)
        assert fit("i@ ?h@HD", t, None) == (0, -1, -1, t.data_ptr(), 15, None)
        h = z(3, 5, 2, 8, dtype=torch.bfloat16)
        assert fit("i@ ?h@HD", t, h) == (0, 2, 8, t.data_ptr(), 15, h.data_ptr())
        assert fit("i@", z()[()])[2] == 1


@pytest.mark.parametrize("spec,make", [
    ("iAB", lambda: (z(3, 5, dtype=torch.int64),)), ("iAB", lambda: (z(3),)), ("iAB", lambda: (z(3, 5, 1),)),
    ("iAB", lambda: (z(5, 3).T,)), ("iAB", lambda: (z(3, 5, device="cpu"),)), ("iAB", lambda: ([1, 2],)),
    ("iAB", lambda: (None,)), ("iAB iA", lambda: (z(3, 5), z(4))), ("iAB iA+", lambda: (z(3, 5), z(3))),
    ("iA+", lambda: (z(),)), ("iAB iAB", lambda: (z(3, 5), z(3, 5, device="cpu"))),
    ("uA", lambda: (z(3),)), ("fA", lambda: (z(3, dtype=torch.float16),)), ("hA", lambda: (z(3, dtype=torch.float16),)),
    ("qNHD", lambda: (z(3, 4, 8, dtype=torch.bfloat16).transpose(1, 2),)),
    ("qNHD", lambda: (z(3, 4, 16, dtype=torch.bfloat16)[:, :, ::2],)),
    ("qNHD", lambda: (z(3, 8, 8, dtype=torch.bfloat16)[:, ::2],)),
    ("i@ h@HD", lambda: (z(3, 5), z(3, 4, 2, 8, dtype=torch.bfloat16))),
    ("i@ h@HD", lambda: (z(3, 5), z(3, 5, 2, dtype=torch.bfloat16))),
    ("iA ?w", lambda: (z(3), z(8, 8).T)), ("iA ?w", lambda: (z(3), z(8, device="cpu"))), ("iA+", lambda: (z(0),)),
])
def test_what_does_not_fit(fits, spec, make):
    args = make()
    assert [fit(spec, *args) for fit in fits] == [None, None]


def test_the_number_of_tensors_is_the_layouts(fits):
    for fit in fits:
        for args in ((z(3),), (z(3), z(3), z(3))):
            with pytest.raises((TypeError, ValueError)):
                fit("iA iA", *args)


@pytest.mark.parametrize("compiled", [True, False])
def test_calls_by_either_form(fits, monkeypatch, compiled):
    """A step through the calls with the compiled checks and with the Python
    ones: the same results, and the same errors."""
    monkeypatch.setattr(qsa, "_fit", fits[0 if compiled else 1])
    torch.manual_seed(3)
    n_slots, h_kv, d, block, page = 512, 2, 128, 16, 64
    kc, vc = z(n_slots, h_kv, d, dtype=torch.uint8), z(n_slots, h_kv, d, dtype=torch.uint8)
    ks, vs = z(n_slots // block, h_kv, dtype=torch.uint8), z(n_slots // block, h_kv, dtype=torch.uint8)
    pt = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    free, n_free = torch.arange(8, dtype=torch.int32, device="cuda"), z(1) + 8
    start, new_len, row_len, row_req, slots = qsa.plan_step(z(2), z(2) + 33, pt, page, free, n_free, 70)
    assert new_len.tolist() == [33, 33] and int(n_free) == 6 and row_req.tolist() == [0] * 33 + [1] * 33 + [-1] * 4
    k = torch.randn(70, h_kv, d, device="cuda").bfloat16()
    qsa.append_kv_fp8(k, k, start, z(2), kc, ks, vc, vs, pt, page)
    got, _ = qsa.gather_kv_fp8(kc, ks, vc, vs, slots)
    assert (got[:66].float() - k[:66].float()).abs().max() <= 2 ** -4 * k.abs().max() and not got[66:].any()
    q = torch.randn(70, 4, d, device="cuda").bfloat16()
    out, lse = qsa.window_attn_fp8(q, kc, ks, vc, vs, start, row_len, pt, page, 256, 256)
    ref, rlse = qsa.sparse_attn_fp8(q[32:33].contiguous(), kc, ks, vc, vs, slots[None, :33].contiguous())
    # one rounding of the output to BF16 (2^-8 of itself) and the parts of the weights (2^-12 of values up to 5)
    assert (out[32].float() - ref[0]).abs().max() <= 2 ** -8 * ref.abs().max() + 2 ** -12 * 6
    assert abs(float(lse[32, 0]) - float(rlse[0, 0])) <= 1e-4
    assert qsa.release_pages(pt, z(2), z(2) + 1, free, n_free) and int(n_free) == 8 and (pt == -1).all()
    with pytest.raises(TypeError, match="k_codes"):
        qsa.gather_kv_fp8(kc.int(), ks, vc, vs, slots)
    with pytest.raises(ValueError, match="contiguous"):
        qsa.window_attn_fp8(q, kc, ks, vc, vs, start, row_len, pt.T.contiguous().T, page, 256, 256)
    with pytest.raises(ValueError, match="fit together"):
        qsa.plan_step(z(3), z(2), pt, page, free, n_free, 70)
    with pytest.raises(ValueError, match="fit together"):
        qsa.plan_step(z(2), z(2), pt, page, free, n_free, 70, row_len=z(69))
    with pytest.raises(ValueError, match="fit together"):
        qsa.sparse_attn_fp8(q, kc, ks[:-1], vc, vs[:-1], z(70, 5))
    torch.cuda.synchronize()
