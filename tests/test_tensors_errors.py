"""Tensors that cannot say where they lie, without a GPU: the compiled checks
of a call's tensors raise what torch raises, as the Python form does, and do
not end the process."""
import subprocess
import sys
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import torch
import sparse_attention_indexer_index_gb300 as qsa
from sparse_attention_indexer_index_gb300._tensors import fit
from torch._subclasses.fake_tensor import FakeTensorMode
caught = []
def look(x):
    for form in (fit, qsa._fit_py):
        try:
            form("iA", x)
        except RuntimeError as e:
            caught.append(str(e))
    return x
with FakeTensorMode():  # a tensor on the device, where there is none
    torch.vmap(look)(torch.empty(3, 5, dtype=torch.int32, device="cuda"))
assert len(caught) == 2 and all("data pointer" in c for c in caught), caught
print("ok")
"""


def test_a_tensor_without_an_address():
    import sparse_attention_indexer_index_gb300 as qsa
    from sparse_attention_indexer_index_gb300 import _build
    qsa.build()
    if not os.path.exists(_build.tensors_path()):
        pytest.skip("the compiled checks were not built (no torch headers here)")
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, (r.returncode, r.stderr[-1500:])


@pytest.mark.gpu
@pytest.mark.parametrize("compiled", [True, False])
def test_sparse_tensors_are_refused(monkeypatch, compiled):
    import sparse_attention_indexer_index_gb300 as qsa
    if compiled:
        pytest.importorskip("sparse_attention_indexer_index_gb300._tensors")
    else:
        monkeypatch.setattr(qsa, "_fit", qsa._fit_py)
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    cache = [z(64, 2, 128), z(4, 2), z(64, 2, 128), z(4, 2)]
    slots = torch.ones(5, dtype=torch.int32, device="cuda")
    qsa.gather_kv_fp8(*cache, slots)
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        qsa.gather_kv_fp8(*cache, slots.to_sparse())
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        qsa.gather_kv_fp8(cache[0], cache[1].to_sparse(), *cache[2:], slots)
    torch.cuda.synchronize()
    assert qsa.device_status(clear=True) == 0
