"""The compiled checks of a call's tensors belong to one torch, without a GPU:
with another they are built anew, and until then the Python form is used."""
import importlib.util
import os
import sys
import types

import pytest

torch = pytest.importorskip("torch")

import sparse_attention_indexer_index_gb300 as qsa
from sparse_attention_indexer_index_gb300 import _build

NAME = qsa.__name__ + "._tensors"


@pytest.fixture
def first_use(monkeypatch):
    """The binding before its first call has chosen a form; gives the choice."""
    spec = importlib.util.find_spec(qsa.__name__)
    fresh = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fresh)

    def choose(**module):
        m = types.ModuleType(NAME)
        m.fit = lambda *a: "compiled"
        m.__dict__.update(module)
        monkeypatch.setitem(sys.modules, NAME, m)
        return "compiled" if fresh._fit("iA", [1]) == "compiled" else "python"
    return choose


def test_the_form_for_this_torch_is_used(first_use):
    assert first_use(torch_version=str(torch.__version__)) == "compiled"


def test_the_form_for_another_torch_is_not_used(first_use):
    assert first_use(torch_version="0." + str(torch.__version__)) == "python"


def test_a_form_that_does_not_say_for_which_is_not_used(first_use):
    assert first_use() == "python"


def test_the_built_form_says_for_which_torch():
    qsa.build()
    if not os.path.exists(_build.tensors_path()):
        pytest.skip("the compiled checks were not built (no torch headers here)")
    from sparse_attention_indexer_index_gb300 import _tensors
    assert _tensors.torch_version == torch.__version__


@pytest.mark.parametrize("stamp", ["same", "other", "none"])
def test_build_by_version_not_by_age(monkeypatch, tmp_path, stamp):
    """A newer file is kept for the same torch and replaced for another one."""
    headers = os.path.join(os.path.dirname(torch.__file__), "include")
    if not os.path.isdir(headers):
        pytest.skip("no torch headers here")
    out = tmp_path / "_tensors.so"
    out.write_bytes(b"")
    os.utime(out, (2 ** 32, 2 ** 32))
    monkeypatch.setattr(_build, "tensors_path", lambda: str(out))
    if stamp != "none":
        (tmp_path / "_tensors.so.torch").write_text(str(torch.__version__) if stamp == "same" else "1.0")
    started = []

    class Compiler:
        returncode = 0

        def __init__(self, cmd, **kw):
            started.append(cmd)
            open(cmd[cmd.index("-o") + 1], "wb").close()

        def communicate(self):
            pass

    monkeypatch.setattr(_build.subprocess, "Popen", Compiler)
    assert _build.build_tensors() == (None if stamp == "same" else str(out))
    assert len(started) == (stamp != "same")
    assert stamp == "same" or any(str(torch.__version__) in c for c in started[0] if c.startswith("-D"))
    assert _build.build_tensors() is None and len(started) == (stamp != "same")  # once
