"""Loads behind griddepcontrol.wait, without a GPU.  A kernel launched as a
programmatic dependent one may run while the kernel before it still writes its
inputs, so behind the wait it has to read them with ordinary loads: a read-only
load, or an asm statement that is not volatile, may be moved ahead."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc")


def code(name):
    """The source without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


WAITING = sorted(f for f in os.listdir(CSRC) if "pdl_wait_primary()" in code(f) and f != "common.cuh")
# The selection kernels load their rows' metadata and pages before the wait, on
# purpose: the scorer does not write them, and lets the selection in only when
# what precedes it has finished.  The scores themselves come behind the wait.
SELECTION = [f for f in WAITING if f.startswith("select")]
# launched after a kernel of the same call, which alone writes what it reads
MERGE = ["sparse_attn.cuh"]


@pytest.mark.parametrize("name", [f for f in WAITING if f not in SELECTION + MERGE])
def test_loads_stay_behind_the_wait(name):
    src = code(name)
    assert "__ldg" not in src and "__restrict__" not in src and ".nc." not in src


@pytest.mark.parametrize("name", SELECTION)
def test_scores_are_read_behind_the_wait(name):
    src = code(name)
    assert not re.search(r"__ldg\((row\b|r\.row\b|gl\b|reinterpret_cast<const float4)", src)
    assert "const float* __restrict__" not in src and ".nc." not in src


@pytest.mark.parametrize("name", [*WAITING, "common.cuh"])
def test_load_statements_are_volatile(name):
    """Volatile statements keep their order, the wait among them."""
    src, n = code(name), 0
    for stmt in re.findall(r"asm\b[^;]*?\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\);", src, re.S):
        if re.search(r"\bld\.global", stmt):
            n += 1
            assert stmt.startswith("asm volatile") and ".nc." not in stmt, stmt
    assert n >= 4 or name != "common.cuh"


def test_the_lists_are_not_empty():
    assert len(WAITING) > 10 and len(SELECTION) == 6 and "window_tc.cuh" in WAITING
