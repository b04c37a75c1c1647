"""Loads behind griddepcontrol.wait, without a GPU.  A kernel launched as a
programmatic dependent one may run while the kernel before it still writes its
inputs, so behind the wait it has to read them with ordinary loads: a read-only
load, or an asm statement that claims no effect on memory, may be moved ahead."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc")


def code(name):
    """The source without its comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["kv4.cuh", "kv_attn.cuh", "kv4_attn.cuh", "window_tc.cuh"])
def test_loads_stay_behind_the_wait(name):
    src = code(name)
    assert "__ldg" not in src and "__restrict__" not in src and ".nc." not in src
    # every global load in an asm statement is volatile and has a memory clobber
    for stmt in re.findall(r"asm\b[^;]*?\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\);", src, re.S):
        if re.search(r"\bld\.global", stmt):
            assert stmt.startswith("asm volatile") and '"memory"' in stmt, stmt
