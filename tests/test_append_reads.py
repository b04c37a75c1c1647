"""append_kv_fp4 and rows behind the last request, without a GPU.  A caller may
pass the most tokens a step can have as n_tok over buffers that hold no more
than the step's own, so the kernel must know a row's request before it reads
the row.  What it loads is read from the source, in order."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc", "kv4.cuh")).read()


def test_rows_are_read_only_once_their_request_is_known():
    k = SRC[SRC.index("append_kv_fp4_kernel(KvWriteArgs a) {"):]
    k = k[:k.index("\n}\n")]
    rows = [m.start() for m in re.finditer(r"ld_stream_32\(a\.[kv]_new", k)]
    assert len(rows) == 2 and len(re.findall(r"a\.[kv]_new", k)) == 2
    assert k.index("if (!ok || r < 0) return;") < k.index("if (r >= a.n_req) return;") < min(rows)
