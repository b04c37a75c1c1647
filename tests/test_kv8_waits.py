"""The waits inside the 8-bit cache attention, without a GPU, by its source:
every one is bounded, and what it answers is looked at."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = re.sub(r"//[^\n]*", "", open(os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc", "kv8_tc.cuh")).read())
KERNEL = SRC[SRC.index("kv8_tc_kernel(const"):SRC.index("kv8_merge_kernel(const")]


def test_no_answer_of_a_wait_is_dropped():
    """A wait that is a statement of its own goes on as if it had come about."""
    calls = list(re.finditer(r"\b(k8_wait|k8_wait_cluster|mbar_wait_bounded|mbar_try_wait|meet|meet_all|met_wait)\(", KERNEL))
    assert len(calls) > 15
    for m in calls:
        before = KERNEL[:m.start()].rstrip()
        assert before[-1] not in ";{}" and not before.endswith("else"), KERNEL[m.start() - 60:m.end() + 40]


def test_products_are_over_before_tensor_memory_is_freed():
    """The last wait of the warp that issues them: as long as every other wait,
    a fault where it runs out."""
    drain = KERNEL[KERNEL.index("k8_commit(&ctl.drain);"):KERNEL.index("tcgen05.dealloc")]
    assert re.match(r"k8_commit\(&ctl\.drain\);\s*if \(!__all_sync\(0xffffffffu, mbar_wait_bounded\(&ctl\.drain, 0u, kK8WaitNs\)\)"
                    r" && lane == 0\) k8_fault\(kFaultWait\);", drain)
    assert re.search(r"constexpr uint64_t kK8WaitNs = 2000000000ull;", SRC)


def test_loops_on_a_barrier_have_a_limit():
    for m in re.finditer(r"while \(!", SRC):
        body = SRC[m.start():m.start() + 300]
        assert "kK8WaitNs" in body, body
    assert len(re.findall(r"while \(!", SRC)) == 2


def test_the_wait_that_spans_a_segment_allows_for_its_blocks():
    """The warp that finds the work waits until a segment is taken up, which is
    when the one before it is done.  That may have 2^23 blocks (2^30 entries), at
    1.5 us or more each: far more than the limit of the other waits."""
    publish = KERNEL[KERNEL.index("auto publish = "):KERNEL.index("bool ok = true;")]
    assert re.search(r"k8_wait\(&ctl\.seg_empty\[sl\], [^;]*, abort, most\)\) return false;\s*most = max\(most, w\.j1 - w\.j0\);", publish)
    assert "t0 > kK8WaitNs + (uint64_t)blocks * kK8BlockNs" in SRC
    limit = [int(re.search(rf"constexpr uint(64|32)_t {n} = (\d+)(ull)?;", SRC).group(2)) for n in ("kK8WaitNs", "kK8BlockNs")]
    assert all(limit[0] + n * limit[1] >= 10 * n * 1500 for n in (1, 1000, 2 ** 23))
