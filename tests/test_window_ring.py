"""The ring of K and V stages of the tensor-core form of window_attn, without a
GPU: the waits of all its roles, replayed over every use of the ring.

A wait by parity on a stage's barrier is sound only where the phase before the
awaited one is known to be over: otherwise it passes at once, on that phase,
and the waiter takes (or writes) another block's stage.  For each wait this
lists what the waiter knows by then and asserts that the earlier phase is among
it.  Sizes and rules are read from the kernel's source."""
import itertools
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "sparse_attention_indexer_index_gb300", "csrc", "window_tc.cuh")).read()


def shape(d):
    """(entries of a block, K stages, entries of a V stage, stages of the ring) at head dim d."""
    n = int(re.search(r"constexpr int kWtN = (\d+);", SRC).group(1))
    assert "static constexpr int kKs = D / 128;" in SRC
    rows = re.search(r"static constexpr int kVRows = D == 256 \? (\d+) : (\d+);", SRC)
    stages = re.search(r"static constexpr int kStages = D == 256 \? (\d+) : (\d+);", SRC)
    i = 1 if d == 256 else 2
    return n, d // 128, int(rows.group(i)), int(stages.group(i))


def uses(d, tiles):
    """The ring's uses in order, as (kind, tile, block, stage of it); tiles: (blocks, entries copied of the last)."""
    n, ks, v_rows, _ = shape(d)
    seq = []
    for t, (blocks, last) in enumerate(tiles):
        def v(b):
            copied = last if b == blocks - 1 else n
            return [("v", t, b, i) for i in range(-(-copied // v_rows))]

        def k(b):
            return [("k", t, b, i) for i in range(ks)]

        seq += k(0)
        for b in range(blocks):
            if b + 1 < blocks:
                seq += k(b + 1)
            seq += v(b)
    return seq


def tile_lists(d):
    n, _, v_rows, _ = shape(d)
    lasts = sorted({8, v_rows, min(n, v_rows + 8), n})
    for blocks in range(1, 17):
        for last in lasts:
            yield [(blocks, last)] * 3
    for a, b, c in itertools.product((1, 2, 3), repeat=3):
        for last in lasts:
            yield [(a, last), (b, n), (c, last), (a, n)]


def zeroing():
    """The part of the softmax in which V rows that no pair sees are zeroed."""
    return re.search(r"// V rows that no pair sees: zeros(.*?)fence_proxy_async_smem", SRC, re.S).group(1)


@pytest.mark.parametrize("d", [128, 256])
def test_stage_numbers_are_those_of_the_source(d):
    """The closed forms by which the copies and the softmax number their stages."""
    assert "Sh::kKs * blk + max(blk - 1, 0) * Sh::kVs" in SRC  # K(blk)
    assert SRC.count("Sh::kKs * min(blk + 2, w.n_blk) + blk * Sh::kVs") == 2  # V(blk)
    assert SRC.count("rs += Sh::kKs * w.n_blk + (w.n_blk - 1) * Sh::kVs + (last + Sh::kVRows - 1) / Sh::kVRows;") == 2
    n, ks, v_rows, _ = shape(d)
    vs = n // v_rows
    for tiles in tile_lists(d):
        at = {u: i for i, u in enumerate(uses(d, tiles))}
        rs = 0
        for t, (blocks, last) in enumerate(tiles):
            for b in range(blocks):
                assert at["k", t, b, 0] == rs + ks * b + max(b - 1, 0) * vs
                assert at["v", t, b, 0] == rs + ks * min(b + 2, blocks) + b * vs
            rs += ks * blocks + (blocks - 1) * vs + -(-last // v_rows)


@pytest.mark.parametrize("d", [128, 256])
def test_waits_of_the_softmax_on_v_stages(d):
    """Before the softmax zeroes rows of V(blk) it waits for `full` of each of
    its stages; by then the stage's use before must be known to have landed.
    S(blk) is there, so what QK(blk) and the products before it read has landed
    (QK(i + 1) is issued before PV(i)); with the wait for PV(blk - 1), what that
    one read too; at a tile's end the last PV is waited for."""
    z = zeroing()
    first_full = z.index("ctl.full")
    waits_pv = re.search(r"ok = blk == 0 \|\| wt_wait\(&ctl\.pv_done\[sl \^ 1\], \(uint32_t\)\(\(x - 1\) >> 1\) & 1u, abort\);",
                         z[:first_full]) is not None
    n_st = shape(d)[3]
    for tiles in tile_lists(d):
        seq = uses(d, tiles)
        for u, (kind, t, b, i) in enumerate(seq):
            if kind != "v" or u < n_st:
                continue
            k0, t0, b0, i0 = seq[u - n_st]
            landed = (t0 < t or (k0 == "k" and b0 <= b) or
                      (k0 == "v" and b0 <= b - (1 if waits_pv else 2)) or
                      (k0 == "v" and b0 == b and i0 < i))  # waited for just before
            assert landed, (tiles, "V", t, b, i, "after", k0, t0, b0, i0)


@pytest.mark.parametrize("d", [128, 256])
def test_waits_of_the_softmax_on_products(d):
    """PV(blk - 1) is waited for by parity too: its barrier's use before is
    PV(blk - 3), which S(blk) covers (QK(blk) is issued after PV(blk - 2))."""
    for blocks in range(1, 17):
        order = ["qk0"]
        for b in range(blocks):
            order += ([f"qk{b + 1}"] if b + 1 < blocks else []) + [f"pv{b}"]
        for b in range(3, blocks):
            assert order.index(f"pv{b - 3}") < order.index(f"qk{b}")


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_waits_of_the_copies_on_empty_stages(d, kind):
    """The copying warp of K (V) waits until use u - kStages is used up before
    it fills the stage again, and must know that u - 2 kStages was.  Stages are
    freed in order, so it knows that of everything up to its own last such wait."""
    n_st = shape(d)[3]
    for tiles in tile_lists(d):
        freed = -1  # the last use known to be used up
        for u, (k, *_) in enumerate(uses(d, tiles)):
            if k != kind or u < n_st:
                continue
            assert u < 2 * n_st or freed >= u - 2 * n_st, (tiles, u)
            freed = u - n_st


def test_what_one_lane_writes_is_ordered_before_the_arrival_of_another():
    """Lane 0 writes a block's list of missing boxes, an elected lane, which may
    be any, announces its copies: the warp meets in between."""
    k = SRC[SRC.index("ctl.bad[(gb + blk) % kWtBadRing] = bad;"):]
    assert "__syncwarp();" in k[:k.index("wt_expect(&ctl.full[st]")]


@pytest.mark.parametrize("d", [128, 256])
def test_products_overwrite_nothing_that_another_may_read(d):
    """Tensor memory: the order in which the pipe runs two MMAs is documented
    only where they share accumulator and shape, so no product may write what an
    earlier one, or the softmax, may still read."""
    n = shape(d)[0]
    cols = re.search(r"static constexpr uint32_t kColS = D, kColP = D \+ kWtN;", SRC)
    assert cols, "S and P lie in different columns"
    o, s, p = range(0, d), range(d, d + n), [range(d + n, d + n + n // 2), range(d + n + n // 2, d + 2 * n)]
    assert p[1].stop <= 512
    assert not (set(o) & set(s) or set(s) & (set(p[0]) | set(p[1])) or set(p[0]) & set(p[1]))
    # where the products and the softmax go
    assert "d = tmem + Sh::kColS;" in SRC and "p = tmem + Sh::kColP + sl * (N / 2) + e0 / 2;" in SRC
    assert "wt_tmem_ld64(lanes + Sh::kColS + 64 * half, s);" in SRC
    assert "wt_tmem_st32(lanes + Sh::kColP + sl * (N / 2) + 32 * half, p);" in SRC
    # QK(x) overwrites S(x - 1): every softmax warp has arrived with it in its registers
    qk = SRC[SRC.index("auto qk = "):SRC.index("auto pv = ")]
    wait = "if (!wait(s ? &ctl.s_free : &ctl.full[st], s ? (uint32_t)(x - 1) & 1u : ph)) return false;"
    # (lanes wait for different barriers, one lane issues)
    assert qk.index(wait) < qk.index("__syncwarp();") < qk.index("tc_fence_after();") < qk.index("wt_mma_qk(")
    assert "const bool s = i == 0 && x > 0 && (lane & 1) != 0;" in qk and "mbar_init(&ctl.s_free, 8);" in SRC
    soft = SRC[SRC.index("wt_tmem_ld64(lanes"):]
    assert soft.index("tc_fence_before();") < soft.index("__syncwarp();") < soft.index("wt_arrive(&ctl.s_free);")
    # P(x) overwrites P(x - 2): S(x) is announced by a commit behind PV(x - 2)
    for blocks in range(1, 17):
        order = []
        for _ in range(2):  # tiles
            x0 = sum(e[0] == "qk" for e in order)
            order.append(("qk", x0))
            for b in range(blocks):
                order += ([("qk", x0 + b + 1)] if b + 1 < blocks else []) + [("pv", x0 + b)]
        for x in range(2, 2 * blocks):
            assert order.index(("pv", x - 2)) < order.index(("qk", x))
            # and its own wait ends: the scores before were announced before
            assert order.index(("qk", x - 1)) < order.index(("qk", x))
