// window_tc.cuh -- attention over a sliding window and the first tokens for
// requests with many rows (prompts, chunks), on the fifth-generation tensor
// cores: the prefill form of window_attn on the BF16 cache.
//
// A tile is R = floor(128 / G) consecutive rows of one request and one KV
// head: its R * G (row, query head) pairs are the 128 rows of the MMA, so the
// heads that share K and V share their tiles too.  Over the keys that any of
// its rows sees, in blocks of N entries:
//     S = Q K^T, P = exp2(c S - c m), O += P V, l += sum P
// with the running maximum m per pair; out = O / l, lse = ln 2 (c m + log2 l).
//
// Bound: 4 D flops per (pair, key), 512 of them per byte of K and V that a
// tile reads: tensor-bound once the copies keep up (64 bytes a clock and SM
// at the full MMA rate).
//
// Design (GB300).  One CTA per SM walks tiles (a static stride).  Where there
// are few tiles, the CTAs of a cluster share one: each takes a part of its
// blocks, and they exchange their sums through shared memory, D / C columns
// to each.  In a CTA:
//  - warp 10 finds the tiles and copies Q (TMA, 3-D boxes: the rows and heads
//    of a tile land as the 128 rows of the MMA operand), a tile ahead;
//  - warps 8 (K) and 11 (V) copy into a ring of 32 KB stages in the order in
//    which they are used, one TMA box of B rows (the largest power of two up
//    to 64 that divides the page) and all the stage's columns a copy.  The
//    instruction takes one box at a time whichever lanes ask (about 100 clocks
//    each: boxes of 16 rows x 64 columns held the tiles at 21 bytes a clock),
//    hence large boxes and two warps.  They follow the page table; a page out
//    of range is copied from beyond the tensor map, which fills zeros.
//  - warp 9 issues the MMAs: S from Q and K in shared memory (both K-major),
//    O from P in tensor memory and V (MN-major: V's rows are keys, the
//    transposition is the descriptor's).  128 entries a block: with 64, S
//    waits for its A operand (measured: 78 clocks a 128x64x16 product with A
//    in tensor memory, where the rate allows 32).
//  - warps 0-7 hold a pair in two threads, 64 entries of a block each: they
//    turn S into P, exchange the maximum through shared memory, and
//    write the outputs.  (One thread a pair took 1,000 clocks for 64 entries,
//    more than a product of D = 128.)
//  - The products go in the order QK(i+1) PV(i), so that a softmax has the
//    time of two products.  No product relies on the order in which the pipe
//    runs MMAs (it is documented for MMAs of one accumulator and shape only):
//    QK(i+1) waits until the softmax holds S(i) in registers, which is while
//    PV(i-1) runs, and P has two buffers apart from S, so that it overwrites
//    nothing that PV(i-1) reads.  P(i) replaces P(i-2): the barrier that
//    announces S(i) covers PV(i-2), issued before QK(i).  (With P(i) in the
//    place of S(i) and two buffers of S, QK(i+1) has to wait for the end of
//    PV(i-1): 72.6 us on the chunk of 4,096 rows instead of 67.7.)
//  - The accumulator is rescaled only when a row's maximum grew by more than
//    2^8 since the last time (the weights stay below 2^8 and the sums are
//    FP32, so nothing is lost); otherwise m stays.
//  - Weights enter the product as BF16 (both operands of it have V's type),
//    2^-8 relative at most, one rounding like that of the output; l sums them
//    before the rounding, in FP32.  Against FP64 the outputs of a chunk are off
//    by 0.0023 (root mean square, relative) where the output's rounding alone
//    gives 0.0017; a second product with the remainders would double PV.
// Tensor memory columns: O [0, D), S 128, P two times 64.
//
// Waits on stages.  The ring's uses are numbered in the order K(0), K(1),
// V(0), K(2), V(1), ... over all tiles; use u is in stage u mod kStages, and
// its phase u / kStages of that stage's barriers.  A wait by parity passes
// wrongly where the phase before the awaited one may still be open, so each
// role has to know by other means that use u - kStages has been there:
//  - warp 9 waits for every use in turn, so for u - kStages itself.
//  - warps 8 and 11 wait for `empty` of u - kStages and must know that u - 2
//    kStages is used up: each use of their own before that was waited for, the
//    gap between two of them is at most kStages, and stages are freed in order.
//  - warps 0-7 wait for some V stages only.  S(blk) is there, so K(0..blk) and
//    V(0..blk-2) were; the second V stage of a block between the first and the
//    last at D = 256 takes the place of the first of V(blk-1), of which that
//    says nothing (copies end in any order).  So they wait for PV(blk-1) first;
//    before block 0, the tile before has been waited for to its end.
// One thread issues all products and commits, and the arrivals of its commits
// come in order: a commit waits for every product before it.
//
// Entries.  With `start` the first window position of the tile rounded down
// to a box, the entries are the boxes of the first tokens before `start`
// (nsr of them, rounded up to a box; all lie below start), then the positions
// from start on.  A pair sees entries [0, a) and [b, c).  V rows that no pair
// of the tile sees are zeroed in shared memory (a weight of 0 times an
// infinity there would be NaN); see wt_redo for those that some pairs see.
//
// Measured (one call after the other over several sets of inputs): a chunk of
// 4,096 rows of 16 heads, 2 KV heads, D = 256, window 1,024: 67.3 us, 1,020
// TFLOP/s, 0.54 of the bf16 rate.  512 tiles make 3.4 rounds of the 152 SMs,
// four in effect.  Windows of 256 to 4,096 take 37.6, 46.9, 67.5, 107 and 192
// us in a graph: 1.2 to 1.3 us a block and round, where its products take 1.33
// at the measured bf16 rate and 1.04 at 64 clocks per 128 x 128 x 16; the rest
// is about 4 us a tile for its start and end.  Seven prompts of D = 128 in
// windows of 500: 43.2 us, 0.24 of the rate: a block takes 0.86 us (in windows
// of 256 to 2,048), its products 0.67, and some 900 short tiles 4 us each for
// their start and end.  32 requests of 6 rows: 25.0 us, 2.8 TB/s; with the L2
// flushed, in a trace: 6 us from the launch to the first copy, 11 us of copies
// at the full HBM rate, then the last block, and 5 us in which a cluster joins.
#pragma once
#include <cuda.h>
#include <string.h>

#include <type_traits>

#include "common.cuh"
#include "kv_attn.cuh"
#include "tc_util.cuh"

namespace qsa {

constexpr int kWtThreads = 384;          // 8 softmax warps; K, MMAs, tiles and Q, V
constexpr int kWtN = 128;                // entries per block
constexpr int kWtStageBytes = 32768;
constexpr int kWtBadRing = 8;
constexpr int kWtTileRing = 3;

// Stage contents.  K: 128 entries x 128 columns (a block of D = 256 takes
// two); V: 64 entries x 256 columns or 128 x 128.  Both as [8-row group][64
// columns][8 rows][128 B], 128-byte swizzled: a box of whole 8-row groups
// fills consecutive bytes.
template <int D>
struct WtShape {
  static constexpr int kKs = D / 128;               // K stages of a block
  static constexpr int kVRows = D == 256 ? 64 : 128;  // entries of a V stage
  static constexpr int kVs = kWtN / kVRows;         // V stages of a full block
  static constexpr uint32_t kKGroup = 2 * 1024, kVGroup = D / 64 * 1024;  // bytes of an 8-row group
  static constexpr uint32_t kColS = D, kColP = D + kWtN;  // S: N columns; P: two buffers of N / 2
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kStages = D == 256 ? 5 : 6;  // of K and V: 224 KB with Q
  static_assert(D + 2 * kWtN <= 512, "tensor memory");
};

struct WtArgs {
  const uint16_t* q;         // rows of h_q * D BF16, ld_q apart
  const uint16_t *k, *v;     // the cache
  int64_t ld_q;
  int64_t n_slots;
  int32_t n_rows, h_q, h_kv, group;
  int32_t rows;              // R: rows per tile
  int32_t n_req;
  const int32_t* req_row_start;
  const int32_t* row_len;
  int32_t max_len, window, n_sink;
  const int32_t* page_table;
  int64_t ld_pt;
  int32_t page_size;
  int32_t box, box_shift;    // B: rows per copy, 8 to 64, dividing the page; its logarithm
  int32_t tile_slots;        // n_rows / R + n_req
  int32_t cluster;           // C: CTAs that share a tile, 1 to 8 (1 from kWtExactReq requests on)
  float c;                   // |scale| log2 e, positive
  uint32_t flip;             // sign bit to flip in S (a negative scale)
  uint16_t* out;             // [n_rows][h_q][D] BF16
  float* lse;                // [n_rows][h_q] or nullptr
  int32_t wait_ms;           // limit of a wait, without what wt_redo adds to it
};

// tcgen05.ld with its wait in one statement, so that no use of the registers
// can be scheduled between the two.
__device__ __forceinline__ void wt_tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wt_tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
        "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
        "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
        "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
        "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void wt_tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
        "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
        "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void wt_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The copies and what announces them: by one elected lane of a whole warp, as the MMAs.
__device__ __forceinline__ void wt_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void wt_arrive(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void wt_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void wt_tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The MMA issuer runs as a whole warp and one elected lane issues: its
// descriptors then live in uniform registers.  (Behind a branch on the lane,
// moving them there took about 85 clocks an MMA, where a 128 x 128 x 16
// product takes 64.)
// A K stage's product: S (+)= Q K^T over 128 columns, eight MMAs of 16 (four
// to a 64-column tile of Q, 16 KB, and to one of the stage's two groups of
// K's, 1 KB).  One statement, one election: eight statements made the chunk of
// 4,096 rows 84.7 us instead of 81.0.
__device__ __forceinline__ void wt_mma_qk(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1024;\n\tadd.u64 b, %2, 64;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1026;\n\tadd.u64 b, %2, 66;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1028;\n\tadd.u64 b, %2, 68;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, 1030;\n\tadd.u64 b, %2, 70;\n\t@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Up to four MMAs of 16 entries, O (+)= P V: P (tensor memory, 8 columns each)
// and V's rows, G descriptor units apart; the first n of them.
template <uint32_t G>
__device__ __forceinline__ void wt_mma_pv(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                          int n) {
  asm volatile(
      "{\n\t.reg .pred p, q, t, u;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "setp.gt.and.s32 u, %5, 0, q;\n\t@u tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "setp.gt.and.s32 u, %5, 1, q;\n\tadd.u32 a, %1, 8;\n\tadd.u64 b, %2, %6;\n\t"
      "@u tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "setp.gt.and.s32 u, %5, 2, q;\n\tadd.u32 a, %1, 16;\n\tadd.u64 b, %2, %7;\n\t"
      "@u tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "setp.gt.and.s32 u, %5, 3, q;\n\tadd.u32 a, %1, 24;\n\tadd.u64 b, %2, %8;\n\t"
      "@u tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(n), "n"(G), "n"(2 * G), "n"(3 * G)
      : "memory");
}
__device__ __forceinline__ void wt_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void wt_tma_4d(void* dst, const CUtensorMap* map, int z, int w, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], "
      "[%5];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// MN-major, 128-byte swizzle: groups of 64 columns 1024 bytes apart, groups
// of 8 rows (the K index) `group` bytes apart.
__device__ __forceinline__ uint64_t wt_desc_mn(uint32_t smem_addr, uint32_t group) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(1024u >> 4) << 16;
  d |= (uint64_t)(group >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

struct WtTile {
  int r, g;            // request, KV head
  int parts;           // CTAs of the cluster that share the tile
  int t0, rows;        // rows t0 .. t0 + rows - 1; 0: nothing to do, -1: no more tiles
  int start, nsr;      // see above
  int j0;              // first box of this CTA's part
  int n_box, n_blk;    // boxes from there on, blocks of N entries of the part
  int ua, ub, uc;      // entries that some pair sees, from the part's first: [0, ua) and [ub, uc)
};

// Tiles of request i; 0 where the grouping is wrong.
__device__ __forceinline__ int wt_request_tiles(const WtArgs& a, int i) {
  if (i >= a.n_req) return 0;
  const int row0 = ld_in(a.req_row_start + i), row1 = ld_in(a.req_row_start + i + 1);
  if (row0 < 0 || row1 < row0 || row1 > a.n_rows) {
    raise_fault(kFaultGrouping);
    return 0;
  }
  return (row1 - row0 + a.rows - 1) / a.rows;
}

// Up to kWtExactReq requests: lane g's number of tiles before requests
// 32 g .. 32 g + 31; the return value is the number of all tiles.
constexpr int kWtExactReq = 1024;
__device__ __forceinline__ int wt_count(const WtArgs& a, int& before) {
  const int lane = threadIdx.x & 31;
  int mine = 0;
#pragma unroll 4
  for (int g = 0; g * 32 < a.n_req; ++g) {
    const int n = __reduce_add_sync(0xffffffffu, wt_request_tiles(a, g * 32 + lane));
    if (lane == g) mine = n;
  }
  int incl = mine;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  before = incl - mine;
  return __shfl_sync(0xffffffffu, incl, 31);
}

// Request of tile `rank`, which becomes the tile's number in the request.
__device__ __forceinline__ int wt_find(const WtArgs& a, int before, int& rank) {
  const int lane = threadIdx.x & 31;
  const int g = 31 - __clz(__ballot_sync(0xffffffffu, before <= rank && lane * 32 < a.n_req));
  rank -= __shfl_sync(0xffffffffu, before, g);
  const int n = wt_request_tiles(a, g * 32 + lane);
  int incl = n;
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, incl > rank)) - 1;
  rank -= __shfl_sync(0xffffffffu, incl - n, l);
  return g * 32 + l;
}

// More requests: slot s, with request r's tiles from slot req_row_start[r] / R
// + r on (enough room, since the requests before it have at most that many
// tiles); slots past a request's last tile are empty (-1).  `rank` becomes the
// tile's number in the request.
__device__ __forceinline__ int wt_find_slot(const WtArgs& a, int s, int& rank) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.n_req + 1;  // the last i with start[i] / R + i <= s, 32 samples a round
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && ld_in(a.req_row_start + lo + i) / a.rows + lo + i <= s;
    const int k = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
    if (step == 1) break;
  }
  if (lo >= a.n_req) return -1;
  rank = s - (ld_in(a.req_row_start + lo) / a.rows + lo);
  return rank < wt_request_tiles(a, lo) ? lo : -1;
}

// Tile `rank` of request r, or this CTA's part of it.  By a whole warp.
__device__ __forceinline__ WtTile wt_tile(const WtArgs& a, int r, int rank, int parts, int part) {
  const int lane = threadIdx.x & 31;
  WtTile w{};
  w.r = r;
  w.parts = parts;
  w.t0 = ld_in(a.req_row_start + r) + rank * a.rows;
  w.rows = min(a.rows, ld_in(a.req_row_start + r + 1) - w.t0);
  const int t0 = w.t0;
  int first = INT32_MAX, last = 0;
  for (int i = lane; i < w.rows; i += 32) {
    const int L = ld_in(a.row_len + t0 + i);
    if (L < 0 || L > a.max_len) {
      raise_fault(kFaultGrouping);
    } else if (L > 0) {
      first = min(first, max(0, L - a.window));
      last = max(last, L);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  if (last == 0) return w;  // rows of no tokens: no blocks
  const int B = a.box;
  w.start = first & ~(B - 1);
  w.nsr = (min(a.n_sink, w.start) + B - 1) & ~(B - 1);
  const int n_box = w.nsr / B + (last - w.start + B - 1) / B, n_blk = (n_box * B + kWtN - 1) / kWtN;
  const int b0 = n_blk * part / parts, e0 = b0 * kWtN;
  w.j0 = e0 / B;
  w.n_box = n_box - w.j0;
  w.n_blk = n_blk * (part + 1) / parts - b0;
  w.ua = min(a.n_sink, last) - e0;
  w.ub = w.nsr + first - w.start - e0;
  w.uc = w.nsr + last - w.start - e0;
  return w;
}

// The part's box j, on a page out of range: a fault if some row of the tile
// attends to one of its positions.  (Where the windows of the rows lie apart,
// boxes between them belong to none.)  A lane with `ask` asks.  The tile comes
// by value: by reference it was kept in memory (prompts 43.5 us instead of 43.1).
__device__ __noinline__ void wt_missing(const WtArgs& a, int t0, int rows, int j0, int nsr, int start, int j, bool ask) {
  const int e = (j0 + j) << a.box_shift;
  const int pos = e < nsr ? e : start + (e - nsr);
  bool seen = false;
  for (int i = 0; ask && i < rows; ++i) {
    const int L = ld_in(a.row_len + t0 + i);
    if (L > 0 && L <= a.max_len) seen |= pos < min(a.n_sink, L) || (pos < L && pos + a.box > L - a.window);
  }
  if (seen) raise_fault(kFaultIndex);
}

struct WtCtl {
  uint64_t full[6], empty[6];
  uint64_t s_full[2], s_free, p_full[2], pv_done[2], q_full, q_empty, drain;
  uint64_t tile_full[kWtTileRing], tile_empty[kWtTileRing];
  uint64_t pair[4];          // the two warps of a lane quarter
  uint64_t join_free, join_full;  // the cluster's CTAs take sums; all sums are here
  WtTile tile[kWtTileRing];
  float mx[2][2][128];       // [block parity][half][pair]: maxima, at the end the sums
  uint32_t bad[kWtBadRing];  // boxes of a block that are out of range
  uint32_t tmem;
  int abort, wait_ms;        // in this order: see wt_wait
};

template <int D>
constexpr int wt_smem_bytes() {  // all of it dynamic, from a 1024-byte boundary
  return WtShape<D>::kQBytes + WtShape<D>::kStages * kWtStageBytes + (int)sizeof(WtCtl);
}

// Pairs of FP32 numbers, one instruction for both.
__device__ __forceinline__ uint64_t wt_pack(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float2 wt_unpack(uint64_t v) {
  return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ uint64_t wt_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t wt_add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The lowest n bits (none below 0, all from 64).
__device__ __forceinline__ uint64_t wt_low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// Bounded wait by a whole warp, which stays together: every branch hangs on a
// vote.  (With branches on a lane's own result the
// chunk of 4,096 rows took 80.2 us instead of 73.4.)
__device__ __forceinline__ bool wt_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    const bool late = global_timer_ns() - t0 > (uint64_t)abort[1] * 1000000u;  // WtCtl::wait_ms
    if (__any_sync(0xffffffffu, late || *abort != 0)) {
      if ((threadIdx.x & 31) == 0) {
        if (*abort == 0) raise_fault(kFaultWait);
        *abort = 1;
      }
      return false;
    }
  }
  return true;
}

// The next tile of the ring, by a whole warp; false: aborted.
__device__ __forceinline__ bool wt_next_tile(WtCtl& ctl, int k, WtTile& w, volatile int* abort) {
  const int sl = k % kWtTileRing;
  if (!wt_wait(&ctl.tile_full[sl], (uint32_t)(k / kWtTileRing) & 1u, abort)) return false;
  w = ctl.tile[sl];
  __syncwarp();
  wt_arrive(&ctl.tile_empty[sl]);
  return true;
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void wt_store32(uint16_t* dst, const uint32_t* y) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]),
               "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
               : "memory");
}
// The cluster barrier, by threads of any branch.
__device__ __forceinline__ void wt_cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void wt_cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// One arrival at every CTA's barrier for what the warp wrote to them.
__device__ __forceinline__ void wt_arrive_all(uint64_t* bar, int n_cta) {
  __syncwarp();
  const int lane = threadIdx.x & 31;
  if (lane < n_cta)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_shared_rank(bar, lane)) : "memory");
}
// Wait (bounded) for arrivals from the cluster: phase 0, by a whole warp.  No
// CTA of it has summed rows once more by then (see wt_redo): tiles are shared
// where there are fewer of them than CTAs, so a shared one is its CTAs' first.
__device__ __forceinline__ bool wt_wait_cluster(uint64_t* bar, volatile int* abort) {
  auto arrived = [&]() -> bool {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar))
        : "memory");
    return done != 0;
  };
  bool ok = true;
  const uint64_t t0 = global_timer_ns();
  while (ok && !arrived()) {
    if (*abort || global_timer_ns() - t0 > (uint64_t)abort[1] * 1000000u) {
      if (!*abort) raise_fault(kFaultWait);
      *abort = 1;
      ok = false;
    }
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void wt_tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

// In a tile, V rows that another row sees meet a weight of 0: where one holds
// an infinity or a NaN, the sum becomes NaN for rows that do not see it.  So an
// output that is not finite though its l is, is summed once more over the
// row's own entries, from the cache: `cols` columns from col0 on of one (row,
// head), by a whole warp, four entries at a time.  m and l come from the row's
// own entries alone.  Slow (a warp takes 270 to 300 clocks an entry, a tile of
// 128 pairs over 65,601 entries 0.3 s), and only then.  The roles that wait for
// this warp meanwhile must not give up: the time it takes is added to the CTA's
// limit as it passes, a millisecond or more at a time (less than that for each
// of a warp's 32 pairs is within the limit as it is).
template <int D>
__device__ __noinline__ void wt_redo(const WtArgs& a, int req, int64_t t, int g, int head, int col0, int cols, float m,
                                     float l, volatile int* abort) {
  constexpr int kPer = D / 32, kU = 4;  // dimensions of a lane, entries at a time
  using Piece = typename std::conditional<D == 256, uint4, uint2>::type;
  const int lane = threadIdx.x & 31;
  const int L = ld_in(a.row_len + t), lo = max(0, L - a.window), n_first = min(a.n_sink, lo);
  const int n = n_first + L - lo;
  uint64_t t0 = global_timer_ns();
  const int32_t* pt = a.page_table + (int64_t)req * a.ld_pt;
  float q[kPer], acc[D / 64] = {};
  for (int j = 0; j < kPer; ++j) q[j] = __uint_as_float((uint32_t)a.q[t * a.ld_q + head * D + lane * kPer + j] << 16);
  for (int e0 = 0; e0 < n; e0 += 32) {
    const uint64_t t1 = global_timer_ns();
    if (t1 - t0 >= 1000000u) {
      if (lane == 0) atomicAdd(const_cast<int*>(abort) + 1, (int)((t1 - t0) / 1000000u) + 1);  // WtCtl::wait_ms
      t0 = t1;
    }
    int64_t own = -1;  // where the lane's entry lies; -1: none, or on a page out of range
    if (e0 + lane < n) {
      const int e = e0 + lane, pos = e < n_first ? e : lo + e - n_first;
      const int64_t page = ld_in(pt + pos / a.page_size);
      if (page >= 0 && (page + 1) * a.page_size <= a.n_slots)
        own = ((page * a.page_size + pos % a.page_size) * a.h_kv + g) * D;
    }
    for (int i0 = 0; i0 < min(32, n - e0); i0 += kU) {
      float x[kU];
      uint16_t v[kU][D / 64];  // loads without a branch: behind one, each waits for itself
      int64_t at[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        at[i] = __shfl_sync(0xffffffffu, own, i0 + i);
        const int64_t from = max(at[i], (int64_t)0);
        const Piece piece = *reinterpret_cast<const Piece*>(a.k + from + lane * kPer);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) v[i][j] = a.v[from + col0 + min(lane + 32 * j, cols - 1)];
        uint32_t w[kPer / 2];
        memcpy(w, &piece, sizeof(piece));
        x[i] = 0.f;
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
          const float2 f = bf16x2_to_float2(w[j]);
          x[i] = fmaf(q[2 * j + 1], f.y, fmaf(q[2 * j], f.x, x[i]));
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int i = 0; i < kU; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        if (at[i] < 0) continue;  // the same in all lanes
        const float p = ka_ex2((__uint_as_float(__float_as_uint(x[i]) ^ a.flip) - m) * a.c);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) acc[j] = fmaf(p, __uint_as_float((uint32_t)v[i][j] << 16), acc[j]);
      }
    }
  }
  uint16_t* out = a.out + (t * a.h_q + head) * D + col0;
  for (int j = 0; j < D / 64; ++j)
    if (lane + 32 * j < cols) out[lane + 32 * j] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[j] / l));
}
// wt_redo for the lanes that ask for it, one after the other.
template <int D>
__device__ __forceinline__ void wt_redo_lanes(const WtArgs& a, const WtTile& w, bool ask, int pair, int col0, int cols,
                                              float m, float l, volatile int* abort) {
  unsigned todo = __ballot_sync(0xffffffffu, ask && l != 0.f && l == l);
  while (todo != 0) {
    const int i = __ffs(todo) - 1;
    todo &= todo - 1;
    const int p = __shfl_sync(0xffffffffu, pair, i), row = p / a.group;
    wt_redo<D>(a, w.r, w.t0 + row, w.g, w.g * a.group + p - row * a.group, __shfl_sync(0xffffffffu, col0, i), cols,
               __shfl_sync(0xffffffffu, m, i), __shfl_sync(0xffffffffu, l, i), abort);
  }
}

// A tile that the cluster's C CTAs shared: out = sum_s f_s O_s / sum_s f_s l_s,
// f_s = exp2(c (m_s - max m)), by the softmax warps.  CTA j writes columns
// [j S, (j + 1) S), S = D / C, and gets them from all (itself too) in its
// ring, which nothing uses any more: [source][4 columns][pair] vectors of
// 4, a source's groups of 4 columns kJoinGroup bytes apart (an odd number of
// vectors: no bank conflicts either way), then the l and m of all pairs.
constexpr int kWtJoinGroup = 129 * 16;
template <int D>
__device__ __forceinline__ void wt_join(const WtArgs& a, const WtTile& w, unsigned char* ring, WtCtl& ctl,
                                        uint32_t lanes, int half, int pair, bool mine, float m, float l, int rank,
                                        volatile int* abort) {
  static_assert(D / 4 * kWtJoinGroup + 8 * 1024 <= WtShape<D>::kStages * kWtStageBytes, "ring");
  const int C = a.cluster, S = D / C, groups = S / 4;
  float* lm = reinterpret_cast<float*>(ring + D / 4 * kWtJoinGroup);  // [source][l, m][pair]
  // this CTA's ring is free: its products are done, and no copy is under way
  wt_arrive_all(&ctl.join_free, C);
  if (!wt_wait_cluster(&ctl.join_free, abort)) return;
#pragma unroll 1
  for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 8) {
    if (w.n_blk == 0) break;  // m says so
    uint32_t o[8];
    wt_tmem_ld8(lanes + c, o);
    const int to = c / S;
    const uint32_t at = map_shared_rank(ring + (rank * groups + (c - to * S) / 4) * kWtJoinGroup + pair * 16, to);
    if (mine) {
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                   "r"(o[3])
                   : "memory");
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + kWtJoinGroup), "r"(o[4]), "r"(o[5]),
                   "r"(o[6]), "r"(o[7])
                   : "memory");
    }
  }
  for (int to = half; to < C; to += 2) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_shared_rank(lm + rank * 256 + pair, to)), "f"(l) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_shared_rank(lm + rank * 256 + 128 + pair, to)), "f"(m)
                 : "memory");
  }
  wt_arrive_all(&ctl.join_full, C);
  if (!wt_wait_cluster(&ctl.join_full, abort)) return;
  const float ninf = -__int_as_float(0x7f800000);
  const int vecs = S / 8, n = w.rows * a.group * vecs;  // 8 columns a thread, a row's next to each other
  for (int i0 = 0; i0 < n; i0 += 256) {
    // behind the end the last one once more, not written: another warp may have summed it again by then
    const bool own = i0 + (int)threadIdx.x < n;
    const int i = own ? i0 + (int)threadIdx.x : n - 1;
    const int p = i / vecs, v = i - p * vecs;
    float mx = ninf, ls = 0.f, acc[8] = {};
    for (int s = 0; s < C; ++s) mx = fmaxf(mx, lm[s * 256 + 128 + p]);
    for (int s = 0; s < C; ++s) {
      const float ms = lm[s * 256 + 128 + p], l_s = lm[s * 256 + p];
      if (l_s == 0.f) continue;  // nothing seen: the sums may hold anything
      const float f = ms == mx ? 1.f : ka_ex2((ms - mx) * a.c);
      ls = fmaf(f, l_s, ls);
      const unsigned char* src = ring + (s * groups + 2 * v) * kWtJoinGroup + p * 16;
      const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + kWtJoinGroup);
      acc[0] = fmaf(f, x.x, acc[0]), acc[1] = fmaf(f, x.y, acc[1]);
      acc[2] = fmaf(f, x.z, acc[2]), acc[3] = fmaf(f, x.w, acc[3]);
      acc[4] = fmaf(f, y.x, acc[4]), acc[5] = fmaf(f, y.y, acc[5]);
      acc[6] = fmaf(f, y.z, acc[6]), acc[7] = fmaf(f, y.w, acc[7]);
    }
    const float inv = ls == 0.f ? 0.f : 1.0f / ls;
    float broken = 0.f;  // NaN once a sum is not finite
#pragma unroll
    for (int j = 0; j < 8; ++j) broken = fmaf(acc[j], 0.f, broken);
    uint32_t y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * j] * inv, acc[2 * j + 1] * inv);
      y[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    const int row = p / a.group;
    const int64_t hq = (int64_t)(w.t0 + row) * a.h_q + (int64_t)w.g * a.group + (p - row * a.group);
    if (own) *reinterpret_cast<uint4*>(a.out + hq * D + rank * S + v * 8) = make_uint4(y[0], y[1], y[2], y[3]);
    if (own && rank == 0 && v == 0 && a.lse != nullptr)
      a.lse[hq] = ls == 0.f ? ninf : mx == ninf ? ls : fmaf(mx, a.c, log2f(ls)) * 0.69314718055994531f;
    __syncwarp();
    wt_redo_lanes<D>(a, w, broken != broken && own, p, rank * S + v * 8, 8, mx, ls, abort);
  }
}

template <int D>
__global__ void __launch_bounds__(kWtThreads, 1)
window_tc_kernel(const __grid_constant__ WtArgs a, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using Sh = WtShape<D>;
  constexpr int N = kWtN;
  constexpr uint32_t kQHalf = 128 * 128;
  extern __shared__ __align__(1024) unsigned char wt_smem[];
  unsigned char* q_buf = wt_smem;
  unsigned char* ring = q_buf + Sh::kQBytes;
  WtCtl& ctl = *reinterpret_cast<WtCtl*>(ring + Sh::kStages * kWtStageBytes);
  if ((smem_u32(wt_smem) & 1023u) != 0) {  // the swizzle atoms need it
    if (threadIdx.x == 0) raise_fault(kFaultWait);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort;
  const float ninf = -__int_as_float(0x7f800000);

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 10 && lane < 3) wt_prefetch(lane == 0 ? &q_map : lane == 1 ? &k_map : &v_map);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 2);   // the MMAs' commit and the issuing warp (which orders `bad`)
      mbar_init(&ctl.p_full[i], 8);
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < kWtTileRing; ++i) {
      mbar_init(&ctl.tile_full[i], 1);
      mbar_init(&ctl.tile_empty[i], 11);  // softmax warps, K, V, MMAs
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ctl.pair[i], 2);
    mbar_init(&ctl.s_free, 8);
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.q_empty, 1);
    mbar_init(&ctl.drain, 1);
    mbar_init(&ctl.join_free, 8 * a.cluster);
    mbar_init(&ctl.join_full, 8 * a.cluster);
    ctl.abort = 0;
    ctl.wait_ms = a.wait_ms;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait_primary();
  const uint32_t tmem = ctl.tmem;
  const int n_cta = a.cluster, rank = n_cta > 1 ? (int)cluster_ctarank() : 0;
  bool met = n_cta == 1;  // the cluster's CTAs all run
  if (n_cta > 1) wt_cluster_arrive();

  if (warp == 10) {
    // ---- tiles and Q ---------------------------------------------------------------
    const bool exact = a.n_req <= kWtExactReq;
    int before = 0;
    const int units = (exact ? wt_count(a, before) : a.tile_slots) * a.h_kv;
    // whole rounds of units, then a last one: shared by the clusters if there are enough
    const int grid = gridDim.x, whole = units / grid * grid;
    const bool share = n_cta > 1 && (units - whole) * n_cta <= grid;
    int k = 0, nq = 0;  // tiles published, Q copies
    auto publish = [&](const WtTile& w) -> bool {
      const int sl = k % kWtTileRing;
      if (k >= kWtTileRing && !wt_wait(&ctl.tile_empty[sl], (uint32_t)(k / kWtTileRing - 1) & 1u, abort)) return false;
      if (lane == 0) {
        ctl.tile[sl] = w;
        mbar_arrive(&ctl.tile_full[sl]);
      }
      ++k;
      return true;
    };
    bool ok = true, end = false;
    for (int u = blockIdx.x; ok && !end; u += grid) {
      end = u >= whole;  // the last round
      const bool part = share && end;
      const int v = part ? whole + (int)blockIdx.x / n_cta : u;
      if (v >= units) break;
      int i = v / a.h_kv;  // the tile's number, then its number in the request
      const int req = exact ? wt_find(a, before, i) : wt_find_slot(a, i, i);
      if (req < 0) continue;
      WtTile w = wt_tile(a, req, i, part ? n_cta : 1, part ? rank : 0);
      w.g = v % a.h_kv;
      ok = publish(w);
      if (!ok) break;
      if (w.n_blk > 0) {
        ok = nq == 0 || wt_wait(&ctl.q_empty, (uint32_t)(nq - 1) & 1u, abort);
        if (!ok) break;
        // boxes of `rows` x `group` x 64; what of the 128 rows they leave is never used
        wt_expect(&ctl.q_full, (uint32_t)(a.rows * a.group * D * 2));
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
          wt_tma_3d(q_buf + h * kQHalf, &q_map, h * 64, w.g * a.group, w.t0, &ctl.q_full);
        ++nq;
      }
    }
    if (ok) {
      WtTile none{};
      none.rows = -1;
      publish(none);
    }
    if (lane == 0 && nq > 0) mbar_wait_bounded(&ctl.q_full, (uint32_t)(nq - 1) & 1u, 20000000ull);
  } else if (warp == 8 || warp == 11) {
    // ---- K (warp 8) and V (warp 11) -----------------------------------------------------
    const bool is_k = warp == 8;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    const int B = a.box, sh = a.box_shift;
    const int per = N >> sh;                       // boxes of a block, at most 16
    const int per_st = is_k ? per : Sh::kVRows >> sh;  // and of a stage
    const uint32_t box_bytes = (uint32_t)B * (is_k ? 256u : D * 2u);
    int gb = 0, rs = 0, done = 0;                  // blocks, ring stages, own last stage + 1 so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      WtTile w;
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      const int32_t* pt = a.page_table + (int64_t)w.r * a.ld_pt;
      const int oob = (int)(a.n_slots >> 3);       // 8-row groups of the map
      // first 8-row group of the block's box `lane`; past the map (zeros)
      // where the page is out of range
      auto lookup = [&](int blk) -> int {
        const int j = blk * per + lane;
        if (blk >= w.n_blk || lane >= per || j >= w.n_box) return 0;
        const int e = (w.j0 + j) << sh;
        const int pos = e < w.nsr ? e : w.start + (e - w.nsr);
        const int pi = pos / a.page_size;
        const int64_t page = ld_in(pt + pi);
        if (page < 0 || (page + 1) * a.page_size > a.n_slots) return oob;
        return (int)((page * a.page_size + (pos - pi * a.page_size)) >> 3);
      };
      int next = lookup(0);
      for (int blk = 0; ok && blk < w.n_blk; ++blk) {
        const int row = next;
        next = lookup(blk + 1);
        const int nb = min(per, w.n_box - blk * per);
        if (is_k) {
          const uint32_t bad = __ballot_sync(0xffffffffu, lane < nb && row == oob);
          if (bad != 0) wt_missing(a, w.t0, w.rows, w.j0, w.nsr, w.start, blk * per + lane, (bad >> lane) & 1u);
          if (lane == 0) ctl.bad[(gb + blk) % kWtBadRing] = bad;
          __syncwarp();  // before the arrivals of whichever lane is elected
        }
        // stages in the order of use: K(0), K(1), V(0), K(2), V(1), ...
        int at = rs + (is_k ? Sh::kKs * blk + max(blk - 1, 0) * Sh::kVs
                            : Sh::kKs * min(blk + 2, w.n_blk) + blk * Sh::kVs);
        const int n_st = is_k ? Sh::kKs : (nb + per_st - 1) / per_st;
        for (int i = 0; ok && i < n_st; ++i, ++at) {
          const int st = at % Sh::kStages;
          const int b0 = is_k ? 0 : i * per_st, n = is_k ? nb : min(per_st, nb - b0);
          ok = at < Sh::kStages || wt_wait(&ctl.empty[st], (uint32_t)(at / Sh::kStages - 1) & 1u, abort);
          if (!ok) break;
          wt_expect(&ctl.full[st], (uint32_t)n * box_bytes);
          for (int j = 0; j < n; ++j)
            wt_tma_4d(ring + st * kWtStageBytes + j * box_bytes, map, w.g * (D / 64) + (is_k ? i * 2 : 0),
                      __shfl_sync(0xffffffffu, row, b0 + j), &ctl.full[st]);
          done = at + 1;
        }
      }
      gb += w.n_blk;
      if (w.n_blk > 0) {
        const int last = min(N, w.n_box * B - (w.n_blk - 1) * N);  // rows copied for the last block
        rs += Sh::kKs * w.n_blk + (w.n_blk - 1) * Sh::kVs + (last + Sh::kVRows - 1) / Sh::kVRows;
      }
    }
    // after an abort: copies under way land before the shared memory is
    // released (else every stage was waited for by its MMAs)
    if (lane == 0 && *abort)
      for (int j = max(0, done - Sh::kStages); j < done; ++j)
        mbar_wait_bounded(&ctl.full[j % Sh::kStages], (uint32_t)(j / Sh::kStages) & 1u, 20000000ull);
  } else if (warp == 9) {
    // ---- MMA issuer --------------------------------------------------------------------
    constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
    constexpr uint32_t kIdescO = kIdescS | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // B is MN-major
    // descriptors: the upper words never change, the lower ones by constants
    const uint64_t q_desc = umma_desc_sw128(smem_u32(q_buf)), k_desc0 = umma_desc_sw128(smem_u32(ring), Sh::kKGroup),
                   v_desc0 = wt_desc_mn(smem_u32(ring), Sh::kVGroup);
    auto add = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };  // stays inside the address field
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wt_wait(bar, parity, abort); };
    int gb = 0, nq = 0;          // blocks and Q copies so far
    int st = 0;                  // next ring stage and its parity
    uint32_t ph = 0;
    bool ok = true;
    auto next_stage = [&]() {
      wt_commit(&ctl.empty[st]);
      if (++st == Sh::kStages) {
        st = 0;
        ph ^= 1u;
      }
    };
    for (int k = 0; ok; ++k) {
      WtTile w;
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      // the same in all lanes, now known to be: the stage counter and the
      // descriptors stay in uniform registers (chunk 76.5 -> 74.7 us at the time, in a graph)
      w.n_blk = __reduce_max_sync(0xffffffffu, w.n_blk);
      w.n_box = __reduce_max_sync(0xffffffffu, w.n_box);
      w.uc = __reduce_max_sync(0xffffffffu, w.uc);
      if (w.n_blk == 0) continue;
      auto n16 = [&](int blk) { return (min(N, w.uc - blk * N) + 15) & ~15; };
      auto qk = [&](int blk) -> bool {
        const int x = gb + blk, sl = x & 1;
        const uint32_t idesc = kIdescS | ((uint32_t)(n16(blk) >> 3) << 17), d = tmem + Sh::kColS;
#pragma unroll
        for (int i = 0; i < Sh::kKs; ++i) {
          // the odd lanes wait until the scores before are read, the even ones for the keys: two
          // waits, one after the other, leave the pipe idle (chunk 70.5 us instead of 67.7)
          const bool s = i == 0 && x > 0 && (lane & 1) != 0;
          if (!wait(s ? &ctl.s_free : &ctl.full[st], s ? (uint32_t)(x - 1) & 1u : ph)) return false;
          if (i == 0) {
            __syncwarp();  // the lane that issues knows what the others waited for
            tc_fence_after();
          }
          const uint64_t kd = add(k_desc0, st * kWtStageBytes), qd = add(q_desc, i * 2 * kQHalf);
          wt_mma_qk(d, qd, kd, idesc, i > 0 ? 1u : 0u);
          next_stage();
        }
        wt_commit(&ctl.s_full[sl]);
        wt_arrive(&ctl.s_full[sl]);
        if (blk + 1 == w.n_blk) wt_commit(&ctl.q_empty);
        return true;
      };
      auto pv = [&](int blk) -> bool {
        const int x = gb + blk, sl = x & 1;
        if (!wait(&ctl.p_full[sl], (uint32_t)(x >> 1) & 1u)) return false;
        tc_fence_after();
        const int n = n16(blk), copied = min(N, w.n_box * a.box - blk * N);
        for (int e0 = 0; e0 < copied; e0 += Sh::kVRows) {
          if (!wait(&ctl.full[st], ph)) return false;
          const uint64_t vd = add(v_desc0, st * kWtStageBytes);
          const uint32_t p = tmem + Sh::kColP + sl * (N / 2) + e0 / 2;
          const int steps = min(Sh::kVRows, n - e0) / 16;  // none for rows past the last key
          const uint32_t first = blk > 0 || e0 > 0 ? 1u : 0u;
#pragma unroll
          for (int c = 0; c < Sh::kVRows / 16; c += 4)
            wt_mma_pv<(2 * Sh::kVGroup >> 4)>(tmem, p + c * 8, add(vd, c * 2 * Sh::kVGroup), kIdescO,
                                              c > 0 ? 1u : first, steps - c);
          next_stage();
        }
        wt_commit(&ctl.pv_done[sl]);
        return true;
      };
      ok = wait(&ctl.q_full, (uint32_t)nq & 1u) && qk(0);
      for (int i = 0; ok && i < w.n_blk; ++i) ok = (i + 1 >= w.n_blk || qk(i + 1)) && pv(i);
      gb += w.n_blk;
      ++nq;
    }
    // every MMA has finished before the memories are released
    wt_commit(&ctl.drain);
    mbar_wait_bounded(&ctl.drain, 0u, 20000000ull);
  } else {
    // ---- softmax and outputs: a pair in two threads ------------------------------------
    const int half = warp >> 2;                   // columns 64 half .. + 63 of S, D/2 half .. of O
    const int pair = (warp & 3) * 32 + lane;      // MMA row = tensor-memory lane
    const int row = pair / a.group, hd = pair - row * a.group;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float thr = 8.0f / a.c;                 // growth of the maximum that forces a rescale
    uint64_t* pair_bar = &ctl.pair[warp & 3];
    int gb = 0, rs = 0, n_pair = 0;               // blocks, ring stages, exchanges so far
    // both warps of the pair have written what comes before
    auto meet = [&]() -> bool {
      __syncwarp();
      wt_arrive(pair_bar);
      const bool ok = wt_wait(pair_bar, (uint32_t)n_pair & 1u, abort);
      ++n_pair;
      return ok;
    };
    bool ok = true, shared = false;
    bool ahead = false;                           // next_len is the next tile's
    int next_len = 0;
    float m = ninf, l = 0.f;
    WtTile w;
    for (int k = 0; ok; ++k) {
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      const bool mine = row < w.rows;
      const int64_t t = w.t0 + row;
      int L = next_len;
      if (!ahead) L = mine ? ld_in(a.row_len + t) : 0;
      if (L < 0 || L > a.max_len) L = 0;
      const int64_t hq = t * a.h_q + (int64_t)w.g * a.group + hd;
      m = ninf;
      l = 0.f;
      // the pair sees entries [0, va) and [vb, vc) of the part
      const int part0 = w.j0 << a.box_shift;
      const int va = min(a.n_sink, L) - part0;
      const int vb = (L > 0 ? w.nsr + max(0, L - a.window) - w.start : 0) - part0;
      const int vc = (L > 0 ? w.nsr + L - w.start : 0) - part0;
      for (int blk = 0; blk < w.n_blk; ++blk) {
        const int x = gb + blk, sl = x & 1;
        const int e0 = blk * N;
        ok = wt_wait(&ctl.s_full[sl], (uint32_t)(x >> 1) & 1u, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t bad = ctl.bad[x % kWtBadRing];
        const int c0 = e0 + 64 * half;            // first entry of this thread
        uint32_t s[64];
        wt_tmem_ld64(lanes + Sh::kColS + 64 * half, s);
        tc_fence_before();
        if (a.flip != 0) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] ^= a.flip;
        }
        if (__any_sync(0xffffffffu, bad != 0 || c0 < vb || c0 + 64 > vc)) {
          uint64_t see = wt_low_bits(va - c0) | (wt_low_bits(vc - c0) & ~wt_low_bits(vb - c0));
          if (bad != 0)
            for (int j = 0; j < 64; j += a.box < 64 ? a.box : 64)
              if ((bad >> ((64 * half + j) >> a.box_shift)) & 1u) see &= ~(wt_low_bits(a.box) << j);
          const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            s[j] = (see0 >> j) & 1u ? s[j] : 0xff800000u;
            s[32 + j] = (see1 >> j) & 1u ? s[32 + j] : 0xff800000u;
          }
        }
        __syncwarp();
        wt_arrive(&ctl.s_free);  // S is in registers
        float mx4[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
        for (int j = 0; j < 64; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(s[j]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        ctl.mx[x & 1][half][pair] = mx;
        ok = meet();
        if (!ok) break;
        tc_fence_after();
        mx = fmaxf(mx, ctl.mx[x & 1][half ^ 1][pair]);
        const bool grow = m != ninf && mx > m + thr;
        if (__any_sync(0xffffffffu, grow)) {
          // O holds every product before this block's
          ok = wt_wait(&ctl.pv_done[sl ^ 1], (uint32_t)((x - 1) >> 1) & 1u, abort);
          if (!ok) break;
          tc_fence_after();
          const float f = m != ninf && mx > m ? ka_ex2((m - mx) * a.c) : 1.0f;
          l *= f;
          if (m != ninf) m = fmaxf(m, mx);
#pragma unroll 1
          for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
            uint32_t o[32];
            wt_tmem_ld32(lanes + c, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            wt_tmem_st32(lanes + c, o);
          }
        }
        if (m == ninf) m = mx;
        const float off = m == ninf ? 0.f : -m * a.c;
        // two entries an instruction but for the exponentials (76 -> 74 us on
        // the chunk, 50 -> 48 on seven prompts, in a graph)
        const uint64_t c2 = wt_pack(a.c, a.c), off2 = wt_pack(off, off);
        uint64_t l2[2] = {0, 0};
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 x = wt_unpack(wt_fma2((uint64_t)s[2 * j + 1] << 32 | s[2 * j], c2, off2));
          const float2 e = make_float2(ka_ex2(x.x), ka_ex2(x.y));
          l2[j & 1] = wt_add2(l2[j & 1], wt_pack(e.x, e.y));
          const __nv_bfloat162 b = __floats2bfloat162_rn(e.x, e.y);
          p[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        const float2 ls = wt_unpack(wt_add2(l2[0], l2[1]));
        l += ls.x + ls.y;
        wt_tmem_st32(lanes + Sh::kColP + sl * (N / 2) + 32 * half, p);
        wt_wait_st();
        tc_fence_before();
        // V rows that no pair sees: zeros
        const int n16 = (min(N, w.uc - e0) + 15) & ~15;
        if (e0 < w.ub || e0 + n16 > w.uc) {
          // the stages' earlier contents have landed: see "Waits on stages"
          ok = blk == 0 || wt_wait(&ctl.pv_done[sl ^ 1], (uint32_t)((x - 1) >> 1) & 1u, abort);
          if (!ok) break;
          const int at = rs + Sh::kKs * min(blk + 2, w.n_blk) + blk * Sh::kVs;  // V's first stage
          for (int v = 0; ok && v * Sh::kVRows < n16; ++v) {
            const int st = (at + v) % Sh::kStages;
            ok = wt_wait(&ctl.full[st], (uint32_t)((at + v) / Sh::kStages) & 1u, abort);
            if (!ok) break;
            unsigned char* vst = ring + st * kWtStageBytes;
            const int ev = e0 + v * Sh::kVRows, rows = min(Sh::kVRows, n16 - v * Sh::kVRows);
            // entries [ua, ub) and from uc on: 16 bytes a lane, all rows of a warp's pass at once
            constexpr int kLanes = D / 8, kPass = 256 / kLanes;
            const int r0 = threadIdx.x / kLanes, col = threadIdx.x % kLanes;
            auto zero = [&](int from, int to) {
              for (int r = max(from - ev, 0) + r0; r < min(to - ev, rows); r += kPass)
                *reinterpret_cast<uint4*>(vst + (r >> 3) * Sh::kVGroup + (col >> 3) * 1024 + (r & 7) * 128 +
                                          (col & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            };
            zero(w.ua, min(w.ub, w.uc));
            zero(max(w.ua, w.uc), ev + rows);
          }
          if (!ok) break;
          fence_proxy_async_smem();
        }
        __syncwarp();
        wt_arrive(&ctl.p_full[sl]);
      }
      if (!ok) break;
      gb += w.n_blk;
      if (w.n_blk > 0) {
        const int last = min(N, w.n_box * a.box - (w.n_blk - 1) * N);  // rows copied for the last block
        rs += Sh::kKs * w.n_blk + (w.n_blk - 1) * Sh::kVs + (last + Sh::kVRows - 1) / Sh::kVRows;
      }
      // the next tile's row lengths under way beside the outputs, if it is known by now
      {
        const int sl = (k + 1) % kWtTileRing;
        ahead = __all_sync(0xffffffffu, mbar_try_wait(&ctl.tile_full[sl], (uint32_t)((k + 1) / kWtTileRing) & 1u));
        if (ahead) next_len = row < ctl.tile[sl].rows ? ld_in(a.row_len + ctl.tile[sl].t0 + row) : 0;
      }
      // ---- outputs ---------------------------------------------------------------------
      float inv = 0.f;
      if (w.n_blk > 0) {
        ctl.mx[gb & 1][half][pair] = l;  // the last block's maxima are in the other one
        ok = meet();
        if (!ok) break;
        l += ctl.mx[gb & 1][half ^ 1][pair];
        ok = meet();  // read, before the next tile's first maxima
        if (!ok) break;
        ok = wt_wait(&ctl.pv_done[(gb - 1) & 1], (uint32_t)((gb - 1) >> 1) & 1u, abort);
        if (!ok) break;
        tc_fence_after();
        inv = l == 0.f ? 0.f : 1.0f / l;
      }
      shared = w.parts > 1;
      if (shared) break;  // the cluster's last tile, and this CTA's
      // 32 columns at a time: two pieces of 32 bytes a lane, exchanged with the
      // next lane so that the two write 64 consecutive bytes of a row (written
      // a row a lane, 16 bytes each, every store met 32 lines: 4,000 clocks a tile)
      const bool odd = (lane & 1) != 0;
      const uint32_t keep = l == 0.f ? 0u : ~0u;  // a row that sees nothing: zeros, whatever the sums hold
      const long long own = mine ? (long long)(hq * D) + half * (D / 2) : -1ll;
      const long long at0 = __shfl_sync(0xffffffffu, own, lane & ~1), at1 = __shfl_sync(0xffffffffu, own, lane | 1);
      __nv_bfloat162 broken2 = __floats2bfloat162_rn(0.f, 0.f);  // NaN once a sum is not finite
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t o[32];
        if (w.n_blk > 0) {
          wt_tmem_ld32(lanes + half * (D / 2) + c, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        uint32_t y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const __nv_bfloat162 b =
              __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
          y[j] = *reinterpret_cast<const uint32_t*>(&b) & keep;
          broken2 = __hfma2(b, __floats2bfloat162_rn(0.f, 0.f), broken2);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // the even lane's second piece <-> the odd lane's first
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? y[j] : y[8 + j], 1);
          if (odd) y[j] = got;
          else y[8 + j] = got;
        }
        const int piece = c + (odd ? 16 : 0);
        if (at0 >= 0) wt_store32(a.out + at0 + piece, y);
        if (at1 >= 0) wt_store32(a.out + at1 + piece, y + 8);
      }
      tc_fence_before();
      __syncwarp();
      wt_redo_lanes<D>(a, w, mine && !(__low2float(broken2) + __high2float(broken2) == 0.f), pair, half * (D / 2), D / 2,
                       m, l, abort);
      if (mine && half == 0 && a.lse != nullptr)
        a.lse[hq] = l == 0.f ? ninf : (m == ninf ? l : (fmaf(m, a.c, log2f(l))) * 0.69314718055994531f);
    }
    if (shared) {
      if (!met) wt_cluster_wait();
      met = true;
      wt_join<D>(a, w, ring, ctl, lanes, half, pair, row < w.rows, m, l, rank, abort);
    }
  }

  // no CTA of the cluster leaves before all have written to each other
  if (n_cta > 1) {
    if (!met) wt_cluster_wait();
    wt_cluster_arrive();
    wt_cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace qsa
