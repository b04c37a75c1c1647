// window_tc.cuh -- attention over a sliding window and the first tokens for
// requests with many rows (prompts, chunks), on the fifth-generation tensor
// cores: the prefill form of window_attn on the BF16 cache.
//
// A tile is 2 R consecutive rows of one request and one KV head, R =
// floor(128 / G): its 2 R * G (row, query head) pairs are the 256 rows of the
// MMA, so the heads that share K and V share their tiles too.  Over the keys
// that any of its rows sees, in blocks of 128 entries:
//     S = Q K^T, P = exp2(c S - c m), O += P V, l += sum P
// with the running maximum m per pair; out = O / l, lse = ln 2 (c m + log2 l).
//
// Bound: 4 D flops per (pair, key): the tensor cores, as long as shared memory
// feeds them.
//
// Design (GB300).  A cluster of two CTAs on a pair of SMs walks tiles (a
// static stride); each holds R rows, half of every K block (64 entries) and
// half of V's columns, and the products are cta_group::2 ones (256 x 128 x 16
// and 256 x D x 16).  One CTA a tile had to copy and read whole K and V
// blocks: per 128 entries at D = 256, 320 KB through shared memory at 128
// bytes a clock, 2,500 clocks for products of 2,048 (measured: about 3,600).
// Per CTA:
//  - warp 10 finds the tiles and copies Q (TMA, 3-D boxes: the rows and heads
//    of a tile land as the rows of the MMA operand), a tile ahead;
//  - warps 8 (K) and 11 (V) copy into a ring of stages in the order in which
//    they are used, one TMA box of B rows (the largest power of two up to 64
//    that divides the page) and all the stage's columns a copy.  The
//    instruction takes one box at a time whichever lanes ask (about 100 clocks
//    each: boxes of 16 rows x 64 columns held the tiles at 21 bytes a clock),
//    hence large boxes and two warps.  They follow the page table; a page out
//    of range is copied from beyond the tensor map, which fills zeros.
//  - warp 9 issues the MMAs in the first CTA: S from Q and K in shared memory
//    (both K-major), O from P in tensor memory and V (MN-major: V's rows are
//    keys, the transposition is the descriptor's).  In the second CTA it tells
//    the first of copies that have landed.
//  - warps 0-7 hold a pair in two threads, 64 entries of a block each: they
//    turn S into P, exchange the maximum through shared memory, and write the
//    outputs.  (One thread a pair took 1,000 clocks for 64 entries.)
//  - The products go in the order QK(i+1) PV(i), so that a softmax has the
//    time of two products.  S has one buffer, free again as soon as the
//    softmax warps hold it in registers; P has two, and the barrier that
//    announces S(i) also covers PV(i-2), which read the one P(i) goes into.
//  - The accumulator is rescaled only when a row's maximum grew by more than
//    2^8 since the last time (the weights stay below 2^8 and the sums are
//    FP32, so nothing is lost); otherwise m stays.
//  - Weights enter the product as BF16, 2^-9 relative at most, one rounding
//    like that of the output; l sums them before the rounding, in FP32.
// Tensor memory columns: O [0, D), S the next 128, P two times 64.
//
// Entries.  With `start` the first window position of the tile rounded down
// to a box, the entries are the boxes of the first tokens before `start`
// (nsr of them, rounded up to a box; all lie below start), then the positions
// from start on.  A pair sees entries [0, a) and [b, c).  V rows that no pair
// of the tile sees are zeroed in shared memory (a weight of 0 times an
// infinity there would be NaN), or left out of the product where 16 of them
// lie together.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "kv_attn.cuh"
#include "tc_util.cuh"

namespace qsa {

constexpr int kWtThreads = 384;          // 8 softmax warps; K, MMAs, tiles and Q, V
constexpr int kWtN = 128;                // entries per block
constexpr int kWtTileRing = 3;

// Stage contents of a CTA.  K: its 64 of the block's entries x D columns; V:
// 128 entries x its half of the columns.  Both as [8-row group][64 columns][8
// rows][128 B], 128-byte swizzled: a box of whole 8-row groups fills
// consecutive bytes.
template <int D>
struct WtShape {
  static constexpr int kStageBytes = 128 * D;
  static constexpr uint32_t kKGroup = D / 64 * 1024, kVGroup = D / 128 * 1024;  // bytes of an 8-row group
  static constexpr uint32_t kColS = D, kColP = D + kWtN;
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kStages = D == 256 ? 4 : 8;  // of K and V
  static constexpr int kOutBytes = 8 * 4096;        // 32 pairs x 64 columns a softmax warp
  static_assert(D + 2 * kWtN <= 512, "tensor memory");
};

struct WtArgs {
  const uint16_t* q;         // rows of h_q * D BF16, ld_q apart
  int64_t ld_q;
  int64_t n_slots;
  int32_t n_rows, h_q, h_kv, group;
  int32_t rows;              // 2 R: rows per tile
  int32_t n_req;
  const int32_t* req_row_start;
  const int32_t* row_len;
  int32_t max_len, window, n_sink;
  const int32_t* page_table;
  int64_t ld_pt;
  int32_t page_size;
  int32_t box, box_shift;    // B: rows per copy, 8 to 64, dividing the page; its logarithm
  int32_t tile_slots;        // n_rows / (2 R) + n_req
  float c;                   // |scale| log2 e, positive
  uint32_t flip;             // sign bit to flip in S (a negative scale)
  uint16_t* out;             // [n_rows][h_q][D] BF16
  float* lse;                // [n_rows][h_q] or nullptr
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

__device__ __forceinline__ void wt_tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// The MMA issuer runs as a whole warp and one elected lane issues: its
// descriptors then live in uniform registers.  (Behind a branch on the lane,
// moving them there took about 85 clocks an MMA, where a 128 x 128 x 16
// product takes 64.)
// D[256][n] (+)= A (shared memory) * B (shared memory), over both CTAs.
__device__ __forceinline__ void wt_mma_ss(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[256][n] (+)= A (tensor memory, BF16 pairs) * B (shared memory).
__device__ __forceinline__ void wt_mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The products so far arrive on this barrier of both CTAs.
__device__ __forceinline__ void wt_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// Arrive on the first CTA's barrier.  What it announces are tensor-memory
// accesses (ordered by tcgen05's own fences) and landed copies; only V rows
// zeroed by threads need a release at cluster scope, which takes about 1,000
// clocks (every arrival with one: 84 -> 103 us for a 4,096-row chunk).
__device__ __forceinline__ void wt_arrive_first(uint64_t* bar, bool wrote = false) {
  const uint32_t to = map_shared_rank(bar, 0);
  if (wrote) asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(to) : "memory");
  else asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(to) : "memory");
}
// tm_wait for an arrival of the other CTA after it wrote to shared memory.
__device__ __forceinline__ bool wt_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wt_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (wt_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!wt_try_wait_cluster(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > 200000000ull) {
      *abort = 1;
      raise_fault(kFaultWait);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void wt_tma_4d(void* dst, const CUtensorMap* map, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
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
  int t0, rows;        // rows t0 .. t0 + rows - 1; 0: nothing to do, -1: no more tiles
  int start, nsr;      // see above
  int n_box, n_blk;    // boxes and blocks of N entries
  int ua, ub, uc;      // entries that some pair sees: [0, ua) and [ub, uc)
  int bad;             // a page of the tile is out of range
};

// First 8-row group of cache box j; -1 where its page is out of range.
__device__ __forceinline__ int wt_box(const WtArgs& a, const WtTile& w, int j) {
  const int e = j << a.box_shift;
  const int pos = e < w.nsr ? e : w.start + (e - w.nsr);
  const int pi = pos / a.page_size;
  const int64_t page = __ldg(a.page_table + (int64_t)w.r * a.ld_pt + pi);
  if (page < 0 || (page + 1) * a.page_size > a.n_slots) return -1;
  return (int)((page * a.page_size + (pos - pi * a.page_size)) >> 3);
}

// Tile of slot s: request r's tiles begin at slot req_row_start[r] / R + r
// (enough room, since the requests before it have at most that many tiles);
// slots past a request's last tile are empty.  By a whole warp.
__device__ __forceinline__ WtTile wt_tile(const WtArgs& a, int s) {
  const int lane = threadIdx.x & 31;
  WtTile w{};
  int lo = 0, n = a.n_req + 1;  // the last i with start[i] / R + i <= s, 32 samples a round
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && __ldg(a.req_row_start + lo + i) / a.rows + lo + i <= s;
    const int k = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    lo += (k - 1) * step;
    n = min(step, n - (k - 1) * step);
    if (step == 1) break;
  }
  if (lo >= a.n_req) return w;
  const int row0 = __ldg(a.req_row_start + lo), row1 = __ldg(a.req_row_start + lo + 1);
  if (row0 < 0 || row1 < row0 || row1 > a.n_rows) {
    if (lane == 0) raise_fault(kFaultGrouping);
    return w;
  }
  const int64_t t0 = row0 + (int64_t)(s - (row0 / a.rows + lo)) * a.rows;
  if (t0 < row0 || t0 >= row1) return w;
  w.r = lo;
  w.t0 = (int)t0;
  w.rows = min(a.rows, row1 - (int)t0);
  int first = INT32_MAX, last = 0;
  for (int i = lane; i < w.rows; i += 32) {
    const int L = __ldg(a.row_len + t0 + i);
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
  w.n_box = w.nsr / B + (last - w.start + B - 1) / B;
  w.n_blk = (w.n_box * B + kWtN - 1) / kWtN;
  w.ua = min(a.n_sink, last);
  w.ub = w.nsr + first - w.start;
  w.uc = w.nsr + last - w.start;
  for (int j = lane; j < w.n_box; j += 32) w.bad |= wt_box(a, w, j) < 0;
  w.bad = __any_sync(0xffffffffu, w.bad != 0);
  if (w.bad && lane == 0) raise_fault(kFaultIndex);
  return w;
}

struct WtCtl {
  uint64_t full[8], empty[8];
  uint64_t peer_full[8], peer_q;  // in the first CTA: the second one's copies have landed
  uint64_t s_full, s_free, p_full[2], pv_done[2], q_full, q_empty, drain;
  uint64_t tile_full[kWtTileRing], tile_empty[kWtTileRing];
  uint64_t pair[4];          // the two warps of a lane quarter
  WtTile tile[kWtTileRing];
  float mx[2][2][128];       // [block parity][half][pair]: maxima, at the end the sums
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr int wt_smem_bytes() {  // all of it dynamic, from a 1024-byte boundary
  return WtShape<D>::kQBytes + WtShape<D>::kStages * WtShape<D>::kStageBytes + WtShape<D>::kOutBytes + (int)sizeof(WtCtl);
}

// The lowest n bits (none below 0, all from 64).
__device__ __forceinline__ uint64_t wt_low_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// The groups of 16 entries of a block that hold one that some pair sees.
__device__ __forceinline__ uint32_t wt_steps(const WtTile& w, int blk) {
  uint32_t use = 0;
#pragma unroll
  for (int c = 0; c < kWtN / 16; ++c) {
    const int e = blk * kWtN + c * 16;
    if (e < w.ua || (e + 16 > w.ub && e < w.uc)) use |= 1u << c;
  }
  return use;
}

// Whether a block may hold V rows that no pair sees.
__device__ __forceinline__ bool wt_edge(const WtTile& w, int blk) {
  return blk * kWtN < w.ub || (blk + 1) * kWtN > w.uc;
}

// The next tile of the ring, by a whole warp; false: aborted.
__device__ __forceinline__ bool wt_next_tile(WtCtl& ctl, int k, WtTile& w, volatile int* abort) {
  const int sl = k % kWtTileRing;
  const bool ok = __all_sync(0xffffffffu, tm_wait(&ctl.tile_full[sl], (uint32_t)(k / kWtTileRing) & 1u, abort));
  if (!ok) return false;
  w = ctl.tile[sl];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&ctl.tile_empty[sl]);
  return true;
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWtThreads, 1)
window_tc_kernel(const __grid_constant__ WtArgs a, const __grid_constant__ CUtensorMap q_map,
                 const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using Sh = WtShape<D>;
  constexpr int N = kWtN;
  constexpr uint32_t kQHalf = 128 * 128;
  extern __shared__ __align__(1024) unsigned char wt_smem[];
  unsigned char* q_buf = wt_smem;
  unsigned char* ring = q_buf + Sh::kQBytes;
  unsigned char* out_buf = ring + Sh::kStages * Sh::kStageBytes;
  WtCtl& ctl = *reinterpret_cast<WtCtl*>(out_buf + Sh::kOutBytes);
  if ((smem_u32(wt_smem) & 1023u) != 0) {  // the swizzle atoms need it (alike in both CTAs)
    if (threadIdx.x == 0) raise_fault(kFaultWait);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  volatile int* abort = &ctl.abort;
  const float ninf = -__int_as_float(0x7f800000);

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
      mbar_init(&ctl.peer_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.p_full[i], 16);   // softmax warps of both CTAs
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < kWtTileRing; ++i) {
      mbar_init(&ctl.tile_full[i], 1);
      mbar_init(&ctl.tile_empty[i], 11);  // softmax warps, K, V, MMAs
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ctl.pair[i], 2);
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.s_free, 16);
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.q_empty, 1);
    mbar_init(&ctl.peer_q, 1);
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are there
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;

  if (warp == 10) {
    // ---- tiles and Q ---------------------------------------------------------------
    const int units = a.tile_slots * a.h_kv, half_rows = a.rows / 2;
    int k = 0, nq = 0;  // tiles published, Q copies
    bool ok = true;
    for (int u = blockIdx.x >> 1; ok; u += gridDim.x >> 1) {
      WtTile w{};
      if (u < units) {
        w = wt_tile(a, u / a.h_kv);
        if (w.rows == 0) continue;
        w.g = u % a.h_kv;
      } else {
        w.rows = -1;
      }
      const int sl = k % kWtTileRing;
      if (k >= kWtTileRing && lane == 0) ok = tm_wait(&ctl.tile_empty[sl], (uint32_t)(k / kWtTileRing - 1) & 1u, abort);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (lane == 0) {
        ctl.tile[sl] = w;
        mbar_arrive(&ctl.tile_full[sl]);
      }
      ++k;
      if (w.rows < 0) break;
      if (w.n_blk > 0 && lane == 0) {
        if (nq > 0) ok = tm_wait(&ctl.q_empty, (uint32_t)(nq - 1) & 1u, abort);
        if (ok) {
          // boxes of R x `group` x 64; what of the 128 rows they leave is never used
          mbar_arrive_expect_tx(&ctl.q_full, (uint32_t)(half_rows * a.group * D * 2));
          for (int h = 0; h < D / 64; ++h)
            wt_tma_3d(q_buf + h * kQHalf, &q_map, h * 64, w.g * a.group, w.t0 + rank * half_rows, &ctl.q_full);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (w.n_blk > 0 && ok) ++nq;
    }
    if (lane == 0 && nq > 0) mbar_wait_bounded(&ctl.q_full, (uint32_t)(nq - 1) & 1u, 20000000ull);
  } else if (warp == 8 || warp == 11) {
    // ---- K (warp 8) and V (warp 11) -----------------------------------------------------
    const bool is_k = warp == 8;
    const CUtensorMap* map = is_k ? &k_map : &v_map;
    const int B = a.box, sh = a.box_shift;
    const int per = N >> sh;                         // boxes of a block, at most 16
    const int per_st = is_k ? per / 2 : per;         // and of a stage
    const int b0 = is_k ? rank * per_st : 0;         // the stage's first box in the block
    const uint32_t box_bytes = (uint32_t)B * (is_k ? D * 2u : (uint32_t)D);
    const int oob = (int)(a.n_slots >> 3);           // 8-row groups of the map: zeros from there on
    int rs = 0, done = 0;                            // ring stages, own last stage + 1 so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      WtTile w;
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      auto lookup = [&](int blk) -> int {
        const int j = blk * per + b0 + lane;
        if (blk >= w.n_blk || lane >= per_st || j >= w.n_box) return -1;
        const int y = wt_box(a, w, j);
        return y < 0 ? oob : y;
      };
      int next = lookup(0);
      for (int blk = 0; ok && blk < w.n_blk; ++blk) {
        const int y = next;
        next = lookup(blk + 1);
        // the order of use: K(0), K(1), V(0), K(2), V(1), ...
        const int at = rs + (is_k ? blk + max(blk - 1, 0) : min(blk + 2, w.n_blk) + blk);
        const int st = at % Sh::kStages;
        const int n = max(0, min(per_st, w.n_box - blk * per - b0));  // 0: none of this CTA's entries
        if (at >= Sh::kStages && lane == 0) ok = tm_wait(&ctl.empty[st], (uint32_t)(at / Sh::kStages - 1) & 1u, abort);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&ctl.full[st], (uint32_t)n * box_bytes);
        __syncwarp();
        if (lane < n)
          wt_tma_4d(ring + st * Sh::kStageBytes + lane * box_bytes, map,
                    w.g * (D / 64) + (is_k ? 0 : rank * (D / 128)), y, &ctl.full[st]);
        done = at + 1;
      }
      rs += 2 * w.n_blk;
    }
    // after an abort: copies under way land before the shared memory is
    // released (else every stage was waited for by its MMAs)
    if (lane == 0 && *abort)
      for (int j = max(0, done - Sh::kStages); j < done; ++j)
        mbar_wait_bounded(&ctl.full[j % Sh::kStages], (uint32_t)(j / Sh::kStages) & 1u, 20000000ull);
  } else if (warp == 9 && rank == 1) {
    // ---- the second CTA's copies, told to the first --------------------------------------
    int rs = 0, nq = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      WtTile w;
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      if (w.n_blk == 0) continue;
      if (lane == 0) {
        ok = tm_wait(&ctl.q_full, (uint32_t)nq & 1u, abort);
        if (ok) wt_arrive_first(&ctl.peer_q);
        for (int i = 0; ok && i < 2 * w.n_blk; ++i) {
          const int st = (rs + i) % Sh::kStages;
          ok = tm_wait(&ctl.full[st], (uint32_t)((rs + i) / Sh::kStages) & 1u, abort);
          if (ok) wt_arrive_first(&ctl.peer_full[st]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      rs += 2 * w.n_blk;
      ++nq;
    }
  } else if (warp == 9) {
    // ---- MMA issuer --------------------------------------------------------------------
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((256u >> 4) << 24);
    constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(N >> 3) << 17);
    constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // B is MN-major
    // descriptors: the upper words never change, the lower ones by constants
    const uint64_t q_desc = umma_desc_sw128(smem_u32(q_buf)), k_desc0 = umma_desc_sw128(smem_u32(ring), Sh::kKGroup),
                   v_desc0 = wt_desc_mn(smem_u32(ring), Sh::kVGroup);
    auto add = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };  // stays inside the address field
    int gb = 0, rs = 0, nq = 0;  // blocks, ring stages and Q copies so far
    bool ok = true;
    for (int k = 0; ok; ++k) {
      WtTile w;
      if (!wt_next_tile(ctl, k, w, abort) || w.rows < 0) break;
      if (w.n_blk == 0) continue;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, tm_wait(bar, parity, abort)); };
      auto landed = [&](int st) {
        const uint32_t ph = (uint32_t)(rs / Sh::kStages) & 1u;
        return wait(&ctl.full[st], ph) && wait(&ctl.peer_full[st], ph);
      };
      auto qk = [&](int blk) -> bool {
        const int x = gb + blk, st = rs % Sh::kStages;
        if (x >= 1 && !wait(&ctl.s_free, (uint32_t)(x - 1) & 1u)) return false;
        if (!landed(st)) return false;
        tc_fence_after();
        const uint64_t kd = add(k_desc0, st * Sh::kStageBytes);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          wt_mma_ss(tmem + Sh::kColS, add(q_desc, (c >> 2) * kQHalf + (c & 3) * 32),
                    add(kd, (c >> 2) * 1024 + (c & 3) * 32), kIdescS, c > 0 ? 1u : 0u);
        wt_commit(&ctl.empty[st]);
        ++rs;
        wt_commit(&ctl.s_full);
        if (blk + 1 == w.n_blk) wt_commit(&ctl.q_empty);
        return true;
      };
      auto pv = [&](int blk) -> bool {
        const int x = gb + blk, sl = x & 1, st = rs % Sh::kStages;
        if (!landed(st)) return false;
        const uint32_t ph = (uint32_t)(x >> 1) & 1u;
        if (wt_edge(w, blk) ? !__all_sync(0xffffffffu, wt_wait_cluster(&ctl.p_full[sl], ph, abort))
                            : !wait(&ctl.p_full[sl], ph))
          return false;
        tc_fence_after();
        const uint64_t vd = add(v_desc0, st * Sh::kStageBytes);
        const uint32_t p = tmem + Sh::kColP + sl * 64;
        const uint32_t use = wt_steps(w, blk);
        uint32_t acc = blk > 0 ? 1u : 0u;
#pragma unroll
        for (int c = 0; c < N / 16; ++c)
          if ((use >> c) & 1u) {
            wt_mma_ts(tmem, p + c * 8, add(vd, c * 2 * Sh::kVGroup), kIdescO, acc);
            acc = 1u;
          }
        wt_commit(&ctl.empty[st]);
        ++rs;
        wt_commit(&ctl.pv_done[sl]);
        return true;
      };
      ok = wait(&ctl.q_full, (uint32_t)nq & 1u) && wait(&ctl.peer_q, (uint32_t)nq & 1u) && qk(0);
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
    const int row = rank * (a.rows / 2) + pair / a.group, hd = pair % a.group;
    const bool held = pair < a.rows / 2 * a.group;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float thr = 8.0f / a.c;                 // growth of the maximum that forces a rescale
    uint64_t* pair_bar = &ctl.pair[warp & 3];
    int gb = 0, rs = 0, n_pair = 0;               // blocks, ring stages, exchanges so far
    // both warps of the pair have written what comes before
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(pair_bar);
      const bool ok = __all_sync(0xffffffffu, tm_wait(pair_bar, (uint32_t)n_pair & 1u, abort));
      ++n_pair;
      return ok;
    };
    auto length = [&](const WtTile& w) -> int {
      if (!held || row >= w.rows) return 0;
      const int L = __ldg(a.row_len + w.t0 + row);
      return L < 0 || L > a.max_len ? 0 : L;
    };
    WtTile w;
    bool ok = wt_next_tile(ctl, 0, w, abort) && w.rows >= 0;
    int L = ok ? length(w) : 0;
    for (int k = 1; ok; ++k) {
      const bool mine = held && row < w.rows;
      const int64_t hq = ((int64_t)w.t0 + row) * a.h_q + (int64_t)w.g * a.group + hd;
      float m = ninf, l = 0.f;
      // the pair sees entries [0, va) and [vb, vc)
      const int va = min(a.n_sink, L);
      const int vb = L > 0 ? w.nsr + max(0, L - a.window) - w.start : 0;
      const int vc = L > 0 ? w.nsr + L - w.start : 0;
      for (int blk = 0; blk < w.n_blk; ++blk) {
        const int x = gb + blk, sl = x & 1;
        const int e0 = blk * N, c0 = e0 + 64 * half;  // c0: first entry of this thread
        ok = __all_sync(0xffffffffu, tm_wait(&ctl.s_full, (uint32_t)x & 1u, abort));
        if (!ok) break;
        tc_fence_after();
        uint32_t s[64];
        wt_tmem_ld64(lanes + Sh::kColS + 64 * half, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) wt_arrive_first(&ctl.s_free);
        if (a.flip != 0) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] ^= a.flip;
        }
        if (__any_sync(0xffffffffu, w.bad != 0 || c0 < vb || c0 + 64 > vc)) {
          uint64_t see = wt_low_bits(va - c0) | (wt_low_bits(vc - c0) & ~wt_low_bits(vb - c0));
          if (w.bad)
            for (int j = 0; j < 64; j += a.box) {
              const int bx = (c0 + j) >> a.box_shift;
              if (bx < w.n_box && wt_box(a, w, bx) < 0) see &= ~(wt_low_bits(a.box) << j);
            }
          const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            s[j] = (see0 >> j) & 1u ? s[j] : 0xff800000u;
            s[32 + j] = (see1 >> j) & 1u ? s[32 + j] : 0xff800000u;
          }
        }
        float mx4[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
        for (int j = 0; j < 64; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], __uint_as_float(s[j]));
        float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        ctl.mx[x & 1][half][pair] = mx;
        ok = meet();
        if (!ok) break;
        mx = fmaxf(mx, ctl.mx[x & 1][half ^ 1][pair]);
        const bool grow = m != ninf && mx > m + thr;
        if (__any_sync(0xffffffffu, grow)) {
          // O holds every product before this block's
          ok = __all_sync(0xffffffffu, tm_wait(&ctl.pv_done[sl ^ 1], (uint32_t)((x - 1) >> 1) & 1u, abort));
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
        float l4[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float p0 = ka_ex2(fmaf(__uint_as_float(s[2 * j]), a.c, off));
          const float p1 = ka_ex2(fmaf(__uint_as_float(s[2 * j + 1]), a.c, off));
          l4[j & 3] += p0 + p1;
          const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
          p[j] = *reinterpret_cast<const uint32_t*>(&b);
        }
        l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
        wt_tmem_st32(lanes + Sh::kColP + sl * 64 + 32 * half, p);
        wt_wait_st();
        tc_fence_before();
        // V rows that no pair sees, where the product takes them: zeros
        const bool edge = wt_edge(w, blk);
        if (edge) {
          const int at = rs + min(blk + 2, w.n_blk) + blk, st = at % Sh::kStages;  // V's stage
          ok = __all_sync(0xffffffffu, tm_wait(&ctl.full[st], (uint32_t)(at / Sh::kStages) & 1u, abort));
          if (!ok) break;
          unsigned char* vst = ring + st * Sh::kStageBytes;
          const uint32_t use = wt_steps(w, blk);
          for (int r = warp; r < N; r += 8) {  // a row a warp, 16 bytes a lane
            const int e = e0 + r;
            if (((use >> (r >> 4)) & 1u) && !(e < w.ua || (e >= w.ub && e < w.uc)) && lane < D / 16)
              *reinterpret_cast<uint4*>(vst + (r >> 3) * Sh::kVGroup + (lane >> 3) * 1024 + (r & 7) * 128 +
                                        (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) wt_arrive_first(&ctl.p_full[sl], edge);
      }
      if (!ok) break;
      gb += w.n_blk;
      rs += 2 * w.n_blk;
      // the next tile's rows, while the last products run
      WtTile nw;
      ok = wt_next_tile(ctl, k, nw, abort);
      if (!ok) break;
      const int nL = nw.rows > 0 ? length(nw) : 0;
      // ---- outputs ---------------------------------------------------------------------
      float inv = 0.f;
      if (w.n_blk > 0) {
        ctl.mx[gb & 1][half][pair] = l;  // the last block's maxima are in the other one
        ok = meet();
        if (!ok) break;
        l += ctl.mx[gb & 1][half ^ 1][pair];
        ok = meet();  // read, before the next tile's first maxima
        if (!ok) break;
        ok = __all_sync(0xffffffffu, tm_wait(&ctl.pv_done[(gb - 1) & 1], (uint32_t)((gb - 1) >> 1) & 1u, abort));
        if (!ok) break;
        tc_fence_after();
        inv = l == 0.f ? 0.f : 1.0f / l;
      }
      // 64 columns at a time through 4 KB of shared memory, so that 8 lanes
      // write 128 consecutive bytes of a row (a row a lane, every store met 32
      // lines: 4,000 clocks a tile)
      unsigned char* stage = out_buf + warp * 4096;
      const int64_t at = mine ? hq * D : -1;
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 64) {
        uint32_t o[64];
        if (w.n_blk > 0) {
          wt_tmem_ld64(lanes + c, o);
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a row that sees nothing writes zeros, whatever the accumulator holds
            const float x0 = l == 0.f ? 0.f : __uint_as_float(o[8 * j + 2 * i]) * inv;
            const float x1 = l == 0.f ? 0.f : __uint_as_float(o[8 * j + 2 * i + 1]) * inv;
            const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
            y[i] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3);
          const int64_t to = __shfl_sync(0xffffffffu, at, r);
          if (to >= 0)
            *reinterpret_cast<uint4*>(a.out + to + c + (lane & 7) * 8) =
                *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
        __syncwarp();
      }
      tc_fence_before();
      if (mine && half == 0 && a.lse != nullptr)
        a.lse[hq] = l == 0.f ? ninf : (m == ninf ? l : (fmaf(m, a.c, log2f(l))) * 0.69314718055994531f);
      w = nw;
      L = nL;
      if (w.rows < 0) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memories are in use any more
  tc_fence_after();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace qsa
