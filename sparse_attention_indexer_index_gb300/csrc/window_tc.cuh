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
// Design (GB300).  One CTA per SM walks tiles (a static stride):
//  - warp 4 copies K and V blocks into two rings of 32 KB stages by TMA, one
//    box of B rows (16, or 8 where the page is not a multiple of 16) x 64
//    columns a copy, 128-byte swizzled in whole 8-row groups.  Boxes follow the page table; a page out of
//    range is copied from beyond the tensor map, which fills zeros.
//  - warp 5 issues the MMAs: S from Q in tensor memory (read once per tile,
//    so K alone crosses shared memory) and K (K-major), O from P in tensor
//    memory and V (MN-major: V's rows are keys, the transposition is the
//    descriptor's).
//  - warps 0-3 hold one pair per thread: they put Q into tensor memory, turn
//    S into P in place, and write the outputs.
//  - Two S buffers: the order PV(i) PV(i+1) QK(i+2) QK(i+3) lets each softmax
//    run beside a product, and by the time a product may overwrite P(i) the
//    one that reads it has long finished (its barrier is waited for).
//  - The accumulator is rescaled only when a row's maximum grew by more than
//    2^8 since the last time (the weights stay below 2^8 and the sums are
//    FP32, so nothing is lost); otherwise m stays.
//  - Weights enter the product as BF16, 2^-9 relative at most, one rounding
//    like that of the output; l sums them before the rounding, in FP32.
// Tensor memory columns: O [0, D), Q [D, 3D/2), S/P two times N after it.
//
// Entries.  With `start` the first window position of the tile rounded down
// to a box, the entries are the boxes of the first tokens before `start`
// (nsr of them, rounded up to a box; all lie below start), then the positions
// from start on.  A pair sees entries [0, a) and [b, c).  V rows that no pair
// of the tile sees are zeroed in shared memory (a weight of 0 times an
// infinity there would be NaN).
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "kv_attn.cuh"
#include "tc_util.cuh"

namespace qsa {

constexpr int kWtThreads = 192;
constexpr int kWtStages = 3;
constexpr int kWtStageBytes = 32768;
constexpr int kWtSmem = 2 * kWtStages * kWtStageBytes + 1024;
constexpr int kWtBadRing = 8;

template <int D>
struct WtShape {
  static constexpr int kN = D == 256 ? 64 : 128;  // entries per block (32 KB of K)
  static constexpr uint32_t kColQ = D, kColS = D + D / 2;
  static_assert(kN * D * 2 == kWtStageBytes && kColS + 2 * kN <= 512, "tensor memory");
};

struct WtArgs {
  const uint16_t* q;         // rows of h_q * D BF16, ld_q apart
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
  int32_t box, box_shift;    // B: rows per copy, 8 or 16, dividing the page; its logarithm
  int32_t tile_slots;        // n_rows / R + n_req
  float c;                   // |scale| log2 e, positive
  uint32_t flip;             // sign bits of q to flip (a negative scale)
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

// D[128][n] += A (tensor memory, BF16 pairs) * B (shared memory).
__device__ __forceinline__ void wt_mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// MN-major, 128-byte swizzle: groups of 64 columns `lbo` bytes apart, groups
// of 8 rows (the K index) 1024 bytes apart.
__device__ __forceinline__ uint64_t wt_desc_mn(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lbo >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

struct WtTile {
  int r;               // request; rows 0: nothing to do
  int t0, rows;        // rows t0 .. t0 + rows - 1
  int start, nsr;      // see above
  int n_box, n_blk;    // boxes and blocks of N entries
  int ua, ub, uc;      // entries that some pair sees: [0, ua) and [ub, uc)
};

// Tile of slot s: request r's tiles begin at slot req_row_start[r] / R + r
// (enough room, since the requests before it have at most that many tiles);
// slots past a request's last tile are empty.  By a whole warp.
template <int N>
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
  w.n_blk = (w.n_box * B + N - 1) / N;
  w.ua = min(a.n_sink, last);
  w.ub = w.nsr + first - w.start;
  w.uc = w.nsr + last - w.start;
  return w;
}

struct WtCtl {
  uint64_t k_full[kWtStages], k_empty[kWtStages], v_full[kWtStages], v_empty[kWtStages];
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, drain;
  uint32_t bad[kWtBadRing];  // boxes of a block that are out of range
  uint32_t tmem;
  int abort;
};

template <int D>
__global__ void __launch_bounds__(kWtThreads, 1)
window_tc_kernel(const __grid_constant__ WtArgs a, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  using Sh = WtShape<D>;
  constexpr int N = Sh::kN;
  constexpr int H = D / 64;                  // 64-column halves of a row
  constexpr uint32_t kHalfBytes = N * 128;
  extern __shared__ __align__(16) unsigned char wt_smem_raw[];
  __shared__ WtCtl ctl;
  unsigned char* base = wt_smem_raw + ((1024u - (smem_u32(wt_smem_raw) & 1023u)) & 1023u);
  unsigned char* k_buf = base;
  unsigned char* v_buf = base + kWtStages * kWtStageBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort;
  const float ninf = -__int_as_float(0x7f800000);

  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWtStages; ++i) {
      mbar_init(&ctl.k_full[i], 1);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 2);   // the MMAs' commit and the issuing thread (which orders `bad`)
      mbar_init(&ctl.p_full[i], 128);
      mbar_init(&ctl.pv_done[i], 1);
    }
    mbar_init(&ctl.q_full, 128);
    mbar_init(&ctl.drain, 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem;
  const int units = a.tile_slots * a.h_kv;

  if (warp == 4) {
    // ---- producer ------------------------------------------------------------
    const int B = a.box, per = N / B;  // boxes per block, at most 32
    int gb = 0;                        // blocks so far
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const WtTile w = wt_tile<N>(a, u / a.h_kv);
      const int g = u % a.h_kv;
      const int32_t* pt = a.page_table + (int64_t)w.r * a.ld_pt;
      // first cache row of the block's box `lane`; n_slots (zeros) where the
      // page is out of range
      auto lookup = [&](int blk) -> int {
        const int j = blk * per + lane;
        if (lane >= per || j >= w.n_box) return 0;
        const int e = j * B;
        const int pos = e < w.nsr ? e : w.start + (e - w.nsr);
        const int pi = pos / a.page_size;
        const int64_t page = __ldg(pt + pi);
        if (page < 0 || (page + 1) * a.page_size > a.n_slots) return (int)a.n_slots;
        return (int)(page * a.page_size) + (pos - pi * a.page_size);
      };
      int next = w.n_blk > 0 ? lookup(0) : 0;
      for (int blk = 0; blk < w.n_blk; ++blk, ++gb) {
        const int row = next;
        if (blk + 1 < w.n_blk) next = lookup(blk + 1);
        const int nb = min(per, w.n_box - blk * per);
        const int st = gb % kWtStages;
        const uint32_t bad = __ballot_sync(0xffffffffu, lane < nb && row == (int)a.n_slots);
        if (bad != 0 && lane == 0) raise_fault(kFaultIndex);
        const int ops = nb * H;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint64_t* full = m == 0 ? &ctl.k_full[st] : &ctl.v_full[st];
          uint64_t* empty = m == 0 ? &ctl.k_empty[st] : &ctl.v_empty[st];
          bool ok = true;
          if (gb >= kWtStages && lane == 0) ok = tm_wait(empty, (uint32_t)(gb / kWtStages - 1) & 1u, abort);
          if (!__shfl_sync(0xffffffffu, ok ? 1 : 0, 0)) goto produced;
          if (lane == 0) {
            if (m == 0) ctl.bad[gb % kWtBadRing] = bad;
            mbar_arrive_expect_tx(full, (uint32_t)ops * (uint32_t)B * 128u);
          }
          __syncwarp();
          unsigned char* dst = (m == 0 ? k_buf : v_buf) + st * kWtStageBytes;
          for (int i0 = 0; i0 < ops; i0 += 32) {
            const int i = i0 + lane;
            const int bx = i / H, hf = i % H;
            const int y = __shfl_sync(0xffffffffu, row, bx & 31);
            if (i < ops)
              tma_load_2d(dst + hf * kHalfBytes + bx * B * 128, m == 0 ? &k_map : &v_map, g * D + hf * 64, y, full);
          }
        }
      }
    }
  produced:
    // every copy has landed before the shared memory is released
    if (lane == 0) {
      for (int j = max(0, gb - kWtStages); j <= gb; ++j) {
        const int st = j % kWtStages;
        const uint32_t ph = (uint32_t)(j / kWtStages) & 1u;
        if (j < gb) {
          mbar_wait_bounded(&ctl.k_full[st], ph, 20000000ull);
          mbar_wait_bounded(&ctl.v_full[st], ph, 20000000ull);
        } else if (*abort) {  // the block whose K copies may be under way
          mbar_wait_bounded(&ctl.k_full[st], ph, 20000000ull);
        }
      }
    }
  } else if (warp == 5) {
    // ---- MMA issuer --------------------------------------------------------------
    constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 4) << 24);
    constexpr uint32_t kIdescO = kIdescS | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // B is MN-major
    int gb = 0, tiles = 0;  // blocks and tiles so far
    bool ok = true;
    for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
      const WtTile w = wt_tile<N>(a, u / a.h_kv);
      if (w.n_blk == 0) continue;
      if (lane == 0) {
        const int entries = w.n_box * a.box;
        auto n16 = [&](int blk) { return (min(N, entries - blk * N) + 15) & ~15; };
        auto qk = [&](int blk) -> bool {
          const int x = gb + blk, st = x % kWtStages, sl = x & 1;
          if (!tm_wait(&ctl.k_full[st], (uint32_t)(x / kWtStages) & 1u, abort)) return false;
          // P of two blocks ago lies in this S buffer
          if (x >= 2 && !tm_wait(&ctl.pv_done[sl], (uint32_t)((x >> 1) - 1) & 1u, abort)) return false;
          tc_fence_after();
          const uint32_t idesc = kIdescS | ((uint32_t)(n16(blk) >> 3) << 17);
          const uint32_t kb = smem_u32(k_buf + st * kWtStageBytes);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            wt_mma_ts(tmem + Sh::kColS + sl * N, tmem + Sh::kColQ + k * 8,
                      umma_desc_sw128(kb + (k >> 2) * kHalfBytes + (k & 3) * 32), idesc, k > 0 ? 1u : 0u);
          umma_commit(&ctl.k_empty[st]);
          umma_commit(&ctl.s_full[sl]);
          mbar_arrive(&ctl.s_full[sl]);
          return true;
        };
        auto pv = [&](int blk) -> bool {
          const int x = gb + blk, st = x % kWtStages, sl = x & 1;
          if (!tm_wait(&ctl.v_full[st], (uint32_t)(x / kWtStages) & 1u, abort)) return false;
          if (!tm_wait(&ctl.p_full[sl], (uint32_t)(x >> 1) & 1u, abort)) return false;
          tc_fence_after();
          const uint32_t vb = smem_u32(v_buf + st * kWtStageBytes);
          const int steps = n16(blk) / 16;
          for (int k = 0; k < steps; ++k)
            wt_mma_ts(tmem, tmem + Sh::kColS + sl * N + k * 8, wt_desc_mn(vb + k * 2048, kHalfBytes), kIdescO,
                      blk > 0 || k > 0 ? 1u : 0u);
          umma_commit(&ctl.v_empty[st]);
          umma_commit(&ctl.pv_done[sl]);
          return true;
        };
        ok = tm_wait(&ctl.q_full, (uint32_t)tiles & 1u, abort);
        ok = ok && qk(0) && (w.n_blk < 2 || qk(1));
        for (int i = 0; ok && i < w.n_blk; i += 2)
          ok = pv(i) && (i + 1 >= w.n_blk || pv(i + 1)) && (i + 2 >= w.n_blk || qk(i + 2)) &&
               (i + 3 >= w.n_blk || qk(i + 3));
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      gb += w.n_blk;
      ++tiles;
    }
    if (lane == 0) {  // every MMA has finished before the memories are released
      umma_commit(&ctl.drain);
      mbar_wait_bounded(&ctl.drain, 0u, 20000000ull);
    }
  } else {
    // ---- softmax, Q and outputs: thread = pair -----------------------------------
    const int pair = threadIdx.x;                 // MMA row = tensor-memory lane
    const int row = pair / a.group, hd = pair - row * a.group;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const float thr = 8.0f / a.c;                 // growth of the maximum that forces a rescale
    int gb = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const WtTile w = wt_tile<N>(a, u / a.h_kv);
      if (w.rows == 0) continue;
      const int g = u % a.h_kv;
      const bool mine = row < w.rows;
      const int64_t t = w.t0 + row;
      int L = mine ? __ldg(a.row_len + t) : 0;
      if (L < 0 || L > a.max_len) L = 0;
      const int64_t hq = t * a.h_q + (int64_t)g * a.group + hd;
      float m = ninf, l = 0.f;
      if (w.n_blk > 0) {
        // Q row -> tensor memory (every earlier product has read the last one)
        const uint16_t* src = a.q + t * a.ld_q + ((int64_t)g * a.group + hd) * D;
#pragma unroll
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = mine ? __ldg(reinterpret_cast<const uint4*>(src + c0 * 2) + i) : make_uint4(0u, 0u, 0u, 0u);
            v[4 * i] = x.x ^ a.flip;
            v[4 * i + 1] = x.y ^ a.flip;
            v[4 * i + 2] = x.z ^ a.flip;
            v[4 * i + 3] = x.w ^ a.flip;
          }
          wt_tmem_st32(lanes + Sh::kColQ + c0, v);
        }
        wt_wait_st();
        tc_fence_before();
        mbar_arrive(&ctl.q_full);
      }
      // the pair sees entries [0, va) and [vb, vc)
      const int va = min(a.n_sink, L);
      const int vb = L > 0 ? w.nsr + max(0, L - a.window) - w.start : 0;
      const int vc = L > 0 ? w.nsr + L - w.start : 0;
      const int entries = w.n_box * a.box;
      bool ok = true;
      for (int blk = 0; blk < w.n_blk; ++blk) {
        const int x = gb + blk, sl = x & 1, st = x % kWtStages;
        const int e0 = blk * N, n = min(N, entries - e0);
        ok = __all_sync(0xffffffffu, tm_wait(&ctl.s_full[sl], (uint32_t)(x >> 1) & 1u, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t bad = ctl.bad[x % kWtBadRing];
        const uint32_t s_col = lanes + Sh::kColS + sl * N;
        uint32_t s[N];
        {
          uint32_t(&s0)[64] = *reinterpret_cast<uint32_t(*)[64]>(s);
          wt_tmem_ld64(s_col, s0);
          if constexpr (N == 128) {
            uint32_t(&s1)[64] = *reinterpret_cast<uint32_t(*)[64]>(s + 64);
            wt_tmem_ld64(s_col + 64, s1);
          }
        }
        if (__any_sync(0xffffffffu, bad != 0 || e0 < vb || e0 + N > vc)) {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const int e = e0 + j;
            const bool see = (e < va || (e >= vb && e < vc)) && !((bad >> (j >> a.box_shift)) & 1u);
            s[j] = see ? s[j] : 0xff800000u;
          }
        }
        float mx = ninf;
#pragma unroll
        for (int j = 0; j < N; ++j) mx = fmaxf(mx, __uint_as_float(s[j]));
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
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t o[32];
            wt_tmem_ld32(lanes + c0, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            wt_tmem_st32(lanes + c0, o);
          }
        }
        if (m == ninf) m = mx;
        const float off = m == ninf ? 0.f : -m * a.c;
#pragma unroll
        for (int c0 = 0; c0 < N; c0 += 64) {
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float p0 = ka_ex2(fmaf(__uint_as_float(s[c0 + 2 * j]), a.c, off));
            const float p1 = ka_ex2(fmaf(__uint_as_float(s[c0 + 2 * j + 1]), a.c, off));
            l += p0 + p1;
            const __nv_bfloat162 b = __floats2bfloat162_rn(p0, p1);
            p[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          wt_tmem_st32(s_col + c0 / 2, p);
        }
        wt_wait_st();
        tc_fence_before();
        // V rows that no pair sees: zeros
        const int n16 = (n + 15) & ~15;
        if (e0 < w.ub || e0 + n16 > w.uc) {
          ok = __all_sync(0xffffffffu, tm_wait(&ctl.v_full[st], (uint32_t)(x / kWtStages) & 1u, abort));
          if (!ok) break;
          unsigned char* vst = v_buf + st * kWtStageBytes;
          constexpr int kPieces = D / 8;  // 16-byte pieces of a row
          for (int i = threadIdx.x; i < n16 * kPieces; i += 128) {
            const int r = i / kPieces, pc = i % kPieces;
            const int e = e0 + r;
            if (!(e < w.ua || (e >= w.ub && e < w.uc)))
              *reinterpret_cast<uint4*>(vst + (pc >> 3) * kHalfBytes + r * 128 + (pc & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        mbar_arrive(&ctl.p_full[sl]);
      }
      if (!ok) break;
      gb += w.n_blk;
      // ---- outputs ----------------------------------------------------------------
      float inv = 0.f;
      if (w.n_blk > 0) {
        ok = __all_sync(0xffffffffu, tm_wait(&ctl.pv_done[(gb - 1) & 1], (uint32_t)((gb - 1) >> 1) & 1u, abort));
        if (!ok) break;
        tc_fence_after();
        inv = l == 0.f ? 0.f : 1.0f / l;
      }
      uint16_t* dst = a.out + hq * D;
#pragma unroll 2
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        if (w.n_blk > 0) {
          wt_tmem_ld32(lanes + c0, o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        if (mine) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            U8 y;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // a row that sees nothing writes zeros, whatever the accumulator holds
              const float x0 = l == 0.f ? 0.f : __uint_as_float(o[16 * j + 2 * i]) * inv;
              const float x1 = l == 0.f ? 0.f : __uint_as_float(o[16 * j + 2 * i + 1]) * inv;
              const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
              y.w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            st_32(dst + c0 + 16 * j, y);
          }
        }
      }
      tc_fence_before();
      if (mine && a.lse != nullptr)
        a.lse[hq] = l == 0.f ? ninf : (m == ninf ? l : (fmaf(m, a.c, log2f(l))) * 0.69314718055994531f);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace qsa
