// kv_attn.cuh -- softmax attention of decode rows over the K/V cache: over
// the slots of a selection (sparse_attn_fp4) or over a sliding window and the
// first tokens (window_attn, window_attn_fp4), on a BF16 or a 4-bit cache.
//
// For row t and query head h (KV head h / G), with j over the row's entries:
//     x_j = scale <q_h, k_j>,  lse = log sum_j exp(x_j),
//     out = sum_j exp(x_j - lse) v_j;   no entry: out = 0, lse = -inf.
//
// Entry e of a row that sees L tokens in a window of W with S first tokens:
// with lo = max(0, L - W) and s = min(S, lo), positions 0 .. s-1, then
// lo .. L-1 (the two never overlap), translated through the page table.
//
// Bound.  Per entry and KV head 4 D bytes (BF16) or 9/8 D bytes (4 bits) are
// read for 4 G D flops, so HBM bounds the BF16 form; on the 4-bit form the
// instructions that unpack 2 D values per entry come close behind.
//
// Design (GB300).
//  - A cluster of C CTAs (1 to 8) serves one (row, KV head): its 16-entry
//    tiles are dealt to the cluster's warps, and the partial results meet
//    through distributed shared memory, so a row needs one launch and no
//    workspace.  Very long rows with too few clusters to fill the GPU also
//    split over n_group clusters and meet in kv_attn_merge_kernel.
//  - Each warp runs alone: a ring of cp.async stages in shared memory, and
//    per tile S = q K^T, the running maximum and sum, and O += P V, both
//    products on the tensor cores (mma.sync m16n8k16, FP32 accumulation);
//    no barrier until the row's end.  Decode has at most 16 heads to a KV
//    head: a 128-row tcgen05 tile would be mostly empty, and the unpacked
//    operands would have to go back through shared memory to reach it.
//  - The 16 rows of an MMA tile hold 8 heads twice: in S the second half is
//    zero, in P V rows 0-7 hold the high parts of the weights and rows 8-15
//    the remainders, so the weights keep 22 (FP16) or 16 (BF16) significant
//    bits at no extra MMA, and the two halves of the accumulator add up.
//  - 4-bit operands: a code times its e4m3 scale is exact in FP16, so K and V
//    enter the MMA without rounding.  q is BF16: it is brought into FP16's
//    range by a power of two per head (exact; a component below 2^-14 of the
//    head's largest loses at most 2^-25 of that largest), which the logit's
//    factor takes back.
//  - The K index of an MMA may be permuted alike in both operands, and so
//    may the columns of V: the permutations are chosen so that lanes read
//    16-byte (V, D = 128: 8-byte) pieces of the stage rows.
#pragma once
#include "common.cuh"
#include "kv4.cuh"

namespace qsa {

constexpr int kKaWarps = 4;
constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaTile = 16;        // entries per warp step
constexpr int kKaMaxCluster = 8;

struct KvAttnArgs {
  const uint16_t* q;         // rows of h_q * D BF16, ld_q apart
  int64_t ld_q;
  const uint8_t *k, *v;      // BF16 rows or codes
  const uint8_t *ks, *vs;    // scales (4-bit cache)
  int64_t n_slots;
  int32_t n_rows, h_q, h_kv, group;
  // entries: a list of slots ...
  const int32_t* slots;      // [n_rows][ld_slots]
  int64_t ld_slots;
  int32_t n_idx;
  // ... or a window
  int32_t n_req;
  const int32_t* req_row_start;
  const int32_t* row_len;
  int32_t max_len, window, n_sink;
  const int32_t* page_table;
  int64_t ld_pt;
  int32_t page_size;
  float scale;               // softmax scale times K's tensor scale
  float v_g;                 // V's tensor scale
  int32_t cluster, n_group;  // CTAs per cluster, clusters per (row, KV head)
  int32_t out_bf16;
  void* out;                 // [n_rows][h_q][D] FP32 or BF16
  float* lse;                // [n_rows][h_q] or nullptr
  float* part;               // n_group > 1: [n_rows][h_q][n_group][D + 2] (m, l, sum), m in base 2
};

template <int D, bool kFp4>
struct KaShape {
  static constexpr int kRow = kFp4 ? D / 2 : D * 2;          // bytes of a K or V row
  static constexpr int kSc = kFp4 ? D / 16 : 0;              // scale bytes of a row
  static constexpr int kStage = kKaTile * (kRow + kSc) * 2;  // bytes of a stage
  static constexpr int kStages = kFp4 ? 4 : 3;
  static constexpr int kCtas = (kFp4 || D == 128) ? 2 : 1;   // resident CTAs the shared memory allows
  // O in shared memory: groups of D/8 columns padded by 4 floats, rows by 4 more
  static constexpr int kGrp = D / 8;
  static constexpr int kORow = 8 * (kGrp + 4) + 4;
};
template <int D, int NT, bool kFp4>
constexpr size_t ka_smem_bytes() {
  using S = KaShape<D, kFp4>;
  const size_t ring = (size_t)kKaWarps * S::kStages * S::kStage;
  const size_t o = (size_t)kKaWarps * NT * 8 * S::kORow * 4;
  return (ring > o ? ring : o);
}
template <int D>
__device__ __forceinline__ int ka_o_col(int d) {
  return (d / (D / 8)) * (D / 8 + 4) + d % (D / 8);
}

__device__ __forceinline__ void ka_cp16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void ka_cp8(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8u : 0u) : "memory");
}
__device__ __forceinline__ float ka_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 ka_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 ka_lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ka_lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ka_lds_u8(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
template <bool kF16>
__device__ __forceinline__ void ka_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t ka_h2(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// Two weights as a high part and the remainder, FP16 or BF16 pairs.
template <bool kF16>
__device__ __forceinline__ void ka_split(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = ka_h2(h);
    lo = ka_h2(__floats2half2_rn(x - f.x, y - f.y));
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const float2 f = bf16x2_to_float2(hi);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

// The row's entries: their number, and the slot of entry e (-1: none).
template <bool kWindow>
struct KaRow {
  int n;             // entries
  const int32_t* p;  // list, or the request's page-table row
  int lo, sinks;     // window
};
template <bool kWindow>
__device__ __forceinline__ int32_t ka_slot(const KvAttnArgs& a, const KaRow<kWindow>& r, int e) {
  if constexpr (!kWindow) {
    if (e >= r.n) return -1;
    const int32_t s = __ldg(r.p + e);
    if (s < 0) return -1;
    if (s >= a.n_slots) {
      raise_fault(kFaultIndex);
      return -1;
    }
    return s;
  } else {
    if (e >= r.n) return -1;
    const int pos = e < r.sinks ? e : r.lo + (e - r.sinks);
    const int pi = pos / a.page_size;
    const int64_t page = __ldg(r.p + pi);  // pi < ld_pt: pos < max_len
    // a page counts only if it lies wholly inside the cache
    if (page < 0 || (page + 1) * a.page_size > a.n_slots) {
      raise_fault(kFaultIndex);
      return -1;
    }
    return (int32_t)(page * a.page_size + (pos - pi * a.page_size));
  }
}

// One warp's part of a (row, KV head): NT tiles of 8 heads.
template <int D, int NT, bool kFp4, bool kWindow>
__global__ void __launch_bounds__(kKaThreads, KaShape<D, kFp4>::kCtas)
kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using Sh = KaShape<D, kFp4>;
  constexpr int KS = D / 16;   // k-steps of S
  constexpr int VN = D / 8;    // n-tiles of O
  // Weights are held as 2^kBias p, clear of FP16's subnormals.  The running
  // maximum follows only when it grew by more than 2^kGrow (a warp has few
  // tiles, and every change rescales the whole accumulator), so a weight is
  // at most 2^(kBias + kGrow) <= 2^15.
  constexpr int kBias = kFp4 ? 10 : 0, kGrow = 5;
  extern __shared__ __align__(128) unsigned char ka_smem[];
  __shared__ uint32_t s_mask[kKaWarps][4];       // valid entries of a stage
  __shared__ float s_m[kKaWarps][NT * 8], s_l[kKaWarps][NT * 8];
  __shared__ float c_m[NT * 8], c_l[NT * 8];     // this CTA's, read by the cluster
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int C = a.cluster;
  const int parts = C * a.n_group;
  const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  const int rank = part % C, grp = part / C;
  const int g = blockIdx.y;
  const float ninf = -__int_as_float(0x7f800000);

  // ---- the row's entries ---------------------------------------------------
  KaRow<kWindow> row;
  if constexpr (kWindow) {
    int L = __ldg(a.row_len + t);
    const int r = warp_row_request(a.req_row_start, a.n_req, t);
    if (r < 0) return;  // behind the last request: the row is left as it was (the same for the whole cluster)
    if (L < 0 || L > a.max_len) {
      raise_fault(kFaultGrouping);
      L = 0;
    }
    row.lo = max(0, L - a.window);
    row.sinks = min(a.n_sink, row.lo);
    row.n = row.sinks + L - row.lo;
    row.p = a.page_table + (int64_t)r * a.ld_pt;
  } else {
    row.n = a.n_idx;
    row.p = a.slots + (int64_t)t * a.ld_slots;
    row.lo = row.sinks = 0;
  }
  const int tiles = (row.n + kKaTile - 1) / kKaTile;
  const int first = part * kKaWarps + warp, stride = parts * kKaWarps;

  // ---- the ring --------------------------------------------------------------
  const uint32_t ring = smem_u32(ka_smem) + (uint32_t)warp * (Sh::kStages * Sh::kStage);
  // Stage layout: K rows, V rows, K scales, V scales.  Rows are swizzled in
  // 16-byte pieces so that the reads below touch all 32 banks.
  auto k_off = [](int r, int c) -> uint32_t {
    if constexpr (kFp4 && D == 128) return (uint32_t)(r * 64 + c * 16);
    else return (uint32_t)(r * Sh::kRow + ((c ^ ((r & 1) << 2)) << 4));
  };
  auto v_off = [](int r, int c) -> uint32_t {
    if constexpr (!kFp4) return (uint32_t)(r * Sh::kRow + ((c ^ (r & 7)) << 4));
    else if constexpr (D == 256) return (uint32_t)(r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4));
    else {  // rows 0, 2, 4, 6 (one per lane of a quad) over both halves of 128 bytes
      const int pr = (r & 12) | ((r & 1) << 1) | ((r >> 1) & 1);
      return (uint32_t)(pr * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4));
    }
  };
  constexpr uint32_t kVBase = kKaTile * Sh::kRow;
  constexpr uint32_t kKsBase = 2 * kKaTile * Sh::kRow;
  constexpr uint32_t kVsBase = kKsBase + kKaTile * Sh::kSc;
  const uint8_t* gk = a.k + (int64_t)g * Sh::kRow;
  const uint8_t* gv = a.v + (int64_t)g * Sh::kRow;
  const int64_t pitch = (int64_t)a.h_kv * Sh::kRow;

  // copies of a tile whose entries' slots lanes 0-15 hold
  auto issue = [&](int stage, int32_t slot) {
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    constexpr int PP = Sh::kRow / 16;            // 16-byte pieces of a row
    const uint32_t valid = __ballot_sync(0xffffffffu, slot >= 0) & 0xffffu;
    if (lane == 0) s_mask[warp][stage] = valid;
#pragma unroll
    for (int u = 0; u < PP / 2; ++u) {           // 16 rows x PP pieces
      const int idx = u * 32 + lane;
      const int r = idx / PP, c = idx % PP;
      const int32_t s = __shfl_sync(0xffffffffu, slot, r);
      const int64_t off = (int64_t)max(s, 0) * pitch + c * 16;
      ka_cp16(base + k_off(r, c), gk + off, s >= 0);
      ka_cp16(base + kVBase + v_off(r, c), gv + off, s >= 0);
    }
    if constexpr (kFp4) {                        // lanes 0-15: K scales, 16-31: V scales
      const int32_t s = __shfl_sync(0xffffffffu, slot, lane & 15);
      const uint8_t* src = (lane < 16 ? a.ks : a.vs) + ((int64_t)max(s, 0) * a.h_kv + g) * Sh::kSc;
      const uint32_t dst = base + (lane < 16 ? kKsBase : kVsBase) + (lane & 15) * Sh::kSc;
      if constexpr (Sh::kSc == 16) ka_cp16(dst, src, s >= 0);
      else ka_cp8(dst, src, s >= 0);
    }
  };
  auto slot_of_tile = [&](int tile) -> int32_t {
    return lane < kKaTile && tile < tiles ? ka_slot<kWindow>(a, row, tile * kKaTile + lane) : -1;
  };
  int32_t pre[Sh::kStages];
#pragma unroll
  for (int i = 0; i < Sh::kStages; ++i) pre[i] = slot_of_tile(first + i * stride);
#pragma unroll
  for (int i = 0; i < Sh::kStages - 1; ++i) {
    if (first + i * stride < tiles) issue(i, pre[i]);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  int32_t next = pre[Sh::kStages - 1];

  // ---- q as A fragments (rows gq: heads; rows gq + 8: zero) -----------------
  // k-step s of lane tq: 4 consecutive dimensions; see the loads of K.
  uint32_t qa[NT][KS][2];
  float mult[NT];  // logit (base 2) = mult * accumulator
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + gq;
    const uint16_t* src = a.q + (int64_t)t * a.ld_q + ((int64_t)g * a.group + h) * D;
    constexpr int kPieces = D / 32;  // 16-byte pieces of q per lane
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      // 4 bits: the lane's K pieces hold 32 dimensions, so its q pieces are
      // 4 consecutive ones; BF16: one piece of 8 of every 32 dimensions
      const int piece = kFp4 ? (tq + 4 * (i >> 2)) * 4 + (i & 3) : tq + 4 * i;
      const uint4 u = h < a.group ? __ldg(reinterpret_cast<const uint4*>(src) + piece) : make_uint4(0u, 0u, 0u, 0u);
      qa[nt][2 * i][0] = u.x;
      qa[nt][2 * i][1] = u.y;
      qa[nt][2 * i + 1][0] = u.z;
      qa[nt][2 * i + 1][1] = u.w;
    }
    mult[nt] = a.scale * 1.4426950408889634f;
    if constexpr (kFp4) {
      uint32_t mx = 0;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        mx = __vmaxu2(mx, __vmaxu2(qa[nt][s][0] & 0x7fff7fffu, qa[nt][s][1] & 0x7fff7fffu));
      uint32_t top = max(mx & 0xffffu, mx >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = min(max((int)(top >> 7), 1), 253) - 127;  // exponent of the head's largest component
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
      mult[nt] *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float2 f = bf16x2_to_float2(qa[nt][s][w]);
          qa[nt][s][w] = ka_h2(__floats2half2_rn(f.x * down, f.y * down));
        }
    }
  }

  float o[NT][VN][4];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = ninf;
    l[nt] = 0.f;
#pragma unroll
    for (int i = 0; i < VN; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
  }

  // ---- tiles -------------------------------------------------------------------
  int stage = 0;
  for (int tile = first; tile < tiles; tile += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kStages - 2) : "memory");
    __syncwarp();
    {  // refill the stage that the previous step emptied
      const int ahead = tile + (Sh::kStages - 1) * stride;
      const int st = stage == 0 ? Sh::kStages - 1 : stage - 1;
      if (ahead < tiles) issue(st, next);
      asm volatile("cp.async.commit_group;" ::: "memory");
      next = slot_of_tile(ahead + stride);
    }
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    const uint32_t valid = s_mask[warp][stage];

    // S = q K^T: 16 entries as two n-tiles of 8 (lane: entry gq of each)
    float s[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[nt][j][0] = s[nt][j][1] = s[nt][j][2] = s[nt][j][3] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = j * 8 + gq;
      if constexpr (kFp4) {
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
          const uint4 w4 = ka_lds16(base + k_off(r, tq + 4 * i));
          const __half2 sc = kv4_scales(ka_lds_u16(base + kKsBase + r * Sh::kSc + 2 * (tq + 4 * i)));
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half2 sk = k < 2 ? __low2half2(sc) : __high2half2(sc);
            __half2 h[4];
            kv4_word(w[k], h);
            uint32_t b[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) b[y] = ka_h2(__hmul2(h[y], sk));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              ka_mma<true>(s[nt][j], qa[nt][i * 8 + 2 * k][0], 0u, qa[nt][i * 8 + 2 * k][1], 0u, b[0], b[1]);
              ka_mma<true>(s[nt][j], qa[nt][i * 8 + 2 * k + 1][0], 0u, qa[nt][i * 8 + 2 * k + 1][1], 0u, b[2], b[3]);
            }
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 w = ka_lds16(base + k_off(r, tq + 4 * i));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            ka_mma<false>(s[nt][j], qa[nt][2 * i][0], 0u, qa[nt][2 * i][1], 0u, w.x, w.y);
            ka_mma<false>(s[nt][j], qa[nt][2 * i + 1][0], 0u, qa[nt][2 * i + 1][1], 0u, w.z, w.w);
          }
        }
      }
    }

    // running maximum and sum; the weights as A fragments (lane: head gq,
    // entries 2 tq, 2 tq + 1 of each n-tile)
    uint32_t pa[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[2][2];
      float mx = ninf;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool ok = (valid >> (8 * j + 2 * tq + e)) & 1u;
          x[j][e] = ok ? s[nt][j][e] * mult[nt] : ninf;
          mx = fmaxf(mx, x[j][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, m[nt] != ninf && mx > m[nt] + (float)kGrow)) {
        const float mn = fmaxf(m[nt], mx);
        const float f = m[nt] == ninf ? 1.f : ka_ex2(m[nt] - mn);  // -inf: nothing yet
        l[nt] *= f;
#pragma unroll
        for (int i = 0; i < VN; ++i)
#pragma unroll
          for (int y = 0; y < 4; ++y) o[nt][i][y] *= f;
        m[nt] = mn;
      }
      if (m[nt] == ninf) m[nt] = mx;
      const float ms = m[nt] == ninf ? 0.f : m[nt] - (float)kBias;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p0 = ka_ex2(x[j][0] - ms), p1 = ka_ex2(x[j][1] - ms);
        l[nt] += p0 + p1;
        ka_split<kFp4>(p0, p1, pa[nt][2 * j], pa[nt][2 * j + 1]);
      }
    }

    // O += P V
    if constexpr (kFp4) {
      // lane: entries 2tq, 2tq+1 (b0) and 2tq+8, 2tq+9 (b1); columns
      // gq * D/8 + i of n-tile i
      const int r0 = 2 * tq;
      constexpr int kW = D / 64;  // 4-byte words of the lane's piece: 4 or 2
      uint32_t w[4][kW];
      uint32_t sc[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + (e & 1) + (e >> 1) * 8;
        if constexpr (D == 256) {
          const uint4 x = ka_lds16(base + kVBase + v_off(r, gq));
          w[e][0] = x.x; w[e][1] = x.y; w[e][2] = x.z; w[e][3] = x.w;
          sc[e] = ka_lds_u16(base + kVsBase + r * Sh::kSc + 2 * gq);
        } else {
          const uint2 x = ka_lds8(base + kVBase + v_off(r, gq >> 1) + (gq & 1) * 8);
          w[e][0] = x.x; w[e][1] = x.y;
          sc[e] = ka_lds_u8(base + kVsBase + r * Sh::kSc + gq);
        }
      }
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        // scales of the word's block for the two entries of each register
        const int sh = 8 * (k / 2);
        const __half2 s0 = kv4_scales(((sc[0] >> sh) & 0xffu) | (((sc[1] >> sh) & 0xffu) << 8));
        const __half2 s1 = kv4_scales(((sc[2] >> sh) & 0xffu) | (((sc[3] >> sh) & 0xffu) << 8));
        const uint32_t e0 = (w[0][k] & 0x0f0f0f0fu) | ((w[1][k] & 0x0f0f0f0fu) << 4);
        const uint32_t o0 = ((w[0][k] >> 4) & 0x0f0f0f0fu) | (w[1][k] & 0xf0f0f0f0u);
        const uint32_t e1 = (w[2][k] & 0x0f0f0f0fu) | ((w[3][k] & 0x0f0f0f0fu) << 4);
        const uint32_t o1 = ((w[2][k] >> 4) & 0x0f0f0f0fu) | (w[3][k] & 0xf0f0f0f0u);
        __half2 he0[4], he1[4], ho0[4], ho1[4];
        kv4_word(e0, he0);
        kv4_word(e1, he1);
        kv4_word(o0, ho0);
        kv4_word(o1, ho1);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t b0 = ka_h2(__hmul2(he0[y], s0)), b1 = ka_h2(__hmul2(he1[y], s1));
          const uint32_t b2 = ka_h2(__hmul2(ho0[y], s0)), b3 = ka_h2(__hmul2(ho1[y], s1));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            ka_mma<true>(o[nt][8 * k + 2 * y], pa[nt][0], pa[nt][1], pa[nt][2], pa[nt][3], b0, b1);
            ka_mma<true>(o[nt][8 * k + 2 * y + 1], pa[nt][0], pa[nt][1], pa[nt][2], pa[nt][3], b2, b3);
          }
        }
      }
    } else {
      // transposed 8x8 matrices: lane l addresses entry l % 16 of column
      // piece 2c + l / 16; columns 8 i + gq of n-tile i
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        uint32_t b[4];
        const int r = lane & 15;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                     : "r"(base + kVBase + v_off(r, 2 * c + (lane >> 4))));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          ka_mma<false>(o[nt][2 * c], pa[nt][0], pa[nt][1], pa[nt][2], pa[nt][3], b[0], b[1]);
          ka_mma<false>(o[nt][2 * c + 1], pa[nt][0], pa[nt][1], pa[nt][2], pa[nt][3], b[2], b[3]);
        }
      }
    }
    stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
  }

  // ---- the CTA's result ------------------------------------------------------------
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 1);
    l[nt] += __shfl_xor_sync(0xffffffffu, l[nt], 2);
    if (tq == 0) {
      s_m[warp][nt * 8 + gq] = m[nt];
      s_l[warp][nt * 8 + gq] = l[nt];
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // also: every ring is free
  float* so = reinterpret_cast<float*>(ka_smem);  // [warp][NT * 8][kORow]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float cm = ninf;
#pragma unroll
    for (int w = 0; w < kKaWarps; ++w) cm = fmaxf(cm, s_m[w][nt * 8 + gq]);
    const float f = cm == ninf ? 0.f : ka_ex2(m[nt] - cm);
    if (warp == 0 && tq == 0) {
      float cl = 0.f;
#pragma unroll
      for (int w = 0; w < kKaWarps; ++w)
        cl += s_l[w][nt * 8 + gq] * (cm == ninf ? 1.f : ka_ex2(s_m[w][nt * 8 + gq] - cm));  // all 0, or a NaN
      c_m[nt * 8 + gq] = cm;
      c_l[nt * 8 + gq] = cl;
    }
    float* dst = so + (size_t)(warp * NT * 8 + nt * 8 + gq) * Sh::kORow;
    if constexpr (kFp4) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < VN; i += 4) {
          float4 x;
          x.x = (o[nt][i][e] + o[nt][i][2 + e]) * f;
          x.y = (o[nt][i + 1][e] + o[nt][i + 1][2 + e]) * f;
          x.z = (o[nt][i + 2][e] + o[nt][i + 2][2 + e]) * f;
          x.w = (o[nt][i + 3][e] + o[nt][i + 3][2 + e]) * f;
          *reinterpret_cast<float4*>(dst + ka_o_col<D>((2 * tq + e) * VN + i)) = x;
        }
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        *reinterpret_cast<float2*>(dst + ka_o_col<D>(8 * i + 2 * tq)) =
            make_float2((o[nt][i][0] + o[nt][i][2]) * f, (o[nt][i][1] + o[nt][i][3]) * f);
    }
  }
  __syncthreads();
  // the four warps' sums into warp 0's rows
  const int heads = a.group;
  for (int idx = tid; idx < heads * (D / 4); idx += kKaThreads) {
    const int h = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float* p0 = so + (size_t)h * Sh::kORow + ka_o_col<D>(d);
    float4 x = *reinterpret_cast<float4*>(p0);
#pragma unroll
    for (int w = 1; w < kKaWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(p0 + (size_t)w * NT * 8 * Sh::kORow);
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
    *reinterpret_cast<float4*>(p0) = x;
  }
  if (C > 1) cluster_sync();
  else __syncthreads();

  // ---- the cluster's result: CTA `rank` writes its share of the columns -------
  const int quads = heads * (D / 4);
  for (int idx = rank * kKaThreads + tid; idx < quads; idx += C * kKaThreads) {
    const int h = idx / (D / 4), d = (idx % (D / 4)) * 4;
    const float* p0 = so + (size_t)h * Sh::kORow + ka_o_col<D>(d);
    float M, Lsum;
    float4 x;
    if (C == 1) {
      M = c_m[h];
      Lsum = c_l[h];
      x = *reinterpret_cast<const float4*>(p0);
    } else {
      float cm[kKaMaxCluster];
      M = ninf;
#pragma unroll
      for (int c = 0; c < kKaMaxCluster; ++c) {
        cm[c] = c < C ? __uint_as_float(ld_dsmem_u32(map_shared_rank(&c_m[h], c))) : ninf;
        M = fmaxf(M, cm[c]);
      }
      Lsum = 0.f;
      x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < kKaMaxCluster; ++c) {
        if (c < C) {
          const float f = cm[c] == ninf ? 0.f : ka_ex2(cm[c] - M);
          Lsum += f * __uint_as_float(ld_dsmem_u32(map_shared_rank(&c_l[h], c)));
          uint32_t y0, y1, y2, y3;
          asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(y0), "=r"(y1), "=r"(y2), "=r"(y3)
                       : "r"(map_shared_rank(p0, c)));
          x.x += f * __uint_as_float(y0);
          x.y += f * __uint_as_float(y1);
          x.z += f * __uint_as_float(y2);
          x.w += f * __uint_as_float(y3);
        }
      }
    }
    const int64_t hq = (int64_t)t * a.h_q + (int64_t)g * a.group + h;
    if (a.n_group > 1) {
      float* pp = a.part + (hq * a.n_group + grp) * (D + 2);
      pp[2 + d] = x.x; pp[3 + d] = x.y; pp[4 + d] = x.z; pp[5 + d] = x.w;
      if (d == 0) {
        pp[0] = M;
        pp[1] = Lsum;
      }
      continue;
    }
    const float inv = Lsum == 0.f ? 0.f : a.v_g / Lsum;
    if (a.out_bf16) {
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(x.x * inv, x.y * inv), b1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + hq * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + hq * D + d) =
          make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    }
    if (d == 0 && a.lse != nullptr)
      a.lse[hq] = Lsum == 0.f ? ninf : (M - (float)kBias + log2f(Lsum)) * 0.69314718055994531f;
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Merge of the n_group partial results of every (row, query head); `bias` is
// the weights' exponent offset of the kernel that wrote them.
template <int D>
__global__ void __launch_bounds__(D)
kv_attn_merge_kernel(const __grid_constant__ KvAttnArgs a, float bias) {
  pdl_wait_primary();
  const int64_t hq = blockIdx.x;
  if (a.n_req > 0) {  // window rows behind the last request are left as they were
    if ((int)(hq / a.h_q) >= __ldg(a.req_row_start + a.n_req)) return;
  }
  const int e = threadIdx.x;
  const float ninf = -__int_as_float(0x7f800000);
  const float* pp = a.part + hq * a.n_group * (D + 2);
  float m = ninf;
  for (int s = 0; s < a.n_group; ++s) m = fmaxf(m, pp[s * (D + 2)]);
  float l = 0.f, o = 0.f;
  for (int s = 0; s < a.n_group; ++s) {
    const float ms = pp[s * (D + 2)];
    const float c = ms == ninf ? 0.f : ka_ex2(ms - m);
    l += pp[s * (D + 2) + 1] * c;
    o += pp[s * (D + 2) + 2 + e] * c;
  }
  const float r = l == 0.f ? 0.f : o * (a.v_g / l);
  if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[hq * D + e] = __float2bfloat16_rn(r);
  else static_cast<float*>(a.out)[hq * D + e] = r;
  if (e == 0 && a.lse != nullptr) a.lse[hq] = l == 0.f ? ninf : (m - bias + log2f(l)) * 0.69314718055994531f;
}

}  // namespace qsa
