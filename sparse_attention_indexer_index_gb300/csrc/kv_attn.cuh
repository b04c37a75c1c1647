// kv_attn.cuh -- softmax attention of decode rows over the K/V cache: over
// the slots of a selection (sparse_attn_fp4) or over a sliding window and the
// first tokens (window_attn, window_attn_fp4).  What the two caches share,
// and the kernel of the BF16 cache; kv4_attn.cuh has the 4-bit one's.
//
// For row t and query head h (KV head h / G), with j over the row's entries:
//     x_j = scale <q_h, k_j>,  lse = log sum_j exp(x_j),
//     out = sum_j exp(x_j - lse) v_j;   no entry: out = 0, lse = -inf.
//
// Entry e of a row that sees L tokens in a window of W with S first tokens:
// with lo = max(0, L - W) and s = min(S, lo), positions 0 .. s-1, then
// lo .. L-1 (the two never overlap), translated through the page table.
//
// Bound.  Per entry and KV head 4 D bytes are read for 4 G D flops: HBM, and
// for a few rows the latency of the chain row -> page -> data -> join.
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
//    no barrier until the row's end.  One row has at most 16 heads to a KV
//    head: a 128-row tcgen05 tile would be mostly empty.
//  - The 16 rows of an MMA tile hold 8 heads twice: in S the second half is
//    zero, in P V rows 0-7 hold the high parts of the weights and rows 8-15
//    the remainders, so the weights keep 16 significant bits at no extra MMA,
//    and the two halves of the accumulator add up.
//  - The K index of an MMA may be permuted alike in both operands: chosen so
//    that lanes read 16-byte pieces of the stage rows.
//
// Measured (BF16, in a graph): a window of 1,028 entries at 16 query heads, 2
// KV heads, D = 256: one row 7.5 us, 32 rows 17.8 us (3.8 TB/s), 64 rows 27.2 us
// (4.9 TB/s: one CTA an SM, whose three stages a warp cannot keep more bytes on
// the way).
#pragma once
#include "common.cuh"
#include "kv4.cuh"

namespace qsa {

constexpr int kKaWarps = 4;
constexpr int kKaThreads = 32 * kKaWarps;
constexpr int kKaTile = 16;        // entries per warp step
constexpr int kKaStages = 3;
constexpr int kKaMaxCluster = 8;
// The running maximum follows only when it grew by more than 2^kKaGrow: a
// warp has few tiles, and every change rescales the whole accumulator.
constexpr int kKaGrow = 5;

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

template <int D>
struct KaShape {
  static constexpr int kRow = D * 2;                  // bytes of a K or V row
  static constexpr int kStage = kKaTile * kRow * 2;   // bytes of a stage
  static constexpr int kCtas = D == 128 ? 2 : 1;      // resident CTAs the shared memory allows
};
// O in shared memory, heads x D floats: groups of GS columns padded by 4
// floats, rows by 4 more, so that the fragments' writes meet no bank twice.
template <int D, int GS>
struct KaOut {
  static constexpr int kRow = D / GS * (GS + 4) + 4;
  static __device__ __forceinline__ int col(int d) { return d / GS * (GS + 4) + d % GS; }
};
template <int D, int NT>
constexpr size_t ka_smem_bytes() {
  const size_t ring = (size_t)kKaWarps * kKaStages * KaShape<D>::kStage;
  const size_t o = (size_t)kKaWarps * NT * 8 * KaOut<D, D / 8>::kRow * 4;
  return ring > o ? ring : o;
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
__device__ __forceinline__ uint32_t ka_lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
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

// The row's entries: their number, and the slot of entry e (-1: none) in two
// parts: what is loaded, and what is made of it, so that no branch waits for
// the load where it is issued (a slot is fetched a step before its copies).
template <bool kWindow>
struct KaRow {
  int n;             // entries
  const int32_t* p;  // list, or the request's page-table row
  int lo, sinks;     // window
};
struct KaFetch {
  int32_t raw;       // slot, or page; -1: no entry
  int32_t off;       // window: offset in the page
};
template <bool kWindow>
__device__ __forceinline__ KaFetch ka_fetch(const KvAttnArgs& a, const KaRow<kWindow>& r, int e) {
  KaFetch f{-1, 0};
  if (e >= r.n) return f;
  if constexpr (kWindow) {
    const int pos = e < r.sinks ? e : r.lo + (e - r.sinks);
    const int pi = pos / a.page_size;  // < ld_pt: pos < max_len
    f.raw = ld_in(r.p + pi);
    f.off = pos - pi * a.page_size;
  } else {
    f.raw = ld_in(r.p + e);
  }
  return f;
}
template <bool kWindow>
__device__ __forceinline__ int32_t ka_slot(const KvAttnArgs& a, const KaRow<kWindow>& r, int e, const KaFetch& f) {
  if (e >= r.n) return -1;
  if constexpr (!kWindow) {
    if (f.raw < 0) return -1;
    if (f.raw >= a.n_slots) {
      raise_fault(kFaultIndex);
      return -1;
    }
    return f.raw;
  } else {
    // a page counts only if it lies wholly inside the cache
    if (f.raw < 0 || ((int64_t)f.raw + 1) * a.page_size > a.n_slots) {
      raise_fault(kFaultIndex);
      return -1;
    }
    return f.raw * a.page_size + f.off;
  }
}

// The row's entries; false: the row lies behind the last request.
template <bool kWindow>
__device__ __forceinline__ bool ka_row(const KvAttnArgs& a, int t, KaRow<kWindow>& row) {
  if constexpr (kWindow) {
    int L = ld_in(a.row_len + t);
    const int r = warp_row_request(a.req_row_start, a.n_req, t);
    if (r < 0) return false;
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
  return true;
}

// Where the CTAs of a cluster join: each CTA pushes its sums into the one
// that writes them, so that a single cluster barrier lies between (reading
// them from the others' shared memory took two, and a round trip between).
template <int D, int NT>
struct KaJoin {
  static constexpr int kQuads = NT * 8 * (D / 4) + kKaMaxCluster;  // of all CTAs together
  float4 sum[kQuads];                     // [source CTA][own quad]
  float2 ml[kKaMaxCluster][NT * 8];       // maximum and sum per source and head
};
// At the kernel's start: every CTA of the cluster runs before any is written to.
__device__ __forceinline__ void ka_cluster_arrive(int c) {
  if (c > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// The cluster's result from its CTAs' sums (so: heads x D in KaOut's layout;
// c_m, c_l: maximum and sum per head; weights hold a factor 2^bias).  Quad i
// (4 columns) of the output is written by CTA i mod C.
template <int D, int NT, int kThreads>
__device__ __forceinline__ void ka_cluster_result(const KvAttnArgs& a, const float* so, const float* c_m,
                                                  const float* c_l, KaJoin<D, NT>& join, int t, int g, int rank,
                                                  int grp, float bias) {
  using Out = KaOut<D, D / 8>;
  const int C = a.cluster;
  const float ninf = -__int_as_float(0x7f800000);
  const int quads = a.group * (D / 4), own = (quads + C - 1) / C;
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();
  if (C > 1) {
    for (int i = threadIdx.x; i < quads; i += kThreads) {
      const float4 x = *reinterpret_cast<const float4*>(so + (size_t)(i / (D / 4)) * Out::kRow + Out::col(i % (D / 4) * 4));
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                       map_shared_rank(&join.sum[rank * own + i / C], (uint32_t)(i % C))),
                   "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                   : "memory");
    }
    for (int i = threadIdx.x; i < C * a.group; i += kThreads) {
      const int h = i % a.group;
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                       map_shared_rank(&join.ml[rank][h], (uint32_t)(i / a.group))),
                   "f"(c_m[h]), "f"(c_l[h])
                   : "memory");
    }
    cluster_sync();
  }
  for (int j = threadIdx.x; j < own; j += kThreads) {
    const int idx = j * C + rank;
    if (idx >= quads) break;
    const int h = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float M, Lsum;
    float4 x;
    if (C == 1) {
      M = c_m[h];
      Lsum = c_l[h];
      x = *reinterpret_cast<const float4*>(so + (size_t)h * Out::kRow + Out::col(d));
    } else {
      M = ninf;
      for (int c = 0; c < C; ++c) M = fmaxf(M, join.ml[c][h].x);
      Lsum = 0.f;
      x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < C; ++c) {
        const float2 ml = join.ml[c][h];
        const float4 y = join.sum[c * own + j];
        const float f = ml.x == ninf ? 0.f : ka_ex2(ml.x - M);
        // a CTA without a weight (or with NaN weights only) has m = -inf
        Lsum += ml.x == ninf ? ml.y : f * ml.y;
        x.x += f * y.x;
        x.y += f * y.y;
        x.z += f * y.z;
        x.w += f * y.w;
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
      a.lse[hq] = Lsum == 0.f ? ninf : (M - bias + log2f(Lsum)) * 0.69314718055994531f;
  }
}

// One warp's part of a (row, KV head): NT tiles of 8 heads.
template <int D, int NT>
__global__ void __launch_bounds__(kKaThreads, KaShape<D>::kCtas)
kv_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using Sh = KaShape<D>;
  using Out = KaOut<D, D / 8>;
  constexpr int KS = D / 16;   // k-steps of S
  constexpr int VN = D / 8;    // n-tiles of O
  extern __shared__ __align__(128) unsigned char ka_smem[];
  __shared__ uint32_t s_mask[kKaWarps][kKaStages];       // valid entries of a stage
  __shared__ float s_m[kKaWarps][NT * 8], s_l[kKaWarps][NT * 8];
  __shared__ float c_m[NT * 8], c_l[NT * 8];     // this CTA's
  __shared__ KaJoin<D, NT> join;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int C = a.cluster;
  const int parts = C * a.n_group;
  const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  const int rank = part % C, grp = part / C;
  const int g = blockIdx.y;
  const float ninf = -__int_as_float(0x7f800000);

  pdl_wait_primary();
  KaRow<true> row;
  if (!ka_row<true>(a, t, row)) return;  // behind the last request (the same for the whole cluster)
  ka_cluster_arrive(C);
  const int tiles = (row.n + kKaTile - 1) / kKaTile;
  const int first = part * kKaWarps + warp, stride = parts * kKaWarps;

  // ---- the ring --------------------------------------------------------------
  const uint32_t ring = smem_u32(ka_smem) + (uint32_t)warp * (kKaStages * Sh::kStage);
  // Stage layout: K rows, V rows.  Rows are swizzled in
  // 16-byte pieces so that the reads below touch all 32 banks.
  auto k_off = [](int r, int c) -> uint32_t {
    return (uint32_t)(r * Sh::kRow + ((c ^ ((r & 1) << 2)) << 4));
  };
  auto v_off = [](int r, int c) -> uint32_t {
    return (uint32_t)(r * Sh::kRow + ((c ^ (r & 7)) << 4));
  };
  constexpr uint32_t kVBase = kKaTile * Sh::kRow;
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
  };
  // lane's entry of a tile (none from kKaTile on, nor past the row's end)
  auto entry = [&](int tile) -> int { return lane < kKaTile && tile < tiles ? tile * kKaTile + lane : INT32_MAX; };
  KaFetch pre[kKaStages];
#pragma unroll
  for (int i = 0; i < kKaStages; ++i) pre[i] = ka_fetch<true>(a, row, entry(first + i * stride));
#pragma unroll
  for (int i = 0; i < kKaStages - 1; ++i) {
    const int tile = first + i * stride;
    if (tile < tiles) issue(i, ka_slot<true>(a, row, entry(tile), pre[i]));
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  KaFetch next = pre[kKaStages - 1];

  // ---- q as A fragments (rows gq: heads; rows gq + 8: zero) -----------------
  // k-step s of lane tq: 4 consecutive dimensions; see the loads of K.
  uint32_t qa[NT][KS][2];
  const float mult = a.scale * 1.4426950408889634f;  // logit (base 2) = mult * accumulator
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + gq;
    const uint16_t* src = a.q + (int64_t)t * a.ld_q + ((int64_t)g * a.group + h) * D;
    constexpr int kPieces = D / 32;  // 16-byte pieces of q per lane
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int piece = tq + 4 * i;  // 8 of every 32 dimensions
      const uint4 u = h < a.group ? ld_in(reinterpret_cast<const uint4*>(src) + piece) : make_uint4(0u, 0u, 0u, 0u);
      qa[nt][2 * i][0] = u.x;
      qa[nt][2 * i][1] = u.y;
      qa[nt][2 * i + 1][0] = u.z;
      qa[nt][2 * i + 1][1] = u.w;
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
    asm volatile("cp.async.wait_group %0;" ::"n"(kKaStages - 2) : "memory");
    __syncwarp();
    {  // refill the stage that the previous step emptied
      const int ahead = tile + (kKaStages - 1) * stride;
      const int st = stage == 0 ? kKaStages - 1 : stage - 1;
      if (ahead < tiles) issue(st, ka_slot<true>(a, row, entry(ahead), next));
      asm volatile("cp.async.commit_group;" ::: "memory");
      next = ka_fetch<true>(a, row, entry(ahead + stride));
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
          x[j][e] = ok ? s[nt][j][e] * mult : ninf;
          mx = fmaxf(mx, x[j][e]);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, m[nt] != ninf && mx > m[nt] + (float)kKaGrow)) {
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
      const float ms = m[nt] == ninf ? 0.f : m[nt];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p0 = ka_ex2(x[j][0] - ms), p1 = ka_ex2(x[j][1] - ms);
        l[nt] += p0 + p1;
        ka_split<false>(p0, p1, pa[nt][2 * j], pa[nt][2 * j + 1]);
      }
    }

    // O += P V
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
    stage = stage + 1 == kKaStages ? 0 : stage + 1;
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
    float* dst = so + (size_t)(warp * NT * 8 + nt * 8 + gq) * Out::kRow;
#pragma unroll
      for (int i = 0; i < VN; ++i)
        *reinterpret_cast<float2*>(dst + Out::col(8 * i + 2 * tq)) =
            make_float2((o[nt][i][0] + o[nt][i][2]) * f, (o[nt][i][1] + o[nt][i][3]) * f);
  }
  __syncthreads();
  // the four warps' sums into warp 0's rows
  const int heads = a.group;
  for (int idx = tid; idx < heads * (D / 4); idx += kKaThreads) {
    const int h = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float* p0 = so + (size_t)h * Out::kRow + Out::col(d);
    float4 x = *reinterpret_cast<float4*>(p0);
#pragma unroll
    for (int w = 1; w < kKaWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(p0 + (size_t)w * NT * 8 * Out::kRow);
      x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
    }
    *reinterpret_cast<float4*>(p0) = x;
  }
  ka_cluster_result<D, NT, kKaThreads>(a, so, c_m, c_l, join, t, g, rank, grp, 0.f);
}

// Merge of the n_group partial results of every (row, query head); `bias` is
// the weights' exponent offset of the kernel that wrote them.
template <int D>
__global__ void __launch_bounds__(D)
kv_attn_merge_kernel(const __grid_constant__ KvAttnArgs a, float bias) {
  pdl_wait_primary();
  const int64_t hq = blockIdx.x;
  if (a.n_req > 0) {  // window rows behind the last request are left as they were
    if ((int)(hq / a.h_q) >= ld_in(a.req_row_start + a.n_req)) return;
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
