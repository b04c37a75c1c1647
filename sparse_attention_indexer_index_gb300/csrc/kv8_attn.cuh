// kv8_attn.cuh -- softmax attention of rows over the 8-bit K/V cache: over the
// slots of a selection (sparse_attn_fp8) or a window (window_attn_fp8).
//
// For row t and query head h (KV head h / G), with j over the row's entries,
// codes kc, vc and the exponents ek, ev of their blocks' scales:
//     x_j = scale 2^ek_j <q_h, kc_j>,  lse = log sum_j exp(x_j),
//     out = sum_j exp(x_j - lse) 2^ev_j vc_j;   no entry: out = 0, lse = -inf.
// So the scales enter once an entry: ek as a factor of the logit, ev as a
// factor of the weight.  The reference of both sums is the running maximum M
// of y_j = x_j + ev_j (in powers of two): the weights 2^(y_j - M) stay within
// FP16 whatever the scales are, and the normaliser sum 2^(x_j - M) within FP32
// (|ev| <= 64).
//
// Bound.  Per entry and KV head 2 D bytes are read for 4 G D flops: HBM, and
// for a few rows the latency of the chain row -> page -> data -> join.
//
// Design (GB300).
//  - A tile is 8 or 16 MT (row, query head) pairs of one KV head: a row's own
//    heads (lists, single rows), or the heads of R rows of one request that
//    see nearly the same window.  A cluster of C CTAs (1 to 8) serves it: its
//    entries are dealt in steps of kStep to the cluster's groups of MT warps,
//    and the partial results meet through distributed shared memory.  Few
//    tiles with many entries split over n_group clusters too and meet in
//    kv_attn_merge_kernel.
//  - The MT warps of a group share a ring of cp.async stages and hold 16 pairs
//    each (one barrier of the group a step); with MT = 1 a warp runs alone.
//  - A code is exact in FP16 (one conversion for two), so K and V enter the
//    MMA (mma.sync m16n8k16, FP32 accumulation) without rounding.  q is
//    brought into FP16's range by a power of two per pair, as on the 4-bit
//    cache; weights are FP16 high parts and remainders (22 bits).  With 8
//    pairs the two fill the 16 rows of one product; with 16 there are two
//    products into the same sums.
//  - K's dimensions and V's columns are permuted so that a lane reads 16-byte
//    pieces of the stage's rows without bank conflicts; V's entries meet in
//    pairs (the MMA's K index) by byte permutations before the conversion.
//  - In a shared tile some pairs do not see some entries: their weight is 0.
//    There a NaN of V counts as 0 in the product, and columns of pairs that
//    see it are set to NaN by a second product of 0/1 marks.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "kv8.cuh"
#include "kv_attn.cuh"

namespace qsa {

constexpr int kK8Bias = 10;   // weights are held as 2^kK8Bias w, w <= 2^kKaGrow

struct Kv8AttnArgs : KvAttnArgs {
  int32_t block_shift;       // log2 of the tokens to a scale
  int32_t rows;              // R: rows per tile (shared tiles)
};

// Warps and shared memory.  Two CTAs an SM, but for 64 pairs of D = 256, whose
// sums alone take 75 KB: there one of 8 warps.  (16 pairs of D = 256 leave
// room for three rings only.)
template <int D, int P, int MT>
struct K8Shape {
  static constexpr bool kWide = MT == 4 && D == 256;
  static constexpr int kCtas = kWide ? 1 : 2;
  static constexpr int kGroups = MT == 1 ? (D == 256 && P == 16 ? 3 : 4) : MT == 2 || kWide ? 2 : 1;  // groups of MT warps
  static constexpr int kThreads = 32 * MT * kGroups;
  static constexpr int kStep = kWide || D == 128 ? 32 : 16;      // entries
  static constexpr int kStage = kStep * D * 2;                   // bytes of K and V
  static constexpr int kStages = MT == 1 ? 3 : MT == 2 || kWide ? 4 : 6;
  static constexpr int kPairs = P * MT;
  static constexpr int kRing = kGroups * kStages * kStage;
  using Out = KaOut<D, D / 8>;
  static constexpr int kSums = MT * kGroups * P * Out::kRow * 4;  // a warp's sums
  static constexpr int kFront = kRing > kSums ? kRing : kSums;
  // what the cluster's other CTAs push here: sums by quads, then maxima and sums by pair
  static constexpr int kJoinQuads = kPairs * (D / 4) + kKaMaxCluster;
  static constexpr int kSmem = kFront + kJoinQuads * 16 + kKaMaxCluster * kPairs * 8;
  static_assert(kSmem <= (kCtas == 2 ? 111 : 222) * 1024, "shared memory");
};

// What a CTA's pairs are: pair p is row p / group, head p mod group of the tile.
struct K8Tile {
  int t0, rows;        // rows; 0: nothing to do
  int n;               // entries
  const int32_t* p;    // list of slots, or the request's page-table row
  int first, ns;       // window: first position behind the first tokens, and their number
};

// Tile `s` of all requests, by a whole warp: request r and the tile's number
// in it.  Up to kK8Exact requests the tiles are counted; else slot s holds
// request r's tiles from slot start[r] / R + r on (enough room: the requests
// before have at most that many), and slots past its last tile are empty.
constexpr int kK8Exact = 1024;
__device__ __forceinline__ int k8_request_tiles(const Kv8AttnArgs& a, int i) {
  if (i >= a.n_req) return 0;
  const int row0 = ld_in(a.req_row_start + i), row1 = ld_in(a.req_row_start + i + 1);
  if (row0 < 0 || row1 < row0 || row1 > a.n_rows) {
    raise_fault(kFaultGrouping);
    return 0;
  }
  return (row1 - row0 + a.rows - 1) / a.rows;
}
__device__ __forceinline__ int k8_find(const Kv8AttnArgs& a, int s, int& rank) {
  const int lane = threadIdx.x & 31;
  if (a.n_req <= kK8Exact) {
    for (int g0 = 0; g0 < a.n_req; g0 += 32) {
      const int n = k8_request_tiles(a, g0 + lane);
      int incl = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
      }
      const uint32_t behind = __ballot_sync(0xffffffffu, incl > s);
      if (behind != 0) {
        const int l = __ffs(behind) - 1;
        rank = s - __shfl_sync(0xffffffffu, incl - n, l);
        return g0 + l;
      }
      s -= __shfl_sync(0xffffffffu, incl, 31);
    }
    return -1;
  }
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
  return rank >= 0 && rank < k8_request_tiles(a, lo) ? lo : -1;
}

template <bool kWindow, bool kShared>
__device__ __forceinline__ K8Tile k8_tile(const Kv8AttnArgs& a, int s) {
  K8Tile w{};
  if constexpr (!kShared) {
    KaRow<kWindow> row;
    if (!ka_row<kWindow>(a, s, row)) return w;  // behind the last request
    w.t0 = s;
    w.rows = 1;
    w.n = row.n;
    w.p = row.p;
    w.first = row.lo;
    w.ns = row.sinks;
  } else {
    const int lane = threadIdx.x & 31;
    int rank = 0;
    const int r = k8_find(a, s, rank);
    if (r < 0) return w;
    w.t0 = ld_in(a.req_row_start + r) + rank * a.rows;
    w.rows = min(a.rows, ld_in(a.req_row_start + r + 1) - w.t0);
    w.p = a.page_table + (int64_t)r * a.ld_pt;
    int first = INT32_MAX, last = 0;
    for (int i = lane; i < w.rows; i += 32) {
      const int L = ld_in(a.row_len + w.t0 + i);
      if (L < 0 || L > a.max_len) {
        raise_fault(kFaultGrouping);
      } else if (L > 0) {
        first = min(first, max(0, L - a.window));
        last = max(last, L);
      }
    }
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (last == 0) return w;  // rows of no tokens: no entries
    w.first = first;
    w.ns = min(a.n_sink, first);
    w.n = w.ns + last - first;
  }
  return w;
}
__device__ __forceinline__ int k8_pos(const K8Tile& w, int e) { return e < w.ns ? e : w.first + (e - w.ns); }

// Whether a row of the tile attends to a position.
__device__ __noinline__ bool k8_seen(const Kv8AttnArgs& a, int t0, int rows, int pos) {
  for (int i = 0; i < rows; ++i) {
    const int L = ld_in(a.row_len + t0 + i);
    if (L > 0 && L <= a.max_len && pos < L && (pos >= L - a.window || pos < a.n_sink)) return true;
  }
  return false;
}

// An entry's slot in two parts, as in kv_attn.cuh: what is loaded, and what is
// made of it (-1: none).
template <bool kWindow>
__device__ __forceinline__ KaFetch k8_fetch(const Kv8AttnArgs& a, const K8Tile& w, int e) {
  KaFetch f{-1, 0};
  if (e >= w.n) return f;
  if constexpr (kWindow) {
    const int pos = k8_pos(w, e);
    const int pi = pos / a.page_size;  // < ld_pt: pos < max_len
    f.raw = ld_in(w.p + pi);
    f.off = pos - pi * a.page_size;
  } else {
    f.raw = ld_in(w.p + e);
  }
  return f;
}
template <bool kWindow, bool kShared>
__device__ __forceinline__ int32_t k8_slot(const Kv8AttnArgs& a, const K8Tile& w, int e, const KaFetch& f) {
  if (e >= w.n) return -1;
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
      if (!kShared || k8_seen(a, w.t0, w.rows, k8_pos(w, e))) raise_fault(kFaultIndex);
      return -1;
    }
    return f.raw * a.page_size + f.off;
  }
}

// An entry's scale bytes, K's in the low byte, and bit 16 where there is one.
__device__ __forceinline__ uint32_t k8_scales(const Kv8AttnArgs& a, int32_t slot, int g) {
  if (slot < 0) return 0u;
  const int64_t at = (int64_t)(slot >> a.block_shift) * a.h_kv + g;
  return (uint32_t)ld_in(a.ks + at) | (uint32_t)ld_in(a.vs + at) << 8 | 0x10000u;
}

template <int D, int P, int MT, bool kWindow>
__global__ void __launch_bounds__(K8Shape<D, P, MT>::kThreads, K8Shape<D, P, MT>::kCtas)
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using Sh = K8Shape<D, P, MT>;
  using Out = typename Sh::Out;
  constexpr bool kShared = kWindow && P == 16;
  constexpr int KS = D / 16, VN = D / 8;       // k-steps of S, n-tiles of O
  constexpr int NP = P / 8;                    // pairs a lane's quad holds
  constexpr int kStep = Sh::kStep, J = kStep / 8, NS = Sh::kStages;
  extern __shared__ __align__(128) unsigned char k8_smem[];
  __shared__ float s_m[MT * Sh::kGroups][P], s_l[MT * Sh::kGroups][P];
  __shared__ float c_m[Sh::kPairs], c_l[Sh::kPairs];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int mt = warp % MT, grp_w = warp / MT;  // M tile, group
  const int C = a.cluster, parts = C * a.n_group;
  const int s_tile = blockIdx.x / parts, part = blockIdx.x - s_tile * parts;
  const int rank = part % C, grp = part / C;
  const int g = blockIdx.y;
  const float ninf = -__int_as_float(0x7f800000);

  pdl_wait_primary();
  const K8Tile w = k8_tile<kWindow, kShared>(a, s_tile);
  if (w.rows == 0) return;  // no such tile (the same for the whole cluster)
  ka_cluster_arrive(C);
  const int steps = (w.n + kStep - 1) / kStep;
  const int first = part * Sh::kGroups + grp_w, stride = parts * Sh::kGroups;
  const int pairs = w.rows * a.group;

  // ---- the group's ring --------------------------------------------------------------
  const uint32_t ring = smem_u32(k8_smem) + (uint32_t)grp_w * (NS * Sh::kStage);
  constexpr uint32_t kVBase = kStep * D;
  auto k_off = [](int r, int c) -> uint32_t { return (uint32_t)(r * D + ((c ^ ((r & 1) << 2)) << 4)); };
  auto v_off = [](int r, int c) -> uint32_t {
    if constexpr (D == 256) return (uint32_t)(r * D + ((c ^ (((r >> 1) & 1) | (((r >> 2) & 1) << 2))) << 4));
    else return (uint32_t)(r * D + ((c ^ (((r >> 1) & 3) << 1)) << 4));
  };
  const uint8_t* gk = a.k + (int64_t)g * D;
  const uint8_t* gv = a.v + (int64_t)g * D;
  const int64_t pitch = (int64_t)a.h_kv * D;
  auto issue = [&](int stage, int32_t slot) {  // lane i holds the slot of the step's entry i
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    constexpr int PP = D / 16, kRows = 32 / PP;  // pieces of a row, rows a warp copies at once
#pragma unroll
    for (int u = 0; u < (kStep / kRows + MT - 1) / MT; ++u) {
      const int r0 = (u * MT + mt) * kRows;
      if (kStep / kRows % MT != 0 && r0 >= kStep) break;
      const int r = r0 + lane / PP, c = lane % PP;
      const int32_t s = __shfl_sync(0xffffffffu, slot, r);
      const int64_t off = (int64_t)max(s, 0) * pitch + c * 16;
      ka_cp16(base + k_off(r, c), gk + off, s >= 0);
      ka_cp16(base + kVBase + v_off(r, c), gv + off, s >= 0);
    }
  };
  auto entry = [&](int step) -> int { return lane < kStep && step < steps ? step * kStep + lane : INT32_MAX; };
  KaFetch pre[NS];
  uint32_t sc[NS];  // sc[i]: scales of the lane's entry i steps ahead
#pragma unroll
  for (int i = 0; i < NS; ++i) pre[i] = k8_fetch<kWindow>(a, w, entry(first + i * stride));
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) {
    const int32_t slot = k8_slot<kWindow, kShared>(a, w, entry(first + i * stride), pre[i]);
    if (first + i * stride < steps) issue(i, slot);
    asm volatile("cp.async.commit_group;" ::: "memory");
    sc[i] = k8_scales(a, slot, g);
  }
  KaFetch next = pre[NS - 1];

  // ---- the pairs: q as A fragments (rows gq, gq + 8), their factors and entries -------
  uint32_t qa[KS][2][NP];
  float mult[NP];              // logit (base 2) = mult * 2^ek * accumulator
  int va[NP], vb[NP], vc[NP];  // shared tiles: the pair sees entries [0, va) and [vb, vc)
#pragma unroll
  for (int np = 0; np < NP; ++np) {
    const int p = mt * P + np * 8 + gq;
    const int row = p / a.group, hd = p - row * a.group;
    const bool ok = p < pairs;
    const uint16_t* src = a.q + (int64_t)(w.t0 + row) * a.ld_q + ((int64_t)g * a.group + hd) * D;
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      // the lane's K pieces hold 16 dimensions each, two of q's
      const int piece = (tq + 4 * (i >> 1)) * 2 + (i & 1);
      const uint4 u = ok ? ld_in(reinterpret_cast<const uint4*>(src) + piece) : make_uint4(0u, 0u, 0u, 0u);
      qa[2 * i][0][np] = u.x;
      qa[2 * i][1][np] = u.y;
      qa[2 * i + 1][0][np] = u.z;
      qa[2 * i + 1][1][np] = u.w;
      mx = __vmaxu2(__vmaxu2(mx, u.x & 0x7fff7fffu), u.y & 0x7fff7fffu);
      mx = __vmaxu2(__vmaxu2(mx, u.z & 0x7fff7fffu), u.w & 0x7fff7fffu);
    }
    uint32_t top = max(mx & 0xffffu, mx >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = min(max((int)(top >> 7), 1), 253) - 127;  // exponent of the pair's largest component
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    mult[np] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float2 f = bf16x2_to_float2(qa[s][y][np]);
        qa[s][y][np] = ka_h2(__floats2half2_rn(f.x * down, f.y * down));
      }
    va[np] = vb[np] = vc[np] = 0;
    if constexpr (kShared) {
      int L = ok ? ld_in(a.row_len + w.t0 + row) : 0;
      if (L > a.max_len) L = 0;
      if (L > 0) {
        va[np] = min(a.n_sink, L);
        vb[np] = w.ns + max(0, L - a.window) - w.first;
        vc[np] = w.ns + L - w.first;
      }
      if (!ok) vc[np] = INT32_MAX;  // nobody's: sees what there is
    }
  }

  float o[VN][4];
  float m[NP], l[NP];
#pragma unroll
  for (int np = 0; np < NP; ++np) {
    m[np] = ninf;
    l[np] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < VN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

  // ---- steps ---------------------------------------------------------------------------
  int stage = 0;
  for (int step = first; step < steps; step += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    if constexpr (MT == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(grp_w + 1), "n"(MT * 32) : "memory");
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    const uint32_t here = sc[0];
    {  // refill the stage that the last step emptied
      const int ahead = step + (NS - 1) * stride;
      const int32_t slot = k8_slot<kWindow, kShared>(a, w, entry(ahead), next);
      if (ahead < steps) issue(stage == 0 ? NS - 1 : stage - 1, slot);
      asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
      for (int i = 0; i + 1 < NS - 1; ++i) sc[i] = sc[i + 1];
      sc[NS - 2] = k8_scales(a, slot, g);
      next = k8_fetch<kWindow>(a, w, entry(ahead + stride));
    }

    // S = q K^T: J n-tiles of 8 entries (lane: entries 2 tq, 2 tq + 1 of each)
    float s[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint4 kw[J];
#pragma unroll
      for (int j = 0; j < J; ++j) kw[j] = ka_lds16(base + k_off(j * 8 + gq, tq + 4 * i));
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const uint32_t x = k == 0 ? kw[j].x : k == 1 ? kw[j].y : k == 2 ? kw[j].z : kw[j].w;
          const int n = 4 * i + k;
          ka_mma<true>(s[j], qa[n][0][0], NP > 1 ? qa[n][0][NP - 1] : 0u, qa[n][1][0], NP > 1 ? qa[n][1][NP - 1] : 0u,
                       ka_h2(kv8_half2(x & 0xffffu)), ka_h2(kv8_half2(x >> 16)));
        }
    }

    // logits, the running maximum, weights and their sum
    uint32_t es[J][2];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) es[j][e] = __shfl_sync(0xffffffffu, here, 8 * j + 2 * tq + e);
    bool part_seen = false;  // some pair of the warp does not see some entry
    if constexpr (kShared) {
      const int e0 = step * kStep;
      bool all = true;
#pragma unroll
      for (int np = 0; np < NP; ++np) all &= e0 + kStep <= va[np] || (e0 >= vb[np] && e0 + kStep <= vc[np]);
      part_seen = !__all_sync(0xffffffffu, all);
    }
    uint32_t hi[NP][J], lo[NP][J];   // weights of the pair: high parts and remainders, entry pairs of the n-tiles
    uint32_t sees[NP];               // bit 2 j + e: the pair sees the lane's entry
#pragma unroll
    for (int np = 0; np < NP; ++np) {
      float x[J][2];
      float mx = ninf;
      sees[np] = 0xffffffffu;
      if (part_seen) {
        sees[np] = 0u;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = step * kStep + 8 * j + 2 * tq + e;
            sees[np] |= (uint32_t)(i < va[np] || (i >= vb[np] && i < vc[np])) << (2 * j + e);
          }
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t f = es[j][e];
          const bool ok = (f & 0x10000u) != 0 && ((sees[np] >> (2 * j + e)) & 1u) != 0;
          x[j][e] = ok ? s[j][2 * np + e] * (mult[np] * __uint_as_float((f & 0xffu) << 23)) : ninf;
          mx = fmaxf(mx, x[j][e] + (float)(int)((f >> 8) & 0xffu));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) - 127.f;
      if (__any_sync(0xffffffffu, m[np] != ninf && mx > m[np] + (float)kKaGrow)) {
        const float mn = fmaxf(m[np], mx);
        const float f = m[np] == ninf ? 1.f : ka_ex2(m[np] - mn);  // -inf: nothing yet
        l[np] *= f;
#pragma unroll
        for (int i = 0; i < VN; ++i) {
          if constexpr (NP == 1) {
            o[i][0] *= f; o[i][1] *= f; o[i][2] *= f; o[i][3] *= f;
          } else {
            o[i][2 * np] *= f; o[i][2 * np + 1] *= f;
          }
        }
        m[np] = mn;
      }
      if (m[np] == ninf) m[np] = mx;
      const float ms = m[np] == ninf ? 0.f : m[np] - (float)kK8Bias;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float p0 = ka_ex2(x[j][0] - ms), p1 = ka_ex2(x[j][1] - ms);
        l[np] += p0 + p1;
        ka_split<true>(p0 * __uint_as_float((es[j][0] & 0xff00u) << 15), p1 * __uint_as_float((es[j][1] & 0xff00u) << 15),
                       hi[np][j], lo[np][j]);
      }
    }

    // O += P V: lane: entries 2tq, 2tq+1 (b0) and 2tq+8, 2tq+9 (b1) of 16;
    // columns gq * VN + i of n-tile i
    uint32_t nans = 0;
    auto product = [&](auto marks_tag, auto part_tag) {
      constexpr bool kMarks = decltype(marks_tag)::value, kPart = decltype(part_tag)::value;
#pragma unroll
      for (int ks = 0; ks < J / 2; ++ks) {
        uint32_t one[2][NP];  // marks: 1 where the pair sees the entry
        if constexpr (kMarks) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int np = 0; np < NP; ++np) {
              const uint32_t b = sees[np] >> (4 * ks + 2 * y);
              one[y][np] = ((b & 1u) ? 0x3c00u : 0u) | ((b & 2u) ? 0x3c000000u : 0u);
            }
        }
#pragma unroll
        for (int half = 0; half < D / 128; ++half) {
          uint32_t vw[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = ks * 16 + 2 * tq + (e & 1) + (e >> 1) * 8;
            const uint4 y = ka_lds16(base + kVBase + v_off(r, D == 256 ? 2 * gq + half : gq));
            vw[e][0] = y.x; vw[e][1] = y.y; vw[e][2] = y.z; vw[e][3] = y.w;
            if constexpr (kPart || kMarks) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t nan = __vcmpeq4(vw[e][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                nans |= nan;
                vw[e][k] = kMarks ? nan & 0x38383838u : vw[e][k] & ~nan;  // 0x38: 1.0
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t b[2][2];  // [entries 2tq.., 2tq+8..][columns 0 and 1, 2 and 3]
            b[0][0] = __byte_perm(vw[0][k], vw[1][k], 0x5140);
            b[0][1] = __byte_perm(vw[0][k], vw[1][k], 0x7362);
            b[1][0] = __byte_perm(vw[2][k], vw[3][k], 0x5140);
            b[1][1] = __byte_perm(vw[2][k], vw[3][k], 0x7362);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int i = half * 16 + 4 * k + c;
              const uint32_t b0 = ka_h2(kv8_half2((b[0][c >> 1] >> (16 * (c & 1))) & 0xffffu));
              const uint32_t b1 = ka_h2(kv8_half2((b[1][c >> 1] >> (16 * (c & 1))) & 0xffffu));
              if constexpr (kMarks) {
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                ka_mma<true>(t, one[0][0], one[0][NP - 1], one[1][0], one[1][NP - 1], b0, b1);
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (t[y] > 0.f) o[i][y] = __int_as_float(0x7fffffff);
              } else if constexpr (NP == 1) {
                ka_mma<true>(o[i], hi[0][2 * ks], lo[0][2 * ks], hi[0][2 * ks + 1], lo[0][2 * ks + 1], b0, b1);
              } else {
                ka_mma<true>(o[i], hi[0][2 * ks], hi[1][2 * ks], hi[0][2 * ks + 1], hi[1][2 * ks + 1], b0, b1);
                ka_mma<true>(o[i], lo[0][2 * ks], lo[1][2 * ks], lo[0][2 * ks + 1], lo[1][2 * ks + 1], b0, b1);
              }
            }
          }
        }
      }
    };
    if constexpr (kShared) {
      if (part_seen) {
        product(std::false_type(), std::true_type());
        if (__any_sync(0xffffffffu, nans != 0)) product(std::true_type(), std::false_type());
      } else {
        product(std::false_type(), std::false_type());
      }
    } else {
      product(std::false_type(), std::false_type());
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
  }

  // ---- the CTA's result ----------------------------------------------------------------
#pragma unroll
  for (int np = 0; np < NP; ++np) {
    l[np] += __shfl_xor_sync(0xffffffffu, l[np], 1);
    l[np] += __shfl_xor_sync(0xffffffffu, l[np], 2);
    if (tq == 0) {
      s_m[warp][np * 8 + gq] = m[np];
      s_l[warp][np * 8 + gq] = l[np];
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();  // also: every ring is free
  float* so = reinterpret_cast<float*>(k8_smem);  // [warp][P][Out::kRow]
#pragma unroll
  for (int np = 0; np < NP; ++np) {
    const int p = np * 8 + gq;
    float cm = ninf;
#pragma unroll
    for (int i = 0; i < Sh::kGroups; ++i) cm = fmaxf(cm, s_m[i * MT + mt][p]);
    const float f = cm == ninf ? 0.f : ka_ex2(m[np] - cm);
    if (grp_w == 0 && tq == 0) {
      float cl = 0.f;
#pragma unroll
      for (int i = 0; i < Sh::kGroups; ++i)
        cl += s_l[i * MT + mt][p] * (cm == ninf ? 1.f : ka_ex2(s_m[i * MT + mt][p] - cm));  // all 0, or a NaN
      c_m[mt * P + p] = cm;
      c_l[mt * P + p] = cl;
    }
    float* dst = so + (size_t)(warp * P + p) * Out::kRow;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < VN; i += 4) {
        float4 y;
        float* z = &y.x;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          z[c] = (NP == 1 ? o[i + c][e] + o[i + c][2 + e] : o[i + c][2 * np + e]) * f;
        *reinterpret_cast<float4*>(dst + Out::col((2 * tq + e) * VN + i)) = y;
      }
  }
  __syncthreads();
  // the groups' sums into the first one's rows
  const int quads = pairs * (D / 4);
  if constexpr (Sh::kGroups > 1) {
    for (int idx = tid; idx < quads; idx += Sh::kThreads) {
      const int p = idx / (D / 4), d = (idx % (D / 4)) * 4;
      float* p0 = so + (size_t)p * Out::kRow + Out::col(d);
      float4 y = *reinterpret_cast<float4*>(p0);
#pragma unroll
      for (int i = 1; i < Sh::kGroups; ++i) {
        const float4 z = *reinterpret_cast<const float4*>(p0 + (size_t)i * MT * P * Out::kRow);
        y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
      }
      *reinterpret_cast<float4*>(p0) = y;
    }
  }
  // ---- the cluster's: each CTA pushes its sums into the one that writes them (quad i of
  // the tile's output: CTA i mod C), so that one cluster barrier lies between -------------
  float4* join = reinterpret_cast<float4*>(k8_smem + Sh::kFront);           // [source CTA][own quad]
  float2* jml = reinterpret_cast<float2*>(join + Sh::kJoinQuads);           // [source CTA][pair]
  const int own = (quads + C - 1) / C;
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();
  if (C > 1) {
    for (int i = tid; i < quads; i += Sh::kThreads) {
      const float4 x = *reinterpret_cast<const float4*>(so + (size_t)(i / (D / 4)) * Out::kRow + Out::col(i % (D / 4) * 4));
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                       map_shared_rank(join + rank * own + i / C, (uint32_t)(i % C))),
                   "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                   : "memory");
    }
    for (int i = tid; i < C * pairs; i += Sh::kThreads) {
      const int p = i % pairs;
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                       map_shared_rank(jml + rank * Sh::kPairs + p, (uint32_t)(i / pairs))),
                   "f"(c_m[p]), "f"(c_l[p])
                   : "memory");
    }
    cluster_sync();
  }
  for (int j = tid; j < own; j += Sh::kThreads) {
    const int idx = j * C + rank;
    if (idx >= quads) break;
    const int p = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float M, Lsum;
    float4 x;
    if (C == 1) {
      M = c_m[p];
      Lsum = c_l[p];
      x = *reinterpret_cast<const float4*>(so + (size_t)p * Out::kRow + Out::col(d));
    } else {
      M = ninf;
      for (int c = 0; c < C; ++c) M = fmaxf(M, jml[c * Sh::kPairs + p].x);
      Lsum = 0.f;
      x = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < C; ++c) {
        const float2 ml = jml[c * Sh::kPairs + p];
        const float4 y = join[c * own + j];
        const float f = ml.x == ninf ? 0.f : ka_ex2(ml.x - M);
        // a CTA without a weight (or with NaN weights only) has m = -inf
        Lsum += ml.x == ninf ? ml.y : f * ml.y;
        x.x += f * y.x;
        x.y += f * y.y;
        x.z += f * y.z;
        x.w += f * y.w;
      }
    }
    const int row = p / a.group;
    const int64_t hq = (int64_t)(w.t0 + row) * a.h_q + (int64_t)g * a.group + (p - row * a.group);
    if (a.n_group > 1) {
      float* pp = a.part + (hq * a.n_group + grp) * (D + 2);
      pp[2 + d] = x.x; pp[3 + d] = x.y; pp[4 + d] = x.z; pp[5 + d] = x.w;
      if (d == 0) {
        pp[0] = M;
        pp[1] = Lsum;
      }
      continue;
    }
    const float inv = Lsum == 0.f ? 0.f : 1.0f / Lsum;
    if (a.out_bf16) {
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(x.x * inv, x.y * inv), b1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + hq * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + hq * D + d) =
          make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    }
    if (d == 0 && a.lse != nullptr)
      a.lse[hq] = Lsum == 0.f ? ninf : (M - (float)kK8Bias + log2f(Lsum)) * 0.69314718055994531f;
  }
}

}  // namespace qsa
