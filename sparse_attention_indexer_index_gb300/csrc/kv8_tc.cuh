// kv8_tc.cuh -- softmax attention of rows over the 8-bit K/V cache on the
// fifth-generation tensor cores: over the slots of a selection
// (sparse_attn_fp8) or a window (window_attn_fp8).
//
// For row t and query head h (KV head h / G), with j over the row's entries,
// codes kc, vc and the exponents ek, ev of their blocks' scales:
//     x_j = scale 2^ek_j <q_h, kc_j>,  lse = log sum_j exp(x_j),
//     out = sum_j exp(x_j - lse) 2^ev_j vc_j;   no entry: out = 0, lse = -inf.
//
// Bound.  Per entry and KV head 2 D bytes are read for 4 G D flops: HBM.  So
// the codes go from HBM to shared memory to the tensor cores as they are; no
// instruction touches one.
//
// Design (GB300).
//  - The products are transposed: entries are the 128 rows of the MMA, the (row,
//    query head) pairs of a tile its columns, 8 to 48 of them.
//        S^T [128 entries][2 N]  = K [128][D] (Q parts)^T
//        O^T [D][parts N]       += V^T [D][128] (P parts)^T
//    A tile is one row's heads, or those of R rows of one request, which see
//    nearly the same window.
//  - Both operands of an MMA (kind::f8f6f4) are e4m3, so q and the weights enter
//    in parts of 4 significant bits, as columns of their own: part i holds what
//    the parts before left, times 32^i, which keeps it clear of e4m3's lower
//    end.  q takes two parts: exact down to 2^-14 of the pair's largest
//    component, off by 2^-22 of that at most below.  Weights take four: off by
//    2^-16 of themselves, or 2^-28 of the largest (with three, 2^-12 and 2^-23,
//    the many small weights of a long row behind a first token that holds
//    nearly all of it were lost, and the normaliser still counted them).  The
//    parts are added in FP32 when S and O are read.
//  - The scales enter once an entry: 2^ek as a factor of the logit, 2^ev of the
//    weight.  The reference of both sums is a running maximum M of y_j = x_j +
//    ev_j (in powers of two): the weights 2^(y_j - M) stay within e4m3 whatever
//    the scales are, the normaliser sum 2^(x_j - M) within FP32 (|ev| <= 64).
//    M follows only when a weight would pass 2^5: then O is rescaled.  Two such
//    M may be 127 apart for the same logits, and the sum be as far from 1 the
//    other way: it is scaled by 2^(d/2) twice (k8_half), as 2^-127 alone is 0.
//  - One CTA an SM.  4 to 12 warps turn S into P: a thread has one entry and 4 to
//    16 pairs, so the sums of weights are its own registers until the end, and
//    the only exchange between threads is the vote on whether M has to grow
//    (taken, with up to 16 pairs, while the weights are computed as if not).
//    One warp issues the MMAs, QK(i+1) before PV(i); two or four copy K and V
//    rows with cp.async into a ring of tiles, in the order in which they are
//    used; one finds the CTA's work.
//  - Work, three ways.  Clusters: where the (tile, KV head) units are few, the C
//    CTAs of a cluster (1 to 8) share one, a part of its blocks each, and join
//    through distributed shared memory; one launch, no workspace.  Shares: the
//    blocks of all units are numbered through, and each CTA takes an equal
//    share of them, wherever that begins and ends, so that requests of any
//    lengths keep all SMs busy; sums of units that several CTAs share meet in
//    kv8_merge_kernel, through the workspace.  A unit's begin costs a CTA two
//    blocks' time (its q, the sums of the unit before, the first M), so every
//    unit is numbered with two blocks more.  Many units: CTAs take whole units
//    in turn.
//  - From one unit to the next: q is prepared, and its first products begin,
//    before the sums of the unit before go out.
//  - Rows of a tile that do not see an entry give it the weight 0.  A NaN of V
//    there is replaced by 0 in shared memory, and noted for the pairs that do
//    see it, whose sum becomes NaN.
// Tensor memory columns: S two times 2 N (48 pairs of D = 256: once), O D / 128
// times parts N.
//
// Measured, us a call in a graph of calls on different inputs (a GB300, copy
// rate 6,784 GB/s; in brackets the form before on mma.sync, where the warps
// unpacked the codes): 32 rows of 2,051 (2 KV heads, D = 256) 17.7 (24.9), 3.9
// TB/s; 192 rows (1 KV head of 16, D = 128) 28.5 (35.9); one row 8.3 (9.6); a
// window of 4,096 for 32 requests 29.0 (36.7), 4.6 TB/s; 32 requests x 6 rows in
// a window of 1,024 24.2 (54.9; 23.0 with three parts to a weight); 8 requests of
// up to 131,072 tokens 125 to 128 (260), 6.0 TB/s; one of 20,011 14.1 (20.6).  A
// block (64 KB) takes 1.15 to 1.4 us with 8 or 16 pairs, what its bytes take of
// HBM's rate, and about 1.5 with 48 (the weights' parts).  The rest is a call's ends: 3 to 4 us from its start to the first S
// (three dependent loads, cold instructions), 2 to 3 for the last sums and the
// join of a cluster, 3 for the merge.  What runs once takes as long as its
// instructions take to arrive: hence loops of few passes are not unrolled and
// rare cases are calls (184 -> 121 KB for 48 pairs, at the time).
//
// Waits on stages.  The ring's uses are numbered in the order K(0), K(1), V(0),
// K(2), V(1), ... of a segment, over all segments; use u is in stage u mod
// kStages, phase u / kStages of that stage's barriers.  Producers and the MMA
// warp wait for every use in turn.  The softmax warps wait for some V tiles
// (shared tiles): S(b) is there, so K(b) = use 2b - 1 of the segment was, and
// all before it; V(b) = use 2b + 2 at most, so the phase before V(b)'s, kStages
// >= 3 uses earlier, is over.
#pragma once
#include "common.cuh"
#include "kv8.cuh"
#include "kv_attn.cuh"
#include "tc_util.cuh"

namespace qsa {

// Shares below so many units, whole units in turn from there on.  Shares keep all
// SMs busy where lengths differ, and cost the merge.  Measured in a graph, whole
// units / shares: 100, 150 and 300 requests of 2,000 to 40,000 tokens 595 / 312,
// 678 / 475, 1294 / 944 us; rows of equal length, at worst 300, 600 and 1,200
// lists of 2,051 on 1 KV head of D = 128 34.7 / 38.9, 63.8 / 68.2, 122.6 / 126.0;
// 1,600 and 2,400 units of 2,051 on 2 heads of D = 256 259 / 259 and 377 / 383.
constexpr int kK8MaxUnits = 1216;
// Tiles, and requests, that a CTA's tables of shares hold.  More of them take whole
// units in turn, whatever their lengths: 304 and 305 of the uneven requests above
// 955 and 1298 us, 400 of them 1495; of equal length no matter (608 windows of
// 4,096 374 us, the copy rate).
constexpr int kK8MaxTiles = 304;
constexpr int kK8Ctas = 152;       // CTAs of shares and whole units at most (one an SM)
constexpr int kK8Bias = 3;         // weights are held as 2^kK8Bias w, w <= 2^kKaGrow
constexpr int kK8SegRing = 2;
constexpr int kK8Lead = 2;         // blocks' time that a unit's begin costs a CTA (shares count it)
constexpr uint64_t kK8WaitNs = 2000000000ull;  // limit of a wait for a few blocks' work (a block takes 1.5 us at most)
constexpr uint32_t kK8BlockNs = 20000;         // and for every block of a segment where one lies in between
constexpr float kK8None = -1e30f;  // M of a pair that has seen nothing (finite: -inf less it is -inf)
enum { kK8Cluster = 0, kK8Shares = 1, kK8Whole = 2 };

struct Kv8AttnArgs : KvAttnArgs {
  int32_t block_shift;       // log2 of the tokens to a scale
  int32_t page_shift;        // log2 of the page size, -1: not a power of two
  int32_t cluster_shift;     // log2 of the CTAs to a cluster
  uint32_t group_inv;        // pair / group = pair * group_inv >> 16
  int32_t rows;              // R: rows per tile
  int32_t tile_slots;        // slots of tiles (see k8_find)
  int32_t mode;              // how the work is dealt
  int32_t n_units;           // (tile, KV head) pairs, for requests of equal length
  int4* jobs;                // [units or CTAs]: what kv8_merge_kernel joins: first CTA (-1: nothing), last CTA, first
                             // row, KV head * 256 + rows
  int32_t jobs_by_unit;      // a job for every unit, or (more units than CTAs) for the CTA where one ends
};

// D = 128 with 8 pairs takes blocks of 256 entries (two products each way),
// whose tiles are as large as those of D = 256: with 128 the fixed costs of a
// block held it at 1.35 us, where its bytes take 0.73.
template <int D, int N, int PARTS, bool kWindow, bool kShared>
struct K8Tc {
  static constexpr int kSub = N <= 16 ? 256 / D : 1;   // products of 128 entries to a block
  static constexpr int kBlock = 128 * kSub;            // entries of a block
  // Pairs of a thread.  16 where there are enough of them: their weights of a part are one 16-byte
  // store, without bank conflicts (48 pairs by 12s: 24.5 us where this took 23.0, with three parts).  4 with 8 pairs of
  // D = 256: twice the warps for the q, the first block and the sums of calls of a few blocks (by 8s:
  // 29.6 us for a window of 4,096, where this takes 28.7).
  static constexpr int kPer = N >= 32 || (N == 16 && kSub == 2) ? 16 : N == 8 && kSub == 1 ? 4 : 8;
  static constexpr int kSlices = N / kPer;             // softmax warps to an entry
  static constexpr int kSoft = 4 * kSub * kSlices;     // softmax warps
  static constexpr int kLoads = (N + kSoft - 1) / kSoft;  // pairs whose q a warp prepares
  static constexpr int kProd = N >= 32 ? 2 : 4;        // producer warps
  static constexpr int kThreads = 32 * (kSoft + 2 + kProd);  // and MMA, work
  // Whether the vote on M is taken beside the weights (with registers to spare) or before them.
  static constexpr bool kAhead = N <= 16 && kPer <= 8;
  static constexpr int kTile = kBlock * D;             // bytes
  static constexpr int kNS = 2 * N, kNP = PARTS * N;   // columns of S (of a product) and of a half of O
  static constexpr int kGroups = (kNP + 31) / 32;      // groups of 32 columns of P
  static constexpr int kPSub = kGroups * 4096;         // P of a product: [group][128 entries][32 B]
  static constexpr int kQ = kNS * D, kP = kSub * kPSub;
  // Buffers of S: two, one where O leaves no room for more (48 pairs of D = 256).  Then S(i + 1) begins
  // when S(i) has been read, which is long before P(i) is there.
  static constexpr int kSBuf = 2 * kSub * kNS + D / 128 * kNP <= 512 ? 2 : 1;
  static constexpr int kColO = kSBuf * kSub * kNS;
  static_assert(kColO + D / 128 * kNP <= 512 && kNS % 16 == 0 && kNP % 16 == 0, "tensor memory");
  struct Seg {
    int t0, rows, r, g;    // first row, rows (-1: no more), request, KV head
    int n, first, ns;      // entries, and where they lie (see k8_pos)
    int j0, j1;            // blocks of the segment
    int slot;              // partial result's slot; -1: the whole unit, or a cluster's part
  };
  struct Ctl {
    uint64_t full[12], empty[12];
    uint64_t s_full[2], s_free[2], p_full[2], pv_done[2], q_full, drain;
    uint64_t met[kSlices + 1];   // softmax warps of a slice, of all
    uint64_t join_full;          // the cluster's softmax warps: their sums are there
    uint64_t seg_full[kK8SegRing], seg_empty[kK8SegRing];
    Seg seg[kK8SegRing];
    alignas(16) float mb[N];     // the reference M, less kK8Bias
    // a pair's words, for segments of even and odd number (one begins before the other's sums are out):
    alignas(16) float mult[2][N];   // logit (base 2) = mult * 2^ek * S
    int out[2][N];                  // (row, query head) of the pair, -1: none
    int4 sees[2][kShared ? N : 1];  // the pair sees entries [0, x) and [y, z)
    uint32_t nan[2][kShared ? N : 1][D / 32];  // columns that a NaN of V reached
    int any_nan[2];
    alignas(16) float wmax[kSoft][kPer];
    float wsum[kSoft][kPer];
    alignas(16) int vote[2][kSoft];          // [block parity]: a weight of the warp's passes the limit
    int scan[32];
    uint32_t tmem;
    int abort;
    int base[kWindow ? kK8MaxTiles + 1 : 1];   // tiles before request r
    int pre[kWindow ? kK8MaxTiles + 1 : 1];    // blocks before tile t, kK8Lead more to each
    int4 tile[kWindow ? kK8MaxTiles : 1];      // its first row, request * 256 + rows, first, n
  };
  // Rows of partial results: D sums, M and L.  In a cluster of up to 16 pairs a CTA writes a pair's row
  // into the memory of the one that joins it, [source][own pair].  With more there is no room, and each
  // keeps its rows, [pair], in its ring, whose last tile has been used by then, for the others to read
  // (48 pairs, 2 CTAs: 1.3 us less than writing there behind one more meeting; 8 pairs: 0.4 us more).
  static constexpr bool kPull = N > 16;
  static constexpr int kJoin = D + 4;
  static constexpr int kFixed = kQ + 2 * kP + (kPull ? 0 : N * kJoin * 4) + (int)sizeof(Ctl) + 1024;
  static constexpr int kFit = (227 * 1024 - kFixed) / kTile;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static_assert(kStages >= 3 && N * kJoin * 4 <= kStages * kTile, "ring");
  static constexpr int kSmem = kFixed + kStages * kTile;
};

// ---- waits and tensor-memory accesses --------------------------------------------------
// (What is rare is kept out of line: a kernel of 100 KB and more fetched its
// instructions for longer than it ran them, where each is run once or twice.)
__device__ __noinline__ void k8_fault(unsigned bits) { raise_fault(bits); }
__device__ __noinline__ bool k8_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int blocks) {
  const uint64_t t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    const bool late = global_timer_ns() - t0 > kK8WaitNs + (uint64_t)blocks * kK8BlockNs;
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
// Bounded wait by a whole warp, which stays together.
__device__ __forceinline__ bool k8_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int blocks = 0) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || k8_wait_long(bar, parity, abort, blocks);
}
// One arrival for a warp, behind what its lanes did.
__device__ __forceinline__ void k8_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// One arrival of the warp at every CTA's barrier for what it wrote to them, and
// the (bounded) wait for all such: phase 0.
__device__ __forceinline__ void k8_arrive_all(uint64_t* bar, int n_cta) {
  __syncwarp();
  const int lane = threadIdx.x & 31;
  if (lane < n_cta)
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(map_shared_rank(bar, lane)) : "memory");
  __syncwarp();
}
// What another CTA of the cluster has in shared memory (several can be on the way, see ld_dsmem_u32).
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ char* map_generic_rank(const void* p, uint32_t rank) {
  uint64_t r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return reinterpret_cast<char*>(r);
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at));
  return v;
}
__device__ __noinline__ bool k8_wait_cluster(uint64_t* bar, volatile int* abort) {
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
  const uint64_t t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, arrived())) {
    const bool late = global_timer_ns() - t0 > kK8WaitNs;
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
__device__ __forceinline__ void k8_ld8(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void k8_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void k8_ld4(uint32_t taddr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void k8_st4(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
template <int n>
__device__ __forceinline__ void k8_ld(uint32_t taddr, uint32_t* v) {  // n columns: 4, 8 or 16
  if constexpr (n == 4) k8_ld4(taddr, v);
  else k8_ld8(taddr, v);
  if constexpr (n == 16) k8_ld8(taddr + 8, v + 8);
}
template <int n>
__device__ __forceinline__ void k8_st(uint32_t taddr, const uint32_t* v) {
  if constexpr (n == 4) k8_st4(taddr, v);
  else k8_st8(taddr, v);
  if constexpr (n == 16) k8_st8(taddr + 8, v + 8);
}
// The wait for loads, through which their registers pass: no use of one can be
// scheduled ahead of it.
template <int n>
__device__ __forceinline__ void k8_wait_ld(uint32_t (&v)[n]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void k8_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void k8_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// Four MMAs of 32 in K, their operands A1 and B1 descriptor units apart, by one
// elected lane of a whole warp (the descriptors stay in uniform registers).
template <int A1, int B1>
__device__ __forceinline__ void k8_mma4(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, t;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, %7;\n\tadd.u64 b, %2, %8;\n\t@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "add.u64 a, %1, %9;\n\tadd.u64 b, %2, %10;\n\t@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "n"(A1), "n"(B1), "n"(2 * A1), "n"(2 * B1), "n"(3 * A1),
      "n"(3 * B1)
      : "memory");
}
// Instruction descriptor: D = F32, A = B = e4m3, M = 128; transposed: the rows
// of A and B in shared memory are the K index (MN-major).
__host__ __device__ constexpr uint32_t k8_idesc(int n, bool transposed) {
  return (1u << 4) | (transposed ? 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// MN-major, 32-byte swizzle: groups of 32 columns `group` bytes apart, rows of
// 32 bytes, groups of 8 rows (the K index) 256 bytes apart.
__device__ __forceinline__ uint64_t k8_desc_p(uint32_t smem_addr, uint32_t group) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(group >> 4) << 16;
  d |= (uint64_t)(256u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)6 << 61;
  return d;
}
// Pairs of FP32 numbers, one instruction for both.
__device__ __forceinline__ uint64_t k8_pair(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float k8_low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float k8_high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t k8_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// ---- entries ---------------------------------------------------------------------------
// Entry e lies at list position e, or (window) at position e below ns, behind
// that at first + e - ns.
template <class Seg>
__device__ __forceinline__ int k8_pos(const Seg& w, int e) {
  return e < w.ns ? e : w.first + (e - w.ns);
}
// Where a window of rows t0 .. t0 + rows - 1 begins and ends: entries, first, ns.
__device__ __noinline__ int3 k8_window(const Kv8AttnArgs& a, int t0, int rows) {
  int lo = INT32_MAX, last = 0;
  bool bad = false;
#pragma unroll 1
  for (int i0 = 0; i0 < rows; i0 += 8) {
    int L[8];  // on the way together
#pragma unroll
    for (int i = 0; i < 8; ++i) L[i] = i0 + i < rows ? ld_in(a.row_len + t0 + i0 + i) : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool ok = L[i] > 0 && L[i] <= a.max_len;
      bad |= L[i] != 0 && !ok;
      lo = min(lo, ok ? max(0, L[i] - a.window) : INT32_MAX);
      last = max(last, ok ? L[i] : 0);
    }
  }
  if (bad) raise_fault(kFaultGrouping);
  const int first = last > 0 ? lo : 0, ns = min(a.n_sink, first);
  return make_int3(last > 0 ? ns + last - first : 0, first, ns);
}
template <int kBlock>
__device__ __forceinline__ int k8_blocks(int n) {
  return max(1, (n + kBlock - 1) / kBlock);
}
// Whether a row of the tile attends to a position.
__device__ __noinline__ bool k8_seen(const Kv8AttnArgs& a, int t0, int rows, int pos) {
#pragma unroll 1
  for (int i = 0; i < rows; ++i) {
    const int L = ld_in(a.row_len + t0 + i);
    if (L > 0 && L <= a.max_len && pos < L && (pos >= L - a.window || pos < a.n_sink)) return true;
  }
  return false;
}
__device__ __noinline__ int k8_divide(int x, int y) { return x / y; }
// An entry's slot in two parts, as in kv_attn.cuh: what is loaded, and what is
// made of it (-1: none).
template <bool kWindow, class Seg>
__device__ __forceinline__ KaFetch k8_fetch(const Kv8AttnArgs& a, const Seg& w, int e) {
  KaFetch f{-1, 0};
  if (e >= w.n) return f;
  if constexpr (kWindow) {
    const int pos = k8_pos(w, e);
    const int pi = a.page_shift >= 0 ? pos >> a.page_shift : k8_divide(pos, a.page_size);  // < ld_pt: pos < max_len
    f.raw = ld_in(a.page_table + (int64_t)w.r * a.ld_pt + pi);
    f.off = pos - pi * a.page_size;
  } else {
    f.raw = ld_in(a.slots + (int64_t)w.t0 * a.ld_slots + e);
  }
  return f;
}
template <bool kWindow, bool kFaults, class Seg>
__device__ __forceinline__ int32_t k8_slot(const Kv8AttnArgs& a, const Seg& w, int e, const KaFetch& f) {
  if (e >= w.n || f.raw < 0) {
    if (kWindow && kFaults && e < w.n && k8_seen(a, w.t0, w.rows, k8_pos(w, e))) k8_fault(kFaultIndex);
    return -1;
  }
  if constexpr (!kWindow) {
    if (f.raw >= a.n_slots) {
      if (kFaults) k8_fault(kFaultIndex);
      return -1;
    }
    return f.raw;
  } else {
    // a page counts only if it lies wholly inside the cache
    if (((int64_t)f.raw + 1) * a.page_size > a.n_slots) {
      if (kFaults && k8_seen(a, w.t0, w.rows, k8_pos(w, e))) k8_fault(kFaultIndex);
      return -1;
    }
    return f.raw * a.page_size + f.off;
  }
}
// An entry's scale bytes as they are loaded: nothing is made of them before the
// block that uses them.
struct K8Scales {
  uint8_t k, v;
  bool valid;
};
__device__ __forceinline__ K8Scales k8_scales(const Kv8AttnArgs& a, int32_t slot, int g) {
  K8Scales f{0, 0, false};
  if (slot < 0) return f;
  const uint64_t at = (uint64_t)(uint32_t)(slot >> a.block_shift) * (uint32_t)a.h_kv + g;
  f.k = ld_in(a.ks + at);
  f.v = ld_in(a.vs + at);
  f.valid = true;
  return f;
}

__device__ __forceinline__ int k8_warp_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}
// ---- the CTA's work ----------------------------------------------------------------------
// arr[0 .. n) becomes the sums before each, arr[n] the sum of all; by the whole CTA.
template <int kThreads>
__device__ __noinline__ void k8_scan(int* arr, int n, int* tmp) {
  const int per = (n + kThreads - 1) / kThreads, i0 = threadIdx.x * per, i1 = min(i0 + per, n);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  int sum = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) sum += arr[i];
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) tmp[warp] = incl;
  __syncthreads();
  int before = incl - sum, all = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = tmp[w];
    if (w < warp) before += v;
    all += v;
  }
#pragma unroll 1
  for (int i = i0; i < i1; ++i) {
    const int v = arr[i];
    arr[i] = before;
    before += v;
  }
  if (threadIdx.x == 0) arr[n] = all;
  __syncthreads();
}
// The last i with arr[i] <= x (arr[0] <= x < arr[n]).
__device__ __forceinline__ int k8_search(const int* arr, int n, int x) {
  int lo = 0, hi = n;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// Tiles of request i; 0 where the grouping is wrong.
__device__ __forceinline__ int k8_request_tiles(const Kv8AttnArgs& a, int i) {
  const int row0 = ld_in(a.req_row_start + i), row1 = ld_in(a.req_row_start + i + 1);
  if (row0 < 0 || row1 < row0 || row1 > a.n_rows) {
    k8_fault(kFaultGrouping);
    return 0;
  }
  return (row1 - row0 + a.rows - 1) / a.rows;
}
// A step d of a reference is 2^d, here its half 2^(d/2): a sum of weights, which
// may be as large as 2^d is small, is multiplied by it twice, a sum of weighted
// values by its square.
__device__ __forceinline__ float k8_half(float d) { return ka_ex2(0.5f * d); }
// A pair's log-sum-exp from M (base 2) and the sum of its weights (without any
// weight, or with NaN only, M = -inf).
__device__ __forceinline__ float k8_lse(float M, float L) {
  const float ninf = -__int_as_float(0x7f800000);
  return L == 0.f ? ninf : (M == ninf ? L : M + log2f(L)) * 0.69314718055994531f;
}
// Request of tile s and the tile's number in it, by a whole warp (-1: none).  Up
// to kK8Exact requests the tiles are counted.  Else a tile has a slot of its own
// among some that are empty, of which there are a.tile_slots: that of its first
// row, where these are all rows' (few rows to a request), or else, for request
// r's tiles, those from start[r] / R + r on (the requests before have at most
// that many tiles, and all have n_rows / R + n_req).
constexpr int kK8Exact = 1024;
// The slots of n_rows rows in tiles of R: as many as tiles at least, whichever
// way they are numbered.
constexpr int64_t k8_tile_slots(int64_t n_rows, int64_t n_req, int R) {
  const int64_t by_request = n_rows / R + n_req;
  return n_rows < by_request ? n_rows : by_request;
}
__device__ __noinline__ int k8_find(const Kv8AttnArgs& a, int s, int& rank) {
  const int lane = threadIdx.x & 31;
  if (a.n_req <= kK8Exact) {
#pragma unroll 1
    for (int g0 = 0; g0 < a.n_req; g0 += 32) {
      const int n = g0 + lane < a.n_req ? k8_request_tiles(a, g0 + lane) : 0;
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
  if (a.tile_slots == a.n_rows) {
    const int r = warp_row_request(a.req_row_start, a.n_req, s);
    if (r < 0) return -1;
    const int in = s - ld_in(a.req_row_start + r);
    rank = in / a.rows;
    return in >= 0 && in == rank * a.rows && rank < k8_request_tiles(a, r) ? r : -1;
  }
  int lo = 0, n = a.n_req + 1;  // the last i with start[i] / R + i <= s, 32 samples a round
#pragma unroll 1
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

template <int D, int N, int PARTS, bool kWindow, bool kShared>
__global__ void __launch_bounds__(K8Tc<D, N, PARTS, kWindow, kShared>::kThreads, 1)
kv8_tc_kernel(const __grid_constant__ Kv8AttnArgs a) {
  using Sh = K8Tc<D, N, PARTS, kWindow, kShared>;
  using Seg = typename Sh::Seg;
  constexpr int H = D / 128, NS = Sh::kNS, NP = Sh::kNP, S = Sh::kStages, kPer = Sh::kPer, kSub = Sh::kSub;
  constexpr int kBlock = Sh::kBlock;
  static_assert(kWindow || !kShared, "lists are not shared");
  extern __shared__ unsigned char k8_raw[];
  unsigned char* const smem = k8_raw + ((1024u - (smem_u32(k8_raw) & 1023u)) & 1023u);  // the swizzle atoms need it
  unsigned char* const ring = smem;
  unsigned char* const q_buf = ring + S * Sh::kTile;
  unsigned char* const p_buf = q_buf + Sh::kQ;
  float* const join = reinterpret_cast<float*>(Sh::kPull ? ring : p_buf + 2 * Sh::kP);
  typename Sh::Ctl& ctl =
      *reinterpret_cast<typename Sh::Ctl*>(p_buf + 2 * Sh::kP + (Sh::kPull ? 0 : N * Sh::kJoin * 4));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &ctl.abort;
  const float ninf = -__int_as_float(0x7f800000);

  // Tiles past those of requests of equal length are there only if lengths differ: their clusters
  // look first, as the SMs are handed on from one to the next of them.
  if (kShared && a.mode == kK8Cluster && (int)(blockIdx.x >> a.cluster_shift) >= a.n_units) {
    pdl_wait_primary();
    int number;
    if (k8_find(a, (int)(blockIdx.x >> a.cluster_shift) / a.h_kv, number) < 0) return;
  }
  if (warp == Sh::kSoft) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&ctl.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {  // a barrier of each kind a lane
    static_assert(S <= 32 && Sh::kSlices < 32, "lanes");
    if (lane < S) {
      mbar_init(&ctl.full[lane], Sh::kProd);
      mbar_init(&ctl.empty[lane], 1);
    }
    if (lane < 2) {
      mbar_init(&ctl.s_full[lane], 1);
      mbar_init(&ctl.s_free[lane], Sh::kSoft);
      mbar_init(&ctl.p_full[lane], Sh::kSoft);
      mbar_init(&ctl.pv_done[lane], 1);
    }
    if (lane <= Sh::kSlices) mbar_init(&ctl.met[lane], lane < Sh::kSlices ? 4 * kSub : Sh::kSoft);
    if (lane < kK8SegRing) {
      mbar_init(&ctl.seg_full[lane], 1);
      mbar_init(&ctl.seg_empty[lane], Sh::kSoft + 1 + Sh::kProd);  // softmax, MMA, producers
    }
    if (lane == 0) {
      mbar_init(&ctl.q_full, Sh::kSoft);
      mbar_init(&ctl.drain, 1);
      mbar_init(&ctl.join_full, Sh::kSoft * a.cluster);
      ctl.abort = 0;
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();  // the next kernel (the merge) may take its place beside this one; it waits for its end
  pdl_wait_primary();
  const uint32_t tmem = ctl.tmem;
  const int C = a.cluster, rank = C > 1 ? (int)cluster_ctarank() : 0;
  bool met = C == 1;  // the cluster's CTAs all run
  if (C > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

  // ---- shares of windows: tiles, and blocks before each --------------------------------------
  // (up to 32 tiles, of up to 32 requests: by the warp that needs them)
  auto tile_blocks = [&](int t) -> int {
    const int r = k8_search(ctl.base, a.n_req, t);
    const int t0 = ld_in(a.req_row_start + r) + (t - ctl.base[r]) * a.rows;
    const int rows = a.rows == 1 ? 1 : min(a.rows, ld_in(a.req_row_start + r + 1) - t0);
    const int3 y = k8_window(a, t0, rows);
    ctl.tile[t] = make_int4(t0, r * 256 + rows, y.y, y.x);
    return k8_blocks<kBlock>(y.x) + kK8Lead;
  };
  const bool few = a.n_req <= 32 && a.tile_slots <= 32;
  int tiles = a.n_rows;
  if constexpr (kWindow) {
    if (a.mode == kK8Shares && !few) {
      // the lengths on their way to L2 beside the requests' starts
      if (threadIdx.x * 32 < a.n_rows) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.row_len + threadIdx.x * 32) : "memory");
#pragma unroll 1
      for (int r = threadIdx.x; r < a.n_req; r += Sh::kThreads) ctl.base[r] = k8_request_tiles(a, r);
      k8_scan<Sh::kThreads>(ctl.base, a.n_req, ctl.scan);
      tiles = min(ctl.base[a.n_req], kK8MaxTiles);
#pragma unroll 1
      for (int t = threadIdx.x; t < tiles; t += Sh::kThreads) ctl.pre[t] = tile_blocks(t);
      k8_scan<Sh::kThreads>(ctl.pre, tiles, ctl.scan);
    }
  }

  auto next_seg = [&](int k, Seg& w) -> bool {
    const int sl = k % kK8SegRing;
    if (!k8_wait(&ctl.seg_full[sl], (uint32_t)(k / kK8SegRing) & 1u, abort)) return false;
    w = ctl.seg[sl];
    k8_arrive(&ctl.seg_empty[sl]);
    return w.rows >= 0;
  };

  if (warp == Sh::kSoft + 1) {
    // ---- the CTA's segments ----------------------------------------------------------------
    // (the rows' lengths on their way to L2 beside the requests' starts)
    if (kWindow && (a.mode != kK8Shares || few) && lane * 32 < a.n_rows && a.n_rows <= 1024)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.row_len + lane * 32) : "memory");
    int k = 0, most = 0;  // segments, and the blocks of the longest
    auto publish = [&](const Seg& w) -> bool {
      const int sl = k % kK8SegRing;
      // a segment is taken up when the one before it is done: that may be a whole long one (the other roles,
      // for which segments lie ready, wait for a few blocks)
      if (k >= kK8SegRing && !k8_wait(&ctl.seg_empty[sl], (uint32_t)(k / kK8SegRing - 1) & 1u, abort, most)) return false;
      most = max(most, w.j1 - w.j0);
      if (lane == 0) {
        ctl.seg[sl] = w;
        mbar_arrive(&ctl.seg_full[sl]);
      }
      if (k > 0 && w.rows > 0) {  // q, and a list's first slots, on their way to L2 while the CTA is busy
#pragma unroll 1
        for (int i = lane; i < w.rows * a.group * (D / 64); i += 32) {
          const int pair = i / (D / 64), row = (int)(pair * a.group_inv >> 16);
          const uint16_t* src = a.q + (int64_t)(w.t0 + row) * a.ld_q + ((int64_t)w.g * a.group + pair - row * a.group) * D;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src + i % (D / 64) * 64) : "memory");
        }
        const int at = w.j0 * kBlock + lane * 32;
        if (!kWindow && lane < 2 * kBlock / 32 && at < w.n)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a.slots + w.t0 * a.ld_slots + at) : "memory");
      }
      ++k;
      return true;
    };
    bool ok = true;
    if (a.mode != kK8Shares) {
      // a cluster's unit, or whole ones in turn
      const bool one = a.mode == kK8Cluster;
      int u = one ? (int)(blockIdx.x >> a.cluster_shift) : (int)blockIdx.x;
      const int end = one ? u + 1 : a.tile_slots * a.h_kv;
#pragma unroll 1
      for (; ok && u < end; u += gridDim.x) {
        Seg w{};
        w.slot = -1;
        const int t = u / a.h_kv;
        w.t0 = t;
        w.g = u - t * a.h_kv;
        w.n = a.n_idx;
        w.rows = 1;
        if constexpr (kWindow) {
          int number = 0;
          if constexpr (kShared) w.r = k8_find(a, t, number);
          else w.r = warp_row_request(a.req_row_start, a.n_req, t);
          if (w.r < 0) continue;               // no such tile
          if constexpr (kShared) {
            w.t0 = ld_in(a.req_row_start + w.r) + number * a.rows;
            w.rows = min(a.rows, ld_in(a.req_row_start + w.r + 1) - w.t0);
          }
          const int3 y = k8_window(a, w.t0, w.rows);
          w.n = y.x;
          w.first = y.y;
          w.ns = y.z;
        }
        const int nb = k8_blocks<kBlock>(w.n);  // at most 2^23
        w.j0 = nb * rank >> a.cluster_shift;
        w.j1 = nb * (rank + 1) >> a.cluster_shift;
        ok = publish(w);
      }
    } else {
      if constexpr (kWindow) {
        if (few) {
          const int own = lane < a.n_req ? k8_request_tiles(a, lane) : 0, upto = k8_warp_scan(own);
          ctl.base[lane] = upto - own;
          tiles = min(__shfl_sync(0xffffffffu, upto, 31), 32);
          __syncwarp();
          const int blocks = lane < tiles ? tile_blocks(lane) : 0, sum = k8_warp_scan(blocks);
          ctl.pre[lane] = sum - blocks;
          if (lane == 31) ctl.pre[32] = sum;
          __syncwarp();
        }
      }
      const int cta = blockIdx.x, ctas = gridDim.x;
      const int4 no_job = make_int4(-1, 0, 0, 0);
      int4 job = no_job;
      const int same = k8_blocks<kBlock>(a.n_idx) + kK8Lead;  // a list's blocks
      const int total = (kWindow ? ctl.pre[tiles] : tiles * same) * a.h_kv;
      // the first `more` CTAs take per + 1 blocks, the others per
      const int per = total / ctas, more = total - per * ctas;
      int b = cta * per + min(cta, more);
      const int end = b + per + (cta < more ? 1 : 0);
#pragma unroll 1
      while (ok && b < end) {
        const int bt = b / a.h_kv;  // at or behind the tile's first block, before its last head's end
        Seg w{};
        w.slot = -1;
        int first_b, nbl, u_tile;              // (nbl: with the lead)
        if constexpr (kWindow) {
          const int t = u_tile = k8_search(ctl.pre, tiles, bt);
          const int4 y = ctl.tile[t];
          first_b = ctl.pre[t];
          nbl = ctl.pre[t + 1] - first_b;
          w.t0 = y.x;
          w.rows = y.y & 255;
          w.r = y.y >> 8;
          w.first = y.z;
          w.n = y.w;
          w.ns = min(a.n_sink, w.first);
        } else {
          w.t0 = u_tile = bt / same;
          w.rows = 1;
          w.n = a.n_idx;
          first_b = w.t0 * same;
          nbl = same;
        }
        const int in = b - first_b * a.h_kv;  // within the tile, head by head
        w.g = in / nbl;
        const int at = in - w.g * nbl, take = min(nbl - at, end - b), nb = nbl - kK8Lead;
        const int unit0 = b - at + kK8Lead;    // the unit's first block
        b += take;
        w.j0 = max(at - kK8Lead, 0);
        w.j1 = max(at + take - kK8Lead, 0);
        if (w.j0 == w.j1) continue;            // nothing but (a part of) the lead
        if (w.j0 > 0) w.slot = 2 * cta;
        else if (w.j1 < nb) w.slot = 2 * cta + 1;
        if (w.j1 == nb) {  // the unit ends here: the job names the first CTA that has a part
          int4 y = no_job;
          if (w.j0 > 0) {
            const int longer = more * (per + 1);
            y = make_int4(unit0 < longer ? unit0 / (per + 1) : more + (unit0 - longer) / per, cta, w.t0, w.g * 256 + w.rows);
          }
          if (!a.jobs_by_unit) {
            if (w.j0 > 0) job = y;
          } else if (lane == 0) {
            a.jobs[u_tile * a.h_kv + w.g] = y;
          }
        }
        ok = publish(w);
      }
      if (!a.jobs_by_unit) {
        if (lane == 0) a.jobs[cta] = job;
      } else if (cta == 0) {  // units that are none
#pragma unroll 1
        for (int u = tiles * a.h_kv + lane; u < a.tile_slots * a.h_kv; u += 32) a.jobs[u] = no_job;
      }
    }
    if (ok) {
      Seg none{};
      none.rows = -1;
      publish(none);
    }
  } else if (warp > Sh::kSoft + 1) {
    // ---- K and V rows ------------------------------------------------------------------------
    const int pw = warp - (Sh::kSoft + 2);
    constexpr int kE = 4 * kSub / Sh::kProd;   // entries of a lane: 32 (kE pw + i) + lane of a block
    constexpr int PP = D / 16, kRows = 32 / PP;  // 16-byte pieces of a row, rows a warp copies at once
    constexpr int kDepth = S - 1;              // tiles on the way
    const int c = lane % PP;
    const uint32_t pitch = (uint32_t)a.h_kv * D;
    int u = 0, told = 0;                       // uses so far, and those known to have landed
    bool ok = true;
    auto signal = [&](int use) {               // the tile of that use has landed
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      k8_arrive(&ctl.full[use % S]);
    };
    auto copy = [&](const uint8_t* src, const int32_t (&slot)[kE]) -> bool {
      const int st = u % S;
      if (u >= S && !k8_wait(&ctl.empty[st], (uint32_t)(u / S - 1) & 1u, abort)) return false;
      __syncwarp();
      // a tile: [D / 128 or kSub][128 entries][128 B]
      const uint32_t dst = smem_u32(ring) + (uint32_t)(st * Sh::kTile + (c >> 3) * 16384);
#pragma unroll
      for (int i = 0; i < kE * 32 / kRows; ++i) {
        const int rr = i * kRows + lane / PP, row = pw * (kE * 32) + rr;
        const int32_t s = __shfl_sync(0xffffffffu, slot[i * kRows / 32], rr & 31);
        ka_cp16(dst + row * 128 + (((c & 7) ^ (row & 7)) << 4), src + (uint64_t)(uint32_t)max(s, 0) * pitch, s >= 0);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      ++u;
#pragma unroll 1
      while (told <= u - kDepth) signal(told++);
      return true;
    };
    auto flush = [&]() {  // (loops of one or two passes, not unrolled)
      asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
      while (told < u) signal(told++);
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      Seg w;
      // the others may have to use what is on the way before the next segment is known
      if (!__all_sync(0xffffffffu, mbar_try_wait(&ctl.seg_full[k % kK8SegRing], (uint32_t)(k / kK8SegRing) & 1u))) flush();
      if (!next_seg(k, w)) break;
      const uint8_t* gk = a.k + (int64_t)w.g * D + c * 16;
      const uint8_t* gv = a.v + (int64_t)w.g * D + c * 16;
      auto entry = [&](int j, int i) -> int {
        return j < w.j1 ? j * kBlock + (pw * kE + i) * 32 + lane : INT32_MAX;
      };
      KaFetch next[kE];
      int32_t last[kE], slot[kE] = {};
#pragma unroll
      for (int i = 0; i < kE; ++i) next[i] = k8_fetch<kWindow>(a, w, entry(w.j0, i));
#pragma unroll 1
      for (int j = w.j0; ok && j <= w.j1; ++j) {  // K(j), V(j - 1)
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          last[i] = slot[i];
          slot[i] = k8_slot<kWindow, true>(a, w, entry(j, i), next[i]);
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) next[i] = k8_fetch<kWindow>(a, w, entry(j + 1, i));
#pragma unroll 1
        for (int v = 0; ok && v < 2; ++v) {    // (one copy of the code: instructions are fetched, too)
          if (v == 0 ? j == w.j1 : j == w.j0) continue;
          int32_t from[kE];
#pragma unroll
          for (int i = 0; i < kE; ++i) from[i] = v == 0 ? slot[i] : last[i];
          ok = copy(v == 0 ? gk : gv, from);
        }
      }
    }
    flush();
  } else if (warp == Sh::kSoft) {
    // ---- MMAs --------------------------------------------------------------------------------
    // K tile: [D / 128 or kSub][128 entries][128 B], Q: [D / 128][2 N][128 B], 128-byte swizzled; V
    // tile like K's, its rows the K index of the product, as those of P: [kSub][groups of 32 columns][128 entries][32
    // B], 32-byte swizzled (a thread's weights lie next to each other)
    const uint64_t k_desc0 = umma_desc_sw128(smem_u32(ring)), q_desc = umma_desc_sw128(smem_u32(q_buf)),
                   p_desc0 = k8_desc_p(smem_u32(p_buf), 4096);
    int x = 0, st = 0;        // blocks so far; next ring stage and its parity
    uint32_t ph = 0;
    bool ok = true;
    auto next_stage = [&]() {
      k8_commit(&ctl.empty[st]);
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      Seg w;
      if (!next_seg(k, w)) break;
      const int nb = __reduce_max_sync(0xffffffffu, w.j1 - w.j0);  // uniform
      ok = k8_wait(&ctl.q_full, (uint32_t)k & 1u, abort);
#pragma unroll 1
      for (int i = 0; ok && i <= nb; ++i) {
        if (i < nb) {  // S(i)
          const int sl = (x + i) & 1, had = x + i - Sh::kSBuf;  // the block that had this buffer
          ok = k8_wait(&ctl.full[st], ph, abort) &&
               (had < 0 || k8_wait(&ctl.s_free[had & 1], (uint32_t)(had >> 1) & 1u, abort));
          if (!ok) break;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int y = 0; y < kSub; ++y)
#pragma unroll
            for (int h = 0; h < H; ++h)
              k8_mma4<2, 2>(tmem + (sl % Sh::kSBuf * kSub + y) * NS, k_desc0 + (uint64_t)((st * Sh::kTile + (h + y) * 16384) >> 4),
                            q_desc + (uint64_t)((h * NS * 128) >> 4), k8_idesc(NS, false), h > 0 ? 1u : 0u);
          next_stage();
          k8_commit(&ctl.s_full[sl]);
        }
        if (i > 0) {  // O += P(i - 1) V(i - 1)
          const int sl = (x + i - 1) & 1;
          ok = k8_wait(&ctl.full[st], ph, abort) && k8_wait(&ctl.p_full[sl], (uint32_t)((x + i - 1) >> 1) & 1u, abort);
          if (!ok) break;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int y = 0; y < kSub; ++y)
#pragma unroll
            for (int h = 0; h < H; ++h)
              k8_mma4<256, 64>(tmem + Sh::kColO + h * NP, k_desc0 + (uint64_t)((st * Sh::kTile + (h + y) * 16384) >> 4),
                              p_desc0 + (uint64_t)((sl * Sh::kP + y * Sh::kPSub) >> 4), k8_idesc(NP, true),
                              i > 1 || y > 0 ? 1u : 0u);
          next_stage();
          k8_commit(&ctl.pv_done[sl]);
        }
      }
      x += nb;
    }
    // every MMA has finished before the memories are released (also where a wait has been given up)
    k8_commit(&ctl.drain);
    if (!__all_sync(0xffffffffu, mbar_wait_bounded(&ctl.drain, 0u, kK8WaitNs)) && lane == 0) k8_fault(kFaultWait);
  } else {
    // ---- softmax and outputs: a thread for an entry and a slice of the pairs --------------------
    const int slice = warp / (4 * kSub), p0 = slice * kPer, sub = (warp >> 2) % kSub;
    const int lane_e = (warp & 3) * 32 + lane, e = sub * 128 + lane_e;  // tensor-memory lane, entry of the block
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    int n_slice = 0, n_all = 0;                // meetings so far
    // (bounded, unlike a named barrier: a warp that gives up holds none up)
    // the slice's warps have written what comes before
    auto met_arrive = [&]() { k8_arrive(&ctl.met[slice]); };
    auto met_wait = [&]() -> bool { return k8_wait(&ctl.met[slice], (uint32_t)n_slice++ & 1u, abort); };
    auto meet = [&]() -> bool {
      met_arrive();
      return met_wait();
    };
    auto meet_all = [&]() -> bool {
      k8_arrive(&ctl.met[Sh::kSlices]);
      return k8_wait(&ctl.met[Sh::kSlices], (uint32_t)n_all++ & 1u, abort);
    };
    constexpr int W = 4 * kSub;                // warps of a slice
    // a segment's loads: q of the warp's pairs, their rows' lengths, the thread's first two entries
    uint32_t qv[Sh::kLoads][H * 2];            // D / 32 dimensions of the lane
    int q_len[Sh::kLoads];
    KaFetch f0, next;
    auto entry = [&](const Seg& w, int j) -> int { return j < w.j1 ? j * kBlock + e : INT32_MAX; };
    auto load = [&](const Seg& w) {
      const int pairs = w.rows * a.group;
#pragma unroll
      for (int i = 0; i < Sh::kLoads; ++i) {
        const int p = warp + i * Sh::kSoft, row = (int)(p * a.group_inv >> 16), hd = p - row * a.group;
#pragma unroll
        for (int y = 0; y < H * 2; ++y) qv[i][y] = 0u;
        q_len[i] = 0;
        if (p < pairs) {
          const uint16_t* src = a.q + (int64_t)(w.t0 + row) * a.ld_q + ((int64_t)w.g * a.group + hd) * D + lane * (D / 32);
          if constexpr (D == 256) {
            const uint4 y = ld_in(reinterpret_cast<const uint4*>(src));
            qv[i][0] = y.x; qv[i][1] = y.y; qv[i][2] = y.z; qv[i][3] = y.w;
          } else {
            const uint2 y = ld_in(reinterpret_cast<const uint2*>(src));
            qv[i][0] = y.x; qv[i][1] = y.y;
          }
          if constexpr (kShared) q_len[i] = ld_in(a.row_len + w.t0 + row);
        }
      }
      f0 = k8_fetch<kWindow>(a, w, entry(w, w.j0));
      next = k8_fetch<kWindow>(a, w, entry(w, w.j0 + 1));
    };
    int x = 0;                                 // blocks so far
    int use = 0;                               // ring uses so far
    Seg w{};
    w.rows = -1;
    bool ok = true;
    float l[kPer];                             // sums of weights
    int nb = 0;
    K8Scales sc{};
#pragma unroll 1
    for (int k = 0;; ++k) {
      // the next segment's q, so that its products begin (those of the one before have been read), then
      // the sums of the one before; nothing of the next is added to them before all warps are through
      Seg after;
      const bool more = next_seg(k, after);
      if (more) load(after);
      if (w.rows >= 0) {                       // (before the loads are waited for)
        // the lanes' sums: half of the pairs go to each half of the lanes, and so on; in the end lane
        // 32 / kPer i has pair i
        float y[kPer];
#pragma unroll
        for (int p = 0; p < kPer; ++p) y[p] = l[p];
#pragma unroll
        for (int d = 16, n = kPer / 2; n > 0; d >>= 1, n >>= 1) {
          const bool up = (lane & d) != 0;
#pragma unroll
          for (int p = 0; p < n; ++p) {
            const float give = up ? y[p] : y[p + n], keep = up ? y[p + n] : y[p];
            y[p] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        }
#pragma unroll
        for (int d = 16 / kPer; d > 0; d >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], d);
        if (lane % (32 / kPer) == 0) ctl.wsum[warp][lane / (32 / kPer)] = y[0];
        met_arrive();
      }
      if (more) {
        const int pairs = after.rows * a.group;
        sc = k8_scales(a, k8_slot<kWindow, false>(a, after, entry(after, after.j0), f0), after.g);
        // q: a warp for a pair, two parts
#pragma unroll
        for (int i = 0; i < Sh::kLoads; ++i) {
          const int p = warp + i * Sh::kSoft;
          if (p >= N) break;
          const int row = (int)(p * a.group_inv >> 16), hd = p - row * a.group;
          uint32_t mx = 0;
#pragma unroll
          for (int y = 0; y < H * 2; ++y) mx = __vmaxu2(mx, qv[i][y] & 0x7fff7fffu);
          const uint32_t top = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
          // the largest component to [128, 256)
          const int ex = min(max((int)(top >> 7), 8), 254) - 127;
          const float up = kv8_pow2(7 - ex);
          uint32_t hi[H], lo[H];
#pragma unroll
          for (int c = 0; c < H; ++c) {
            uint32_t h2[2], l2[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float2 f = bf16x2_to_float2(qv[i][2 * c + y]);
              f.x *= up;
              f.y *= up;
              h2[y] = kv8_pack2(f.x, f.y);
              const float2 b = __half22float2(kv8_half2(h2[y]));
              l2[y] = kv8_pack2((f.x - b.x) * 32.f, (f.y - b.y) * 32.f);
            }
            hi[c] = h2[0] | h2[1] << 16;
            lo[c] = l2[0] | l2[1] << 16;
          }
          // rows p and N + p of [D / 128][2 N][128 B], swizzled by row mod 8 (N is a multiple of 8)
          const int d = lane * (D / 32), kh = d >> 7, ch = (d & 127) >> 4;
          unsigned char* dst = q_buf + kh * NS * 128 + p * 128 + ((ch ^ (p & 7)) << 4) + (d & 15);
          if constexpr (D == 256) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + N * 128) = make_uint2(lo[0], lo[1]);
          } else {
            *reinterpret_cast<uint32_t*>(dst) = hi[0];
            *reinterpret_cast<uint32_t*>(dst + N * 128) = lo[0];
          }
          if (lane == 0) {
            // an infinity or a NaN in q shows in the whole pair
            ctl.mult[k & 1][p] = top >= 0x7f80u ? __int_as_float(0x7fffffff)
                                         : a.scale * 1.4426950408889634f * kv8_pow2(ex - 7);
            ctl.out[k & 1][p] = p < pairs ? (after.t0 + row) * a.h_q + after.g * a.group + hd : -1;
            if constexpr (kShared) {
              int4 s = make_int4(0, 0, 0, 0);
              const int L = q_len[i];
              if (p >= pairs) s.z = INT32_MAX;   // nobody's: sees what there is
              else if (L > 0 && L <= a.max_len)
                s = make_int4(min(a.n_sink, L), after.ns + max(0, L - a.window) - after.first,
                              after.ns + L - after.first, 0);
              ctl.sees[k & 1][p] = s;
            }
          }
          if constexpr (kShared)
            if (lane < D / 32) ctl.nan[k & 1][p][lane] = 0u;
        }
        if (threadIdx.x == 0) ctl.any_nan[k & 1] = 0;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        k8_arrive(&ctl.q_full);
      }
      if (w.rows >= 0) {
        // ---- outputs: a thread for a column of O ---------------------------------------------
        ok = met_wait() && (nb == 0 || k8_wait(&ctl.pv_done[(x - 1) & 1], (uint32_t)((x - 1) >> 1) & 1u, abort));
        if (!ok) break;
        __syncwarp();
        tc_fence_after();
        const bool nans = kShared && ctl.any_nan[(k - 1) & 1] != 0;
        // a pair a lane: its M, sum and place
        const int lp = min(lane, kPer - 1);
        float sum_l = 0.f;
#pragma unroll
        for (int i = 0; i < W; ++i) sum_l += ctl.wsum[slice * W + i][lp];
        const float m_l = nb > 0 && ctl.mb[p0 + lp] != kK8None ? ctl.mb[p0 + lp] : ninf;
        const int hq_l = ctl.out[(k - 1) & 1][p0 + lp];
        const int own = N >> a.cluster_shift;  // pairs that a CTA of the cluster writes: rank, rank + C, ...
        // where the pair's sums go: to the joining CTA, the partial results, or (times 1 / L) the output.
        // (One address for all three: code that runs once takes as long as its instructions to arrive.)
        const bool done = C == 1 && w.slot < 0;
        const bool half = kWindow && done;     // BF16
        char* to_l = nullptr;
        float inv_l = 1.f;
        if (hq_l >= 0) {
          const int p = p0 + lp;
          if (C > 1) {
            float* mine = join + (Sh::kPull ? p : rank * own + (p >> a.cluster_shift)) * Sh::kJoin;
            to_l = Sh::kPull ? reinterpret_cast<char*>(mine) : map_generic_rank(mine, (uint32_t)(p & (C - 1)));
          } else if (!done) {
            to_l = reinterpret_cast<char*>(a.part + ((int64_t)w.slot * N + p) * Sh::kJoin);
          } else {
            to_l = static_cast<char*>(a.out) + (int64_t)hq_l * (D * (kWindow ? 2 : 4));
            inv_l = sum_l == 0.f ? 0.f : 1.0f / sum_l;
          }
          if ((warp & 3) == 0 && sub == 0 && lane < kPer) {  // M, L and lse by one warp
            if (!done) *reinterpret_cast<float2*>(to_l + 4 * D) = make_float2(m_l, sum_l);
            else if (a.lse != nullptr) a.lse[hq_l] = k8_lse(m_l, sum_l);
          }
        }
        // (the sub-blocks' warps take a half of the pairs each)
#pragma unroll 1
        for (int c0 = kPer / kSub * sub; c0 < kPer / kSub * (sub + 1); c0 += 4) {
          float sum[H][4];
#pragma unroll
          for (int h = 0; h < H; ++h) {
            uint32_t v[PARTS * 4];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) k8_ld4(lanes + Sh::kColO + h * NP + i * N + p0 + c0, v + i * 4);
            k8_wait_ld(v);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float o = __uint_as_float(v[(PARTS - 1) * 4 + y]);
#pragma unroll
              for (int i = PARTS - 2; i >= 0; --i) o = fmaf(o, 0.03125f, __uint_as_float(v[i * 4 + y]));
              sum[h][y] = nb > 0 ? o : 0.f;      // no block: nothing was written there
            }
          }
          if (nans) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
              for (int h = 0; h < H; ++h)
                if ((ctl.nan[(k - 1) & 1][kShared ? p0 + c0 + y : 0][h * 4 + (lane_e >> 5)] >> (lane_e & 31)) & 1u)
                  sum[h][y] = __int_as_float(0x7fffffff);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            char* to = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to_l), c0 + y));
            const float inv = __shfl_sync(0xffffffffu, inv_l, c0 + y);
            if (to == nullptr) continue;
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const float o = sum[h][y] * inv;
              if (half) reinterpret_cast<__nv_bfloat16*>(to)[h * 128 + lane_e] = __float2bfloat16_rn(o);
              else reinterpret_cast<float*>(to)[h * 128 + lane_e] = o;
            }
          }
        }
        if (C > 1) {
          k8_arrive_all(&ctl.join_full, C);
          ok = k8_wait_cluster(&ctl.join_full, abort);
          if (!ok) break;
          // a warp for 128 columns of a pair, or (more than 16 pairs) for all, four sources at a time
          constexpr int kCols = N <= 16 ? 128 : D, V = kCols / 128;
#pragma unroll 1
          for (int i = warp; i < own * (D / kCols); i += Sh::kSoft) {
            const int p = i / (D / kCols) * C + rank, col = i % (D / kCols) * kCols + lane * 4;
            if (p >= w.rows * a.group) break;
            float M = ninf, L = 0.f, sum[V * 4] = {};
#pragma unroll 1
            for (int c0 = 0; c0 < C; c0 += 4) {
              float v[4][V * 4], m[4], l4[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                m[c] = ninf;
                l4[c] = 0.f;
#pragma unroll
                for (int y = 0; y < V * 4; ++y) v[c][y] = 0.f;
                if (c0 + c >= C) continue;
                const uint32_t from = Sh::kPull ? map_shared_rank(join + p * Sh::kJoin, (uint32_t)(c0 + c))
                                                : smem_u32(join + ((c0 + c) * own + (p >> a.cluster_shift)) * Sh::kJoin);
#pragma unroll
                for (int y = 0; y < V; ++y) {
                  const float4 f = ld_cluster_f4(from + 4 * (col + y * 128));
                  v[c][y * 4] = f.x; v[c][y * 4 + 1] = f.y; v[c][y * 4 + 2] = f.z; v[c][y * 4 + 3] = f.w;
                }
                const float2 f = ld_cluster_f2(from + 4 * D);
                m[c] = f.x;
                l4[c] = f.y;
              }
              const float top = fmaxf(M, fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
              const float hm = M == ninf ? 1.f : k8_half(M - top), fm = hm * hm;
              M = top;
              L = L * hm * hm;
#pragma unroll
              for (int y = 0; y < V * 4; ++y) sum[y] *= fm;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (c0 + c >= C) break;
                const float h = m[c] == ninf ? 0.f : k8_half(m[c] - M), f = h * h;
                L += m[c] == ninf ? l4[c] : l4[c] * h * h;  // without a weight (or with NaN only) M = -inf
#pragma unroll
                for (int y = 0; y < V * 4; ++y) sum[y] = fmaf(f, v[c][y], sum[y]);
              }
            }
            const float inv = L == 0.f ? 0.f : 1.0f / L;
            const int64_t at = (int64_t)ctl.out[(k - 1) & 1][p] * D + col;
#pragma unroll
            for (int y = 0; y < V; ++y) {
              const float4 o = make_float4(sum[y * 4] * inv, sum[y * 4 + 1] * inv, sum[y * 4 + 2] * inv, sum[y * 4 + 3] * inv);
              if constexpr (kWindow) {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at + y * 128) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
              } else {
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + y * 128) = o;
              }
            }
            if (col == 0 && a.lse != nullptr)
              a.lse[ctl.out[(k - 1) & 1][p]] = k8_lse(M, L);
          }
        }
        tc_fence_before();
      }
      if (!more) break;
      w = after;
      nb = w.j1 - w.j0;
      ok = meet_all();                         // the pairs' words are there, M's are free
      if (!ok) break;
      int4 both = make_int4(0, 0, 0, 0);       // shared tiles: every pair sees entries [0, x) and [y, z)
      if constexpr (kShared) {
        int va = INT32_MAX, vb = 0, vc = INT32_MAX;
#pragma unroll 1
        for (int p = lane; p < w.rows * a.group; p += 32) {
          const int4 y = ctl.sees[k & 1][p];
          va = min(va, y.x);
          vb = max(vb, y.y);
          vc = min(vc, y.z);
        }
        both = make_int4(__reduce_min_sync(0xffffffffu, va), __reduce_max_sync(0xffffffffu, vb),
                         __reduce_min_sync(0xffffffffu, vc), 0);
      }

      if (!met) {                              // (here it has long come about, and costs nothing)
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        met = true;
      }
#pragma unroll
      for (int p = 0; p < kPer; ++p) l[p] = 0.f;
#pragma unroll 1
      for (int b = 0; ok && b < nb; ++b, ++x) {
        const int sl = x & 1, j = w.j0 + b;
        ok = k8_wait(&ctl.s_full[sl], (uint32_t)(x >> 1) & 1u, abort);
        if (!ok) break;
        __syncwarp();
        tc_fence_after();
        uint32_t v[2 * kPer];
        k8_ld<kPer>(lanes + (sl % Sh::kSBuf * kSub + sub) * NS + p0, v);
        k8_ld<kPer>(lanes + (sl % Sh::kSBuf * kSub + sub) * NS + N + p0, v + kPer);
        // meanwhile the scales of the next block, slots of the one behind it
        const K8Scales now = sc;
        sc = k8_scales(a, k8_slot<kWindow, false>(a, w, entry(w, j + 1), next), w.g);
        next = k8_fetch<kWindow>(a, w, entry(w, j + 2));
        const float kf = __uint_as_float((uint32_t)now.k << 23), vf = __uint_as_float((uint32_t)now.v << 23);
        const float ev = (float)((int)now.v - 127);
        const int i_e = j * kBlock + e;
        bool part = false;                     // a pair of the tile does not see an entry of the block
        uint32_t sees = 0;                     // then: the thread's pairs that see its entry
        if constexpr (kShared) {
          const int b0 = j * kBlock, b1 = min(b0 + kBlock, w.n);
          part = !(b1 <= both.x || (b0 >= both.y && b1 <= both.z));
          if (part) {
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
              const int4 y = ctl.sees[k & 1][p0 + p];
              sees |= (uint32_t)(i_e < y.x || (i_e >= y.y && i_e < y.z)) << p;
            }
          }
        }
        float t[kPer];                         // logits (base 2); -inf where the pair does not see the entry
        k8_wait_ld(v);
        tc_fence_before();
        k8_arrive(&ctl.s_free[sl]);
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
          t[p] = fmaf(__uint_as_float(v[kPer + p]), 0.03125f, __uint_as_float(v[p])) * (ctl.mult[k & 1][p0 + p] * kf);
          if (!now.valid) t[p] = ninf;
        }
        if (part) {
#pragma unroll
          for (int p = 0; p < kPer; ++p)
            if (((sees >> p) & 1u) == 0) t[p] = ninf;
        }
        if (x >= 2) {
          ok = k8_wait(&ctl.pv_done[sl], (uint32_t)((x - 2) >> 1) & 1u, abort);  // P's buffer
          if (!ok) break;
        }
        unsigned char* const pb = p_buf + sl * Sh::kP + sub * Sh::kPSub + lane_e * 32;
        const int flip = (lane_e >> 2) & 1;    // the swizzle of the thread's row
        // A weight is 2^(t - M + kK8Bias); where one times its V scale would pass
        // 2^(kKaGrow + kK8Bias), M has to grow.  With registers to spare, whether it
        // has to is asked beside the weights, which go on as if not.  (One copy of
        // the code for all passes: instructions are fetched, too.)
        const float limit = (float)(kKaGrow + kK8Bias) - ev;
        auto vote = [&](bool grow) -> bool {   // of the slice's warps; ok: it came about
          const bool any = __any_sync(0xffffffffu, grow);
          if (lane == 0) ctl.vote[sl][warp] = any;
          ok = meet();
          if (!ok) return false;
          int votes = 0;
#pragma unroll
          for (int i = 0; i < W; ++i) votes |= ctl.vote[sl][slice * W + i];
          return votes != 0;
        };
        float was[Sh::kAhead ? kPer : 1];
        bool again = b == 0;                   // the first block has no M yet
        if constexpr (Sh::kAhead) {
#pragma unroll
          for (int p = 0; p < kPer; ++p) was[p] = l[p];
        } else if (!again) {
          bool grow = false;
#pragma unroll
          for (int p = 0; p < kPer; ++p) grow |= t[p] - ctl.mb[p0 + p] > limit;
          again = vote(grow);
          if (!ok) break;
        }
#pragma unroll 1
        while (ok) {
          if (again) {
            // M of the pairs that pass the limit, or had none, becomes the block's maximum; O and l follow
            const bool first = b == 0;
#pragma unroll
            for (int p = 0; p < kPer; ++p) {
              float top;
              asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(t[p] + ev));
              if (lane == 0) ctl.wmax[warp][p] = top;
            }
            ok = meet();
            if (!ok) break;
            // a pair a lane
            const int lp = min(lane, kPer - 1);
            float top = ctl.wmax[slice * W][lp];
#pragma unroll
            for (int i = 1; i < W; ++i) top = fmaxf(top, ctl.wmax[slice * W + i][lp]);
            top -= (float)kK8Bias;
            const float old = first ? kK8None : ctl.mb[p0 + lp];
            const float mn = top > old + (float)kKaGrow ? top : old;
            if (!first) {
              const float hl = old == kK8None ? 1.f : k8_half(old - mn), fl = hl * hl;
              float f[kPer];
#pragma unroll
              for (int p = 0; p < kPer; ++p) {
                const float h = __shfl_sync(0xffffffffu, hl, p);
                // (a second exchange with 16 pairs a thread, where the product spilled 30 bytes more: 192 x 2051 28.4 us
                // instead of 30.5; with fewer the product, 127.6 instead of 129.1 us for 8 long requests)
                f[p] = Sh::kAhead ? h * h : __shfl_sync(0xffffffffu, fl, p);
                l[p] = (Sh::kAhead ? was[Sh::kAhead ? p : 0] : l[p]) * h * h;
              }
              // O holds every product before this block's
              ok = meet() && k8_wait(&ctl.pv_done[sl ^ 1], (uint32_t)((x - 1) >> 1) & 1u, abort);
              if (!ok) break;
              __syncwarp();
              tc_fence_after();
              if (sub == 0) {
#pragma unroll 1
                for (int i = 0; i < H * PARTS; ++i) {
                  const uint32_t at = lanes + Sh::kColO + i / PARTS * NP + i % PARTS * N + p0;
                  uint32_t o[kPer];
                  k8_ld<kPer>(at, o);
                  k8_wait_ld(o);
#pragma unroll
                  for (int y = 0; y < kPer; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f[y]);
                  k8_st<kPer>(at, o);
                }
                k8_wait_st();
              }
              tc_fence_before();
            }
            // every warp of the slice writes the same, once all have read what was there
            if (lane < kPer) ctl.mb[p0 + lane] = mn;
            __syncwarp();
          }
          // the weights: their sums, and parts of 4 bits for the product
          bool grow = false;
          uint32_t words[PARTS][kPer / 4];
#pragma unroll
          for (int p = 0; p < kPer; p += 4) {
            uint64_t r01, r23;
            float r[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float u = t[p + y] - ctl.mb[p0 + p + y];
              if constexpr (Sh::kAhead) grow |= u > limit;
              r[y] = ka_ex2(u);
              l[p + y] += r[y];
              r[y] *= vf;
            }
            r01 = k8_pair(r[0], r[1]);
            r23 = k8_pair(r[2], r[3]);
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
              const uint32_t c0 = kv8_pack2(k8_low(r01), k8_high(r01)), c1 = kv8_pack2(k8_low(r23), k8_high(r23));
              words[i][p / 4] = c0 | c1 << 16;
              if (i + 1 < PARTS) {  // (r - what the part holds) * 32
                const __half2 m32 = __floats2half2_rn(-32.f, -32.f);
                const float2 b0 = __half22float2(__hmul2(kv8_half2(c0), m32)), b1 = __half22float2(__hmul2(kv8_half2(c1), m32));
                r01 = k8_fma2(r01, k8_pair(32.f, 32.f), k8_pair(b0.x, b0.y));
                r23 = k8_fma2(r23, k8_pair(32.f, 32.f), k8_pair(b1.x, b1.y));
              }
            }
          }
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            if constexpr (kPer == 16) {
              const int n = i * N + p0;
              *reinterpret_cast<uint4*>(pb + (n >> 5) * 4096 + ((((n >> 4) & 1) ^ flip) << 4)) =
                  make_uint4(words[i][0], words[i][1], words[i][2], words[i][3]);
            } else if constexpr (kPer == 4) {
              const int n = i * N + p0;
              *reinterpret_cast<uint32_t*>(pb + (n >> 5) * 4096 + ((((n >> 4) & 1) ^ flip) << 4) + (n & 15)) = words[i][0];
            } else {
              const int n = i * N + p0;
              *reinterpret_cast<uint2*>(pb + (n >> 5) * 4096 + ((((n >> 4) & 1) ^ flip) << 4) + (n & 15)) =
                  make_uint2(words[i][0], words[i][1]);
            }
          }
          if (again || !Sh::kAhead) break;
          again = vote(grow);
          if (!again) break;
        }
        if (!ok) break;
        // NaN of V where some pair does not see the entry
        if constexpr (kShared) {
          if (part && slice == 0) {
            const int at = use + (nb == 1 ? 1 : b + 1 == nb ? 2 * nb - 1 : 2 * b + 2);
            ok = k8_wait(&ctl.full[at % S], (uint32_t)(at / S) & 1u, abort);
            if (!ok) break;
            // entries that some pairs see and others do not, one after the other by the whole warp: D / 32
            // codes a lane
            uint32_t todo = __ballot_sync(0xffffffffu, now.valid && !(i_e < both.x || (i_e >= both.y && i_e < both.z)));
#pragma unroll 1
            while (todo != 0) {
              const int f = __ffs(todo) - 1;
              todo &= todo - 1;
              const int ef = e - lane + f, at_e = i_e - lane + f, d0 = lane * (D / 32), c = d0 >> 4;
              uint32_t* word = reinterpret_cast<uint32_t*>(ring + (at % S) * Sh::kTile + ef * 128 + (c >> 3) * 16384 +
                                                           (((c & 7) ^ (ef & 7)) << 4) + (d0 & 15));
#pragma unroll
              for (int y = 0; y < D / 128; ++y) {
                const uint32_t bad = __vcmpeq4(word[y] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                if (bad == 0) continue;
                word[y] &= ~bad;
                // columns d0 + 4 y .. + 3
                const uint32_t bits = ((bad & 1u) | (bad >> 7 & 2u) | (bad >> 14 & 4u) | (bad >> 21 & 8u)) << ((d0 + 4 * y) & 31);
#pragma unroll 1
                for (int p = 0; p < w.rows * a.group; ++p) {
                  const int4 s4 = ctl.sees[k & 1][p];
                  if (at_e < s4.x || (at_e >= s4.y && at_e < s4.z)) atomicOr(&ctl.nan[k & 1][p][(d0 + 4 * y) >> 5], bits);
                }
                ctl.any_nan[k & 1] = 1;
              }
              __syncwarp();
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        k8_arrive(&ctl.p_full[sl]);
      }
      if (!ok) break;
      use += 2 * nb;

    }
  }

  // no CTA of the cluster leaves before all have read each other's sums
  if (C > 1) {
    if (!met) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == Sh::kSoft)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Units that several CTAs shared: out = sum_s f_s O_s / sum_s f_s l_s, f_s =
// 2^(M_s - max M).  CTA (i, y, z) works for job i.
// Few parts to a unit: its threads are D columns of 1024 / D pairs, which add
// up their parts by themselves.  Many (kMany): 64 columns of one pair, for which
// 16 groups take the parts in turn and meet in shared memory.
constexpr int kK8MergeThreads = 1024;
template <int D, bool kMany>
__global__ void __launch_bounds__(kK8MergeThreads)
kv8_merge_kernel(const __grid_constant__ Kv8AttnArgs a, int n) {
  constexpr int kCols = kMany ? 64 : D, G = kK8MergeThreads / kCols;
  __shared__ float s_m[kMany ? G : 1], s_l[kMany ? G : 1], s_o[kMany ? G : 1][64];
  const int grp = threadIdx.x / kCols;
  const int p = kMany ? blockIdx.y : blockIdx.y * G + grp, d = blockIdx.z * kCols + threadIdx.x % kCols;
  const float ninf = -__int_as_float(0x7f800000);
  pdl_launch_dependents();
  // A first pass of one warp loads and stores nothing: it runs beside the kernel before, and brings
  // the instructions of the second.
#pragma unroll 1
  for (bool live = threadIdx.x >= 32;; live = true) {
    if (live) pdl_wait_primary();
    int4 job = make_int4(0, 0, 0, 1);
    if (live) job = ld_in(a.jobs + blockIdx.x);
    const int k = job.y;
    if (job.x < 0 || (live && p >= (job.w & 255) * a.group)) return;  // (with kMany the whole CTA)
    // the first part begins the unit (its CTA's second slot), the others come from within it
    auto part = [&](int c) -> const float* {
      return a.part + ((int64_t)(2 * c + (c == job.x ? 1 : 0)) * n + p) * (D + 4);
    };
    float m = ninf, l = 0.f, o = 0.f;
    auto add = [&](float ms, float ls, float os) {  // with M at least ms
      const float h = ms == ninf ? 0.f : k8_half(ms - m);
      l += ms == ninf ? ls : ls * h * h;  // without a weight (or with NaN only) M = -inf
      o = fmaf(h * h, os, o);
    };
    constexpr int kStep = kMany ? G : 1, kU = 4;
#pragma unroll 1
    for (int c0 = job.x + (kMany ? grp : 0); c0 <= k; c0 += kU * kStep) {
      float2 ml[kU];
      float os[kU];  // on the way together
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const float* pp = part(min(c0 + i * kStep, k));
        ml[i] = live ? ld_in(reinterpret_cast<const float2*>(pp + D)) : make_float2(0.f, 1.f);
        os[i] = live ? ld_in(pp + d) : 0.f;
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kU; ++i) mn = fmaxf(mn, c0 + i * kStep <= k ? ml[i].x : ninf);
      const float g = m == ninf ? 1.f : k8_half(m - mn);  // (nothing or a NaN yet)
      l = l * g * g;
      o *= g * g;
      m = mn;
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (c0 + i * kStep <= k) add(ml[i].x, ml[i].y, os[i]);
    }
    if constexpr (kMany) {
      const int col = threadIdx.x % 64;
      if (live) {
        s_o[grp][col] = o;
        if (col == 0) {
          s_m[grp] = m;
          s_l[grp] = l;
        }
        __syncthreads();
        if (grp != 0) return;
      }
#pragma unroll
      for (int i = 1; i < G; ++i) m = fmaxf(m, s_m[i]);
      l = o = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) add(s_m[i], s_l[i], s_o[i][col]);
    }
    const int row = (int)(p * a.group_inv >> 16);
    const int64_t hq = (int64_t)(job.z + row) * a.h_q + (int64_t)(job.w >> 8) * a.group + (p - row * a.group);
    const float r = l == 0.f ? 0.f : o / l;
    const float lse = k8_lse(m, l);
    if (live) {
      if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[hq * D + d] = __float2bfloat16_rn(r);
      else static_cast<float*>(a.out)[hq * D + d] = r;
      if (d == 0 && a.lse != nullptr) a.lse[hq] = lse;
      return;
    }
  }
}

}  // namespace qsa
