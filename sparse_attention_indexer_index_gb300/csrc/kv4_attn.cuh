// kv4_attn.cuh -- softmax attention of rows over the 4-bit K/V cache: over
// the slots of a selection (sparse_attn_fp4) or a window (window_attn_fp4).
// The formulas, the entries, the cluster per (row, KV head) and its join are
// kv_attn.cuh's.
//
// Bound.  Per entry and KV head 9/8 D bytes are read and 2 D values unpacked
// (a conversion and a product with the scale per two of them) for 4 G D
// flops: the instructions, not HBM, set the time.
//
// Design (GB300).
//  - A warp takes 32 entries a step, with no barrier before the row's end:
//    four independent chains of products form S, one reduction serves 32
//    weights a head, and O += P V follows in two steps of 16.
//  - A team of two warps, each with half of O's columns, fits 16 warps on an
//    SM instead of 8 but pays a barrier and spills: 24.6 against 22.8 us for
//    32 rows of 2,051 entries (G = 8, D = 256).
//  - A code times its e4m3 scale is exact in FP16, so K and V enter the MMA
//    (mma.sync m16n8k16, FP32 accumulation) without rounding.  q is BF16: it
//    is brought into FP16's range by a power of two per head (exact; a
//    component below 2^-14 of the head's largest loses at most 2^-25 of that
//    largest), which the logit's factor takes back.
//  - The 16 rows of an MMA tile hold 8 heads twice: in S the second half is
//    zero (unless a KV head has more than 8), in P V rows 0-7 hold the high
//    parts of the weights and rows 8-15 the remainders (22 significant bits),
//    and the two halves of the accumulator add up.
//  - K's dimensions and V's columns are permuted so that a lane reads 16-byte
//    pieces of K rows and 16- or 8-byte pieces of V rows; V's entries come in
//    pairs (the K index of the MMA), which are interleaved nibble by nibble
//    before the conversion.
//
// Measured (one call after the other; 16 query heads): 32 rows of 2,051 entries, 2 KV heads
// of D = 256: 16.4 us, 2.4 TB/s; 192 rows, 1 KV head of D = 128: 33.2 us, 1.8
// TB/s; 32 windows of 4,100 entries, 2 KV heads of D = 256: 27.5 us, 2.8 TB/s;
// one row 8.7 us.  From 32 rows of 2,051, 4,102, 8,204 and 16,408 entries (15.6,
// 25.4, 43.9, 80.1 us in a graph) the middle of a row goes at 4.2 TB/s, 0.62 of
// the copy rate, and the chain from the launch to the first keys and the join
// take 7 us.  There (16,408 entries) the ALU is 42 %, the tensor pipe 40 % and
// the issue slots 40 % busy, on 8 warps an SM (250 registers a thread): too few
// to cover the waits between dependent instructions.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "kv4.cuh"
#include "kv_attn.cuh"

namespace qsa {

constexpr int kK4Warps = 4;
constexpr int kK4Threads = 32 * kK4Warps;
constexpr int kK4Step = 32;     // entries per warp step
constexpr int kK4Stages = 2;     // a step takes longer than the copies of the next
// Weights are held as 2^kK4Bias p, clear of FP16's subnormals; with the lazy
// maximum a weight is at most 2^(kK4Bias + kKaGrow) = 2^15.
constexpr int kK4Bias = 10;

template <int D>
struct K4Shape {
  static constexpr int kRow = D / 2, kSc = D / 16;         // bytes of a row's codes and scales
  static constexpr uint32_t kV = kK4Step * kRow, kKs = 2 * kK4Step * kRow, kVs = kKs + kK4Step * kSc;
  static constexpr int kStage = kK4Step * (kRow + kSc) * 2;
};
template <int D, int NT>
constexpr size_t k4_smem_bytes() {
  const size_t ring = (size_t)kK4Warps * kK4Stages * K4Shape<D>::kStage;
  const size_t o = (size_t)kK4Warps * NT * 8 * KaOut<D, D / 8>::kRow * 4;
  return ring > o ? ring : o;
}

template <int D, int NT, bool kWindow>
__global__ void __launch_bounds__(kK4Threads, 2)
kv4_attn_kernel(const __grid_constant__ KvAttnArgs a) {
  using Sh = K4Shape<D>;
  using Out = KaOut<D, D / 8>;
  constexpr int KS = D / 16, VN = D / 8;
  extern __shared__ __align__(128) unsigned char k4_smem[];
  __shared__ float s_m[kK4Warps][NT * 8], s_l[kK4Warps][NT * 8];
  __shared__ float c_m[NT * 8], c_l[NT * 8];      // this CTA's
  __shared__ KaJoin<D, NT> join;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const int parts = a.cluster * a.n_group;
  const int t = blockIdx.x / parts, part = blockIdx.x - t * parts;
  const int g = blockIdx.y;
  const float ninf = -__int_as_float(0x7f800000);

  pdl_wait_primary();
  KaRow<kWindow> row;
  if (!ka_row<kWindow>(a, t, row)) return;  // behind the last request (the same for the whole cluster)
  ka_cluster_arrive(a.cluster);
  const int steps = (row.n + kK4Step - 1) / kK4Step;
  const int first = part * kK4Warps + warp, stride = parts * kK4Warps;

  // ---- q as A fragments (rows gq: heads; rows gq + 8: zero) -----------------------
  uint32_t qa[NT][KS][2];
  float mult[NT];  // logit (base 2) = mult * accumulator
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int h = nt * 8 + gq;
    const uint16_t* src = a.q + (int64_t)t * a.ld_q + ((int64_t)g * a.group + h) * D;
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      // the lane's K pieces hold 32 dimensions each, four of q's
      const int piece = (tq + 4 * (i >> 2)) * 4 + (i & 3);
      const uint4 u = h < a.group ? ld_in(reinterpret_cast<const uint4*>(src) + piece) : make_uint4(0u, 0u, 0u, 0u);
      qa[nt][2 * i][0] = u.x;
      qa[nt][2 * i][1] = u.y;
      qa[nt][2 * i + 1][0] = u.z;
      qa[nt][2 * i + 1][1] = u.w;
      mx = __vmaxu2(__vmaxu2(mx, u.x & 0x7fff7fffu), u.y & 0x7fff7fffu);
      mx = __vmaxu2(__vmaxu2(mx, u.z & 0x7fff7fffu), u.w & 0x7fff7fffu);
    }
    uint32_t top = max(mx & 0xffffu, mx >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = min(max((int)(top >> 7), 1), 253) - 127;  // exponent of the head's largest component
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
    mult[nt] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float2 f = bf16x2_to_float2(qa[nt][s][w]);
        qa[nt][s][w] = ka_h2(__floats2half2_rn(f.x * down, f.y * down));
      }
  }

  // ---- the warp's ring: K codes, V codes, K scales, V scales of 32 entries -----
  const uint32_t ring = smem_u32(k4_smem) + (uint32_t)warp * (kK4Stages * Sh::kStage);
  // rows in 16-byte pieces, permuted so that the reads below meet no bank twice
  auto k_off = [](int r, int c) -> uint32_t {
    if constexpr (D == 128) return (uint32_t)(r * 64 + c * 16);
    else return (uint32_t)(r * 128 + ((c ^ ((r & 1) << 2)) << 4));
  };
  auto v_off = [](int r, int c) -> uint32_t {
    if constexpr (D == 256) return (uint32_t)(r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4));
    else {  // rows 0, 2, 4, 6 (one per lane of a quad) over both halves of 128 bytes
      const int pr = (r & 28) | ((r & 1) << 1) | ((r >> 1) & 1);
      return (uint32_t)(pr * 64 + ((c ^ (((r >> 2) & 1) << 1)) << 4));
    }
  };
  const uint8_t* gk = a.k + (int64_t)g * Sh::kRow;
  const uint8_t* gv = a.v + (int64_t)g * Sh::kRow;
  const uint8_t* gks = a.ks + (int64_t)g * Sh::kSc;
  const uint8_t* gvs = a.vs + (int64_t)g * Sh::kSc;
  const int64_t pitch = (int64_t)a.h_kv * Sh::kRow, pitch_s = (int64_t)a.h_kv * Sh::kSc;

  // copies of 32 entries, a slot a lane
  auto issue = [&](int stage, int32_t slot) {
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    constexpr int PP = Sh::kRow / 16;            // 16-byte pieces of a row: 8 or 4
#pragma unroll
    for (int u = 0; u < PP; ++u) {
      const int r = u * (32 / PP) + lane / PP, c = lane % PP;
      const int32_t s = __shfl_sync(0xffffffffu, slot, r);
      const int64_t off = (int64_t)max(s, 0) * pitch + c * 16;
      ka_cp16(base + k_off(r, c), gk + off, s >= 0);
      ka_cp16(base + Sh::kV + v_off(r, c), gv + off, s >= 0);
    }
    const int64_t off = (int64_t)max(slot, 0) * pitch_s;
    if constexpr (Sh::kSc == 16) {
      ka_cp16(base + Sh::kKs + lane * 16, gks + off, slot >= 0);
      ka_cp16(base + Sh::kVs + lane * 16, gvs + off, slot >= 0);
    } else {
      ka_cp8(base + Sh::kKs + lane * 8, gks + off, slot >= 0);
      ka_cp8(base + Sh::kVs + lane * 8, gvs + off, slot >= 0);
    }
  };
  // a slot is fetched a step before its copies; mask[i]: valid entries i steps ahead
  auto entry = [&](int step) -> int { return step < steps ? step * kK4Step + lane : INT32_MAX; };
  KaFetch pre[kK4Stages];
  uint32_t mask[kK4Stages];
#pragma unroll
  for (int i = 0; i < kK4Stages; ++i) pre[i] = ka_fetch<kWindow>(a, row, entry(first + i * stride));
#pragma unroll
  for (int i = 0; i < kK4Stages - 1; ++i) {
    const int32_t slot = ka_slot<kWindow>(a, row, entry(first + i * stride), pre[i]);
    if (first + i * stride < steps) issue(i, slot);
    asm volatile("cp.async.commit_group;" ::: "memory");
    mask[i] = __ballot_sync(0xffffffffu, slot >= 0);
  }
  KaFetch next = pre[kK4Stages - 1];

  float o[NT][VN][4];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = ninf;
    l[nt] = 0.f;
#pragma unroll
    for (int i = 0; i < VN; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
  }

  // ---- steps -----------------------------------------------------------------------
  int stage = 0;
  for (int step = first; step < steps; step += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kK4Stages - 2) : "memory");
    __syncwarp();
    const uint32_t base = ring + (uint32_t)stage * Sh::kStage;
    const uint32_t valid = mask[0];
    {  // refill the stage that the last step emptied
      const int ahead = step + (kK4Stages - 1) * stride;
      const int32_t slot = ka_slot<kWindow>(a, row, entry(ahead), next);
      if (ahead < steps) issue(stage == 0 ? kK4Stages - 1 : stage - 1, slot);
      asm volatile("cp.async.commit_group;" ::: "memory");
      mask[kK4Stages - 1] = __ballot_sync(0xffffffffu, slot >= 0);
#pragma unroll
      for (int i = 0; i + 1 < kK4Stages; ++i) mask[i] = mask[i + 1];
      next = ka_fetch<kWindow>(a, row, entry(ahead + stride));
    }

    // J / 4 of a step: a last step of up to 16 entries takes half the work
    // (a selection of 512 blocks and 3 pending tokens ends in one of 3)
    auto attend = [&](auto j_tag) {
      constexpr int J = decltype(j_tag)::value;
      // S = q K^T: J n-tiles of 8 entries (lane: entry gq of each); rows gq:
      // heads 0-7, rows gq + 8: heads 8-15 or zero
      float s[J][4];
#pragma unroll
      for (int j = 0; j < J; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 128; ++i) {
        uint4 w4[J];
        __half2 sc[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          w4[j] = ka_lds16(base + k_off(j * 8 + gq, tq + 4 * i));
          sc[j] = kv4_scales(ka_lds_u16(base + Sh::kKs + (j * 8 + gq) * Sh::kSc + 2 * (tq + 4 * i)));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const uint32_t w = k == 0 ? w4[j].x : k == 1 ? w4[j].y : k == 2 ? w4[j].z : w4[j].w;
            const __half2 sk = k < 2 ? __low2half2(sc[j]) : __high2half2(sc[j]);
            __half2 h[4];
            kv4_word(w, h);
            uint32_t b[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) b[y] = ka_h2(__hmul2(h[y], sk));
            const int n = i * 8 + 2 * k;
            ka_mma<true>(s[j], qa[0][n][0], NT > 1 ? qa[NT - 1][n][0] : 0u, qa[0][n][1], NT > 1 ? qa[NT - 1][n][1] : 0u,
                         b[0], b[1]);
            ka_mma<true>(s[j], qa[0][n + 1][0], NT > 1 ? qa[NT - 1][n + 1][0] : 0u, qa[0][n + 1][1],
                         NT > 1 ? qa[NT - 1][n + 1][1] : 0u, b[2], b[3]);
          }
      }

      // running maximum and sum; the weights as A fragments (lane: head gq,
      // entries 2 tq, 2 tq + 1 of each n-tile)
      uint32_t pa[NT][J / 2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float x[J][2];
        float mx = ninf;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x[j][e] = (valid >> (8 * j + 2 * tq + e)) & 1u ? s[j][2 * nt + e] * mult[nt] : ninf;
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
        const float ms = m[nt] == ninf ? 0.f : m[nt] - (float)kK4Bias;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float p0 = ka_ex2(x[j][0] - ms), p1 = ka_ex2(x[j][1] - ms);
          l[nt] += p0 + p1;
          ka_split<true>(p0, p1, pa[nt][j >> 1][2 * (j & 1)], pa[nt][j >> 1][2 * (j & 1) + 1]);
        }
      }

      // O += P V: lane: entries 2tq, 2tq+1 (b0) and 2tq+8, 2tq+9 (b1) of 16;
      // columns gq * VN + i of n-tile i
#pragma unroll
      for (int ks = 0; ks < J / 2; ++ks) {
        constexpr int kW = D / 64;  // 4-byte words of the lane's piece: 4 or 2
        uint32_t w[4][kW], sc[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = ks * 16 + 2 * tq + (e & 1) + (e >> 1) * 8;
          if constexpr (D == 256) {
            const uint4 y = ka_lds16(base + Sh::kV + v_off(r, gq));
            w[e][0] = y.x; w[e][1] = y.y; w[e][2] = y.z; w[e][3] = y.w;
            sc[e] = ka_lds_u16(base + Sh::kVs + r * Sh::kSc + 2 * gq);
          } else {
            const uint2 y = ka_lds8(base + Sh::kV + v_off(r, gq >> 1) + (gq & 1) * 8);
            w[e][0] = y.x; w[e][1] = y.y;
            sc[e] = ka_lds_u8(base + Sh::kVs + r * Sh::kSc + gq);
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
              ka_mma<true>(o[nt][8 * k + 2 * y], pa[nt][ks][0], pa[nt][ks][1], pa[nt][ks][2], pa[nt][ks][3], b0, b1);
              ka_mma<true>(o[nt][8 * k + 2 * y + 1], pa[nt][ks][0], pa[nt][ks][1], pa[nt][ks][2], pa[nt][ks][3], b2, b3);
            }
          }
        }
      }
    };
    if ((valid >> 16) != 0) attend(std::integral_constant<int, 4>());
    else attend(std::integral_constant<int, 2>());
    stage = stage + 1 == kK4Stages ? 0 : stage + 1;
  }

  // ---- the CTA's result ----------------------------------------------------------------
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
  float* so = reinterpret_cast<float*>(k4_smem);  // [warp][NT * 8][Out::kRow]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float cm = ninf;
#pragma unroll
    for (int w = 0; w < kK4Warps; ++w) cm = fmaxf(cm, s_m[w][nt * 8 + gq]);
    const float f = cm == ninf ? 0.f : ka_ex2(m[nt] - cm);
    if (warp == 0 && tq == 0) {
      float cl = 0.f;
#pragma unroll
      for (int w = 0; w < kK4Warps; ++w)
        cl += s_l[w][nt * 8 + gq] * (cm == ninf ? 1.f : ka_ex2(s_m[w][nt * 8 + gq] - cm));  // all 0, or a NaN
      c_m[nt * 8 + gq] = cm;
      c_l[nt * 8 + gq] = cl;
    }
    float* dst = so + (size_t)(warp * NT * 8 + nt * 8 + gq) * Out::kRow;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < VN; i += 4) {
        float4 y;
        y.x = (o[nt][i][e] + o[nt][i][2 + e]) * f;
        y.y = (o[nt][i + 1][e] + o[nt][i + 1][2 + e]) * f;
        y.z = (o[nt][i + 2][e] + o[nt][i + 2][2 + e]) * f;
        y.w = (o[nt][i + 3][e] + o[nt][i + 3][2 + e]) * f;
        *reinterpret_cast<float4*>(dst + Out::col((2 * tq + e) * VN + i)) = y;
      }
  }
  __syncthreads();
  // the warps' sums into warp 0's rows
  for (int idx = tid; idx < a.group * (D / 4); idx += kK4Threads) {
    const int h = idx / (D / 4), d = (idx % (D / 4)) * 4;
    float* p0 = so + (size_t)h * Out::kRow + Out::col(d);
    float4 y = *reinterpret_cast<float4*>(p0);
#pragma unroll
    for (int w = 1; w < kK4Warps; ++w) {
      const float4 z = *reinterpret_cast<const float4*>(p0 + (size_t)w * NT * 8 * Out::kRow);
      y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
    }
    *reinterpret_cast<float4*>(p0) = y;
  }
  ka_cluster_result<D, NT, kK4Threads>(a, so, c_m, c_l, join, t, g, part % a.cluster, part / a.cluster, (float)kK4Bias);
}

}  // namespace qsa
