// kv8.cuh -- the 8-bit KV cache: its format, the kernel that quantises K and V
// rows as they are written, and the kernel that reads rows back.
//
// Format.  A physical KV slot holds, per KV head, D e4m3 codes; B consecutive
// slots (a block: a power of two that divides the page) share one scale per
// head, a power of two in a byte:
//     codes  [n_slots][h_kv][D]     scales [n_slots / B][h_kv]
//     value = e4m3(code) * 2^(scale - 127)
// A code has 4 significant bits whatever the scale, so the scale only places
// the codes' range (2^-9 to 448): a power of two loses nothing against
// max|x| / 448 but up to one binade at the lower end, makes every value exact
// in BF16, and lets the attention put it into the logits (K) and the weights
// (V) as an exponent, once an entry and not once a value.
//
// Writing.  A block's scale is the smallest 2^e with max|x| <= 448 2^e over its
// finite values, e between -64 and 63; code = e4m3(x / 2^e) (nearest even,
// saturating).  A block that holds earlier tokens keeps at least the scale it
// has; where a new token makes it grow by 2^k, the earlier codes are rounded
// to the new scale: code / 2^k, exact but below 2^-6.  An infinity or a NaN
// takes no part in the maximum and becomes a NaN, alone.
//
// Bound.  Writing reads 2 B a value and writes 1, reading back the reverse: HBM
// for prompts, latency for a step.  60,374 tokens (2 KV heads, D = 256) take
// 64.7 us written and read back, 0.94 of the copy rate (6,784 GB/s); a step of 32
// tokens 4.2 us in a graph, two launches.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kv_util.cuh"

namespace qsa {

constexpr int kKv8Threads = 256;
constexpr int kKv8MinExp = -64, kKv8MaxExp = 63;

// The scale byte of a block whose largest finite |x| has BF16 bits `top`:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int kv8_scale_byte(uint32_t top) {
  const int e = (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, kKv8MinExp), kKv8MaxExp) + 127;
}
__device__ __forceinline__ float kv8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ uint32_t kv8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The low two codes of a word -> an FP16 pair (exact).
__device__ __forceinline__ __half2 kv8_half2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}

struct Kv8WriteArgs {
  const uint16_t *k_new, *v_new;  // [n_tok] rows of h_kv * D BF16, ld_k / ld_v apart
  int64_t ld_k, ld_v;
  int32_t n_tok, h_kv, d;
  int32_t chunk;                 // tokens whose units a CTA serves
  const int32_t* req_tok_start;  // [n_req+1]
  const int32_t* req_first_pos;  // [n_req]
  int32_t n_req;
  const int32_t* page_table;
  int64_t ld_pt;
  int32_t page_size, block_shift, per_shift;  // log2 of the pieces of 8 values to a row
  int64_t n_slots;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
};

// K and V rows quantised into their slots.  A unit is what the call writes of
// one block, for one head of K or V; it belongs to the CTA that has its first
// token among its `chunk` tokens.  The unit's values stay in registers between
// the maximum and the codes (kPieces * 8 of them a thread, a whole block at
// most), so they are read once.  Issue slots were the limit of the large calls
// (74 % busy, 143 instructions for 8 values): with addresses that only step on
// and the scaling as one BF16 pair product it is 86 (39 -> 32 us for 60,374
// tokens).
template <int kPieces>
__global__ void __launch_bounds__(kKv8Threads, kPieces <= 8 ? 4 : 2)
append_kv_fp8_kernel(const __grid_constant__ Kv8WriteArgs a) {
  __shared__ uint32_t s_top[2][kKv8Threads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int B = 1 << a.block_shift, per = a.d >> 3;  // pieces of 8 values to a row
  pdl_wait_primary();
  int t = (int)(blockIdx.x * (uint32_t)a.chunk);
  const int stop = min(t + a.chunk, a.n_tok);
  int r = warp_row_request(a.req_tok_start, a.n_req, t);
  if (r < 0) return;  // behind the last request
  const uint16_t* src = is_v ? a.v_new : a.k_new;
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  uint8_t* scales = is_v ? a.v_scales : a.k_scales;
  // the thread's first row and column of a unit; the next piece is `step` rows on
  const int row0 = tid >> a.per_shift, col = (tid & (per - 1)) * 8, step = kKv8Threads >> a.per_shift;
  int turn = 0;
  while (t < stop && r < a.n_req) {
    const int s0 = ld_in(a.req_tok_start + r), s1 = min(ld_in(a.req_tok_start + r + 1), a.n_tok);
    const int first = ld_in(a.req_first_pos + r);
    if (t >= s1) {
      ++r;
      continue;
    }
    const int64_t pos = (int64_t)first + (t - s0);
    if (pos < 0 || pos > INT32_MAX) {
      if (tid == 0) raise_fault(kFaultIndex);
      t = pos < 0 ? (int)min((int64_t)s1, t - pos) : s1;  // on to position 0, if it comes
      continue;
    }
    const int t0 = t, in = (int)pos & (B - 1);  // the token's place in its block
    t = min(t0 + B - in, s1);                   // (at most 2^31: t0 < n_tok, checked by the host)
    if (t0 != s0 && in != 0) continue;          // the block is another CTA's, or done
    const int lo = (int)pos - in;               // the block's first position
    const int pi = lo / a.page_size;
    const int64_t page = pi < a.ld_pt ? ld_in(a.page_table + (int64_t)r * a.ld_pt + pi) : -1;
    // the unit's values, rows t0 .. t - 1, on the way beside the page and the block's scale
    const int rows = t - t0;
    uint4 x[kPieces];
    const uint16_t* from = src + (int64_t)(t0 + row0) * ld + (int64_t)h * a.d + col;
#pragma unroll
    for (int i = 0; i < kPieces; ++i, from += (int64_t)step * ld) {
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (row0 + i * step < rows) x[i] = ld_stream_16(from);
    }
    const int64_t slot = page * a.page_size + (lo - pi * a.page_size);
    if (page < 0 || slot + B > a.n_slots) {
      if (tid == 0) raise_fault(kFaultIndex);
      continue;
    }
    const int64_t at = (slot >> a.block_shift) * a.h_kv + h;
    const int old = in != 0 ? (int)ld_in(scales + at) : 0;  // the scale of the block's earlier tokens
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[j])));  // not a NaN
    }
    auto reduce = [&](uint32_t v) -> uint32_t {
      v = __reduce_max_sync(0xffffffffu, v);
      if (lane == 0) s_top[turn][warp] = v;
      __syncthreads();
      uint32_t y = s_top[turn][0];
#pragma unroll
      for (int w = 1; w < kKv8Threads / 32; ++w) y = max(y, s_top[turn][w]);
      turn ^= 1;  // the next one's words: this one's are read before the next barrier
      return y;
    };
    const uint32_t mb = *reinterpret_cast<const uint32_t*>(&m);
    uint32_t top = reduce(max(mb & 0xffffu, mb >> 16));
    const bool inf = top >= 0x7f80u;
    if (inf) {  // once more without the infinities, which become NaN
      uint32_t f = 0;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t l = w[j] & 0x7fffu, u = (w[j] >> 16) & 0x7fffu;
          f = max(f, max(l < 0x7f80u ? l : 0u, u < 0x7f80u ? u : 0u));
          w[j] |= (l == 0x7f80u ? 0x7fffu : 0u) | (u == 0x7f80u ? 0x7fff0000u : 0u);
        }
        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      top = reduce(f);
    }
    const int byte = max(kv8_scale_byte(top), old);
    // x / 2^e: exact in BF16, but for what is 0 in e4m3 anyway
    const __nv_bfloat162 down = __float2bfloat162_rn(kv8_pow2(127 - byte));
    uint8_t* to = codes + ((slot + in + row0) * a.h_kv + h) * a.d + col;
    const int64_t to_step = (int64_t)step * a.h_kv * a.d;
#pragma unroll
    for (int i = 0; i < kPieces; ++i, to += to_step) {
      if (row0 + i * step >= rows) break;
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), down);
        const float2 f = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(&y));
        c[j] = kv8_pack2(f.x, f.y);
      }
      *reinterpret_cast<uint2*>(to) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    }
    if (in != 0 && byte > old) {  // the earlier tokens' codes to the new scale
      const float f = kv8_pow2(max(old - byte, -126));
      for (int p = tid; p < in * per; p += kKv8Threads) {
        const int row = p >> a.per_shift;
        uint2* at8 = reinterpret_cast<uint2*>(codes + ((slot + row) * a.h_kv + h) * a.d + (p & (per - 1)) * 8);
        const uint2 v = ld_in(at8);
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 g = __half22float2(kv8_half2(((j < 2 ? v.x : v.y) >> (16 * (j & 1))) & 0xffffu));
          c[j] = kv8_pack2(g.x * f, g.y * f);
        }
        *at8 = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
      }
    }
    if (tid == 0) scales[at] = (uint8_t)byte;
  }
}

struct Kv8ReadArgs {
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t n_slots;
  int32_t h_kv, per;     // pieces of 16 values to a head's row
  int32_t block_shift;
  const int32_t* slots;  // [n]
  int64_t n;
  uint16_t *k_out, *v_out;  // [n][h_kv][D] BF16
};

// 16 codes and their scale -> 16 BF16 values (exact).
__device__ __forceinline__ U8 kv8_read(const uint4& c, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  U8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(kv8_half2((w[i >> 1] >> (16 * (i & 1))) & 0xffffu));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return r;
}

// Rows read back at slots: one thread per 16 values of K and of V.  Per value
// 1 B read and 2 B written: HBM-bound.
__global__ void __launch_bounds__(kKvThreads)
gather_kv_fp8_kernel(const __grid_constant__ Kv8ReadArgs a) {
  const uint32_t u = blockIdx.x * kKvThreads + threadIdx.x;
  const uint32_t row = (uint32_t)(a.h_kv * a.per);  // pieces of a slot
  if (u >= (uint32_t)a.n * row) return;             // 32 bits: checked by the host
  pdl_wait_primary();
  const uint32_t i = u / row, b = u - i * row;
  const int32_t s = ld_in(a.slots + i);
  U8 k{}, v{};
  if (s >= 0 && s < a.n_slots) {
    const int64_t at = (int64_t)s * row + b;
    const int64_t sc = (int64_t)(s >> a.block_shift) * a.h_kv + b / (uint32_t)a.per;
    const uint4 ck = ld_in(reinterpret_cast<const uint4*>(a.k_codes) + at);
    const uint4 cv = ld_in(reinterpret_cast<const uint4*>(a.v_codes) + at);
    const uint32_t sk = ld_in(a.k_scales + sc), sv = ld_in(a.v_scales + sc);
    k = kv8_read(ck, sk);
    v = kv8_read(cv, sv);
  } else if (s >= 0 && b == 0) {
    raise_fault(kFaultIndex);
  }
  st_32(a.k_out + (int64_t)u * 16, k);
  st_32(a.v_out + (int64_t)u * 16, v);
}

}  // namespace qsa
