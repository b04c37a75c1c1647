// kv4.cuh -- the 4-bit KV cache: its format, the kernel that quantises K and
// V rows as they are written, and the kernel that reads rows back.
//
// Format.  A physical KV slot holds, per KV head, D e2m1 values (two to a
// byte, the even dimension in the low nibble) and one e4m3 scale per block
// of 16 of them:
//     codes  [n_slots][h_kv][D/2]     scales [n_slots][h_kv][D/16]
//     value = e2m1(code) * e4m3(scale) * g
// g is one scale for the whole tensor, a power of two given by the caller.
// 4.5 bits a value.  e2m1 has a 2-bit and e4m3 a 4-bit significand, so a
// value has at most 6 significant bits: the product is exact in FP16 without
// g (largest 6 * 448 = 2688, smallest 2^-10) and exact in BF16 with it.
// Reading the cache therefore rounds nothing; only writing does.
//
// Writing a block x[0..15]:
//     scale = e4m3(max|x| / g / 6)     (nearest even; max|x| / g is exact)
//     code  = e2m1(x / g / scale)      (nearest even, saturating at 6)
// x / g is a BF16 number y (8 significant bits), and a rounding border of
// either step times 6 or the scale a number z of at most 7: if y is not z,
// they differ by at least 2^-8 relative.  So no division is needed: y times
// a reciprocal (off by 2^-22 at most) is rounded to FP16 first, which puts a
// quotient on a border exactly there and moves no other across one.  (With
// 17 divisions a block the kernel took 37 us where it took 31.)  A block
// whose scale rounds to zero holds zeros; a block with an infinity or a NaN
// gets the NaN scale and reads back as NaN, so that a broken row shows
// instead of being clipped.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "kv_util.cuh"

namespace qsa {

constexpr int kKvBlock = 16;     // values per scale

// Eight FP32 values -> their codes, the first in the low nibble.
__device__ __forceinline__ uint32_t kv4_pack(const float2 (&q)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
  return r;
}

// One block of 16 BF16 values -> its codes (8 bytes) and scale byte.
__device__ __forceinline__ uint2 kv4_quantise(const U8& x, float inv_g, uint8_t& scale) {
  // max |x|; NaN wins over infinities, both over numbers
  __nv_bfloat162 m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t p = x.w[2 * i] & 0x7fff7fffu, q = x.w[2 * i + 1] & 0x7fff7fffu;
    m[i] = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&p), *reinterpret_cast<const __nv_bfloat162*>(&q));
  }
  m[0] = __hmax2_nan(__hmax2_nan(m[0], m[1]), __hmax2_nan(m[2], m[3]));
  const float top = __bfloat162float(__hmax_nan(__low2bfloat16(m[0]), __high2bfloat16(m[0])));
  uint2 c = make_uint2(0u, 0u);
  if (!(top < __int_as_float(0x7f800000))) {
    scale = 0x7f;
    return c;
  }
  // quotients by way of FP16, see the top of the file
  scale = (uint8_t)__nv_cvt_halfraw_to_fp8(__float2half_rn(top * inv_g * (1.0f / 6.0f)), __NV_SATFINITE, __NV_E4M3);
  const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)scale, __NV_E4M3)));
  if (s == 0.f) return c;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r *= inv_g;  // a power of two: exact
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_float2(x.w[4 * h + i]);
      q[i] = __half22float2(__floats2half2_rn(f.x * r, f.y * r));
    }
    (h == 0 ? c.x : c.y) = kv4_pack(q);
  }
  return c;
}

// The eight codes of a word -> four FP16 pairs, byte by byte (exact).
__device__ __forceinline__ void kv4_word(uint32_t w, __half2 (&h)[4]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const __half2*>(&r[i]);
}
// Two scale bytes -> two FP16 scales (exact).
__device__ __forceinline__ __half2 kv4_scales(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}

// One block's codes and scale -> 16 BF16 values.
__device__ __forceinline__ U8 kv4_read(uint2 codes, uint32_t scale, float g) {
  const __half2 s = kv4_scales(scale | (scale << 8));
  const uint32_t c[2] = {codes.x, codes.y};
  __half2 h[2][4];
  kv4_word(c[0], h[0]);
  kv4_word(c[1], h[1]);
  U8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(__hmul2(h[i >> 2][i & 3], s));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * g, f.y * g);
    r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return r;
}

struct KvWriteArgs {
  const uint16_t* k_new;         // [n_tok] rows of h_kv * D BF16, ld_k apart
  const uint16_t* v_new;
  int64_t ld_k, ld_v;
  int32_t n_tok, h_kv;
  int32_t blocks;                // blocks of a token: h_kv * D / 16
  const int32_t* req_tok_start;  // [n_req+1]
  const int32_t* req_first_pos;  // [n_req]
  int32_t n_req;
  const int32_t* page_table;
  int64_t ld_pt;
  int32_t page_size;
  int64_t n_slots;
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  float k_inv, v_inv;            // 1 / g
};

// K and V rows quantised into their slots.  One thread per block of 16 of K
// and the same block of V.  Per block 64 B read and 18 B written.  60,374 rows
// of 2 x 256: 26.4 us, 6.0 TB/s, 0.89 of the copy rate (two and four blocks a
// thread took 32 and 37 us where one took 31); a decode step
// is a chain of dependent loads (request, position, page), the data beside the
// last two of them.
__global__ void __launch_bounds__(kKvThreads)
append_kv_fp4_kernel(KvWriteArgs a) {
  const uint32_t u0 = blockIdx.x * kKvThreads + (threadIdx.x & ~31);
  const uint32_t total = (uint32_t)a.n_tok * (uint32_t)a.blocks;  // 32 bits: checked by the host
  if (u0 >= total) return;  // the whole warp
  pdl_wait_primary();
  const uint32_t u = u0 + (threadIdx.x & 31);
  const bool ok = u < total;
  const int t = ok ? (int)(u / (uint32_t)a.blocks) : a.n_tok - 1;
  const int b = ok ? (int)(u - (uint32_t)t * (uint32_t)a.blocks) : 0;
  int r = warp_row_request(a.req_tok_start, a.n_req, (int)(u0 / (uint32_t)a.blocks));  // of the warp's first token
  if (!ok || r < 0) return;  // r < 0: behind the last request, as the rest of the warp
  while (r < a.n_req && t >= ld_in(a.req_tok_start + r + 1)) ++r;  // a warp may span tokens
  if (r >= a.n_req) return;
  // not before: rows behind the last request may lie past the end of the buffers
  const U8 kx = ld_stream_32(a.k_new + (int64_t)t * a.ld_k + b * kKvBlock);
  const U8 vx = ld_stream_32(a.v_new + (int64_t)t * a.ld_v + b * kKvBlock);
  const int64_t pos = (int64_t)ld_in(a.req_first_pos + r) + (t - ld_in(a.req_tok_start + r));
  const int pi = pos < 0 || pos > INT32_MAX ? INT32_MAX : (int)pos / a.page_size;
  if (pi >= a.ld_pt) {
    raise_fault(kFaultIndex);
    return;
  }
  const int64_t page = ld_in(a.page_table + (int64_t)r * a.ld_pt + pi);
  const int64_t slot = page * a.page_size + ((int)pos - pi * a.page_size);
  if (page < 0 || slot >= a.n_slots) {
    raise_fault(kFaultIndex);
    return;
  }
  const int64_t at = slot * a.blocks + b;
  uint8_t sk, sv;
  const uint2 ck = kv4_quantise(kx, a.k_inv, sk);
  const uint2 cv = kv4_quantise(vx, a.v_inv, sv);
  reinterpret_cast<uint2*>(a.k_codes)[at] = ck;
  reinterpret_cast<uint2*>(a.v_codes)[at] = cv;
  a.k_scales[at] = sk;
  a.v_scales[at] = sv;
}

struct KvReadArgs {
  const uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  int64_t n_slots;
  int32_t blocks;        // blocks of a slot
  const int32_t* slots;  // [n]
  int64_t n;
  float k_g, v_g;
  uint16_t *k_out, *v_out;  // [n][h_kv][D] BF16
};

// Rows read back at slots: one thread per block of 16 of K and of V.  Per
// block 18 B read and 64 B written, HBM-bound: 131,072 rows of 512 values take
// 52.5 us, 6.6 TB/s, 0.97 of a plain copy's rate; 12,306 selected rows 5.7 us.
__global__ void __launch_bounds__(kKvThreads)
gather_kv_fp4_kernel(KvReadArgs a) {
  const uint32_t u = blockIdx.x * kKvThreads + threadIdx.x;
  if (u >= (uint32_t)a.n * (uint32_t)a.blocks) return;  // 32 bits: checked by the host
  pdl_wait_primary();
  const uint32_t i = u / (uint32_t)a.blocks;
  const int b = (int)(u - i * (uint32_t)a.blocks);
  const int32_t s = ld_in(a.slots + i);
  U8 k{}, v{};
  if (s >= 0 && s < a.n_slots) {
    const int64_t at = (int64_t)s * a.blocks + b;
    const uint2 ck = ld_in(reinterpret_cast<const uint2*>(a.k_codes) + at);
    const uint2 cv = ld_in(reinterpret_cast<const uint2*>(a.v_codes) + at);
    const uint32_t sk = ld_in(a.k_scales + at), sv = ld_in(a.v_scales + at);
    k = kv4_read(ck, sk, a.k_g);
    v = kv4_read(cv, sv, a.v_g);
  } else if (s >= 0 && b == 0) {
    raise_fault(kFaultIndex);
  }
  st_32(a.k_out + (int64_t)u * kKvBlock, k);
  st_32(a.v_out + (int64_t)u * kKvBlock, v);
}

}  // namespace qsa
