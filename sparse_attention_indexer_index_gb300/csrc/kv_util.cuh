// kv_util.cuh -- what the kernels on the K/V caches share: 32-byte accesses
// and the request of a row.
#pragma once
#include "common.cuh"

namespace qsa {

constexpr int kKvThreads = 128;  // threads per CTA of the caches' write and read kernels

// 32 bytes in one instruction (32-byte aligned), read once.  As ld_in, it stays
// where it is written.
struct U8 {
  uint32_t w[8];
};
__device__ __forceinline__ U8 ld_stream_32(const void* p) {
  U8 r;
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void st_32(void* p, const U8& r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
               "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}

// Request of row t by a whole warp: the r with start[r] <= t < start[r+1],
// or -1 when t lies behind start[n_req] (or before start[0]).  32 samples a
// round, so one round trip to memory for up to 32 requests and two for up to
// 1024 (a binary search takes five and ten).
__device__ __forceinline__ int warp_row_request(const int32_t* start, int n_req, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_req + 1;  // candidates lo .. lo + n - 1 of the last start <= t
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && ld_in(start + lo + i) <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));  // starts do not decrease
    if (c == 0) return -1;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (step == 1) break;
  }
  return lo < n_req ? lo : -1;
}

}  // namespace qsa
