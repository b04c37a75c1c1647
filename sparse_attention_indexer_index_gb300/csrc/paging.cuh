// paging.cuh -- a step's rows, slots and pages from the requests' lengths, and
// pages given back: the bookkeeping between two steps, without the host.
//
// With P tokens a page, request r holds ctx tokens in ceil(ctx / P) pages and
// gets n more: start = exclusive sum of n, and the pages from ceil(ctx / P) to
// ceil((ctx + n) / P) of its row of the table come from the end of a list of
// free pages, in the requests' order.  Row i of the step (request r, position
// p = ctx + i - start) sees p + 1 tokens and has slot table[p / P] P + p mod P.
// A request gets all of its pages or none.  Requests that do not fit the list,
// or the rows, are the last ones that need any: sums of what is needed do not
// decrease, so that both tests are comparisons with a running sum.
//
// Bound.  A few bytes a request and twelve a row: latency.  plan_step_kernel
// is one CTA, in which a warp takes 32 requests at a time (a request a lane
// for the sums and small tables, a request a warp for many pages); it also
// writes the rows where they are few, else step_rows_kernel follows.
#pragma once
#include "common.cuh"

namespace qsa {

constexpr int kStepThreads = 1024;
constexpr int kStepMaxGroups = 2048;  // of 32 requests
constexpr int kStepRowsThreads = 256;
constexpr int kStepOneCta = 4096;     // rows that plan_step_kernel writes itself

struct StepArgs {
  const int32_t* ctx_len;    // [n_req]
  const int32_t* n_new;      // [n_req]
  int32_t n_req;
  int32_t* page_table;       // [n_req][ld_pt]
  int64_t ld_pt;
  int32_t page_size;
  const int32_t* free_pages; // [n_pool]
  int32_t n_pool;
  int32_t* n_free;           // [1]
  int32_t n_tok;
  int32_t* req_row_start;    // [n_req + 1]
  int32_t* new_len;          // [n_req]
  int32_t* row_len;          // [n_tok]
  int32_t* row_req;          // [n_tok] or nullptr
  int32_t* slots;            // [n_tok]
};

// Sums that stop at a limit above every value that matters: associative, and
// no sum of 65,535 counts passes 32 bits.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b, uint32_t top) {
  return min(a + b, top);  // a, b <= top <= 2^31
}
__device__ __forceinline__ uint32_t warp_sat_scan(uint32_t v, uint32_t top) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v = sat_add(v, o, top);
  }
  return v;
}

// What request r needs.
struct StepNeed {
  int ctx;
  uint32_t n, pages;   // rows, new pages
  int from;            // index of the first new page
  bool ok;             // its positions exist
};
__device__ __forceinline__ StepNeed step_need(const StepArgs& a, int r) {
  StepNeed x{0, 0u, 0u, 0, true};
  if (r >= a.n_req) return x;
  x.ctx = ld_in(a.ctx_len + r);
  const int n = ld_in(a.n_new + r);
  if (n < 0 || x.ctx < 0) {
    raise_fault(kFaultGrouping);
    x.ok = false;
  }
  x.n = (uint32_t)max(n, 0);
  if (!x.ok || n == 0) return x;
  // in 64 bits: positions end below 2^31, the page behind them need not
  const int64_t end = ((int64_t)x.ctx + n + a.page_size - 1) / a.page_size;
  const int64_t from = ((int64_t)x.ctx + a.page_size - 1) / a.page_size;
  if (end > a.ld_pt || (int64_t)x.ctx + n > INT32_MAX) {
    raise_fault(kFaultIndex);
    x.ok = false;
    return x;
  }
  x.from = (int)from;
  x.pages = (uint32_t)min(end - from, (int64_t)INT32_MAX);
  return x;
}

// 32 rows from t0 on, by a whole warp.
__device__ __forceinline__ void step_rows(const StepArgs& a, int t0) {
  const int lane = threadIdx.x & 31;
  const int t = t0 + lane;
  // the last request that starts at or before t0: 32 samples a round
  int lo = 0, n = a.n_req + 1;
  while (true) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && ld_in(a.req_row_start + lo + i) <= t0;
    const int c = max(1, __popc(__ballot_sync(0xffffffffu, le)));
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (step == 1) break;
  }
  // the lane's own: it moves past the starts behind `lo` that are at or before
  // t, 32 of them a round (more than one where requests without rows lie between)
  int r = lo, base = lo;
  do {
    const int i = base + 1 + lane;
    const int s = i <= a.n_req ? ld_in(a.req_row_start + i) : INT32_MAX;
    int c = 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (__shfl_sync(0xffffffffu, s, c + d - 1) <= t) c += d;
    if (__shfl_sync(0xffffffffu, s, c) <= t) ++c;
    if (r == base) r += c;
    base += 32;
  } while (__any_sync(0xffffffffu, r == base));
  if (t >= a.n_tok) return;
  int len = 0, slot = -1, req = -1;
  if (r < a.n_req) {
    req = r;
    const int ctx = ld_in(a.ctx_len + r);
    if (ld_in(a.new_len + r) != ctx) {  // else refused: it has rows, but no slots
      const int pos = ctx + (t - ld_in(a.req_row_start + r));
      const int pi = pos / a.page_size;
      const int page = ld_in(a.page_table + (int64_t)r * a.ld_pt + pi);
      const int64_t s = (int64_t)page * a.page_size + (pos - pi * a.page_size);
      len = pos + 1;
      if (page >= 0 && s <= INT32_MAX) slot = (int)s;
      else raise_fault(kFaultIndex);
    }
  }
  a.row_len[t] = len;
  a.slots[t] = slot;
  if (a.row_req != nullptr) a.row_req[t] = req;
}

__global__ void __launch_bounds__(kStepThreads)
plan_step_kernel(const __grid_constant__ StepArgs a) {
  __shared__ uint32_t s_tok[kStepMaxGroups], s_pg[kStepMaxGroups];
  __shared__ uint32_t s_all[2], s_taken;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.n_req + 31) / 32;
  const uint32_t top_t = (uint32_t)a.n_tok + 1u, top_p = (uint32_t)a.n_pool + 1u;
  pdl_wait_primary();
  int n_free = ld_in(a.n_free);
  if (n_free < 0 || n_free > a.n_pool) {
    if (threadIdx.x == 0) raise_fault(kFaultGrouping);
    n_free = 0;
  }
  // sums of 32 requests
  StepNeed x{0, 0u, 0u, 0, true};
  uint32_t it = 0, ip = 0;
  for (int g = warp; g < groups; g += kStepThreads / 32) {
    x = step_need(a, g * 32 + lane);
    it = warp_sat_scan(min(x.n, top_t), top_t);
    ip = warp_sat_scan(min(x.pages, top_p), top_p);
    if (lane == 31) {
      s_tok[g] = it;
      s_pg[g] = ip;
    }
  }
  if (threadIdx.x == 0) s_taken = 0;
  __syncthreads();
  // and before them
  if (warp == 0) {
    uint32_t ct = 0, cp = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      const uint32_t vt = g < groups ? s_tok[g] : 0u, vp = g < groups ? s_pg[g] : 0u;
      const uint32_t st = sat_add(warp_sat_scan(vt, top_t), ct, top_t);
      const uint32_t sp = sat_add(warp_sat_scan(vp, top_p), cp, top_p);
      uint32_t bt = __shfl_up_sync(0xffffffffu, st, 1), bp = __shfl_up_sync(0xffffffffu, sp, 1);
      if (lane == 0) {
        bt = ct;
        bp = cp;
      }
      if (g < groups) {
        s_tok[g] = bt;
        s_pg[g] = bp;
      }
      ct = __shfl_sync(0xffffffffu, st, 31);
      cp = __shfl_sync(0xffffffffu, sp, 31);
    }
    if (lane == 0) {
      s_all[0] = ct;
      s_all[1] = cp;
    }
  }
  __syncthreads();
  const bool fits = s_all[0] <= (uint32_t)a.n_tok && s_all[1] <= (uint32_t)n_free;
  const bool keep = groups <= kStepThreads / 32;  // one group a warp: still in registers
  uint32_t taken = s_all[1];
  // the request's sums up to itself, and whether it is served
  auto ends = [&](int g, uint32_t& et, uint32_t& ep) -> bool {
    if (!keep) {
      x = step_need(a, g * 32 + lane);
      it = warp_sat_scan(min(x.n, top_t), top_t);
      ip = warp_sat_scan(min(x.pages, top_p), top_p);
    }
    et = sat_add(s_tok[g], it, top_t);
    ep = sat_add(s_pg[g], ip, top_p);
    return x.ok && et <= (uint32_t)a.n_tok && (x.pages == 0 || ep <= (uint32_t)n_free);
  };
  if (!fits) {  // the pages of those that are served
    if (threadIdx.x == 0) raise_fault(kFaultCapacity);
    for (int g = warp; g < groups; g += kStepThreads / 32) {
      uint32_t et, ep;
      const bool served = ends(g, et, ep);
      const uint32_t most = __reduce_max_sync(0xffffffffu, served && x.pages > 0 ? ep : 0u);
      if (lane == 0) atomicMax(&s_taken, most);
    }
    __syncthreads();
    taken = s_taken;
  }
  const int base = n_free - (int)taken;
  for (int g = warp; g < groups; g += kStepThreads / 32) {
    const int r = g * 32 + lane;
    uint32_t et, ep;
    const bool served = ends(g, et, ep);
    uint32_t b = __shfl_up_sync(0xffffffffu, it, 1);
    b = lane == 0 ? s_tok[g] : sat_add(s_tok[g], b, top_t);
    if (r < a.n_req) {
      a.req_row_start[r] = (int)min(b, (uint32_t)a.n_tok);
      if (r == a.n_req - 1) a.req_row_start[a.n_req] = (int)min(et, (uint32_t)a.n_tok);
      a.new_len[r] = served ? x.ctx + (int)x.n : x.ctx;
    }
    // pages: a warp for a request
    uint32_t todo = __ballot_sync(0xffffffffu, served && x.pages > 0);
    while (todo != 0) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int pages = (int)__shfl_sync(0xffffffffu, x.pages, l), from = __shfl_sync(0xffffffffu, x.from, l);
      const int at = base + (int)__shfl_sync(0xffffffffu, ep, l) - pages;
      int32_t* row = a.page_table + (int64_t)(g * 32 + l) * a.ld_pt + from;
#pragma unroll 4
      for (int i = lane; i < pages; i += 32) row[i] = ld_in(a.free_pages + at + i);
    }
  }
  if (a.n_req == 0 && threadIdx.x == 0) a.req_row_start[0] = 0;
  __syncthreads();  // starts, lengths and pages are read below
  if (threadIdx.x == 0 && taken > 0) *a.n_free = base;
  if (a.n_tok <= kStepOneCta)
    for (int t0 = warp * 32; t0 < a.n_tok; t0 += kStepThreads) step_rows(a, t0);
}

__global__ void __launch_bounds__(kStepRowsThreads)
step_rows_kernel(const __grid_constant__ StepArgs a) {
  pdl_wait_primary();
  const int t0 = (blockIdx.x * kStepRowsThreads + threadIdx.x) & ~31;
  if (t0 < a.n_tok) step_rows(a, t0);
}

struct ReleaseArgs {
  int32_t* page_table;       // [n_req][ld_pt]
  int64_t ld_pt;
  int32_t n_req;
  const int32_t* from_page;  // [n_req]
  const int32_t* to_page;    // [n_req]
  int32_t* free_pages;       // [n_pool]
  int32_t n_pool;
  int32_t* n_free;           // [1]
};

// Pages given back: entries from_page .. to_page - 1 of a request's row go to
// the end of the list in the requests' order and become -1 in the table.  One
// CTA: a warp counts what 32 requests give, and after the sums moves it; a
// request of more than kReleaseFew entries takes the whole warp.
constexpr int kReleaseFew = 4;
__global__ void __launch_bounds__(kStepThreads)
release_pages_kernel(const __grid_constant__ ReleaseArgs a) {
  __shared__ uint32_t s_pg[kStepMaxGroups];
  __shared__ uint32_t s_all;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.n_req + 31) / 32;
  const uint32_t top = (uint32_t)a.n_pool + 1u;
  pdl_wait_primary();
  int n_free = ld_in(a.n_free);
  if (n_free < 0 || n_free > a.n_pool) {  // an unusable list takes nothing
    if (threadIdx.x == 0) raise_fault(kFaultGrouping);
    n_free = a.n_pool;
  }
  const uint32_t room = (uint32_t)(a.n_pool - n_free);
  // the lane's entries of group g
  auto range = [&](int g, int& from, int& n) {
    const int r = g * 32 + lane;
    from = n = 0;
    if (r >= a.n_req) return;
    const int f = ld_in(a.from_page + r), t = ld_in(a.to_page + r);
    if (f >= t) return;
    if (f < 0 || t > a.ld_pt) {
      raise_fault(kFaultIndex);
      return;
    }
    from = f;
    n = t - f;
  };
  // the pages among them
  auto count = [&](int g, int from, int n) -> uint32_t {
    const int32_t* row = a.page_table + (int64_t)(g * 32 + lane) * a.ld_pt + from;
    uint32_t c = 0;
    if (n > 0 && n <= kReleaseFew) {
#pragma unroll
      for (int i = 0; i < kReleaseFew; ++i)
        if (i < n) c += ld_in(row + i) >= 0;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, n > kReleaseFew);
    while (todo != 0) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int nn = __shfl_sync(0xffffffffu, n, l);
      const int32_t* rw = a.page_table + (int64_t)(g * 32 + l) * a.ld_pt + __shfl_sync(0xffffffffu, from, l);
      uint32_t s = 0;
#pragma unroll 4
      for (int i = lane; i < nn; i += 32) s += ld_in(rw + i) >= 0;
      s = __reduce_add_sync(0xffffffffu, s);
      if (lane == l) c = s;
    }
    return c;
  };
  int from = 0, n = 0;
  uint32_t c = 0, ic = 0;
  for (int g = warp; g < groups; g += kStepThreads / 32) {
    range(g, from, n);
    c = count(g, from, n);
    ic = warp_sat_scan(min(c, top), top);
    if (lane == 31) s_pg[g] = ic;
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t carry = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int g = g0 + lane;
      const uint32_t s = sat_add(warp_sat_scan(g < groups ? s_pg[g] : 0u, top), carry, top);
      uint32_t b = __shfl_up_sync(0xffffffffu, s, 1);
      if (lane == 0) b = carry;
      if (g < groups) s_pg[g] = b;
      carry = __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) s_all = carry;
  }
  __syncthreads();
  for (int g = warp; g < groups; g += kStepThreads / 32) {
    if (groups > kStepThreads / 32) {  // else still in registers
      range(g, from, n);
      c = count(g, from, n);
      ic = warp_sat_scan(min(c, top), top);
    }
    uint32_t at = __shfl_up_sync(0xffffffffu, ic, 1);  // pages given back before the request's
    at = lane == 0 ? s_pg[g] : sat_add(s_pg[g], at, top);
    if (n > 0 && n <= kReleaseFew) {
      int32_t* row = a.page_table + (int64_t)(g * 32 + lane) * a.ld_pt + from;
      for (int i = 0; i < n; ++i) {
        const int page = ld_in(row + i);
        if (page < 0) continue;
        if (at < room) {
          a.free_pages[n_free + at] = page;
          row[i] = -1;
        }
        ++at;
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, n > kReleaseFew);
    while (todo != 0) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int nn = __shfl_sync(0xffffffffu, n, l);
      uint32_t b = __shfl_sync(0xffffffffu, at, l);
      int32_t* rw = a.page_table + (int64_t)(g * 32 + l) * a.ld_pt + __shfl_sync(0xffffffffu, from, l);
      for (int i0 = 0; i0 < nn; i0 += 32) {
        const int i = i0 + lane;
        const int page = i < nn ? ld_in(rw + i) : -1;
        const uint32_t has = __ballot_sync(0xffffffffu, page >= 0);
        const uint32_t mine = b + __popc(has & ((1u << lane) - 1u));
        if (page >= 0 && mine < room) {
          a.free_pages[n_free + mine] = page;
          rw[i] = -1;
        }
        b += __popc(has);
      }
    }
  }
  if (threadIdx.x == 0) {
    if (s_all > room) raise_fault(kFaultCapacity);
    if (s_all > 0 && room > 0) *a.n_free = n_free + (int)min(s_all, room);
  }
}

}  // namespace qsa
