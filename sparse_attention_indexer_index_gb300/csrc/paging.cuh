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
// Bound.  A few bytes a request and twelve a row: latency.  plan_step_kernel is
// one cluster of up to 8 CTAs.  Each computes all sums (a warp takes 32 requests
// at a time, a request a lane); up to 2,048 requests they stay in shared memory
// as a table, by which the first CTA hands out the pages, one a thread, and all
// of them write the rows, one a thread, or four on the way together.  More
// requests: a warp for a request's pages, and step_rows_kernel for the rows.
// Plan and release in a graph: 32 decode requests 5.4 us, 1,500 of 0 to 6 tokens
// 10.2 (one CTA, sums taken twice: 15.9), 37 prompts of some 65,000 tokens in all
// 14.3 (one warp for a request's pages and rows: 35.7).
#pragma once
#include <type_traits>

#include "common.cuh"

namespace qsa {

constexpr int kStepThreads = 1024;
constexpr int kStepMaxGroups = 2048;  // of 32 requests
constexpr int kStepRowsThreads = 256;
constexpr int kStepMaxCluster = 8;
constexpr int kStepTable = 2048;      // requests whose sums it keeps

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
  int32_t cluster;           // CTAs that write rows; 0: step_rows_kernel does
  int32_t page_shift;        // log2 of the page size, -1: not a power of two
};
// Whole pages in x tokens (x below 2^32).
__device__ __forceinline__ uint32_t step_pages(const StepArgs& a, uint32_t x) {
  return a.page_shift >= 0 ? x >> a.page_shift : x / (uint32_t)a.page_size;
}

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
  // (positions end below 2^31, so that sums with the page size stay below 2^32)
  const uint32_t up = (uint32_t)(a.page_size - 1);
  if ((uint32_t)x.ctx + (uint32_t)n > (uint32_t)INT32_MAX || step_pages(a, (uint32_t)x.ctx + (uint32_t)n + up) > a.ld_pt) {
    raise_fault(kFaultIndex);
    x.ok = false;
    return x;
  }
  x.from = (int)step_pages(a, (uint32_t)x.ctx + up);
  x.pages = step_pages(a, (uint32_t)x.ctx + (uint32_t)n + up) - (uint32_t)x.from;
  return x;
}

// Row t of request r (-1: none) at position pos (-1: refused, it has rows but no
// slots), on that page.
__device__ __forceinline__ void step_row(const StepArgs& a, int t, int r, int pos, int page) {
  int len = 0, slot = -1;
  if (pos >= 0) {
    const int64_t s = (int64_t)page * a.page_size + (pos - (int)step_pages(a, (uint32_t)pos) * a.page_size);
    len = pos + 1;
    if (page >= 0 && s <= INT32_MAX) slot = (int)s;
    else raise_fault(kFaultIndex);
  }
  a.row_len[t] = len;
  a.slots[t] = slot;
  if (a.row_req != nullptr) a.row_req[t] = r;
}
// The last i in [0, n) with arr[i] <= x; arr does not decrease, arr[0] <= x.
__device__ __forceinline__ int step_search(const int* arr, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (arr[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
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
  const bool real = r < a.n_req;
  const int ctx = real ? ld_in(a.ctx_len + r) : 0;
  const int pos = real && ld_in(a.new_len + r) != ctx ? ctx + t - ld_in(a.req_row_start + r) : -1;
  step_row(a, t, real ? r : -1, pos, pos >= 0 ? ld_in(a.page_table + (int64_t)r * a.ld_pt + step_pages(a, (uint32_t)pos)) : -1);
}

__global__ void __launch_bounds__(kStepThreads, 1)
plan_step_kernel(const __grid_constant__ StepArgs a) {
  __shared__ uint32_t s_tok[kStepMaxGroups], s_pg[kStepMaxGroups];
  __shared__ uint32_t s_all[2], s_taken;
  // up to kStepTable requests: sums of rows and of pages handed out before each, its tokens
  __shared__ int s_start[kStepTable + 1], s_page[kStepTable + 1], s_ctx[kStepTable];
  const bool table = a.n_req <= kStepTable;
  const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (a.n_req + 31) / 32, warps = blockDim.x / 32;
  const uint32_t top_t = (uint32_t)a.n_tok + 1u, top_p = (uint32_t)a.n_pool + 1u;
  pdl_wait_primary();
  int n_free = ld_in(a.n_free);
  // sums of 32 requests (n_free is looked at behind them: the loads are on the way together); a warp's
  // first two groups, all that a table has, stay in registers
  constexpr int kKeep = 2;
  StepNeed x[kKeep];
  uint32_t it[kKeep], ip[kKeep];
#pragma unroll
  for (int y = 0; y < kKeep; ++y) x[y] = step_need(a, (warp + y * warps) * 32 + lane);
  auto sums = [&](int g, const StepNeed& n, uint32_t& t, uint32_t& p) {
    t = warp_sat_scan(min(n.n, top_t), top_t);
    p = warp_sat_scan(min(n.pages, top_p), top_p);
    if (lane == 31 && g < groups) {
      s_tok[g] = t;
      s_pg[g] = p;
    }
  };
#pragma unroll
  for (int y = 0; y < kKeep; ++y)
    if (y == 0 || warps < groups) sums(warp + y * warps, x[y], it[y], ip[y]);
  const bool keep = groups <= kKeep * warps;
  if (!keep) {
#pragma unroll 1
    for (int g = warp + kKeep * warps; g < groups; g += warps) {
      uint32_t t, p;
      sums(g, step_need(a, g * 32 + lane), t, p);
    }
  }
  if (n_free < 0 || n_free > a.n_pool) {
    if (threadIdx.x == 0) raise_fault(kFaultGrouping);
    n_free = 0;
  }
  // every CTA has read it before the first one writes it
  if (a.cluster > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
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
  uint32_t taken = s_all[1];
  // the sums up to request 32 g + lane itself, and whether it is served
  auto ends = [&](int g, const StepNeed& n, uint32_t t, uint32_t p, uint32_t& et, uint32_t& ep) -> bool {
    et = sat_add(s_tok[g], t, top_t);
    ep = sat_add(s_pg[g], p, top_p);
    return n.ok && et <= (uint32_t)a.n_tok && (n.pages == 0 || ep <= (uint32_t)n_free);
  };
  // f(group, what its requests need, sums within the group) for the warp's groups
  auto each = [&](auto f) {
    StepNeed n = x[0];
    uint32_t t = it[0], p = ip[0];
#pragma unroll 1
    for (int g = warp; g < groups; g += warps) {
      f(g, n, t, p);
      n = x[1];
      t = it[1];
      p = ip[1];
      if (!keep && g + warps < groups && g >= warps) {  // (the third and on)
        n = step_need(a, (g + warps) * 32 + lane);
        t = warp_sat_scan(min(n.n, top_t), top_t);
        p = warp_sat_scan(min(n.pages, top_p), top_p);
      }
    }
  };
  if (!fits) {  // the pages of those that are served
    if (threadIdx.x == 0) raise_fault(kFaultCapacity);
    each([&](int g, const StepNeed& n, uint32_t t, uint32_t p) {
      uint32_t et, ep;
      const bool served = ends(g, n, t, p, et, ep);
      const uint32_t most = __reduce_max_sync(0xffffffffu, served && n.pages > 0 ? ep : 0u);
      if (lane == 0) atomicMax(&s_taken, most);
    });
    __syncthreads();
    taken = s_taken;
  }
  const int base = n_free - (int)taken;
  each([&](int g, const StepNeed& x, uint32_t it, uint32_t ip) {
    const int r = g * 32 + lane;
    uint32_t et, ep;
    const bool served = ends(g, x, it, ip, et, ep);
    uint32_t b = __shfl_up_sync(0xffffffffu, it, 1);
    b = lane == 0 ? s_tok[g] : sat_add(s_tok[g], b, top_t);
    if (r < a.n_req && rank == 0) {
      a.req_row_start[r] = (int)min(b, (uint32_t)a.n_tok);
      if (r == a.n_req - 1) a.req_row_start[a.n_req] = (int)min(et, (uint32_t)a.n_tok);
      a.new_len[r] = served ? x.ctx + (int)x.n : x.ctx;
    }
    if (table) {
      // (pages of refused requests count nothing, and lie behind all others)
      uint32_t bp = __shfl_up_sync(0xffffffffu, ip, 1);
      bp = lane == 0 ? s_pg[g] : sat_add(s_pg[g], bp, top_p);
      if (r < a.n_req) {
        s_start[r] = (int)min(b, (uint32_t)a.n_tok);
        s_page[r] = (int)min(bp, taken);
        s_ctx[r] = served && x.n > 0 ? x.ctx : -1;
      }
      return;
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
  });
  if (table) __syncthreads();
  if (table && rank == 0) {
    for (int i = threadIdx.x; i < (int)taken; i += blockDim.x) {
      const int r = step_search(s_page, a.n_req, i);  // it has pages, and is served
      const int from = (int)step_pages(a, (uint32_t)s_ctx[r] + (uint32_t)(a.page_size - 1));
      a.page_table[(int64_t)r * a.ld_pt + from + (i - s_page[r])] = ld_in(a.free_pages + base + i);
    }
  }
  if (a.cluster > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x == 0) {
    if (a.n_req == 0) a.req_row_start[0] = 0;
    if (taken > 0) *a.n_free = base;
  }
  if (a.cluster == 0) return;  // no table, or no rows
  const int rows = (int)min(s_all[0], (uint32_t)a.n_tok), stride = a.cluster * blockDim.x;
  int top = 1;
  while (2 * top < a.n_req) top *= 2;
  // K rows a thread, on the way together: one where that is all, else four (each a piece of code of its
  // own: what runs once has to be fetched first)
  auto write = [&](auto k, int first) {
    constexpr int K = decltype(k)::value;
    const int t0 = first + threadIdx.x;
    int r[K], pos[K], page[K];
#pragma unroll
    for (int y = 0; y < K; ++y) r[y] = 0;
#pragma unroll 1
    for (int d = top; d > 0; d >>= 1)  // the last request that starts at or before the row
#pragma unroll
      for (int y = 0; y < K; ++y)
        if (r[y] + d < a.n_req && s_start[r[y] + d] <= t0 + y * stride) r[y] += d;
#pragma unroll
    for (int y = 0; y < K; ++y) {
      const int t = t0 + y * stride;
      pos[y] = page[y] = -1;
      if (t >= rows) {
        r[y] = -1;
        continue;
      }
      const int ctx = s_ctx[r[y]];
      if (ctx < 0) continue;
      pos[y] = ctx + t - s_start[r[y]];
      const int pi = (int)step_pages(a, (uint32_t)pos[y]), held = (int)step_pages(a, (uint32_t)ctx + (uint32_t)(a.page_size - 1));
      page[y] = ld_in(pi < held ? a.page_table + (int64_t)r[y] * a.ld_pt + pi : a.free_pages + base + s_page[r[y]] + (pi - held));
    }
#pragma unroll
    for (int y = 0; y < K; ++y)
      if (t0 + y * stride < a.n_tok) step_row(a, t0 + y * stride, r[y], pos[y], page[y]);
  };
  int first = rank * blockDim.x;
#pragma unroll 1
  for (; first + stride < a.n_tok; first += 4 * stride) write(std::integral_constant<int, 4>{}, first);
  if (first < a.n_tok) write(std::integral_constant<int, 1>{}, first);
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
// CTA, 2,048 requests at a time: a thread counts what a request with few
// entries gives, a warp one with many; then the sums, and the pages move in the
// same way.
constexpr int kReleaseFew = 4;
constexpr int kReleaseBatch = 2 * kStepThreads;
__global__ void __launch_bounds__(kStepThreads)
release_pages_kernel(const __grid_constant__ ReleaseArgs a) {
  __shared__ int s_from[kReleaseBatch], s_n[kReleaseBatch];  // a request's entries
  __shared__ uint32_t s_count[kReleaseBatch];                // its pages, then those before it
  __shared__ int s_many[kReleaseBatch];                      // requests with many entries
  __shared__ int s_n_many;
  __shared__ uint32_t s_warp[kStepThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int threads = blockDim.x, batch = 2 * threads;
  const uint32_t top = (uint32_t)a.n_pool + 1u;
  pdl_wait_primary();
  int n_free = ld_in(a.n_free);                              // (looked at behind the first loads of a batch)
  uint32_t before = 0;                                       // pages of the batches before
  for (int r0 = 0; r0 < a.n_req; r0 += batch) {
    const int m = min(batch, a.n_req - r0);
    if (tid == 0) s_n_many = 0;
    __syncthreads();
    int few[2][kReleaseFew];                                 // pages of the thread's requests with few entries
    int from[2], n[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int i = z * threads + tid;
      from[z] = i < m ? ld_in(a.from_page + r0 + i) : 0;
      n[z] = i < m ? ld_in(a.to_page + r0 + i) : 0;
    }
    if (n_free < 0 || n_free > a.n_pool) {                   // an unusable list takes nothing
      if (tid == 0) raise_fault(kFaultGrouping);
      n_free = a.n_pool;
    }
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      if (from[z] < n[z] && (from[z] < 0 || n[z] > a.ld_pt)) raise_fault(kFaultIndex);
      const bool some = from[z] < n[z] && from[z] >= 0 && n[z] <= a.ld_pt;
      n[z] = some ? n[z] - from[z] : 0;
      from[z] = some ? from[z] : 0;
      const int32_t* row = a.page_table + (int64_t)(r0 + z * threads + tid) * a.ld_pt + from[z];
#pragma unroll
      for (int y = 0; y < kReleaseFew; ++y) {
        few[z][y] = -1;
        if (y < n[z] && n[z] <= kReleaseFew) few[z][y] = ld_in(row + y);
      }
    }
    const uint32_t room = (uint32_t)(a.n_pool - n_free);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int i = z * threads + tid;
      uint32_t c = 0;
#pragma unroll
      for (int y = 0; y < kReleaseFew; ++y) c += few[z][y] >= 0;
      if (n[z] > kReleaseFew) s_many[atomicAdd(&s_n_many, 1)] = i;  // (in any order)
      s_from[i] = from[z];
      s_n[i] = n[z];
      s_count[i] = c;
    }
    __syncthreads();
    const int n_many = s_n_many;
    for (int j = warp; j < n_many; j += threads / 32) {
      const int i = s_many[j], n = s_n[i];
      const int32_t* row = a.page_table + (int64_t)(r0 + i) * a.ld_pt + s_from[i];
      uint32_t c = 0;
#pragma unroll 4
      for (int y = lane; y < n; y += 32) c += ld_in(row + y) >= 0;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) s_count[i] = c;
    }
    __syncthreads();
    // sums before each request: two neighbours a thread
    const uint32_t c0 = min(s_count[2 * tid], top), c1 = min(s_count[2 * tid + 1], top);
    const uint32_t incl = warp_sat_scan(sat_add(c0, c1, top), top);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t base = before, all = before;
    for (int w = 0; w < threads / 32; ++w) {
      if (w == warp) base = all;
      all = sat_add(all, s_warp[w], top);
    }
    const uint32_t prev = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane > 0) base = sat_add(base, prev, top);
    s_count[2 * tid] = base;
    s_count[2 * tid + 1] = sat_add(base, c0, top);
    before = all;
    __syncthreads();
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int i = z * threads + tid;
      uint32_t at = s_count[i];
      int32_t* row = a.page_table + (int64_t)(r0 + i) * a.ld_pt + s_from[i];
#pragma unroll
      for (int y = 0; y < kReleaseFew; ++y) {
        if (few[z][y] < 0) continue;
        if (at < room) {
          a.free_pages[n_free + at] = few[z][y];
          row[y] = -1;
        }
        ++at;
      }
    }
    for (int j = warp; j < n_many; j += threads / 32) {
      const int i = s_many[j], n = s_n[i];
      uint32_t at = s_count[i];
      int32_t* row = a.page_table + (int64_t)(r0 + i) * a.ld_pt + s_from[i];
      for (int y0 = 0; y0 < n; y0 += 128) {                  // four loads on the way together
        int page[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int y = y0 + z * 32 + lane;
          page[z] = y < n ? ld_in(row + y) : -1;
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t has = __ballot_sync(0xffffffffu, page[z] >= 0);
          const uint32_t mine = sat_add(at, __popc(has & ((1u << lane) - 1u)), top);
          if (page[z] >= 0 && mine < room) {
            a.free_pages[n_free + mine] = page[z];
            row[y0 + z * 32 + lane] = -1;
          }
          at = sat_add(at, __popc(has), top);
        }
      }
    }
  }
  if (tid == 0) {
    const uint32_t room = (uint32_t)(a.n_pool - n_free);
    if (before > room) raise_fault(kFaultCapacity);
    if (before > 0 && room > 0) *a.n_free = n_free + (int)min(before, room);
  }
}

}  // namespace qsa
