// kv8_api.cu -- the extern "C" entry points of the 8-bit KV cache, of the
// attention over it, and of the paging calls: host-side argument checks,
// launch shapes, and launches on the caller's stream.  Contracts are in
// include/qsa.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "../../include/qsa.h"
#include "common.cuh"
#include "host_util.cuh"
#include "kv_host.cuh"
#include "kv8.cuh"
#include "kv8_tc.cuh"
#include "paging.cuh"

using namespace qsa;

namespace {

// The kernel of a tile's pairs, and its shape.
struct K8Kernel {
  void (*fn)(Kv8AttnArgs);
  int threads, smem, pairs, block;
};
template <int D, int N, int PARTS, bool kWindow, bool kShared>
constexpr K8Kernel k8() {
  using Sh = K8Tc<D, N, PARTS, kWindow, kShared>;
  return {kv8_tc_kernel<D, N, PARTS, kWindow, kShared>, Sh::kThreads, Sh::kSmem, N, Sh::kBlock};
}
// Lists and windows of single rows (up to 8 heads to a KV head, up to 16), and
// the rows of a request together: 8, 16, 32 or 48 pairs.
enum { kList8 = 0, kList16 = 1, kRow8 = 2, kTile8 = 3, kTile16 = 4, kTile32 = 5, kTile48 = 6, kK8Kinds = 7 };
constexpr K8Kernel kK8Kernels[kK8Kinds][2] = {
    {k8<128, 8, 4, false, false>(), k8<256, 8, 4, false, false>()},
    {k8<128, 16, 4, false, false>(), k8<256, 16, 4, false, false>()},
    {k8<128, 8, 4, true, false>(), k8<256, 8, 4, true, false>()},
    {k8<128, 8, 4, true, true>(), k8<256, 8, 4, true, true>()},
    {k8<128, 16, 4, true, true>(), k8<256, 16, 4, true, true>()},
    {k8<128, 32, 4, true, true>(), k8<256, 32, 4, true, true>()},
    {k8<128, 48, 4, true, true>(), k8<256, 48, 4, true, true>()},
};

// Per-device one-time set-up: the shared-memory opt-in of the kernels, and how
// many of their clusters run at once.
struct Kv8Device {
  int sms;  // 0: not set up
  int clusters[kK8Kinds][2][kKaMaxCluster + 1];
};
Kv8Device g_kv8_dev[kMaxDevices];
std::mutex g_mu;

qsa_status kv8_device(const Kv8Device** out) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QSA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  Kv8Device& d = g_kv8_dev[dev];
  if (d.sms == 0) {
    bool ok = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    for (int i = 0; ok && i < kK8Kinds * 2; ++i) {
      const K8Kernel& k = kK8Kernels[i / 2][i % 2];
      ok = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) == cudaSuccess;
      for (int c = 1; ok && c <= kKaMaxCluster; c *= 2)
        ok = resident_clusters(k.fn, k.threads, (size_t)k.smem, c, sms, &d.clusters[i / 2][i % 2][c]);
    }
    if (!ok) {
      cudaGetLastError();
      return QSA_ERR_CUDA;
    }
    d.sms = sms;
  }
  *out = &d;
  return QSA_OK;
}

bool kv8_shape_ok(int32_t h_q, int32_t h_kv, int32_t d) {
  return h_q > 0 && h_kv > 0 && h_kv <= 65535 && h_q % h_kv == 0 && h_q / h_kv <= 16 && (d == 128 || d == 256);
}

// The scales' block: a power of two that divides the page (page_size 0: no pages).
qsa_status check_block(int32_t block_tokens, int32_t page_size, int64_t n_slots) {
  if (block_tokens < 4 || block_tokens > 128 || (block_tokens & (block_tokens - 1)) != 0) return QSA_ERR_UNSUPPORTED;
  if (page_size % block_tokens != 0) return QSA_ERR_UNSUPPORTED;
  return n_slots % block_tokens == 0 ? QSA_OK : QSA_ERR_INVALID_ARG;
}
int log2_of(int32_t x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// The cache's four arrays (any of them may be NULL with n_slots 0); scales are
// read byte by byte.
qsa_status check_cache8(const void* kc, const void* ks, const void* vc, const void* vs, int64_t n_slots) {
  if (n_slots < 0 || n_slots > INT32_MAX) return QSA_ERR_INVALID_ARG;
  if (n_slots > 0 && (!kc || !ks || !vc || !vs)) return QSA_ERR_INVALID_ARG;
  return aligned16(kc) && aligned16(vc) ? QSA_OK : QSA_ERR_INVALID_ARG;
}

// How a call is cut into tiles, and how the work is dealt.
struct K8Form {
  int kind, rows;      // kernel, rows per tile
  int64_t tile_slots;  // slots of tiles (see k8_find): as many as tiles at least
  int64_t units;       // (tile, KV head) pairs, for requests of equal length
  int64_t blocks;      // of a unit, where a tile's rows are neighbours
  bool cluster, share; // clusters, shares, else whole units
};
// Clusters where the units are few and their blocks, shared by the CTAs of a
// cluster, few as well; shares of the blocks where units are long; whole units
// where they are many.  The parts' way through memory, and the second kernel,
// count as 9 blocks, which is what they take where all SMs read at HBM's rate; up
// to 4 units only a few would, in clusters of 8 at most, and it is 3 (with 1 a
// list of 2,051 takes 7.6 us instead of 8.2, but the host, which has a workspace
// to find and a second kernel to launch, 4 us more).  Measured in a graph,
// clusters / shares: 38 lists of 2,051 on 2 heads of D = 256 19.6 / 22.9 us, 50 of
// 4,000 39.2 / 41.6, 4 of 9,000 15.7 / 16.2, 14 windows of 16,000 43.5 / 48.7; one
// list of 5,000 10.4 / 7.8, of 9,000 14.9 / 8.8, 2 of 6,000 12.1 / 9.7.  In a stream
// of calls, where the host's time for shares shows, those three take 11.9 / 14 to
// 17, 16.2 / 13 to 18 and 13.3 / 19 to 21: decode steps are captured.
// The choice follows from the arguments alone, as the workspace does: for 152 SMs,
// of which clusters of 2 fill 152 at once, of 4 144 and of 8 120.  144 stands for
// all sizes here; a launch takes the sizes that fit the device (launch_k8): with 73
// to 76 units clusters of 2 where this counts on single CTAs, with 16 to 18 units
// clusters of 4 where it counts on 8.
// `most` is what the rows of a tile can span in any order.
K8Form finish(int kind, int d, int rows, int64_t tile_slots, int64_t units, int64_t n_req, int64_t entries, int64_t most) {
  K8Form f{kind, rows, tile_slots, units, 1, false, false};
  const int block = kK8Kernels[kind][d == 256].block;
  f.blocks = std::max<int64_t>(1, (entries + block - 1) / block);
  const bool list = kind <= kList16;
  const bool fits = units < kK8MaxUnits && (list || (tile_slots <= kK8MaxTiles && n_req <= kK8MaxTiles)) &&
                    // blocks are counted in 32 bits (there are at most two slots to a unit)
                    units * ((most + block - 1) / block + 1 + kK8Lead) < INT32_MAX / 2;
  int c = 1;
  while (c < kKaMaxCluster && units * 2 * c <= 144 && f.blocks >= 2 * c) c *= 2;
  const int64_t rounds = (units * c + 151) / 152;
  const int64_t by_cluster = rounds * ((f.blocks + c - 1) / c);
  const int64_t by_share = (units * (f.blocks + kK8Lead) + 151) / 152 + (units <= 4 ? 3 : 9);
  f.cluster = rounds == 1 && (by_cluster <= by_share || !fits);
  f.share = !f.cluster && fits;
  return f;
}
K8Form list_form(int32_t n_rows, int32_t h_q, int32_t h_kv, int32_t d, int64_t n_idx) {
  return finish(h_q / h_kv > 8 ? kList16 : kList8, d, 1, n_rows, (int64_t)n_rows * h_kv, 0, n_idx, n_idx);
}
K8Form window_form(int32_t n_rows, int32_t n_req, int32_t max_rows_per_req, int32_t h_q, int32_t h_kv, int32_t d,
                   int32_t max_len, int32_t window, int32_t n_sink) {
  const int group = h_q / h_kv;
  const int64_t entries = window_entries(max_len, window, n_sink);
  if (max_rows_per_req <= 1 && group <= 8)
    return finish(kRow8, d, 1, n_rows, (int64_t)n_rows * h_kv, n_req, entries, entries);
  const int64_t pairs = (int64_t)std::max(max_rows_per_req, 1) * group;
  const int kind = pairs <= 8 ? kTile8 : pairs <= 16 ? kTile16 : pairs <= 32 ? kTile32 : kTile48;
  const int rows = kK8Kernels[kind][0].pairs / group;
  const int64_t slots = k8_tile_slots(n_rows, n_req, rows);
  const int64_t per_req = ((int64_t)n_rows + n_req - 1) / n_req;
  // (a tile of rows in any order may span more than a row)
  return finish(kind, d, rows, slots, std::min<int64_t>(slots, (int64_t)n_req * ((per_req + rows - 1) / rows)) * h_kv, n_req,
                std::min<int64_t>(max_len, entries + rows), rows == 1 ? entries : max_len);
}

// The jobs, then two partial results a CTA.
constexpr size_t kJobBytes = (kK8Ctas * sizeof(int4) + 255) / 256 * 256;
size_t form_bytes(const K8Form& f, int32_t d) {
  return f.share ? kJobBytes + (size_t)2 * kK8Ctas * kK8Kernels[f.kind][0].pairs * (d + 4) * 4 : 0;
}

qsa_status launch_k8(const K8Form& f, Kv8AttnArgs& a, int d, void* workspace, cudaStream_t stream) {
  const Kv8Device* dev = nullptr;
  if (qsa_status st = kv8_device(&dev)) return st;
  const K8Kernel& k = kK8Kernels[f.kind][d == 256];
  a.group = a.h_q / a.h_kv;
  a.rows = f.rows;
  const int64_t slots = f.tile_slots * a.h_kv;
  if (slots > INT32_MAX / kKaMaxCluster || (int64_t)a.n_rows * a.h_q > INT32_MAX) return QSA_ERR_UNSUPPORTED;
  a.tile_slots = (int32_t)f.tile_slots;
  a.jobs = static_cast<int4*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kJobBytes);
  const int sms = std::min(dev->sms, kK8Ctas);
  a.cluster = 1;
  int64_t grid = std::min<int64_t>(sms, slots);
  a.mode = kK8Whole;
  if (f.share) {
    a.mode = kK8Shares;
    grid = sms;
    a.jobs_by_unit = slots <= sms;
  } else if (f.cluster) {
    // as many CTAs to a unit as run at once
    a.mode = kK8Cluster;
    const int* at_once = dev->clusters[f.kind][d == 256];
    while (a.cluster < kKaMaxCluster && f.units <= at_once[2 * a.cluster] && f.blocks >= 2 * a.cluster) a.cluster *= 2;
    grid = slots * a.cluster;
    a.n_units = (int32_t)f.units;
  }
  a.cluster_shift = log2_of(a.cluster);
  a.group_inv = (65536 + a.group - 1) / a.group;  // exact for pairs below 4,096
  const ClusterLaunch l(dim3((unsigned)grid), k.threads, (size_t)k.smem, a.cluster, stream);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k.fn, a);
  if (e == cudaSuccess && f.share) {
    // parts of a unit, with blocks of equal number to every CTA; lengths may differ
    const bool many = f.blocks > 8 * (f.units * (f.blocks + kK8Lead) / grid + 1);
    const int cols = many ? 64 : d, pairs = f.rows * a.group;
    const dim3 shape((unsigned)(a.jobs_by_unit ? slots : grid), (unsigned)(many ? pairs : (pairs * d + kK8MergeThreads - 1) / kK8MergeThreads),
                     (unsigned)(d / cols));
    e = launch_pdl(d == 256 ? (many ? kv8_merge_kernel<256, true> : kv8_merge_kernel<256, false>)
                            : (many ? kv8_merge_kernel<128, true> : kv8_merge_kernel<128, false>),
                   shape, dim3(kK8MergeThreads), 0, stream, a, k.pairs);
  }
  return launched(e);
}

void set_cache(Kv8AttnArgs& a, const void* kc, const void* ks, const void* vc, const void* vs, int32_t block_tokens) {
  a.k = static_cast<const uint8_t*>(kc);
  a.v = static_cast<const uint8_t*>(vc);
  a.ks = static_cast<const uint8_t*>(ks);
  a.vs = static_cast<const uint8_t*>(vs);
  a.block_shift = log2_of(block_tokens);
  a.page_shift = a.page_size > 0 && (a.page_size & (a.page_size - 1)) == 0 ? log2_of(a.page_size) : -1;
}

qsa_status check_requests(int32_t n_req) {
  if (n_req < 0) return QSA_ERR_INVALID_ARG;
  return n_req > 65535 ? QSA_ERR_UNSUPPORTED : QSA_OK;
}

}  // namespace

namespace qsa {
bool kv8_fault_word(cudaStream_t stream, bool clear, unsigned* bits) {
  if (cudaMemcpyFromSymbolAsync(bits, g_fault_word, sizeof(*bits), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return false;
  if (clear && *bits) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbolAsync(g_fault_word, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess ||
        cudaStreamSynchronize(stream) != cudaSuccess)
      return false;
  }
  return true;
}
}  // namespace qsa

extern "C" {

qsa_status qsa_plan_step(const int32_t* ctx_len, const int32_t* n_new, int32_t n_req, int32_t* page_table,
                         int64_t ld_pt, int32_t page_size, const int32_t* free_pages, int32_t n_pool, int32_t* n_free,
                         int32_t n_tok, int32_t* req_row_start, int32_t* new_len, int32_t* row_len, int32_t* row_req,
                         int32_t* slots, void* stream) {
  if (qsa_status st = check_requests(n_req)) return st;
  if (n_tok < 0 || n_pool < 0 || ld_pt < 0 || page_size <= 0) return QSA_ERR_INVALID_ARG;
  if (page_size % kBlock != 0 || n_tok > (1 << 30) || n_pool == INT32_MAX) return QSA_ERR_UNSUPPORTED;
  if (!req_row_start || !n_free || (n_pool > 0 && !free_pages)) return QSA_ERR_INVALID_ARG;
  if (n_req > 0 && (!ctx_len || !n_new || !page_table || !new_len)) return QSA_ERR_INVALID_ARG;
  if (n_tok > 0 && (!row_len || !slots)) return QSA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)ctx_len, (const void*)n_new, (const void*)page_table, (const void*)free_pages,
                        (const void*)n_free, (const void*)req_row_start, (const void*)new_len, (const void*)row_len,
                        (const void*)row_req, (const void*)slots})
    if (!aligned4(p)) return QSA_ERR_INVALID_ARG;
  if (new_len != nullptr && new_len == ctx_len) return QSA_ERR_INVALID_ARG;  // the rows are found with both
  StepArgs a{ctx_len, n_new, n_req, page_table, ld_pt, page_size, free_pages, n_pool, n_free,
             n_tok, req_row_start, new_len, row_len, row_req, slots, 0,
             (page_size & (page_size - 1)) == 0 ? log2_of(page_size) : -1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool table = n_req <= kStepTable;
  // a thread for a request, for a page that the step may take, and for a row
  const int want = std::max({n_req, n_tok / page_size + n_req, table ? n_tok : 0});
  const int threads = std::min(kStepThreads, std::max(128, (want + 31) / 32 * 32));
  if (table) {
    a.cluster = 1;
    while (a.cluster < kStepMaxCluster && n_tok > a.cluster * threads) a.cluster *= 2;
  }
  const ClusterLaunch l(dim3((unsigned)std::max(a.cluster, 1)), threads, 0, std::max(a.cluster, 1), s);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, plan_step_kernel, a);
  if (e == cudaSuccess && !table && n_tok > 0)
    e = launch_pdl(step_rows_kernel, dim3((unsigned)((n_tok + kStepRowsThreads - 1) / kStepRowsThreads)),
                   dim3(kStepRowsThreads), 0, s, a);
  return launched(e);
}

qsa_status qsa_release_pages(int32_t* page_table, int64_t ld_pt, int32_t n_req, const int32_t* from_page,
                             const int32_t* to_page, int32_t* free_pages, int32_t n_pool, int32_t* n_free,
                             void* stream) {
  if (qsa_status st = check_requests(n_req)) return st;
  if (n_pool < 0 || ld_pt < 0) return QSA_ERR_INVALID_ARG;
  if (n_pool == INT32_MAX) return QSA_ERR_UNSUPPORTED;
  if (n_req == 0) return QSA_OK;
  if (!page_table || !from_page || !to_page || !n_free || (n_pool > 0 && !free_pages)) return QSA_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(from_page) || !aligned4(to_page) || !aligned4(free_pages) || !aligned4(n_free))
    return QSA_ERR_INVALID_ARG;
  const ReleaseArgs a{page_table, ld_pt, n_req, from_page, to_page, free_pages, n_pool, n_free};
  // two requests a thread, but some warps for requests of many pages
  const int threads = n_req <= 32 ? 256 : kStepThreads;
  return launched(launch_pdl(release_pages_kernel, dim3(1), dim3((unsigned)threads), 0, static_cast<cudaStream_t>(stream), a));
}

qsa_status qsa_append_kv_fp8(const void* k_new, const void* v_new, int64_t ld_k, int64_t ld_v, int32_t n_tok,
                             int32_t h_kv, int32_t head_dim, const int32_t* req_tok_start,
                             const int32_t* req_first_pos, int32_t n_req, const int32_t* page_table, int64_t ld_pt,
                             int32_t page_size, int32_t block_tokens, void* k_codes, void* k_scales, void* v_codes,
                             void* v_scales, int64_t n_slots, void* stream) {
  if (n_tok < 0 || h_kv <= 0) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_requests(n_req)) return st;
  if ((head_dim != 128 && head_dim != 256) || h_kv > 65535 || n_tok > (1 << 30)) return QSA_ERR_UNSUPPORTED;
  if (page_size <= 0) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_block(block_tokens, page_size, n_slots)) return st;
  if (n_tok == 0 || n_req == 0) return QSA_OK;
  if (!k_new || !v_new || !req_tok_start || !req_first_pos) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_paging(page_table, ld_pt, page_size, 0)) return st;
  if (qsa_status st = check_cache8(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  const int64_t row = (int64_t)h_kv * head_dim;
  if (!aligned16(k_new) || !aligned16(v_new) || ld_k % 8 != 0 || ld_v % 8 != 0 || ld_k < row || ld_v < row)
    return QSA_ERR_INVALID_ARG;
  Kv8WriteArgs a{};
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.n_tok = n_tok;
  a.h_kv = h_kv;
  a.d = head_dim;
  a.req_tok_start = req_tok_start;
  a.req_first_pos = req_first_pos;
  a.n_req = n_req;
  a.page_table = page_table;
  a.ld_pt = ld_pt;
  a.page_size = page_size;
  a.block_shift = log2_of(block_tokens);
  a.per_shift = head_dim == 256 ? 5 : 4;
  a.n_slots = n_slots;
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.k_scales = static_cast<uint8_t*>(k_scales);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.v_scales = static_cast<uint8_t*>(v_scales);
  // tokens to a CTA: one, until the CTAs are many rounds; a block at most
  a.chunk = 1;
  while (a.chunk < block_tokens && (int64_t)n_tok * h_kv * 2 > (int64_t)a.chunk * 152 * 32) a.chunk *= 2;
  const dim3 grid((unsigned)((n_tok + a.chunk - 1) / a.chunk), (unsigned)h_kv, 2);
  const int pieces = block_tokens * head_dim / 8 / kKv8Threads;  // a block's, per thread
  const auto kernel = pieces <= 1   ? append_kv_fp8_kernel<1>
                      : pieces <= 2 ? append_kv_fp8_kernel<2>
                      : pieces <= 4 ? append_kv_fp8_kernel<4>
                      : pieces <= 8 ? append_kv_fp8_kernel<8>
                                    : append_kv_fp8_kernel<16>;
  return launched(launch_pdl(kernel, grid, dim3(kKv8Threads), 0, static_cast<cudaStream_t>(stream), a));
}

qsa_status qsa_gather_kv_fp8(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                             int64_t n_slots, int32_t h_kv, int32_t head_dim, int32_t block_tokens,
                             const int32_t* slots, int64_t n, void* k_out, void* v_out, void* stream) {
  if (n < 0 || h_kv <= 0) return QSA_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || h_kv > 65535) return QSA_ERR_UNSUPPORTED;
  if (qsa_status st = check_block(block_tokens, 0, n_slots)) return st;
  if (n == 0) return QSA_OK;
  if (!slots || !k_out || !v_out || !aligned4(slots) || !aligned32(k_out) || !aligned32(v_out))
    return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_cache8(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  Kv8ReadArgs a{};
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.k_scales = static_cast<const uint8_t*>(k_scales);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.n_slots = n_slots;
  a.h_kv = h_kv;
  a.per = head_dim / 16;
  a.block_shift = log2_of(block_tokens);
  a.slots = slots;
  a.n = n;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  const int64_t row = (int64_t)h_kv * a.per;
  // pieces are counted in 32 bits (2^32 of them would be 137 GB of output each)
  if (n > (int64_t)(UINT32_MAX - 4 * kKvThreads) / row) return QSA_ERR_UNSUPPORTED;
  const int64_t ctas = (n * row + kKvThreads - 1) / kKvThreads;
  return launched(launch_pdl(gather_kv_fp8_kernel, dim3((unsigned)ctas), dim3(kKvThreads), 0,
                             static_cast<cudaStream_t>(stream), a));
}

size_t qsa_sparse_attn_fp8_workspace_size(int32_t n_rows, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t n_idx) {
  if (n_rows <= 0 || n_idx < 0 || !kv8_shape_ok(h_q, h_kv, head_dim)) return 0;
  return form_bytes(list_form(n_rows, h_q, h_kv, head_dim, n_idx), head_dim);
}

qsa_status qsa_sparse_attn_fp8(const void* q, int64_t ld_q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, int64_t n_slots, int32_t block_tokens,
                               int32_t n_rows, int32_t h_q, int32_t h_kv, int32_t head_dim, const int32_t* slots,
                               int64_t ld_slots, int32_t n_idx, float scale, float* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (n_rows < 0 || n_idx < 0 || ld_slots < n_idx) return QSA_ERR_INVALID_ARG;
  if (!kv8_shape_ok(h_q, h_kv, head_dim)) return QSA_ERR_UNSUPPORTED;
  if (qsa_status st = check_block(block_tokens, 0, n_slots)) return st;
  if (!std::isfinite(scale)) return QSA_ERR_INVALID_ARG;
  if (n_rows == 0) return QSA_OK;
  if (!q || !out || (n_idx > 0 && !slots) || !aligned16(q) || !aligned16(out) || (lse && !aligned4(lse)) ||
      !aligned4(slots))
    return QSA_ERR_INVALID_ARG;
  if (ld_q < (int64_t)h_q * head_dim || ld_q % 8 != 0) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_cache8(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  if (qsa_status st = check_workspace(qsa_sparse_attn_fp8_workspace_size(n_rows, h_q, h_kv, head_dim, n_idx), workspace,
                                      workspace_bytes))
    return st;
  Kv8AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.ld_q = ld_q;
  set_cache(a, k_codes, k_scales, v_codes, v_scales, block_tokens);
  a.n_slots = n_slots;
  a.n_rows = n_rows;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.slots = slots;
  a.ld_slots = ld_slots;
  a.n_idx = n_idx;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  if (n_idx > (1 << 30)) return QSA_ERR_UNSUPPORTED;  // entry indices stay clear of 2^31
  return launch_k8(list_form(n_rows, h_q, h_kv, head_dim, n_idx), a, head_dim, workspace, static_cast<cudaStream_t>(stream));
}

size_t qsa_window_attn_fp8_workspace_size(int32_t n_rows, int32_t n_req, int32_t max_rows_per_req, int32_t h_q,
                                          int32_t h_kv, int32_t head_dim, int32_t max_len, int32_t window,
                                          int32_t n_sink) {
  if (n_rows <= 0 || n_req <= 0 || max_len < 0 || window < 1 || n_sink < 0 || !kv8_shape_ok(h_q, h_kv, head_dim))
    return 0;
  return form_bytes(window_form(n_rows, n_req, max_rows_per_req, h_q, h_kv, head_dim, max_len, window, n_sink), head_dim);
}

qsa_status qsa_window_attn_fp8(const void* q, int64_t ld_q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, int64_t n_slots, int32_t block_tokens,
                               int32_t n_req, const int32_t* req_row_start, int32_t n_rows, const int32_t* row_len,
                               int32_t max_len, int32_t max_rows_per_req, int32_t h_q, int32_t h_kv, int32_t head_dim,
                               const int32_t* page_table, int64_t ld_pt, int32_t page_size, int32_t window,
                               int32_t n_sink, float scale, void* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (qsa_status st = check_window(q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, max_rows_per_req,
                                   h_q, h_kv, head_dim, page_table, ld_pt, page_size, window, n_sink, scale, out, lse,
                                   kv8_shape_ok(h_q, h_kv, head_dim)))
    return st;
  if (qsa_status st = check_block(block_tokens, n_rows > 0 ? page_size : 0, n_slots)) return st;
  if (n_rows == 0) return QSA_OK;
  if (qsa_status st = check_cache8(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  if (qsa_status st = check_workspace(qsa_window_attn_fp8_workspace_size(n_rows, n_req, max_rows_per_req, h_q, h_kv,
                                                                         head_dim, max_len, window, n_sink),
                                      workspace, workspace_bytes))
    return st;
  if (max_len > (1 << 30)) return QSA_ERR_UNSUPPORTED;  // entry indices stay clear of 2^31
  Kv8AttnArgs a{};
  set_window(a, q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, h_q, h_kv, page_table, ld_pt,
             page_size, window, n_sink, out, lse);
  set_cache(a, k_codes, k_scales, v_codes, v_scales, block_tokens);
  a.scale = scale;
  return launch_k8(window_form(n_rows, n_req, max_rows_per_req, h_q, h_kv, head_dim, max_len, window, n_sink), a, head_dim, workspace,
                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
