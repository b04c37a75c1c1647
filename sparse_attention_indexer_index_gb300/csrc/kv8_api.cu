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
#include "kv8_attn.cuh"
#include "paging.cuh"

using namespace qsa;

namespace {

// The kernel of a tile's pairs, and its shape.
struct K8Kernel {
  void (*fn)(Kv8AttnArgs);
  int threads, smem;
  int entries;  // entries of a CTA per step
};
template <int D, int P, int MT, bool kWindow>
constexpr K8Kernel k8() {
  using Sh = K8Shape<D, P, MT>;
  return {kv8_attn_kernel<D, P, MT, kWindow>, Sh::kThreads, Sh::kSmem, Sh::kStep * Sh::kGroups};
}
// Single rows of up to 8 heads to a KV head, rows of up to 16 (a list; in a
// window they are tiles of 16 pairs), tiles of 16 to 64 pairs.
enum { kList8 = 0, kList16 = 1, kWindow8 = 2, kTiles = 3, kK8Kinds = 7 };
constexpr K8Kernel kK8Kernels[kK8Kinds][2] = {
    {k8<128, 8, 1, false>(), k8<256, 8, 1, false>()},   {k8<128, 16, 1, false>(), k8<256, 16, 1, false>()},
    {k8<128, 8, 1, true>(), k8<256, 8, 1, true>()},     {k8<128, 16, 1, true>(), k8<256, 16, 1, true>()},
    {k8<128, 16, 2, true>(), k8<256, 16, 2, true>()},   {k8<128, 16, 3, true>(), k8<256, 16, 3, true>()},
    {k8<128, 16, 4, true>(), k8<256, 16, 4, true>()},
};

// Per-device one-time set-up: the shared-memory opt-in of the kernels, and
// how many of their clusters run at once.
struct Kv8Device {
  bool ready;
  int clusters[kK8Kinds][2][kKaMaxCluster + 1];
};
Kv8Device g_kv8_dev[kMaxDevices];
std::mutex g_mu;

qsa_status kv8_device(const Kv8Device** out) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QSA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  Kv8Device& d = g_kv8_dev[dev];
  if (!d.ready) {
    bool ok = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    for (int i = 0; ok && i < kK8Kinds * 2; ++i) {
      const K8Kernel& k = kK8Kernels[i / 2][i % 2];
      ok = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem) == cudaSuccess;
      for (int c = 1; ok && c <= kKaMaxCluster; ++c)
        ok = resident_clusters(k.fn, k.threads, (size_t)k.smem, c, sms, &d.clusters[i / 2][i % 2][c]);
    }
    if (!ok) {
      cudaGetLastError();
      return QSA_ERR_CUDA;
    }
    d.ready = true;
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

// How a window call is cut into tiles: single rows with up to 8 heads to a KV
// head, else as many pairs as a request's rows have, 16 to 64 a tile.
struct K8Form {
  int kind, rows;   // kernel, rows per tile
  int64_t slots;    // tiles at most
  int64_t units;    // tiles times KV heads for requests of equal length
};
K8Form window_form(int32_t n_rows, int32_t n_req, int32_t max_rows_per_req, int32_t h_q, int32_t h_kv) {
  const int group = h_q / h_kv;
  if (max_rows_per_req <= 1 && group <= 8) return {kWindow8, 1, n_rows, (int64_t)n_rows * h_kv};
  const int64_t pairs = (int64_t)std::max(max_rows_per_req, 1) * group;
  const int mt = (int)std::min<int64_t>(4, (pairs + 15) / 16);
  const int rows = 16 * mt / group;
  const int64_t per_req = ((int64_t)n_rows + n_req - 1) / n_req;
  return {kTiles + mt - 1, rows, n_rows / rows + (int64_t)n_req,
          std::min<int64_t>(n_rows, (int64_t)n_req * ((per_req + rows - 1) / rows)) * h_kv};
}

size_t part_bytes(int64_t n_rows, int32_t h_q, int32_t d, int n_group) {
  return n_group > 1 ? (size_t)(n_rows * h_q * n_group * (d + 2) * 4) : 0;
}

qsa_status launch_k8(int kind, Kv8AttnArgs& a, int d, int64_t tiles, int64_t units, int64_t entries, void* workspace,
                     cudaStream_t stream) {
  const Kv8Device* dev = nullptr;
  if (qsa_status st = kv8_device(&dev)) return st;
  const K8Kernel& k = kK8Kernels[kind][d == 256];
  a.group = a.h_q / a.h_kv;
  a.v_g = 1.0f;
  a.n_group = ka_groups(units, entries);
  a.cluster = a.n_group > 1 ? kKaMaxCluster : ka_cluster(units, entries, k.entries, dev->clusters[kind][d == 256]);
  a.part = static_cast<float*>(workspace);
  const int64_t ctas = tiles * a.cluster * a.n_group;
  if (ctas > INT32_MAX || (int64_t)a.n_rows * a.h_q > INT32_MAX) return QSA_ERR_UNSUPPORTED;
  if (entries > (1 << 30)) return QSA_ERR_UNSUPPORTED;  // entry indices stay clear of 2^31
  const ClusterLaunch l(dim3((unsigned)ctas, (unsigned)a.h_kv), k.threads, (size_t)k.smem, a.cluster, stream);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k.fn, a);
  if (e == cudaSuccess && a.n_group > 1) e = launch_merge(a, d, (float)kK8Bias, stream);
  return launched(e);
}

void set_cache(Kv8AttnArgs& a, const void* kc, const void* ks, const void* vc, const void* vs, int32_t block_tokens) {
  a.k = static_cast<const uint8_t*>(kc);
  a.v = static_cast<const uint8_t*>(vc);
  a.ks = static_cast<const uint8_t*>(ks);
  a.vs = static_cast<const uint8_t*>(vs);
  a.block_shift = log2_of(block_tokens);
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
  const StepArgs a{ctx_len, n_new, n_req, page_table, ld_pt, page_size, free_pages, n_pool, n_free,
                   n_tok, req_row_start, new_len, row_len, row_req, slots};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(plan_step_kernel, dim3(1), dim3(kStepThreads), 0, s, a);
  if (e == cudaSuccess && n_tok > kStepOneCta)
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
  return launched(launch_pdl(release_pages_kernel, dim3(1), dim3(kStepThreads), 0, static_cast<cudaStream_t>(stream), a));
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
  if (n_rows <= 0 || n_idx <= 0 || !kv8_shape_ok(h_q, h_kv, head_dim)) return 0;
  return part_bytes(n_rows, h_q, head_dim, ka_groups((int64_t)n_rows * h_kv, n_idx));
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
  a.rows = 1;
  a.out = out;
  a.lse = lse;
  return launch_k8(h_q / h_kv > 8 ? kList16 : kList8, a, head_dim, n_rows, (int64_t)n_rows * h_kv, n_idx, workspace,
                   static_cast<cudaStream_t>(stream));
}

size_t qsa_window_attn_fp8_workspace_size(int32_t n_rows, int32_t n_req, int32_t max_rows_per_req, int32_t h_q,
                                          int32_t h_kv, int32_t head_dim, int32_t max_len, int32_t window,
                                          int32_t n_sink) {
  if (n_rows <= 0 || n_req <= 0 || max_len <= 0 || window < 1 || n_sink < 0 || !kv8_shape_ok(h_q, h_kv, head_dim))
    return 0;
  const K8Form f = window_form(n_rows, n_req, max_rows_per_req, h_q, h_kv);
  return part_bytes(n_rows, h_q, head_dim, ka_groups(f.units, window_entries(max_len, window, n_sink)));
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
  const K8Form f = window_form(n_rows, n_req, max_rows_per_req, h_q, h_kv);
  Kv8AttnArgs a{};
  set_window(a, q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, h_q, h_kv, page_table, ld_pt,
             page_size, window, n_sink, out, lse);
  set_cache(a, k_codes, k_scales, v_codes, v_scales, block_tokens);
  a.scale = scale;
  a.rows = f.rows;
  return launch_k8(f.kind, a, head_dim, f.slots, f.units, window_entries(max_len, window, n_sink), workspace,
                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
