// kv_api.cu -- the extern "C" entry points of the 4-bit KV cache and of the
// attention over a window: host-side argument checks, launch shapes, and
// launches on the caller's stream.  Contracts are in include/qsa.h.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "../../include/qsa.h"
#include "common.cuh"
#include "host_util.cuh"
#include "kv_host.cuh"
#include "kv4.cuh"
#include "kv_attn.cuh"
#include "kv4_attn.cuh"
#include "window_tc.cuh"

using namespace qsa;

namespace {

// The kernel of a cache type, head dim and head tiles, and its shape.
struct KaKernel {
  void (*fn)(KvAttnArgs);
  int threads;
  size_t smem;
  int entries;  // entries of a CTA per step
};
template <int D, int NT>
constexpr KaKernel ka_bf16() {
  return {kv_attn_kernel<D, NT>, kKaThreads, ka_smem_bytes<D, NT>(), kKaTile * kKaWarps};
}
template <int D, int NT, bool kWindow>
constexpr KaKernel ka_fp4() {
  return {kv4_attn_kernel<D, NT, kWindow>, kK4Threads, k4_smem_bytes<D, NT>(), kK4Step * kK4Warps};
}
// [cache: BF16 window, 4-bit window, 4-bit list][D = 128 with up to 8 heads, up to 16, D = 256]
const KaKernel kKaKernels[3][3] = {
    {ka_bf16<128, 1>(), ka_bf16<128, 2>(), ka_bf16<256, 1>()},
    {ka_fp4<128, 1, true>(), ka_fp4<128, 2, true>(), ka_fp4<256, 1, true>()},
    {ka_fp4<128, 1, false>(), ka_fp4<128, 2, false>(), ka_fp4<256, 1, false>()},
};
bool set_ka_smem() {
  for (const auto& row : kKaKernels)
    for (const KaKernel& k : row)
      if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem) != cudaSuccess)
        return false;
  return true;
}

// Per-device one-time set-up: the shared-memory opt-in of the kernels, and
// how many of their clusters run at once.
constexpr int kWtMaxCluster = 8;
struct KvDevice {
  int sms;                             // 0: not set up
  int ka[3][3][kKaMaxCluster + 1];     // clusters of c CTAs at once
  int wt[2][kWtMaxCluster + 1];        // D = 128, D = 256
};
KvDevice g_kv_dev[kMaxDevices];
std::mutex g_mu;

bool set_up(KvDevice& d, int sms) {
  if (!set_ka_smem() ||
      cudaFuncSetAttribute(window_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, wt_smem_bytes<128>()) != cudaSuccess ||
      cudaFuncSetAttribute(window_tc_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, wt_smem_bytes<256>()) != cudaSuccess)
    return false;
  for (int i = 0; i < 9; ++i) {
    const KaKernel& k = kKaKernels[i / 3][i % 3];
    for (int c = 1; c <= kKaMaxCluster; ++c)
      if (!resident_clusters(k.fn, k.threads, k.smem, c, sms, &d.ka[i / 3][i % 3][c])) return false;
  }
  for (int c = 1; c <= kWtMaxCluster; c *= 2)
    if (!resident_clusters(window_tc_kernel<128>, kWtThreads, wt_smem_bytes<128>(), c, sms, &d.wt[0][c]) ||
        !resident_clusters(window_tc_kernel<256>, kWtThreads, wt_smem_bytes<256>(), c, sms, &d.wt[1][c]))
      return false;
  return true;
}

qsa_status kv_device(const KvDevice** out) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QSA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  KvDevice& d = g_kv_dev[dev];
  if (d.sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !set_up(d, sms)) {
      cudaGetLastError();
      return QSA_ERR_CUDA;
    }
    d.sms = sms;
  }
  *out = &d;
  return QSA_OK;
}

// A tensor scale: a positive power of two between 2^-64 and 2^63.
bool scale_ok(float g) {
  int e = 0;
  return std::isfinite(g) && g > 0.f && std::frexp(g, &e) == 0.5f && e >= -63 && e <= 64;
}

// Heads and head dims of the calls here: 128 with up to 16 query heads per
// KV head, 256 with up to 8.
bool kv_shape_ok(int32_t h_q, int32_t h_kv, int32_t d) {
  if (h_q <= 0 || h_kv <= 0 || h_kv > 65535 || h_q % h_kv != 0) return false;
  const int group = h_q / h_kv;
  return (d == 128 && group <= 16) || (d == 256 && group <= 8);
}

// Clusters per (row, KV head).  One, unless the clusters of 8 CTAs are too
// few to fill the GPU and a row is long enough to pay for the merge launch.
// The size of the workspace follows from it, so it depends on the arguments
// alone (152 SMs, two CTAs each).
int ka_groups(int64_t units, int64_t entries) {
  const int64_t fill = 304 / (units * kKaMaxCluster);
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(fill, 16), entries / 4096));
}

// CTAs per cluster: the least of waves * (steps + start and end, about 4).
// How many clusters run at once is the device's answer: on 152 SMs, 16
// clusters of 7 do not where a CTA fills an SM (1,028 entries of D = 256: 23.7
// us, in clusters of 6, which do, 17.6).
int ka_cluster(int64_t units, int64_t entries, const KaKernel& k, const int* resident) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int c = 1; c <= kKaMaxCluster && resident[c] > 0; ++c) {
    const int64_t waves = (units + resident[c] - 1) / resident[c];
    const int64_t steps = (entries + (int64_t)k.entries * c - 1) / ((int64_t)k.entries * c);
    const int64_t cost = waves * (steps + 4);
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

enum { kKaBf16Window = 0, kKaFp4Window = 1, kKaFp4List = 2 };

qsa_status launch_ka(int cache, KvAttnArgs& a, int d, int64_t entries, void* workspace, cudaStream_t stream) {
  const int64_t units = (int64_t)a.n_rows * a.h_kv;
  a.group = a.h_q / a.h_kv;
  const int shape = d == 256 ? 2 : a.group > 8 ? 1 : 0;
  const KaKernel& k = kKaKernels[cache][shape];
  const KvDevice* dev = nullptr;
  if (qsa_status st = kv_device(&dev)) return st;
  a.n_group = ka_groups(units, entries);
  a.cluster = a.n_group > 1 ? kKaMaxCluster : ka_cluster(units, entries, k, dev->ka[cache][shape]);
  a.part = static_cast<float*>(workspace);
  if ((int64_t)a.n_rows * std::max(a.cluster * a.n_group, a.h_q) > INT32_MAX) return QSA_ERR_UNSUPPORTED;
  if (entries > (1 << 30)) return QSA_ERR_UNSUPPORTED;  // entry indices stay clear of 2^31
  const ClusterLaunch l(dim3((unsigned)((int64_t)a.n_rows * a.cluster * a.n_group), (unsigned)a.h_kv), k.threads, k.smem,
                        a.cluster, stream);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, k.fn, a);
  if (e == cudaSuccess && a.n_group > 1)
    e = launch_pdl(d == 256 ? kv_attn_merge_kernel<256> : kv_attn_merge_kernel<128>,
                   dim3((unsigned)((int64_t)a.n_rows * a.h_q)), dim3((unsigned)d), 0, stream, a,
                   cache == kKaBf16Window ? 0.0f : (float)kK4Bias);
  return launched(e);
}

// The cache [n_slots][h_kv * D] BF16 for window_tc_kernel, as [row / 8][64
// columns][row % 8][64 BF16], 128-byte swizzled: a box takes `box` rows and
// `groups` groups of 64 columns; 8-row groups past the end read as zeros.
bool encode_cache_map(CUtensorMap* m, const void* cache, int64_t n_slots, int64_t cols, int box, int groups) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {64, 8, (cuuint64_t)cols / 64, (cuuint64_t)n_slots / 8};
  const cuuint64_t strides[3] = {(cuuint64_t)cols * 2, 128, (cuuint64_t)cols * 16};
  const cuuint32_t bx[4] = {64, 8, (cuuint32_t)groups, (cuuint32_t)box / 8};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(cache), dims, strides, bx, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries [n_rows][h_q][D]: a tile's rows x the heads of a KV head x 64
// columns a box; rows past the end read as zeros.
bool encode_q_map(CUtensorMap* m, const WtArgs& a, int d) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)a.h_q, (cuuint64_t)a.n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)a.ld_q * 2};
  const cuuint32_t bx[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), dims, strides, bx, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs that share a tile, where there are few: a single tile of 9 blocks takes
// 19.8 us on one CTA, 17.9 on two, 14.8 on four, 13.7 on eight, one of 33
// blocks 51.3, 33.6, 22.8 and 17.9 (in a graph), as long as all clusters run at
// once (16 tiles of 9 blocks: 27.0 us in eights, which do not, 15.1 in fours).
// From 65 tiles on, one CTA a tile, launched without the
// cluster attribute: sharing the last round's gained nothing (the 512 tiles of
// a 4,096-row chunk: 85 us either way at the time), and a cluster launch cost 1 us.  How
// many tiles there are is known on the device only; the estimate takes
// requests of equal length.
int wt_cluster(const WtArgs& a, const int* resident) {
  if (a.n_req > kWtExactReq) return 1;
  const int64_t per_req = ((int64_t)a.n_rows + a.n_req - 1) / a.n_req;
  const int64_t tiles = a.n_req * ((per_req + a.rows - 1) / a.rows) * a.h_kv;
  const int64_t blocks = (std::min<int64_t>(a.max_len, (int64_t)a.window + a.n_sink + a.rows) + kWtN - 1) / kWtN;
  int c = 1;
  while (c < kWtMaxCluster && tiles <= std::min(64, resident[2 * c]) && blocks >= std::max(4, 2 * c)) c *= 2;
  return c;
}

// Where rows share a tile of keys the tensor cores win, except on little work,
// where the form for single rows starts and ends sooner and spreads over more
// SMs: of window 1,024 and D = 256, 2 KV heads (in a graph, single-row form
// against this one) 1 request of 6 rows 7.8 against 14.0 us, 8 of 2 10.0
// against 14.4, 8 of 4 15.0 against 14.5, 32 of 3 45 against 23, 32 of 6 69
// against 24; of window 4,096 8 of 4 43 against 25; of window 128 8 of 6 7.2
// against 11.0, 32 of 6 20.3 against 11.3.  The line is drawn through the
// columns that the single rows would read of K, in one round of CTAs, for up
// to 16 rows a request.
//
// One row a request shares no keys: the single-row form, whatever the work.
// Single-row form / this one in us, in a graph, 1, 8, 32, 64, 128 requests:
//   D = 256, window 128     6.0/10.6   6.1/10.9   6.9/11.0   7.5/13.6  16.6/23.0
//            window 1,024   7.7/13.3   8.0/14.3  18.0/22.6  27.2/31.1  53.1/54.6
//            window 4,096  14.2/17.3  19.2/24.6  46.8/50.4  83.5/86.3   171/167
//   D = 128, window 128     4.5/9.2    4.5/9.5    5.5/10.2   5.6/16.7  12.2/29.2
//            window 1,024   5.9/12.0   6.7/13.4  15.9/21.3  24.7/35.4  46.7/62.6
//            window 4,096   9.6/15.7  15.8/23.4  44.2/49.4  80.6/97.5   158/192
// (2 KV heads of D = 256, 4 of 128.)
constexpr int kWtFewRows = 16;
constexpr int64_t kWtFewColumns = 20 << 20;
bool wt_serves(const KvAttnArgs& k, int d, int32_t max_rows_per_req, int64_t entries) {
  if (max_rows_per_req <= 1 || k.page_size % 8 != 0 || k.n_slots < 8) return false;
  const int64_t units = (int64_t)k.n_rows * k.h_kv;
  return max_rows_per_req > kWtFewRows || units > 152 * (256 / d) ||
         units * d > kWtFewColumns / std::max<int64_t>(1, entries);
}

// The tensor-core form of window_attn; QSA_ERR_UNSUPPORTED where it cannot serve.
qsa_status launch_window_tc(const KvAttnArgs& k, int d, cudaStream_t stream) {
  WtArgs a{};
  a.q = k.q;
  a.k = reinterpret_cast<const uint16_t*>(k.k);
  a.v = reinterpret_cast<const uint16_t*>(k.v);
  a.ld_q = k.ld_q;
  a.n_slots = k.n_slots;
  a.n_rows = k.n_rows;
  a.h_q = k.h_q;
  a.h_kv = k.h_kv;
  a.group = k.h_q / k.h_kv;
  a.rows = 128 / a.group;
  a.n_req = k.n_req;
  a.req_row_start = k.req_row_start;
  a.row_len = k.row_len;
  a.max_len = k.max_len;
  a.window = k.window;
  a.n_sink = k.n_sink;
  a.page_table = k.page_table;
  a.ld_pt = k.ld_pt;
  a.page_size = k.page_size;
  a.box_shift = 3;
  while (a.box_shift < 6 && k.page_size % (2 << a.box_shift) == 0) ++a.box_shift;
  a.box = 1 << a.box_shift;
  a.tile_slots = k.n_rows / a.rows + k.n_req;
  a.c = std::max(std::fabs(k.scale) * 1.4426950408889634f, 1e-30f);
  a.flip = k.scale < 0.f ? 0x80000000u : 0u;
  a.out = static_cast<uint16_t*>(k.out);
  a.lse = k.lse;
  // the longest wait is for a whole tile: blocks of 128 entries at about a microsecond, with room
  a.wait_ms = 200 + k.max_len / 4096;
  const int64_t units = (int64_t)a.tile_slots * a.h_kv;
  if (units > (1 << 30) || k.max_len > (1 << 30)) return QSA_ERR_UNSUPPORTED;
  const KvDevice* dev = nullptr;
  if (qsa_status st = kv_device(&dev)) return st;
  CUtensorMap q_map, k_map, v_map;
  if (!encode_q_map(&q_map, a, d) || !encode_cache_map(&k_map, k.k, k.n_slots, (int64_t)k.h_kv * d, a.box, 2) ||
      !encode_cache_map(&v_map, k.v, k.n_slots, (int64_t)k.h_kv * d, a.box, d / 64))
    return QSA_ERR_UNSUPPORTED;
  a.cluster = wt_cluster(a, dev->wt[d == 256]);
  const ClusterLaunch l(dim3((unsigned)(std::min<int64_t>(units, dev->sms / a.cluster) * a.cluster)), kWtThreads,
                        d == 256 ? wt_smem_bytes<256>() : wt_smem_bytes<128>(), a.cluster, stream);
  return launched(cudaLaunchKernelEx(&l.cfg, d == 256 ? window_tc_kernel<256> : window_tc_kernel<128>, a, q_map, k_map,
                                     v_map));
}

size_t ka_workspace(int64_t n_rows, int32_t h_q, int32_t h_kv, int32_t d, int64_t entries) {
  if (n_rows <= 0 || entries <= 0 || !kv_shape_ok(h_q, h_kv, d)) return 0;
  const int ng = ka_groups(n_rows * h_kv, entries);
  return ng > 1 ? (size_t)(n_rows * h_q * ng * (d + 2) * 4) : 0;
}

// The 4-bit cache's four arrays (any of them may be NULL with n_slots 0).
qsa_status check_cache4(const void* kc, const void* ks, const void* vc, const void* vs, int64_t n_slots) {
  if (n_slots < 0 || n_slots > INT32_MAX) return QSA_ERR_INVALID_ARG;
  if (n_slots > 0 && (!kc || !ks || !vc || !vs)) return QSA_ERR_INVALID_ARG;
  return aligned16(kc) && aligned16(ks) && aligned16(vc) && aligned16(vs) ? QSA_OK : QSA_ERR_INVALID_ARG;
}

}  // namespace

namespace qsa {
bool kv_fault_word(cudaStream_t stream, bool clear, unsigned* bits) {
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

qsa_status qsa_append_kv_fp4(const void* k_new, const void* v_new, int64_t ld_k, int64_t ld_v, int32_t n_tok,
                             int32_t h_kv, int32_t head_dim, const int32_t* req_tok_start,
                             const int32_t* req_first_pos, int32_t n_req, const int32_t* page_table, int64_t ld_pt,
                             int32_t page_size, float k_scale, float v_scale, void* k_codes, void* k_scales,
                             void* v_codes, void* v_scales, int64_t n_slots, void* stream) {
  if (n_tok < 0 || n_req < 0 || h_kv <= 0) return QSA_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || h_kv > 65535 || n_req > 65535) return QSA_ERR_UNSUPPORTED;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return QSA_ERR_INVALID_ARG;
  if (n_tok == 0 || n_req == 0) return QSA_OK;
  if (!k_new || !v_new || !req_tok_start || !req_first_pos) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_paging(page_table, ld_pt, page_size, 0)) return st;
  if (qsa_status st = check_cache4(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  const int64_t row = (int64_t)h_kv * head_dim;
  if (!aligned32(k_new) || !aligned32(v_new) || ld_k % 16 != 0 || ld_v % 16 != 0 || ld_k < row || ld_v < row)
    return QSA_ERR_INVALID_ARG;
  KvWriteArgs a{};
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.n_tok = n_tok;
  a.h_kv = h_kv;
  a.blocks = h_kv * (head_dim / kKvBlock);
  a.req_tok_start = req_tok_start;
  a.req_first_pos = req_first_pos;
  a.n_req = n_req;
  a.page_table = page_table;
  a.ld_pt = ld_pt;
  a.page_size = page_size;
  a.n_slots = n_slots;
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.k_scales = static_cast<uint8_t*>(k_scales);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.v_scales = static_cast<uint8_t*>(v_scales);
  a.k_inv = 1.0f / k_scale;
  a.v_inv = 1.0f / v_scale;
  const int64_t units = (int64_t)n_tok * a.blocks;
  if (units > (int64_t)UINT32_MAX - 4 * kKvThreads) return QSA_ERR_UNSUPPORTED;  // counted in 32 bits
  const ClusterLaunch l(dim3((unsigned)((units + kKvThreads - 1) / kKvThreads)), kKvThreads, 0, 1,
                        static_cast<cudaStream_t>(stream));
  return launched(cudaLaunchKernelEx(&l.cfg, append_kv_fp4_kernel, a));
}

qsa_status qsa_gather_kv_fp4(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                             int64_t n_slots, int32_t h_kv, int32_t head_dim, const int32_t* slots, int64_t n,
                             float k_scale, float v_scale, void* k_out, void* v_out, void* stream) {
  if (n < 0 || h_kv <= 0) return QSA_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || h_kv > 65535) return QSA_ERR_UNSUPPORTED;
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return QSA_ERR_INVALID_ARG;
  if (n == 0) return QSA_OK;
  if (!slots || !k_out || !v_out || !aligned4(slots) || !aligned32(k_out) || !aligned32(v_out))
    return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_cache4(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  KvReadArgs a{};
  a.k_codes = static_cast<const uint8_t*>(k_codes);
  a.k_scales = static_cast<const uint8_t*>(k_scales);
  a.v_codes = static_cast<const uint8_t*>(v_codes);
  a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.n_slots = n_slots;
  a.blocks = h_kv * (head_dim / kKvBlock);
  a.slots = slots;
  a.n = n;
  a.k_g = k_scale;
  a.v_g = v_scale;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  // blocks are counted in 32 bits (2^32 of them would be 137 GB of output each)
  if (n > (int64_t)(UINT32_MAX - 4 * kKvThreads) / a.blocks) return QSA_ERR_UNSUPPORTED;
  const int64_t ctas = (n * a.blocks + kKvThreads - 1) / kKvThreads;
  const ClusterLaunch l(dim3((unsigned)ctas), kKvThreads, 0, 1, static_cast<cudaStream_t>(stream));
  return launched(cudaLaunchKernelEx(&l.cfg, gather_kv_fp4_kernel, a));
}

size_t qsa_sparse_attn_fp4_workspace_size(int32_t n_rows, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t n_idx) {
  return ka_workspace(n_rows, h_q, h_kv, head_dim, n_idx);
}

qsa_status qsa_sparse_attn_fp4(const void* q, int64_t ld_q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, int64_t n_slots, int32_t n_rows, int32_t h_q,
                               int32_t h_kv, int32_t head_dim, const int32_t* slots, int64_t ld_slots, int32_t n_idx,
                               float scale, float k_scale, float v_scale, float* out, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (n_rows < 0 || n_idx < 0 || ld_slots < n_idx) return QSA_ERR_INVALID_ARG;
  if (!kv_shape_ok(h_q, h_kv, head_dim)) return QSA_ERR_UNSUPPORTED;
  if (!scale_ok(k_scale) || !scale_ok(v_scale) || !std::isfinite(scale)) return QSA_ERR_INVALID_ARG;
  if (n_rows == 0) return QSA_OK;
  if (!q || !out || (n_idx > 0 && !slots) || !aligned16(q) || !aligned16(out) || (lse && !aligned4(lse)) ||
      !aligned4(slots))
    return QSA_ERR_INVALID_ARG;
  if (ld_q < (int64_t)h_q * head_dim || ld_q % 8 != 0) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_cache4(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  if (qsa_status st = check_workspace(ka_workspace(n_rows, h_q, h_kv, head_dim, n_idx), workspace, workspace_bytes))
    return st;
  KvAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.ld_q = ld_q;
  a.k = static_cast<const uint8_t*>(k_codes);
  a.v = static_cast<const uint8_t*>(v_codes);
  a.ks = static_cast<const uint8_t*>(k_scales);
  a.vs = static_cast<const uint8_t*>(v_scales);
  a.n_slots = n_slots;
  a.n_rows = n_rows;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.slots = slots;
  a.ld_slots = ld_slots;
  a.n_idx = n_idx;
  a.scale = scale * k_scale;
  a.v_g = v_scale;
  a.out = out;
  a.lse = lse;
  return launch_ka(kKaFp4List, a, head_dim, n_idx, workspace, static_cast<cudaStream_t>(stream));
}

size_t qsa_window_attn_workspace_size(int32_t n_rows, int32_t h_q, int32_t h_kv, int32_t head_dim, int32_t max_len,
                                      int32_t window, int32_t n_sink) {
  if (window < 1 || n_sink < 0) return 0;
  return ka_workspace(n_rows, h_q, h_kv, head_dim, window_entries(max_len, window, n_sink));
}

qsa_status qsa_window_attn(const void* q, int64_t ld_q, const void* k_cache, const void* v_cache, int64_t n_slots,
                           int32_t n_req, const int32_t* req_row_start, int32_t n_rows, const int32_t* row_len,
                           int32_t max_len, int32_t max_rows_per_req, int32_t h_q, int32_t h_kv, int32_t head_dim,
                           const int32_t* page_table, int64_t ld_pt, int32_t page_size, int32_t window, int32_t n_sink,
                           float scale, void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (qsa_status st = check_window(q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, max_rows_per_req,
                                   h_q, h_kv, head_dim, page_table, ld_pt, page_size, window, n_sink, scale, out,
                                   lse, kv_shape_ok(h_q, h_kv, head_dim)))
    return st;
  if (n_rows == 0) return QSA_OK;
  if ((n_slots > 0 && (!k_cache || !v_cache)) || !aligned16(k_cache) || !aligned16(v_cache)) return QSA_ERR_INVALID_ARG;
  const int64_t entries = window_entries(max_len, window, n_sink);
  if (qsa_status st = check_workspace(ka_workspace(n_rows, h_q, h_kv, head_dim, entries), workspace, workspace_bytes))
    return st;
  KvAttnArgs a{};
  set_window(a, q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, h_q, h_kv, page_table, ld_pt,
             page_size, window, n_sink, out, lse);
  a.k = static_cast<const uint8_t*>(k_cache);
  a.v = static_cast<const uint8_t*>(v_cache);
  a.scale = scale;
  a.v_g = 1.0f;
  if (wt_serves(a, head_dim, max_rows_per_req, entries)) {
    const qsa_status tc = launch_window_tc(a, head_dim, static_cast<cudaStream_t>(stream));
    if (tc != QSA_ERR_UNSUPPORTED) return tc;
  }
  return launch_ka(kKaBf16Window, a, head_dim, entries, workspace, static_cast<cudaStream_t>(stream));
}

qsa_status qsa_window_attn_fp4(const void* q, int64_t ld_q, const void* k_codes, const void* k_scales,
                               const void* v_codes, const void* v_scales, int64_t n_slots, int32_t n_req,
                               const int32_t* req_row_start, int32_t n_rows, const int32_t* row_len, int32_t max_len,
                               int32_t max_rows_per_req, int32_t h_q, int32_t h_kv, int32_t head_dim,
                               const int32_t* page_table, int64_t ld_pt, int32_t page_size, int32_t window,
                               int32_t n_sink, float scale, float k_scale, float v_scale, void* out, float* lse,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!scale_ok(k_scale) || !scale_ok(v_scale)) return QSA_ERR_INVALID_ARG;
  if (qsa_status st = check_window(q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, max_rows_per_req,
                                   h_q, h_kv, head_dim, page_table, ld_pt, page_size, window, n_sink, scale, out,
                                   lse, kv_shape_ok(h_q, h_kv, head_dim)))
    return st;
  if (n_rows == 0) return QSA_OK;
  if (qsa_status st = check_cache4(k_codes, k_scales, v_codes, v_scales, n_slots)) return st;
  const int64_t entries = window_entries(max_len, window, n_sink);
  if (qsa_status st = check_workspace(ka_workspace(n_rows, h_q, h_kv, head_dim, entries), workspace, workspace_bytes))
    return st;
  KvAttnArgs a{};
  set_window(a, q, ld_q, n_slots, n_req, req_row_start, n_rows, row_len, max_len, h_q, h_kv, page_table, ld_pt,
             page_size, window, n_sink, out, lse);
  a.k = static_cast<const uint8_t*>(k_codes);
  a.v = static_cast<const uint8_t*>(v_codes);
  a.ks = static_cast<const uint8_t*>(k_scales);
  a.vs = static_cast<const uint8_t*>(v_scales);
  a.scale = scale * k_scale;
  a.v_g = v_scale;
  return launch_ka(kKaFp4Window, a, head_dim, entries, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
