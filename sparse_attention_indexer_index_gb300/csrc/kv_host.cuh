// kv_host.cuh -- host-side helpers of the calls on the K/V cache: launches,
// clusters, and the arguments that the calls share.
#pragma once
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "host_util.cuh"
#include "kv_attn.cuh"

namespace qsa {

constexpr int kMaxDevices = 64;

// A launch of clusters of c CTAs along x (c = 1: without that attribute), as
// all here a programmatic dependent one: it may be set up while the kernel
// before it in the stream ends.  Every kernel waits for that one's results
// (griddepcontrol.wait) before it touches global memory.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2] = {};
  ClusterLaunch(dim3 grid, int threads, size_t smem, int c, cudaStream_t stream) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
  }
  ClusterLaunch(const ClusterLaunch&) = delete;
};

inline qsa_status launched(cudaError_t e) {
  if (e == cudaSuccess) return QSA_OK;
  cudaGetLastError();
  return QSA_ERR_CUDA;
}

template <class F>
bool resident_clusters(F fn, int threads, size_t smem, int c, int sms, int* n) {
  if (c == 1) {  // without the attribute
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, fn, threads, smem) != cudaSuccess) return false;
    *n *= sms;
    return *n > 0;
  }
  const ClusterLaunch l(dim3((unsigned)c), threads, smem, c, nullptr);
  return cudaOccupancyMaxActiveClusters(n, fn, &l.cfg) == cudaSuccess;
}

inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

inline int64_t window_entries(int32_t max_len, int32_t window, int32_t n_sink) {
  return std::min<int64_t>(max_len, (int64_t)window + n_sink);
}

inline qsa_status check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (need == 0) return QSA_OK;
  if (!workspace || bytes < need) return QSA_ERR_WORKSPACE_TOO_SMALL;
  return aligned16(workspace) ? QSA_OK : QSA_ERR_INVALID_ARG;
}

// Arguments that the window calls share; shape_ok: heads and head dim.
inline qsa_status check_window(const void* q, int64_t ld_q, int64_t n_slots, int32_t n_req, const int32_t* req_row_start,
                        int32_t n_rows, const int32_t* row_len, int32_t max_len, int32_t max_rows_per_req, int32_t h_q,
                        int32_t h_kv, int32_t d, const int32_t* page_table, int64_t ld_pt, int32_t page_size,
                        int32_t window, int32_t n_sink, float scale, const void* out, const void* lse, bool shape_ok) {
  if (!std::isfinite(scale)) return QSA_ERR_INVALID_ARG;
  if (window < 1 || n_sink < 0 || max_rows_per_req < 0 || n_slots < 0 || n_slots > INT32_MAX) return QSA_ERR_INVALID_ARG;
  if (!shape_ok) return QSA_ERR_UNSUPPORTED;
  if (qsa_status st = check_rows(n_req, req_row_start, n_rows, row_len, max_len)) return st;
  if (n_rows == 0) return QSA_OK;
  if (qsa_status st = check_paging(page_table, ld_pt, page_size, max_len)) return st;
  if (!q || !out || !aligned16(q) || !aligned32(out) || (lse && !aligned4(lse))) return QSA_ERR_INVALID_ARG;
  if (ld_q < (int64_t)h_q * d || ld_q % 8 != 0) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

inline void set_window(KvAttnArgs& a, const void* q, int64_t ld_q, int64_t n_slots, int32_t n_req,
                const int32_t* req_row_start, int32_t n_rows, const int32_t* row_len, int32_t max_len, int32_t h_q,
                int32_t h_kv, const int32_t* page_table, int64_t ld_pt, int32_t page_size, int32_t window,
                int32_t n_sink, void* out, float* lse) {
  a.q = static_cast<const uint16_t*>(q);
  a.ld_q = ld_q;
  a.n_slots = n_slots;
  a.n_rows = n_rows;
  a.h_q = h_q;
  a.h_kv = h_kv;
  a.n_req = n_req;
  a.req_row_start = req_row_start;
  a.row_len = row_len;
  a.max_len = max_len;
  a.window = window;
  a.n_sink = n_sink;
  a.page_table = page_table;
  a.ld_pt = ld_pt;
  a.page_size = page_size;
  a.out_bf16 = 1;
  a.out = out;
  a.lse = lse;
}

}  // namespace qsa
