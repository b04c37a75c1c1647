// host_util.cuh -- host-side helpers shared by the library's translation
// units: argument checks, launches, the tensor-map encoder.
#pragma once
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "../../include/qsa.h"
#include "common.cuh"

namespace qsa {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Launch with programmatic stream serialisation: the grid may become
// resident before the previous kernel on the stream finishes; every kernel
// launched this way executes griddepcontrol.wait before reading its inputs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// cuTensorMapEncodeTiled, reached through the runtime's driver entry point
// (the library does not link libcuda directly).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

inline qsa_status check_rows(int32_t n_req, const int32_t* req_row_start, int32_t n_rows,
                      const int32_t* row_len, int32_t max_len) {
  if (n_req < 0 || n_rows < 0 || max_len < 0) return QSA_ERR_INVALID_ARG;
  if (n_rows > 0 && (n_req < 1 || !req_row_start || !row_len)) return QSA_ERR_INVALID_ARG;
  if (n_req > 65535) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

inline qsa_status check_paging(const int32_t* page_table, int64_t ld_pt, int32_t page_size,
                        int32_t max_len) {
  if (!page_table || page_size <= 0 || ld_pt < 0) return QSA_ERR_INVALID_ARG;
  if (page_size % kBlock != 0) return QSA_ERR_UNSUPPORTED;
  if (max_len > 0 && (int64_t)(max_len - 1) / page_size >= ld_pt) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

// Fault word of kv_api.cu's kernels: read into *bits, and cleared if asked
// and non-zero; synchronises the stream.
bool kv_fault_word(cudaStream_t stream, bool clear, unsigned* bits);

}  // namespace qsa
