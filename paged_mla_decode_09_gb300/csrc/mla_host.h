// Host helpers of the newer entry points: alignment and device checks and the
// tensor maps over cache and query rows.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <mutex>
#include <utility>

#include "mla_decode.h"

namespace mla {
namespace host {

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int device_ok(int device) {
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess) {
    cudaGetLastError();
    return MLA_ERR_CUDA;
  }
  return major == 10 && minor == 3 ? MLA_OK : MLA_ERR_DEVICE;
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A 3-D map over rows of `row_bytes`: (128 bytes of a row, rows, 128-byte
// columns), read in boxes of 128 bytes x box_rows x box_cols that land as
// [column][row][128 bytes] with the 128-byte swizzle.
inline bool map3(CUtensorMap* m, const void* base, int64_t rows, int row_bytes, int esz, int cols, int box_rows, int box_cols) {
  cuuint64_t gdim[3] = {static_cast<cuuint64_t>(128 / esz), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(cols)};
  cuuint64_t gstr[2] = {static_cast<cuuint64_t>(row_bytes), 128};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / esz), static_cast<cuuint32_t>(box_rows),
                       static_cast<cuuint32_t>(box_cols)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode_fn()(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                     const_cast<void*>(base), gdim, gstr, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
inline bool map2(CUtensorMap* m, const void* base, int64_t rows, int width, int esz, int box_x, int box_rows,
          CUtensorMapSwizzle swz) {
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstr[1] = {static_cast<cuuint64_t>(width) * esz};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_x), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  return encode_fn()(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : (esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16), 2,
                     const_cast<void*>(base), gdim, gstr, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// scale * log2(e) * kv_scale rounded to fp32 once: the factor of every score,
// so that its error (2^-24 relative) is that of one rounding.  It has to be
// finite and above 0: 0 times an infinity, of a masked score or of the factor,
// is a NaN.
inline float log2_scale(float scale, float kv_scale) {
  return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074 * static_cast<double>(kv_scale));
}
inline bool scale_ok(float scale, float kv_scale, bool f8) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return false;
  if (f8 && (!(kv_scale > 0.f) || !std::isfinite(kv_scale))) return false;
  const float c = log2_scale(scale, f8 ? kv_scale : 1.f);
  return c > 0.f && std::isfinite(c);
}

// Launches a kernel with programmatic stream serialization: it may begin while
// the kernel before it in the stream ends, and waits for that one's results
// (griddep_wait) before it touches any.  Kernels that begin a call do so at
// their very start, before they let the call's next kernel launch.
template <typename... Params, typename... Args>
inline cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                              unsigned cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Raises a kernel's dynamic shared memory limit, once per device.
template <int kTag, typename Kernel>
inline cudaError_t allow_smem(Kernel* kernel, int bytes, int device) {
  static std::mutex mu;
  static bool done[64] = {};
  std::lock_guard<std::mutex> lk(mu);
  if (device >= 0 && device < 64 && done[device]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && device >= 0 && device < 64) done[device] = true;
  return e;
}

}  // namespace host
}  // namespace mla
