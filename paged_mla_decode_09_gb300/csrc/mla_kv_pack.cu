// The cache write that precedes a decode step (see include/mla_kv_pack.h):
// the new tokens' latent rows, quantised to e4m3 (or copied for a bf16
// cache), scattered through the page table.  One warp per 4 rows: a row is
// 72 chunks of 16 bytes (8 bf16 values), so each lane reads and writes 9
// chunks, all loads first; the kernel streams at close to the copy rate of
// HBM.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "mla_e4m3.cuh"
#include "mla_kv_pack.h"

namespace {

constexpr int kRowVals = 576;              // c_kv (512) | k_pe (64)
constexpr int kPageRows = 64;              // tokens per page
constexpr int kChunks = kRowVals * 2 / 16;  // 16-byte chunks of a bf16 row
constexpr int kRowsPerWarp = 4;            // 4 x 72 chunks = 9 per lane
constexpr int kPer = kRowsPerWarp * kChunks / 32;
constexpr int kWarps = 8;                  // warps per block

__device__ __forceinline__ uint4 ldg_nc_v4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<uint64_t>(p)));
  return v;
}

}  // namespace

namespace mla {

template <bool kF8>
__global__ void __launch_bounds__(kWarps * 32)
    mla_kv_pack_kernel(const uint4* __restrict__ rows, const int32_t* __restrict__ page_table,
                       const int32_t* __restrict__ seq_lens, int batch, int num_new, int num_pages, int max_pages,
                       int stride, e4m3::Scale sc, uint8_t* __restrict__ cache, int32_t* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t nrows = static_cast<int64_t>(batch) * num_new;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRowsPerWarp;
  if (row0 >= nrows) return;
  // lanes 0..3 find the cache slot of rows row0 .. row0 + 3 (-1: not written)
  int64_t my_slot = -1;
  if (lane < kRowsPerWarp && row0 + lane < nrows) {
    const int64_t row = row0 + lane;
    const int b = static_cast<int>(row / num_new), i = static_cast<int>(row % num_new);
    const int L = seq_lens[b];
    if (L < num_new || L > max_pages * kPageRows) {
      atomicOr(status, MLA_DEV_BAD_SEQ_LEN);
    } else {
      const int t = L - num_new + i;  // position of the token in its sequence
      const int page = page_table[static_cast<int64_t>(b) * stride + t / kPageRows];
      if (page < 0 || page >= num_pages) atomicOr(status, MLA_DEV_BAD_PAGE_ID);
      else my_slot = static_cast<int64_t>(page) * kPageRows + t % kPageRows;
    }
  }
  // chunk c = lane + 32 k of the warp's 4 rows (they are contiguous in the
  // input): row c / 72, chunk c % 72 of it; all loads first
  const uint4* src = rows + row0 * kChunks;
  const int64_t avail = (nrows - row0) * kChunks;  // chunks of this warp that exist
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (lane + 32 * k < avail) v[k] = ldg_nc_v4(src + lane + 32 * k);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int c = lane + 32 * k;
    const int rq = c / kChunks, cc = c % kChunks;
    const int64_t sl = __shfl_sync(0xffffffffu, my_slot, rq);  // the slot of this chunk's row
    if (c >= avail || sl < 0) continue;
    if constexpr (kF8) {
      reinterpret_cast<uint2*>(cache + sl * kRowVals)[cc] = e4m3::e4m3x8(v[k], sc);  // 8 codes per chunk
    } else {
      reinterpret_cast<uint4*>(cache + sl * kRowVals * 2)[cc] = v[k];
    }
  }
}

}  // namespace mla

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" int mla_kv_pack(const mla_kv_pack_dims* d, const void* rows, const int32_t* page_table,
                           const int32_t* seq_lens, float kv_scale, void* kv_cache, int32_t* status, void* stream) {
  if (!d || !rows || !page_table || !seq_lens || !kv_cache || !status) return MLA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->num_new < 1 || d->num_pages < 1 || d->max_pages_per_req < 1 ||
      d->page_table_stride < d->max_pages_per_req)
    return MLA_ERR_INVALID_ARG;
  if (d->kv_dtype != MLA_KV_BF16 && d->kv_dtype != MLA_KV_FP8_E4M3) return MLA_ERR_UNSUPPORTED;
  const bool f8 = d->kv_dtype == MLA_KV_FP8_E4M3;
  if (f8 && !mla::e4m3::scale_ok(kv_scale)) return MLA_ERR_INVALID_ARG;
  if (!aligned(rows, 16) || !aligned(kv_cache, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(status, 4))
    return MLA_ERR_ALIGNMENT;
  if (static_cast<int64_t>(d->max_pages_per_req) * kPageRows > INT_MAX) return MLA_ERR_INVALID_ARG;
  const int64_t n = static_cast<int64_t>(d->batch) * d->num_new;
  const int64_t blocks = (n + kWarps * kRowsPerWarp - 1) / (kWarps * kRowsPerWarp);
  if (blocks > INT_MAX) return MLA_ERR_INVALID_ARG;
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (major != 10 || minor != 3) return MLA_ERR_DEVICE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const mla::e4m3::Scale sc = mla::e4m3::scale_of(f8 ? kv_scale : 1.0f);
  const uint4* src = static_cast<const uint4*>(rows);
  uint8_t* dst = static_cast<uint8_t*>(kv_cache);
  if (f8)
    mla::mla_kv_pack_kernel<true><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(
        src, page_table, seq_lens, d->batch, d->num_new, d->num_pages, d->max_pages_per_req, d->page_table_stride,
        sc, dst, status);
  else
    mla::mla_kv_pack_kernel<false><<<static_cast<unsigned>(blocks), kWarps * 32, 0, s>>>(
        src, page_table, seq_lens, d->batch, d->num_new, d->num_pages, d->max_pages_per_req, d->page_table_stride,
        sc, dst, status);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
