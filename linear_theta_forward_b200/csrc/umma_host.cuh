// Host side of the tensor-core launches: TMA descriptors and the one-time,
// per-context kernel set-up.
#pragma once

#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace theta {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn(cudaError_t* e) {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  static cudaError_t status = cudaSuccess;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    status = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    if (status == cudaSuccess && q != cudaDriverEntryPointSuccess) status = cudaErrorSymbolNotFound;
    fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  *e = status;
  return fn;
}

// 2-D tensor [rows, cols] of bf16 (or, elem_bytes 1, of bytes), row pitch =
// cols, box [box_rows, box_cols]; out-of-bounds elements of a box read as
// zero and are not written.
inline int make_map_box(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int box_rows, int box_cols,
                        CUtensorMapSwizzle swizzle, cudaError_t* ce, int elem_bytes = 2) {
  EncodeTiledFn enc = encode_fn(ce);
  if (!enc) return THETA_ERR_CUDA;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)cols * elem_bytes};
  cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(m, elem_bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    *ce = cudaErrorInvalidValue;
    return THETA_ERR_CUDA;
  }
  return THETA_OK;
}

// Per-context, per-kernel launch configuration: dynamic shared memory opt-in,
// non-portable cluster sizes, and the number of co-resident CTAs per SM,
// checked against tensor-memory capacity (co-resident CTAs must never need
// more columns than an SM has, or allocation would stall).
struct KernelInfo {
  bool ready = false;
  int blocks_per_sm = 0;
  int max_cluster = 1;
};

template <typename Kern>
inline cudaError_t prepare_kernel(KernelInfo* info, int device, Kern kern, int threads, int smem, int tmem_cols,
                                  bool clusters) {
  std::lock_guard<std::mutex> lk(setup_mutex());
  if (info->ready) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // all of the unified L1/shared array as shared memory: the stage rings are
  // what keeps loads in flight, and the residency count below relies on it
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  if (clusters) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  // Co-resident CTAs per SM, from shared memory (the binding limit for these
  // kernels; the occupancy API under-reports kernels that use cluster
  // instructions). Tensor memory must cover all of them, or allocation
  // would stall.
  int dev_smem = 0, reserved = 0;
  e = cudaDeviceGetAttribute(&dev_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, device);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, device);
  if (e != cudaSuccess) return e;
  int blocks = dev_smem / (smem + reserved);
  const int by_threads = 2048 / threads;
  if (blocks > by_threads) blocks = by_threads;
  if (blocks < 1) return cudaErrorInvalidConfiguration;
  if (blocks * tmem_cols > 512) blocks = 512 / tmem_cols;  // never counted on beyond tensor memory
  int api_blocks = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&api_blocks, kern, threads, smem);
  if (e != cudaSuccess) return e;
  if (api_blocks * tmem_cols > 512) return cudaErrorInvalidConfiguration;
  info->blocks_per_sm = blocks;
  info->max_cluster = 1;
  if (clusters) {
    // the largest cluster (16, else 8) that the GPU can place at all; a
    // refused query sets the thread's last error, which is cleared below only
    // when no earlier error was pending (the caller's must not be lost)
    const bool pending = cudaPeekAtLastError() != cudaSuccess;
    bool refused = false;
    for (int cs = 16; cs >= 8 && info->max_cluster == 1; cs /= 2) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(cs, 1, 1);
      cfg.blockDim = dim3(threads, 1, 1);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = cs;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      const cudaError_t q = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (q == cudaSuccess && n > 0) info->max_cluster = cs;
      if (q != cudaSuccess) refused = true;
    }
    if (refused && !pending) cudaGetLastError();  // a refused query is not an error of this call
    if (info->max_cluster == 1) return cudaErrorInvalidConfiguration;
  }
  info->ready = true;
  return cudaSuccess;
}

// Largest power-of-two split (<= 16) that keeps every CTA resident in one
// wave and leaves each split at least 4 K blocks.
inline int pick_splits(int64_t tiles, int kb, int capacity, int max_cluster) {
  int s = 1;
  while (2 * s <= max_cluster && tiles * (2 * s) <= capacity && kb / (2 * s) >= 4) s *= 2;
  return s;
}

}  // namespace theta
