// What the handle-free operators (grouped_gemm.cu, nvfp4_gemv.cu) share on
// the host: the current device's properties, looked up once, and tensor maps
// (whose encoder moe_api.cu uses, too).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_b200.h"

namespace moe {

constexpr int kMaxDevices = 64;

inline bool aligned_to(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// The current device and its SM count; MOE_ERR_DEVICE when none is current
// or it is not sm_100.
inline moe_status current_device(int* dev, int* sms) {
  static std::atomic<int> cached[kMaxDevices];  // SM count, -1 = not sm_100, 0 = not looked up
  if (cudaGetDevice(dev) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_DEVICE;
  }
  if (*dev < 0 || *dev >= kMaxDevices) return MOE_ERR_DEVICE;
  int n = cached[*dev].load(std::memory_order_relaxed);
  if (n == 0) {
    int major = 0, count = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_DEVICE;
    }
    n = major == 10 && count > 1 ? count : -1;
    cached[*dev].store(n, std::memory_order_relaxed);
  }
  if (n < 0) return MOE_ERR_DEVICE;
  *sms = n;
  return MOE_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_tiled() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Encodes a map.  The driver's call wants a current context, which a host
// thread has only once a runtime call bound the device's primary one to it:
// without one, bind it and try again.
template <typename F>
inline bool encode_bound(const F& encode) {
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    r = encode();
  }
  return r == CUDA_SUCCESS;
}

// 3-D map of a row-major tensor [groups, rows, inner]: box = one span (128
// bytes, or 64) of the inner extent x box_rows rows of one group, swizzled over
// the span or not; loads zero-fill beyond each extent, stores leave it out.
// Strides in bytes, multiples of 16.
inline bool make_map_3d(CUtensorMap* m, CUtensorMapDataType type, uint32_t elem_bytes,
                        const void* base, uint64_t inner, uint64_t rows, uint64_t groups,
                        uint64_t row_stride, uint64_t group_stride, uint32_t box_rows,
                        uint32_t span = 128, bool swizzle = true) {
  const EncodeTiledFn enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[3] = {inner, rows, groups};
  const cuuint64_t strides[2] = {row_stride, group_stride};
  const cuuint32_t box[3] = {span / elem_bytes, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return encode_bound([&] {
    return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               !swizzle      ? CU_TENSOR_MAP_SWIZZLE_NONE
               : span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                             : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

}  // namespace moe
