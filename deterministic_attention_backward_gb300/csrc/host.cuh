// host.cuh -- host-side helpers shared by the extern "C" translation units: the driver's
// tensor-map encoder, device properties, pointer checks and the limit of a bounded wait.
#pragma once
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "dash_attn.h"

namespace dash {

// ------------------------------------------------------------------ driver entry point
inline PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
inline std::once_flag g_encode_once;

inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  std::call_once(g_encode_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

// [B, S, Hx, D] bf16 viewed as a 4-D tensor (D, Hx, S, B); box = 64 columns x 1 head x 128
// (or `rows`) rows x 1 batch, 128-byte swizzle: one box lands in shared memory as that many rows
// of 128 bytes.
// Rows of a tile past S (S not a multiple of 128) are outside the tensor and read as zeros.
inline bool make_bshd_map(CUtensorMap *m, const void *base, int B, int S, int Hx, int D,
                          int rows = kTile) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hx, (cuuint64_t)S, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hx * D * 2,
                                 (cuuint64_t)S * Hx * D * 2};
  const cuuint32_t box[4] = {(cuuint32_t)kBoxCols, 1, (cuuint32_t)rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------------ device properties
struct DevInfo {
  int sms = 0, major = 0, minor = 0;
};
inline std::mutex g_dev_mu;
inline DevInfo g_dev[64];

inline dash_status_t device_info(DevInfo *out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DASH_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DevInfo &d = g_dev[dev];
  if (d.sms == 0) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
      d.sms = 0;
      return DASH_ERR_CUDA;
    }
  }
  *out = d;
  // kernels are built for sm_103a only
  return (d.major == 10 && d.minor == 3) ? DASH_OK : DASH_ERR_UNSUPPORTED;
}

// Lets kKernel have `bytes` of dynamic shared memory on the current device; asked once per device.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (set.load() >> dev & 1)) return e;
  const cudaError_t f =
      cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (f == cudaSuccess) set.fetch_or(1ull << dev);
  return f;
}

// ------------------------------------------------------------------ checks
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr size_t kStatusBytes = 256;  // a workspace's status block

// Limit of one bounded wait inside the kernels (dash_attn_set_wait_limit).
inline std::atomic<unsigned long long> g_wait_ns{2000000000ull};

}  // namespace dash
