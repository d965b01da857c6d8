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

// The bytes of a tensor, as runs of `run` bytes whose begins lie on up to three steps, the
// narrowest first.
struct Bytes {
  uintptr_t at = 0;
  long long run = 0;
  int dims = 0;
  long long step[3] = {}, count[3] = {};
  long long span() const {  // from the first byte to behind the last
    long long s = run;
    for (int i = 0; i < dims; ++i) s += step[i] * (count[i] - 1);
    return s;
  }
};
// One block, or `count` runs of `run` elements at a stride of `stride` elements, and so on
// outwards.  A null pointer has no bytes.
inline Bytes bytes_of(const void *p, int size, long long run) {
  Bytes b;
  b.at = reinterpret_cast<uintptr_t>(p);
  b.run = p ? run * size : 0;
  return b;
}
inline Bytes along(Bytes b, int size, long long stride, long long count) {
  long long step = stride * size;
  if (count <= 1 || step == 0) return b;
  if (step < 0) b.at += (uintptr_t)(step * (count - 1)), step = -step;
  int i = b.dims++;
  for (; i > 0 && b.step[i - 1] > step; --i)
    b.step[i] = b.step[i - 1], b.count[i] = b.count[i - 1];
  b.step[i] = step, b.count[i] = count;
  return b;
}
// Steps that continue what lies inside them become longer runs, or more of them.
inline Bytes flat(const Bytes &b) {
  Bytes r = b;
  r.dims = 0;
  for (int i = 0; i < b.dims; ++i) {
    const int k = r.dims - 1;
    if (k < 0 && b.step[i] == r.run)
      r.run *= b.count[i];
    else if (k >= 0 && b.step[i] == r.step[k] * r.count[k])
      r.count[k] *= b.count[i];
    else
      r.step[k + 1] = b.step[i], r.count[k + 1] = b.count[i], r.dims = k + 2;
  }
  return r;
}
// Whether two tensors have a byte in common.  Gives up (false) after `tries` comparisons of parts,
// which takes strides that hardly occur.
inline bool share_parts(const Bytes &a, const Bytes &b, int &tries) {
  if (a.at + a.span() <= b.at || b.at + b.span() <= a.at || !a.run || !b.run) return false;
  if (a.at == b.at || (a.dims == 0 && b.dims == 0)) return true;
  if (a.dims > 0 && b.dims > 0 && a.step[a.dims - 1] == b.step[b.dims - 1]) {
    const long long step = a.step[a.dims - 1], n = a.count[a.dims - 1], m = b.count[b.dims - 1];
    Bytes pa = a, pb = b;
    --pa.dims, --pb.dims;
    if (pa.span() <= step && pb.span() <= step) {
      // part i of a begins `behind` bytes after part i + by of b, and may reach part i + by + 1
      const long long d = (long long)(a.at - b.at);
      const long long behind = (d % step + step) % step, by = (d - behind) / step;
      auto meet = [&](long long k) {  // whether a part i of a has a part i + k of b
        return (k < 0 ? -k : 0) < (n < m - k ? n : m - k);
      };
      pa.at = b.at + (uintptr_t)behind;
      if (meet(by) && share_parts(pa, pb, tries)) return true;
      pb.at = b.at + (uintptr_t)step;
      return meet(by + 1) && share_parts(pa, pb, tries);
    }
  }
  if (a.dims < b.dims || (a.dims == b.dims && a.step[a.dims - 1] < b.step[b.dims - 1]))
    return share_parts(b, a, tries);
  Bytes part = a;  // a's parts along its widest step, those that reach b
  const long long step = a.step[a.dims - 1], n = a.count[a.dims - 1];
  part.dims = a.dims - 1;
  const long long below = (long long)(b.at - a.at) - part.span();
  const long long last = ((long long)(b.at - a.at) + b.span() - 1) / step;
  for (long long i = below < 0 ? 0 : below / step + 1; i < n && i <= last; ++i) {
    if (--tries < 0) return false;
    part.at = a.at + (uintptr_t)(i * step);
    if (share_parts(part, b, tries)) return true;
  }
  return false;
}
inline bool share(const Bytes &a, const Bytes &b) {
  if (a.at + a.span() <= b.at || b.at + b.span() <= a.at) return false;
  int tries = 4096;
  return share_parts(flat(a), flat(b), tries);
}
// Whether none of the outputs shares memory with another or with one of `reads`.
template <int N, int M>
bool apart(const Bytes (&outs)[N], const Bytes (&reads)[M]) {
  for (int i = 0; i < N; ++i) {
    for (int k = 0; k < i; ++k)
      if (share(outs[i], outs[k])) return false;
    for (const Bytes &r : reads)
      if (share(outs[i], r)) return false;
  }
  return true;
}

constexpr size_t kStatusBytes = 256;  // a workspace's status block

// Limit of one bounded wait inside the kernels (dash_attn_set_wait_limit).
inline std::atomic<unsigned long long> g_wait_ns{2000000000ull};

}  // namespace dash
