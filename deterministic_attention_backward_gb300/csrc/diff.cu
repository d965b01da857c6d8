// diff.cu -- the extern "C" entries of differential attention: argument checks, workspace
// carving, tensor maps, launches.
#include "diff.cuh"

#include <cmath>

#include "dash_attn.h"
#include "host.cuh"

namespace dash {
namespace {

int tiles(int S) { return (S + kTile - 1) / kTile; }

dash_status_t check_diff(int B, int S, int H, int group, int d) {
  if (B <= 0 || S <= 0 || H <= 0 || group <= 0 || d <= 0 || H % group) return DASH_ERR_INVALID;
  if (d != 32 && d != 64) return DASH_ERR_UNSUPPORTED;
  // row numbers and grids are 32-bit
  if ((long long)B * tiles(S) * kTile >= (1LL << 30) || (long long)B * H * tiles(S) >= (1LL << 27))
    return DASH_ERR_UNSUPPORTED;
  return DASH_OK;
}

struct DiffWorkspace {
  uint32_t *status;
  float *rowv, *dlam_part;
  size_t total;
};
DiffWorkspace carve(void *ws, int B, int S, int H) {
  const size_t ntiles = (size_t)B * H * tiles(S);
  char *base = static_cast<char *>(ws);
  DiffWorkspace w{};
  size_t off = 0;
  w.status = reinterpret_cast<uint32_t *>(base);
  off += kStatusBytes;
  w.rowv = reinterpret_cast<float *>(base + off);
  off = align256(off + ntiles * kRowVecs * kTile * sizeof(float));
  w.dlam_part = reinterpret_cast<float *>(base + off);
  w.total = align256(off + ntiles * sizeof(float));
  return w;
}

bool lam_ok(const void *lam, int dtype) {
  return lam && (dtype == DASH_BF16 || dtype == DASH_FP32) &&
         (reinterpret_cast<uintptr_t>(lam) & (dtype == DASH_FP32 ? 3 : 1)) == 0;
}

}  // namespace
}  // namespace dash

extern "C" {

size_t dash_diff_fwd_workspace_bytes(int B, int S, int H, int d) {
  return dash::check_diff(B, S, H, 1, d) == DASH_OK ? dash::kStatusBytes : 0;
}

size_t dash_diff_bwd_workspace_bytes(int B, int S, int H, int d) {
  return dash::check_diff(B, S, H, 1, d) == DASH_OK ? dash::carve(nullptr, B, S, H).total : 0;
}

dash_status_t dash_diff_fwd(const void *q, const void *k, const void *v, const void *lam, void *o,
                            void *o2, float *lse, int B, int S, int H, int group, int d,
                            float scale, dash_mask_t mask, dash_dtype_t lam_dtype,
                            int lam_per_token, void *workspace, size_t workspace_bytes,
                            dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_diff(B, S, H, group, d);
  if (st != DASH_OK) return st;
  if (mask != DASH_MASK_FULL && mask != DASH_MASK_CAUSAL) return DASH_ERR_INVALID;
  const void *ptrs[] = {q, k, v, o, o2};
  for (const void *ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return DASH_ERR_INVALID;
  if (!lse || !aligned4(lse) || !lam_ok(lam, lam_dtype)) return DASH_ERR_INVALID;
  if (!workspace || workspace_bytes < kStatusBytes || !aligned16(workspace))
    return DASH_ERR_WORKSPACE;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  const int Hkv = H / group;
  CUtensorMap tq, tk, tv;
  if (!make_bshd_map(&tq, q, B, S, H, 2 * d) || !make_bshd_map(&tk, k, B, S, Hkv, 2 * d) ||
      !make_bshd_map(&tv, v, B, S, Hkv, 2 * d))
    return DASH_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, kStatusBytes, s) != cudaSuccess) return DASH_ERR_CUDA;
  DiffFwdParams p{};
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.o2 = static_cast<__nv_bfloat16 *>(o2);
  p.lse = lse;
  p.lam = lam;
  p.status = static_cast<uint32_t *>(workspace);
  p.B = B, p.S = S, p.H = H, p.Hkv = Hkv, p.G = group, p.N = tiles(S);
  p.causal = mask == DASH_MASK_CAUSAL;
  p.lam_f32 = lam_dtype == DASH_FP32;
  p.lam_token = lam_per_token != 0;
  p.wait_ns = g_wait_ns.load();
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)d)) * kLog2e;
  return launch_diff_fwd(d, tq, tk, tv, p, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status_t dash_diff_bwd(const void *q, const void *k, const void *v, const void *o,
                            const void *o2, const void *dout, const float *lse, const void *lam,
                            void *dq, void *dk, void *dv, void *dlam, int B, int S, int H,
                            int group, int d, float scale, dash_mask_t mask,
                            dash_dtype_t lam_dtype, int lam_per_token, void *workspace,
                            size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_diff(B, S, H, group, d);
  if (st != DASH_OK) return st;
  if (mask != DASH_MASK_FULL && mask != DASH_MASK_CAUSAL) return DASH_ERR_INVALID;
  const void *ptrs[] = {q, k, v, o, o2, dout, dq, dk, dv};
  for (const void *ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return DASH_ERR_INVALID;
  if (!lse || !aligned4(lse) || !lam_ok(lam, lam_dtype) || !lam_ok(dlam, lam_dtype))
    return DASH_ERR_INVALID;
  const DiffWorkspace w = carve(workspace, B, S, H);
  if (!workspace || !aligned16(workspace) || workspace_bytes < w.total) return DASH_ERR_WORKSPACE;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  const int Hkv = H / group;
  CUtensorMap tq, tk, tv, tdo;
  // Q and dO stream through dK/dV's kernel by half tiles, K and V are read by whole ones
  if (!make_bshd_map(&tq, q, B, S, H, 2 * d, kTile / 2) ||
      !make_bshd_map(&tk, k, B, S, Hkv, 2 * d) || !make_bshd_map(&tv, v, B, S, Hkv, 2 * d) ||
      !make_bshd_map(&tdo, dout, B, S, H, 2 * d, kTile / 2))
    return DASH_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, kStatusBytes, s) != cudaSuccess) return DASH_ERR_CUDA;
  DiffBwdParams p{};
  p.o = static_cast<const __nv_bfloat16 *>(o);
  p.o2 = static_cast<const __nv_bfloat16 *>(o2);
  p.dout = static_cast<const __nv_bfloat16 *>(dout);
  p.lse = lse;
  p.lam = lam;
  p.rowv = w.rowv;
  p.dlam_part = w.dlam_part;
  p.status = w.status;
  p.dq = static_cast<__nv_bfloat16 *>(dq);
  p.dk = static_cast<__nv_bfloat16 *>(dk);
  p.dv = static_cast<__nv_bfloat16 *>(dv);
  p.dlam = dlam;
  p.B = B, p.S = S, p.H = H, p.Hkv = Hkv, p.G = group, p.N = tiles(S);
  p.causal = mask == DASH_MASK_CAUSAL;
  p.lam_f32 = lam_dtype == DASH_FP32;
  p.lam_token = lam_per_token != 0;
  p.wait_ns = g_wait_ns.load();
  p.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)d);
  p.scale_log2 = p.scale * kLog2e;
  const cudaError_t e =
      launch_diff_bwd(d, tq, tk, tv, tdo, p, s);
  return e == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
