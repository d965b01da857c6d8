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

// How dK/dV's tiles (128 keys of a KV head, in descending order of their work) become CTAs.  Whole
// tiles leave the GPU idle at the end: 512 equal ones take four rounds on 152 SMs, the last of
// them a third full.  So the tiles behind the last round that they fill (causal: the last two,
// as a light tile follows a heavy one) are cut into equal pieces, whose sums a small kernel adds,
// where an estimate says that this is shorter.  Measured, dK/dV's kernels of 32 head pairs of 64
// with 8 KV heads: 1 x 8192 full 1803 -> 1615 us, 1 x 2048 causal 130 -> 91 us, 1 x 512 full
// 34 -> 18 us.  The pieces decide the order of the sums, so they follow from the sizes and the
// mask, not from the GPU that runs.
constexpr int kSplitSMs = 152, kMaxPieces = 4 * kSplitSMs, kMaxPiecesPerTile = 8;
struct Cut {
  int whole, pieces;
};
Cut cut_tiles(int B, int S, int Hkv, int group, int d, bool causal) {
  const int N = tiles(S), heads = B * Hkv, all = heads * N;
  const int round = (causal ? 2 : 1) * kSplitSMs;
  Cut c{all / round * round, 1};
  const int rest = all - c.whole;
  if (rest == 0) return c;
  // In steps of 64 queries (0.87 us): a CTA costs 5 beside its own, the additional kernel 5 and
  // what its reads take.
  const float own = 5.f;
  auto steps = [&](int n) {  // of tile n of the rest
    return 2.f * group * (causal ? N - (c.whole + n) / heads : N);
  };
  const float most = steps(0);
  float best = 0.f, total = 0.f;
  for (int k = 1; k <= kMaxPiecesPerTile && (k == 1 || rest * k <= kMaxPieces); ++k) {
    const float piece = most / k + own;
    float t;
    if (!causal) {
      t = (rest * k + kSplitSMs - 1) / kSplitSMs * (std::ceil(most / k) + own);
    } else if (k == 1) {  // the lightest of the first round is followed first
      t = piece;
      for (int n = kSplitSMs; n < rest; ++n)
        t = std::fmax(t, steps(n) + steps(2 * kSplitSMs - 1 - n) + 2 * own);
      for (int n = 0; n < rest; ++n) total += steps(n);
    } else {  // an even share, and half a piece of unevenness
      t = std::fmax(piece, (total + rest * k * own) / kSplitSMs + 0.5f * piece);
    }
    if (k > 1) t += 5.f + rest * k * d * 3e-4f;
    if (k == 1 || t < 0.97f * best) best = t, c.pieces = k;
  }
  if (c.pieces == 1) c.whole = all;
  return c;
}

struct DiffWorkspace {
  uint32_t *status;
  float *rowv, *dlam_part, *kv_part;
  size_t total;
};
DiffWorkspace carve(void *ws, int B, int S, int H, int d) {
  const size_t ntiles = (size_t)B * H * tiles(S);
  char *base = static_cast<char *>(ws);
  DiffWorkspace w{};
  size_t off = 0;
  w.status = reinterpret_cast<uint32_t *>(base);
  off += kStatusBytes;
  w.rowv = reinterpret_cast<float *>(base + off);
  off = align256(off + ntiles * kRowVecs * kTile * sizeof(float));
  w.dlam_part = reinterpret_cast<float *>(base + off);
  off = align256(off + ntiles * sizeof(float));
  w.kv_part = reinterpret_cast<float *>(base + off);
  const size_t pieces = ntiles * kMaxPiecesPerTile;
  w.total = off + (pieces < kMaxPieces ? pieces : kMaxPieces) * kTile * 4 * d * sizeof(float);
  return w;
}

bool lam_ok(const void *lam, int dtype) {
  return lam && (dtype == DASH_BF16 || dtype == DASH_FP32) &&
         (reinterpret_cast<uintptr_t>(lam) & (dtype == DASH_FP32 ? 3 : 1)) == 0;
}

// dash_diff_withhold: the kernel (0: none), and above it the block.
std::atomic<long long> g_withhold{0};
int withheld(int kernel) {
  const long long w = g_withhold.load();
  return (w & 3) == kernel ? (int)(w >> 2) : -1;
}

// The bytes of a bf16 tensor of `heads` heads of 2d, and of the weights.
Bytes heads_of(const void *p, int B, int S, int heads, int d) {
  return bytes_of(p, 2, (long long)B * S * heads * 2 * d);
}
Bytes weights_of(const void *p, int B, int S, int H, int dtype, bool per_token) {
  return bytes_of(p, dtype == DASH_FP32 ? 4 : 2, per_token ? (long long)B * S * H : H);
}

}  // namespace
}  // namespace dash

extern "C" {

dash_status_t dash_diff_withhold(int kernel, int block) {
  if (kernel < 0 || kernel > 3 || block < 0) return DASH_ERR_INVALID;
  dash::g_withhold.store((long long)block << 2 | kernel);
  return DASH_OK;
}

size_t dash_diff_fwd_workspace_bytes(int B, int S, int H, int d) {
  return dash::check_diff(B, S, H, 1, d) == DASH_OK ? dash::kStatusBytes : 0;
}

size_t dash_diff_bwd_workspace_bytes(int B, int S, int H, int d) {
  return dash::check_diff(B, S, H, 1, d) == DASH_OK ? dash::carve(nullptr, B, S, H, d).total : 0;
}

dash_status_t dash_diff_fwd(const void *q, const void *k, const void *v, const void *lam, void *o,
                            void *o2, float *lse, int B, int S, int H, int group, int d,
                            float scale, dash_mask_t mask, dash_dtype_t lam_dtype,
                            int lam_per_token, void *workspace, size_t workspace_bytes,
                            dash_stream_t stream) {
  return dash_diff_fwd_rest(q, k, v, lam, o, o2, nullptr, lse, B, S, H, group, d, scale, mask,
                            lam_dtype, lam_per_token, workspace, workspace_bytes, stream);
}

dash_status_t dash_diff_fwd_rest(const void *q, const void *k, const void *v, const void *lam,
                                 void *o, void *o2, void *rest, float *lse, int B, int S, int H,
                                 int group, int d, float scale, dash_mask_t mask,
                                 dash_dtype_t lam_dtype, int lam_per_token, void *workspace,
                                 size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_diff(B, S, H, group, d);
  if (st != DASH_OK) return st;
  if (mask != DASH_MASK_FULL && mask != DASH_MASK_CAUSAL) return DASH_ERR_INVALID;
  const void *ptrs[] = {q, k, v, o, o2};
  for (const void *ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return DASH_ERR_INVALID;
  if (!lse || !aligned4(lse) || !lam_ok(lam, lam_dtype) || !aligned16(rest))
    return DASH_ERR_INVALID;
  if (!workspace || workspace_bytes < kStatusBytes || !aligned16(workspace))
    return DASH_ERR_WORKSPACE;
  const int Hkv = H / group;
  const Bytes outs[] = {heads_of(o, B, S, H, d), heads_of(o2, B, S, H, d),
                        heads_of(rest, 2 * B, S, H, d),
                        bytes_of(lse, 4, (long long)B * 2 * H * S),
                        bytes_of(workspace, 1, kStatusBytes)};
  const Bytes reads[] = {heads_of(q, B, S, H, d), heads_of(k, B, S, Hkv, d),
                         heads_of(v, B, S, Hkv, d),
                         weights_of(lam, B, S, H, lam_dtype, lam_per_token)};
  if (!apart(outs, reads)) return DASH_ERR_INVALID;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  CUtensorMap tq, tk, tv;
  if (!make_bshd_map(&tq, q, B, S, H, 2 * d) || !make_bshd_map(&tk, k, B, S, Hkv, 2 * d) ||
      !make_bshd_map(&tv, v, B, S, Hkv, 2 * d))
    return DASH_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(workspace, 0, kStatusBytes, s) != cudaSuccess) return DASH_ERR_CUDA;
  DiffFwdParams p{};
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.o2 = static_cast<__nv_bfloat16 *>(o2);
  p.rest = static_cast<__nv_bfloat16 *>(rest);
  p.lse = lse;
  p.lam = lam;
  p.status = static_cast<uint32_t *>(workspace);
  p.taken = p.status + 32;  // a sector of its own in the status block
  p.B = B, p.S = S, p.H = H, p.Hkv = Hkv, p.G = group, p.N = tiles(S);
  p.causal = mask == DASH_MASK_CAUSAL;
  p.lam_f32 = lam_dtype == DASH_FP32;
  p.lam_token = lam_per_token != 0;
  p.wait_ns = g_wait_ns.load();
  p.withhold = withheld(1);
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)d)) * kLog2e;
  return launch_diff_fwd(d, tq, tk, tv, p, dev.sms, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status_t dash_diff_bwd(const void *q, const void *k, const void *v, const void *o,
                            const void *o2, const void *dout, const float *lse, const void *lam,
                            void *dq, void *dk, void *dv, void *dlam, int B, int S, int H,
                            int group, int d, float scale, dash_mask_t mask,
                            dash_dtype_t lam_dtype, int lam_per_token, void *workspace,
                            size_t workspace_bytes, dash_stream_t stream) {
  return dash_diff_bwd_rest(q, k, v, o, o2, nullptr, dout, lse, lam, dq, dk, dv, dlam, B, S, H,
                            group, d, scale, mask, lam_dtype, lam_per_token, workspace,
                            workspace_bytes, stream);
}

dash_status_t dash_diff_bwd_rest(const void *q, const void *k, const void *v, const void *o,
                                 const void *o2, const void *rest, const void *dout,
                                 const float *lse, const void *lam, void *dq, void *dk, void *dv,
                                 void *dlam, int B, int S, int H, int group, int d, float scale,
                                 dash_mask_t mask, dash_dtype_t lam_dtype, int lam_per_token,
                                 void *workspace, size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_diff(B, S, H, group, d);
  if (st != DASH_OK) return st;
  if (mask != DASH_MASK_FULL && mask != DASH_MASK_CAUSAL) return DASH_ERR_INVALID;
  const void *ptrs[] = {q, k, v, o, o2, dout, dq, dk, dv};
  for (const void *ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return DASH_ERR_INVALID;
  if (!lse || !aligned4(lse) || !lam_ok(lam, lam_dtype) || !lam_ok(dlam, lam_dtype) ||
      !aligned16(rest))
    return DASH_ERR_INVALID;
  const DiffWorkspace w = carve(workspace, B, S, H, d);
  if (!workspace || !aligned16(workspace) || workspace_bytes < w.total) return DASH_ERR_WORKSPACE;
  const int Hkv = H / group;
  const Bytes outs[] = {heads_of(dq, B, S, H, d), heads_of(dk, B, S, Hkv, d),
                        heads_of(dv, B, S, Hkv, d),
                        weights_of(dlam, B, S, H, lam_dtype, lam_per_token),
                        bytes_of(workspace, 1, (long long)w.total)};
  const Bytes reads[] = {heads_of(q, B, S, H, d), heads_of(k, B, S, Hkv, d),
                         heads_of(v, B, S, Hkv, d), heads_of(o, B, S, H, d),
                         heads_of(o2, B, S, H, d), heads_of(rest, 2 * B, S, H, d),
                         heads_of(dout, B, S, H, d),
                         bytes_of(lse, 4, (long long)B * 2 * H * S),
                         weights_of(lam, B, S, H, lam_dtype, lam_per_token)};
  if (!apart(outs, reads)) return DASH_ERR_INVALID;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  CUtensorMap tq, tk, tv, tdo;
  // Q and dO stream through dK/dV's kernel by half tiles, K and V are read by whole ones
  if (!make_bshd_map(&tq, q, B, S, H, 2 * d, kTile / 2) ||
      !make_bshd_map(&tk, k, B, S, Hkv, 2 * d) || !make_bshd_map(&tv, v, B, S, Hkv, 2 * d) ||
      !make_bshd_map(&tdo, dout, B, S, H, 2 * d, kTile / 2))
    return DASH_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DiffBwdParams p{};
  p.o = static_cast<const __nv_bfloat16 *>(o);
  p.o2 = static_cast<const __nv_bfloat16 *>(o2);
  p.rest = static_cast<const __nv_bfloat16 *>(rest);
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
  p.withhold_dq = withheld(2), p.withhold_dkv = withheld(3);
  p.scale = scale > 0.f ? scale : 1.0f / std::sqrt((float)d);
  p.scale_log2 = p.scale * kLog2e;
  const Cut cut = cut_tiles(B, S, Hkv, group, d, p.causal);
  p.kv_whole = cut.whole, p.kv_pieces = cut.pieces;
  p.kv_part = w.kv_part;
  return launch_diff_bwd(d, tq, tk, tv, tdo, p, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
