// rope.cu -- rotary positions.  Pair p of a head (elements p and p + rot/2 in the half
// layout, 2p and 2p + 1 in the interleaved one) is turned by the angle
//     a = position * inv_freq[p]:   (x, y) -> m (x cos a - y sin a,  y cos a + x sin a)
// with m the magnitude; the gradient is the same turn by -a.  Elements past rot pass through.
//
// The angle of a far position does not survive fp32 (position 2^20 at one radian a position is
// off by 0.03 rad) and fp64 runs at 1/64 of the fp32 rate here, so the phase is an integer:
// inv_freq / (2 pi) becomes a 128-bit fraction of a turn, the product with the position is
// taken modulo 2^128 -- whole turns fall off exactly, for negative positions too -- and the top
// 32 bits, as a signed fraction of half turns, go through sincospif: over all 64-bit positions the
// angle is off by the rounding of that fraction to fp32, 2^-25 half turns, and what it is cut by.
//
// Bound by memory: every element is read and written once.  A CTA takes kTok tokens, forms
// each (token, pair) phase once in shared memory and uses it for all heads of the token; q, k
// and v go in one launch (v unturned), so that strided views of a qkv product become the
// contiguous tensors attention reads in a single pass.  Measured on 2 x 8192 tokens of 32 + 8 + 8
// heads of 128 in bf16: 65 us, 6.2 TB/s, 91 % of a plain copy's rate; one token 3.5 us, a launch.
#include "angle.cuh"
#include "common.cuh"
#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRot = 1024;

struct RopePart {
  const void *in;
  void *out;
  long long ib, it, ih, ob, ot, oh;  // strides in elements: batch, token, head
  int units;                         // work units per head
  int end;                           // units of this part and the ones before it, per token
  int turn;                          // work units per head that turn (the others copy)
  unsigned magic;                    // ceil(2^32 / units)
};
struct RopeParams {
  RopePart part[3];
  const double *inv_freq;
  const void *pos;
  long long pos_b, pos_t, start;
  float magnitude;
  int pos64, S, tokens, rot, back, nparts, units;
  unsigned magic;  // ceil(2^32 / units)
};

// n / d by the magic ceil(2^32 / d): exact while n d < 2^32.
__device__ __forceinline__ unsigned div_by(unsigned n, unsigned d, unsigned magic, bool exact) {
  return exact ? n / d : (d == 1 ? n : __umulhi(n, magic));
}

template <typename T, int V, bool kHalf, int kTok>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];  // [kTok][rot / 2] (cos, sin) times the magnitude
  const int half = p.rot / 2;
  const int t0 = blockIdx.x * kTok;
  const int ntok = min(kTok, p.tokens - t0);
  for (int i = threadIdx.x; i < ntok * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    const int tok = t0 + t, b = tok / p.S, s = tok - b * p.S;
    long long pos = p.start + s;
    if (p.pos) {
      const long long at = b * p.pos_b + s * p.pos_t;
      pos = p.pos64 ? static_cast<const long long *>(p.pos)[at]
                    : (long long)static_cast<const int *>(p.pos)[at];
    }
    const double f = p.inv_freq[pair];
    const int phase = (int)(uint32_t)(((u128)(__int128)pos * turns_of(f)) >> 96);
    float sn, c;
    sincospif((float)phase * (1.0f / 2147483648.0f), &sn, &c);
    if (!isfinite(f)) c = sn = NAN;
    cs[i] = make_float2(c * p.magnitude, (p.back ? -sn : sn) * p.magnitude);
  }
  __syncthreads();
  const unsigned items = (unsigned)ntok * p.units;
  for (unsigned i = threadIdx.x; i < items; i += kThreads) {
    const unsigned t = kTok == 1 ? 0 : div_by(i, p.units, p.magic, V == 1);
    unsigned r = i - t * p.units;
    int k = 0;
    if (p.nparts > 1 && r >= (unsigned)p.part[0].end) k = 1;
    if (p.nparts > 2 && r >= (unsigned)p.part[1].end) k = 2;
    const RopePart &q = p.part[k];
    if (k) r -= p.part[k - 1].end;
    const unsigned h = div_by(r, q.units, q.magic, V == 1);
    const int u = r - h * q.units;
    const int tok = t0 + t, b = tok / p.S, s = tok - b * p.S;
    const T *in = static_cast<const T *>(q.in) + b * q.ib + s * q.it + h * q.ih;
    T *out = static_cast<T *>(q.out) + b * q.ob + s * q.ot + h * q.oh;
    if (u < q.turn) {
      const int e0 = kHalf ? u * V : 2 * u * V, e1 = kHalf ? half + u * V : e0 + V;
      float x[V], y[V];
      unpack<T, V>(load_pack<T, V>(in + e0), x);
      unpack<T, V>(load_pack<T, V>(in + e1), y);
      const float2 *c = cs + t * half + u * V;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // the e-th pair of this unit: across the two vectors, or neighbours within one
        constexpr bool kAcross = kHalf || V == 1;
        float &a = kAcross ? x[e] : (2 * e < V ? x[(2 * e) % V] : y[(2 * e) % V]);
        float &d = kAcross ? y[e] : (2 * e < V ? x[(2 * e + 1) % V] : y[(2 * e + 1) % V]);
        const float2 w = c[e];
        // fused and unfused roundings fixed, so that both vector widths give the same bits
        const float na = fmaf(a, w.x, -__fmul_rn(d, w.y));
        d = fmaf(d, w.x, __fmul_rn(a, w.y));
        a = na;
      }
      store_pack<T, V>(out + e0, pack<T, V>(x));
      store_pack<T, V>(out + e1, pack<T, V>(y));
    } else {
      const int e = (u + q.turn) * V;  // units past the turned ones: rot = 2 turn V on
      store_pack<T, V>(out + e, load_pack<T, V>(in + e));
    }
  }
}

template <typename T, int V, bool kHalf>
cudaError_t launch(const RopeParams &p, int sms, cudaStream_t s) {
  // Several tokens share a CTA once every SM has work without it.
  const int kTok = p.tokens >= 8 * sms && p.rot <= 512 ? 4 : 1;
  const size_t smem = (size_t)kTok * (p.rot / 2) * sizeof(float2);
  const unsigned grid = (unsigned)((p.tokens + kTok - 1) / kTok);
  if (kTok == 4)
    rope_kernel<T, V, kHalf, 4><<<grid, kThreads, smem, s>>>(p);
  else
    rope_kernel<T, V, kHalf, 1><<<grid, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_layout(const RopeParams &p, bool half, int sms, cudaStream_t s) {
  return half ? launch<T, V, true>(p, sms, s) : launch<T, V, false>(p, sms, s);
}

}  // namespace
}  // namespace dash

extern "C" dash_status_t dash_rope(const dash_rope_part_t *parts, int nparts, int B, int S,
                                   int rot, dash_rope_layout_t layout, dash_dtype_t dtype,
                                   const double *inv_freq, float magnitude, const void *positions,
                                   int positions64, long long pos_stride_b, long long pos_stride_t,
                                   long long start, int backward, dash_stream_t stream) {
  using namespace dash;
  if (!parts || nparts < 1 || nparts > 3 || B <= 0 || S <= 0 || rot <= 0 || (rot & 1))
    return DASH_ERR_INVALID;
  if (layout != DASH_ROPE_HALF && layout != DASH_ROPE_INTERLEAVED) return DASH_ERR_INVALID;
  if (dtype != DASH_BF16 && dtype != DASH_FP16 && dtype != DASH_FP32) return DASH_ERR_INVALID;
  if (!inv_freq || (reinterpret_cast<uintptr_t>(inv_freq) & 7)) return DASH_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(positions) & (positions64 ? 7 : 3)) return DASH_ERR_INVALID;
  Bytes in[3], out[3];
  const int size = dtype == DASH_FP32 ? 4 : 2, vec = 16 / size, psize = positions64 ? 8 : 4;
  for (int i = 0; i < nparts; ++i) {
    const dash_rope_part_t &q = parts[i];
    if (!q.in || !q.out || q.heads <= 0 || q.D <= 0 || (q.turn && q.D < rot))
      return DASH_ERR_INVALID;
    auto lies = [&](const void *at, const long long *stride) {
      const long long count[3] = {B, S, q.heads};
      Bytes b = bytes_of(at, size, q.D);
      for (int k = 0; k < 3; ++k) b = along(b, size, stride[k], count[k]);
      return b;
    };
    in[i] = lies(q.in, q.in_stride), out[i] = lies(q.out, q.out_stride);
  }
  if (rot > kMaxRot || (long long)B * S >= (1LL << 31) - 4) return DASH_ERR_UNSUPPORTED;
  const Bytes angles[2] = {
      bytes_of(inv_freq, 8, rot / 2),
      along(along(bytes_of(positions, psize, 1), psize, pos_stride_t, S), psize, pos_stride_b, B)};
  for (int i = 0; i < nparts; ++i) {  // an output is its input, as it lies, or what nothing else is
    const dash_rope_part_t &q = parts[i];
    bool in_place = q.in == q.out;
    for (int k = 0; k < 3; ++k) in_place = in_place && q.in_stride[k] == q.out_stride[k];
    for (int k = 0; k < nparts; ++k)
      if ((k < i && share(out[i], out[k])) || ((k != i || !in_place) && share(out[i], in[k])))
        return DASH_ERR_INVALID;
    if (share(out[i], angles[0]) || share(out[i], angles[1])) return DASH_ERR_INVALID;
  }
  bool wide = rot % (2 * vec) == 0;
  long long units = 0;
  for (int i = 0; i < nparts; ++i) {
    const dash_rope_part_t &q = parts[i];
    const uintptr_t at = reinterpret_cast<uintptr_t>(q.in) | reinterpret_cast<uintptr_t>(q.out);
    if (at & (size - 1)) return DASH_ERR_INVALID;
    const long long any = q.in_stride[0] | q.in_stride[1] | q.in_stride[2] | q.out_stride[0] |
                          q.out_stride[1] | q.out_stride[2] | q.D;
    wide = wide && !(at & 15) && any % vec == 0;
    units += (long long)q.heads * q.D;
  }
  if (units >= (1LL << 28)) return DASH_ERR_UNSUPPORTED;
  // 4 tokens of a CTA are numbered with 32 bits and divided by a 32-bit reciprocal
  if (units / vec >= (1 << 15)) wide = false;
  DevInfo dev;
  dash_status_t st = device_info(&dev);
  if (st != DASH_OK) return st;
  RopeParams p{};
  const int V = wide ? vec : 1;
  int end = 0;
  for (int i = 0; i < nparts; ++i) {
    const dash_rope_part_t &q = parts[i];
    RopePart &r = p.part[i];
    r.in = q.in;
    r.out = q.out;
    r.ib = q.in_stride[0], r.it = q.in_stride[1], r.ih = q.in_stride[2];
    r.ob = q.out_stride[0], r.ot = q.out_stride[1], r.oh = q.out_stride[2];
    r.turn = q.turn ? rot / (2 * V) : 0;
    r.units = (q.turn ? q.D - rot : q.D) / V + r.turn;
    r.end = end += q.heads * r.units;
    r.magic = (unsigned)(((1ull << 32) + r.units - 1) / r.units);
  }
  p.units = end;
  p.magic = (unsigned)(((1ull << 32) + end - 1) / end);
  p.inv_freq = inv_freq;
  p.pos = positions;
  p.pos64 = positions64;
  p.pos_b = pos_stride_b;
  p.pos_t = pos_stride_t;
  p.start = start;
  p.magnitude = magnitude;
  p.S = S;
  p.tokens = B * S;
  p.rot = rot;
  p.back = backward != 0;
  p.nparts = nparts;
  const bool half = layout == DASH_ROPE_HALF;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DASH_BF16)
    e = wide ? launch_layout<__nv_bfloat16, 8>(p, half, dev.sms, s)
             : launch_layout<__nv_bfloat16, 1>(p, half, dev.sms, s);
  else if (dtype == DASH_FP16)
    e = wide ? launch_layout<__half, 8>(p, half, dev.sms, s)
             : launch_layout<__half, 1>(p, half, dev.sms, s);
  else
    e = wide ? launch_layout<float, 4>(p, half, dev.sms, s)
             : launch_layout<float, 1>(p, half, dev.sms, s);
  return e == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}
