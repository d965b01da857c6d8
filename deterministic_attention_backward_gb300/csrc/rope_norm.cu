// rope_norm.cu -- the norm of every head of q and k with the rotary turn behind it, and its gradient.
//   forward   x^ = x rstd(x),  rstd = (mean(x^2) + eps)^-1/2 over a head,  y = R(w x^)
//   backward  dz = R^T dy,  dx = rstd (w dz - x^ mean(w dz x^)),  dw = sum of dz x^ over all heads
// with R the turn of rope.cu (pairs of the first rot elements, magnitude included).
//
// Bound by memory: forward every element in and out once, backward dy and x in and dx out; rstd is
// formed again there (x is read anyway).  A group of lanes holds a head in registers, a lane two
// vectors: the two sides of its pairs, so that the turn needs no exchange, and the norm's sums (of
// x^2 and of w dz x, from which mean(w dz x^) follows) go through shuffles together.  The lane's
// cosines and sines stay in registers for the heads of a token that the group goes through; the next
// heads are on their way by asynchronous copies into rings of its threads' own.  A CTA takes heads of q, of k or of v only
// (v is copied), so that a thread has one set of weights and one of sums of dw; the CTAs' sums are
// added in order by a second kernel, their number follows from the sizes.
#include "angle.cuh"
#include "common.cuh"
#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 512;
constexpr int kForwardPerSm = 3, kBackPerSm = 2;  // CTAs, for their registers

struct HeadPart {
  const void *x, *dy, *w;            // w null: ones
  void *out;
  float *dw;                         // [ctas][D] sums
  long long xb, xt, xh, gb, gt, gh;  // strides in elements: batch, token, head
  long long ob, ot, oh;
  int heads, D;
  int units, turn;  // pairs of vectors of a head, the ones that turn
  int lanes;        // of a group
  int each, blocks; // heads of a token that a group takes at a time, times that
  int cta0, ctas;
  int normed;
};
struct HeadParams {
  HeadPart part[3];
  const double *inv_freq;
  const void *pos;
  long long pos_b, pos_t, start, tokens;
  float magnitude, eps;
  int pos64, S, rot, nparts, wf32;
};

// A thread's own copies into shared memory: 16 bytes, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T, int V>
__device__ __forceinline__ void load_if(const T *p, bool on, float (&f)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = on ? to_f32<T>(p[e]) : 0.f;
}

// The V pairs of two vectors turned by (cos, sin).
template <int V, bool kHalf>
__device__ __forceinline__ void turn_pairs(float (&x)[V], float (&y)[V], const float2 (&cs)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    constexpr bool kAcross = kHalf || V == 1;
    float &a = kAcross ? x[e] : (2 * e < V ? x[(2 * e) % V] : y[(2 * e) % V]);
    float &d = kAcross ? y[e] : (2 * e < V ? x[(2 * e + 1) % V] : y[(2 * e + 1) % V]);
    const float na = fmaf(a, cs[e].x, -__fmul_rn(d, cs[e].y));
    d = fmaf(d, cs[e].x, __fmul_rn(a, cs[e].y));
    a = na;
  }
}

// Heads on their way to a group, in a ring of its own in shared memory (single elements are loaded
// when they are needed).
template <int V, int R, bool kBack>
constexpr int kRingStages = V == 1 ? 0 : (kBack ? 4 : 6) / R;
template <int V, int R, bool kBack>
constexpr int kRingBytes = kRingStages<V, R, kBack> * (kBack ? 4 : 2) * R * kThreads * 16;

// R pairs of vectors a lane.
template <typename T, int V, int R, bool kHalf, bool kBack>
__global__ void __launch_bounds__(kThreads, kBack ? kBackPerSm : kForwardPerSm)
    heads_kernel(const __grid_constant__ HeadParams p) {
  constexpr int N = kRingStages<V, R, kBack>, kVecs = (kBack ? 4 : 2) * R;
  extern __shared__ uint4 shared[];
  uint4 *ring = shared + threadIdx.x;                                     // [N][kVecs][kThreads]
  u128 *turns = reinterpret_cast<u128 *>(shared + N * kVecs * kThreads);  // [rot / 2]
  float *by = reinterpret_cast<float *>(turns + p.rot / 2);  // magnitude, NaN for a bad frequency
  const int cta = blockIdx.x;
  const int k = p.nparts > 2 && cta >= p.part[2].cta0   ? 2
                : p.nparts > 1 && cta >= p.part[1].cta0 ? 1
                                                        : 0;
  const HeadPart &q = p.part[k];
  const int G = q.lanes, in_group = threadIdx.x & (G - 1);
  int e0[R], e1[R];
  bool has0[R], has1[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int u = in_group + r * G;
    const bool across = kHalf && u < q.turn;
    e0[r] = across ? u * V : 2 * u * V;
    e1[r] = across ? p.rot / 2 + u * V : e0[r] + V;
    has0[r] = u < q.units && e0[r] < q.D;
    has1[r] = u < q.units && e1[r] < q.D;
  }
  const int per_warp = 32 / G, per_cta = kThreads / G;
  const long long items = p.tokens * q.blocks, step = (long long)q.ctas * per_cta;
  // all lanes of a warp go round together, as they meet in the shuffles
  const long long begin =
      (long long)(cta - q.cta0) * per_cta + (threadIdx.x >> 5) * per_warp;
  const int mine = (threadIdx.x & 31) / G;

  // where an item's heads lie; `heads` of them are there
  struct Place {
    const T *x, *dy;
    int heads, b, s;
  };
  auto place = [&](long long i0) {
    const long long item = i0 + mine;
    Place w{static_cast<const T *>(q.x), static_cast<const T *>(q.dy), 0, 0, 0};
    if (item < items) {
      const int tok = (int)(item / q.blocks), h0 = (int)(item - (long long)tok * q.blocks) * q.each;
      w.b = tok / p.S, w.s = tok - w.b * p.S;
      w.heads = min(q.each, q.heads - h0);
      w.x += w.b * q.xb + w.s * q.xt + h0 * q.xh;
      if constexpr (kBack)
        if (q.normed) w.dy += w.b * q.gb + w.s * q.gt + h0 * q.gh;
    }
    return w;
  };
  // the head that is brought in next
  long long ahead0 = begin;
  int ahead_h = 0;
  Place ahead = place(begin);
  auto bring = [&](int slot) {
    if constexpr (N > 0) {
      const bool live = ahead_h < ahead.heads;
      const uint32_t at =
          (uint32_t)__cvta_generic_to_shared(ring + slot * kVecs * kThreads);
      const T *x = ahead.x + ahead_h * q.xh, *dy = ahead.dy + ahead_h * q.gh;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        copy16(at + (2 * r) * kThreads * 16, x + e0[r], live && has0[r]);
        copy16(at + (2 * r + 1) * kThreads * 16, x + e1[r], live && has1[r]);
        if constexpr (kBack)
          if (q.normed) {
            copy16(at + (2 * R + 2 * r) * kThreads * 16, dy + e0[r], live && has0[r]);
            copy16(at + (2 * R + 2 * r + 1) * kThreads * 16, dy + e1[r], live && has1[r]);
          }
      }
      copies_end();
      if (++ahead_h == q.each) ahead_h = 0, ahead0 += step, ahead = place(ahead0);
    }
  };
#pragma unroll
  for (int i = 0; i < N - 1; ++i) bring(i);

  if (q.turn) {
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) {
      const double f = p.inv_freq[i];
      turns[i] = turns_of(f);
      by[i] = isfinite(f) ? p.magnitude : NAN;
    }
    __syncthreads();
  }
  float w0[R][V], w1[R][V], s0[kBack ? R : 1][V] = {}, s1[kBack ? R : 1][V] = {};
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w0[r][e] = w1[r][e] = 1.f;
      if (q.w && p.wf32) {
        if (has0[r]) w0[r][e] = static_cast<const float *>(q.w)[e0[r] + e];
        if (has1[r]) w1[r][e] = static_cast<const float *>(q.w)[e1[r] + e];
      } else if (q.w) {
        if (has0[r]) w0[r][e] = to_f32<T>(static_cast<const T *>(q.w)[e0[r] + e]);
        if (has1[r]) w1[r][e] = to_f32<T>(static_cast<const T *>(q.w)[e1[r] + e]);
      }
    }
  const float inv_d = 1.f / (float)q.D;
  int slot = 0;
  for (long long i0 = begin; i0 < items; i0 += step) {
    const Place at = place(i0);
    const int h0 = (int)((i0 + mine) % q.blocks) * q.each;
    T *out = static_cast<T *>(q.out) + at.b * q.ob + at.s * q.ot + h0 * q.oh;
    float2 cs[R][V];
    if (q.turn) {
      long long pos = p.start + at.s;
      if (p.pos) {
        const long long i = at.b * p.pos_b + at.s * p.pos_t;
        pos = p.pos64 ? static_cast<const long long *>(p.pos)[i]
                      : (long long)static_cast<const int *>(p.pos)[i];
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int u = in_group + r * G;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          cs[r][e] = make_float2(1.f, 0.f);
          if (u < q.turn) {
            const int pair = u * V + e;
            const int phase = (int)(uint32_t)(((u128)(__int128)pos * turns[pair]) >> 96);
            float sn, c;
            sincospif((float)phase * (1.0f / 2147483648.0f), &sn, &c);
            cs[r][e] = make_float2(c * by[pair], (kBack ? -sn : sn) * by[pair]);
          }
        }
      }
    }
    for (int h = 0; h < q.each; ++h) {
      float x0[R][V], x1[R][V], g0[kBack ? R : 1][V], g1[kBack ? R : 1][V];
      const bool live = h < at.heads;
      T *row = out + h * q.oh;
      if constexpr (N > 0) {
        bring(slot == 0 ? N - 1 : slot - 1);
        copies_wait<N - 1>();
        const uint4 *v = ring + slot * kVecs * kThreads;
        slot = slot + 1 == N ? 0 : slot + 1;
        if (!q.normed) {  // (a part's: the same for the whole CTA)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (live && has0[r]) *reinterpret_cast<uint4 *>(row + e0[r]) = v[2 * r * kThreads];
            if (live && has1[r]) *reinterpret_cast<uint4 *>(row + e1[r]) = v[(2 * r + 1) * kThreads];
          }
          continue;
        }
        auto take = [&](int i, float (&f)[V]) {
          const uint4 raw = v[i * kThreads];
          unpack<T, V>(*reinterpret_cast<const Pack<T, V> *>(&raw), f);
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {
          take(2 * r, x0[r]);
          take(2 * r + 1, x1[r]);
          if constexpr (kBack) {
            take(2 * R + 2 * r, g0[r]);
            take(2 * R + 2 * r + 1, g1[r]);
          }
        }
      } else {
        const T *x = at.x + h * q.xh;
        if (!q.normed) {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              if (live && has0[r]) row[e0[r] + e] = x[e0[r] + e];
              if (live && has1[r]) row[e1[r] + e] = x[e1[r] + e];
            }
          continue;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          load_if<T, V>(x + e0[r], live && has0[r], x0[r]);
          load_if<T, V>(x + e1[r], live && has1[r], x1[r]);
          if constexpr (kBack) {
            load_if<T, V>(at.dy + h * q.gh + e0[r], live && has0[r], g0[r]);
            load_if<T, V>(at.dy + h * q.gh + e1[r], live && has1[r], g1[r]);
          }
        }
      }
      float ss = 0.f, sg = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (kBack) {
          if (in_group + r * G < q.turn) turn_pairs<V, kHalf>(g0[r], g1[r], cs[r]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ss = fmaf(x0[r][e], x0[r][e], ss);
          ss = fmaf(x1[r][e], x1[r][e], ss);
          if constexpr (kBack) {
            sg = fmaf(g0[r][e] * w0[r][e], x0[r][e], sg);
            sg = fmaf(g1[r][e] * w1[r][e], x1[r][e], sg);
          }
        }
      }
      for (int o = G >> 1; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if constexpr (kBack) sg += __shfl_xor_sync(0xffffffffu, sg, o);
      }
      const float rstd = live ? rsqrtf(fmaf(ss, inv_d, p.eps)) : 0.f;
      if constexpr (kBack) {
        const float mean = rstd * rstd * (sg * inv_d);  // mean(w dz x^) rstd, x^ = x rstd
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            s0[r][e] = fmaf(g0[r][e], x0[r][e] * rstd, s0[r][e]);
            s1[r][e] = fmaf(g1[r][e], x1[r][e] * rstd, s1[r][e]);
            g0[r][e] = rstd * fmaf(-x0[r][e], mean, g0[r][e] * w0[r][e]);
            g1[r][e] = rstd * fmaf(-x1[r][e], mean, g1[r][e] * w1[r][e]);
          }
          if (live && has0[r]) store_pack<T, V>(row + e0[r], pack<T, V>(g0[r]));
          if (live && has1[r]) store_pack<T, V>(row + e1[r], pack<T, V>(g1[r]));
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x0[r][e] *= rstd * w0[r][e];
            x1[r][e] *= rstd * w1[r][e];
          }
          if (in_group + r * G < q.turn) turn_pairs<V, kHalf>(x0[r], x1[r], cs[r]);
          if (live && has0[r]) store_pack<T, V>(row + e0[r], pack<T, V>(x0[r]));
          if (live && has1[r]) store_pack<T, V>(row + e1[r], pack<T, V>(x1[r]));
        }
      }
    }
  }
  if constexpr (kBack) {
    if constexpr (N > 0) copies_wait<0>();
    if (!q.dw) return;
    // the groups' sums [group][D], added in order
    float *sums = reinterpret_cast<float *>(shared);
    __syncthreads();
    const int group = threadIdx.x / G;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (has0[r]) sums[group * q.D + e0[r] + e] = s0[r][e];
        if (has1[r]) sums[group * q.D + e1[r] + e] = s1[r][e];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < q.D; c += kThreads) {
      float t = 0.f;
      for (int g = 0; g < per_cta; ++g) t += sums[g * q.D + c];
      q.dw[(long long)(cta - q.cta0) * q.D + c] = t;
    }
  }
}

// The CTAs' sums: 8 runs of CTAs for each column, then the runs, in order.
struct HeadSums {
  const float *part[2];
  void *out[2];
  int ctas[2], D, f32;
};
template <typename T>
__global__ void __launch_bounds__(256) heads_sums_kernel(const __grid_constant__ HeadSums p) {
  __shared__ float sums[8][32];
  const int k = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  if (!p.out[k]) return;
  const int per = (p.ctas[k] + 7) / 8, end = min(p.ctas[k], (run + 1) * per);
  float t = 0.f;
  if (c < p.D)
    for (int i = run * per; i < end; ++i) t += p.part[k][(long long)i * p.D + c];
  sums[run][threadIdx.x & 31] = t;
  __syncthreads();
  if (run > 0 || c >= p.D) return;
  for (int r = 1; r < 8; ++r) t += sums[r][threadIdx.x];
  if (p.f32)
    static_cast<float *>(p.out[k])[c] = t;
  else
    static_cast<T *>(p.out[k])[c] = from_f32<T>(t);
}

// ------------------------------------------------------------------ host
constexpr int kSms = 152;  // of a GB300: the number of CTAs, and so dw's sums, follow from the sizes

int lanes_of(int units) {
  int g = 1;
  while (g < units && g < 32) g *= 2;
  return g;
}
// Shares out the CTAs among the parts, by the bytes that they move, and the heads of a token among
// groups.
void deal(HeadParams &p, int V, bool back) {
  auto cost = [&](const HeadPart &q) {
    return (long long)q.heads * q.D * (back && q.normed ? 3 : 2);
  };
  long long all = 0;
  for (int i = 0; i < p.nparts; ++i) all += cost(p.part[i]);
  int cta = 0;
  for (int i = 0; i < p.nparts; ++i) {
    HeadPart &q = p.part[i];
    q.turn = q.normed ? p.rot / (2 * V) : 0;
    q.units = q.turn + (q.D / V - 2 * q.turn + 1) / 2;
    q.lanes = lanes_of(q.units);
    const int groups = kThreads / q.lanes;
    long long share = kSms * (back ? kBackPerSm : kForwardPerSm) * cost(q) / all;
    if (share < 1) share = 1;
    // as many heads of a token to a group as leave every group something, 16 at most: cosines and
    // sines are formed once for them
    long long each = p.tokens * q.heads / (share * groups);
    each = each < 1 ? 1 : each > 16 ? 16 : each;
    if (each > q.heads) each = q.heads;
    q.blocks = (int)((q.heads + each - 1) / each);
    q.each = (q.heads + q.blocks - 1) / q.blocks;
    const long long want = (p.tokens * q.blocks + groups - 1) / groups;
    q.ctas = (int)(want < share ? want : share);
    q.cta0 = cta;
    cta += q.ctas;
  }
}
int ctas_of(const HeadParams &p) { return p.part[p.nparts - 1].cta0 + p.part[p.nparts - 1].ctas; }

template <typename T, int V, int R, bool kHalf, bool kBack>
cudaError_t launch(const HeadParams &p, cudaStream_t s) {
  constexpr int kRing = kRingBytes<V, R, kBack>;
  size_t smem = kRing + (size_t)p.rot / 2 * 20;
  if (kBack)
    for (int i = 0; i < p.nparts; ++i) {
      const size_t sums = (size_t)(kThreads / p.part[i].lanes) * p.part[i].D * 4;
      if (p.part[i].dw && sums > smem) smem = sums;
    }
  // (kMaxD / 2 pairs at most)
  const cudaError_t e =
      allow_smem<heads_kernel<T, V, R, kHalf, kBack>>(kRing + kMaxD / 2 * 20 + 16384);
  if (e != cudaSuccess) return e;
  heads_kernel<T, V, R, kHalf, kBack><<<ctas_of(p), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int V, int R>
cudaError_t launch_v(const HeadParams &p, bool half, bool back, cudaStream_t s) {
  if (half)
    return back ? launch<T, V, R, true, true>(p, s) : launch<T, V, R, true, false>(p, s);
  return back ? launch<T, V, R, false, true>(p, s) : launch<T, V, R, false, false>(p, s);
}
template <typename T>
cudaError_t launch_t(const HeadParams &p, bool wide, bool half, bool back, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  int units = 0;
  for (int i = 0; i < p.nparts; ++i) units = p.part[i].units > units ? p.part[i].units : units;
  if (!wide) return units <= 32 ? launch_v<T, 1, 1>(p, half, back, s)
                                : launch_v<T, 1, 8>(p, half, back, s);
  if constexpr (V == 4)
    if (units > 32) return launch_v<T, V, 2>(p, half, back, s);
  return launch_v<T, V, 1>(p, half, back, s);
}

struct Lay {
  Bytes x[3], dy[3], out[3];
};

// Checks and fills everything but the addresses of partial sums.
dash_status_t fill(HeadParams &p, bool &wide, Lay &lay, const dash_rope_part_t *parts,
                   const dash_rope_part_t *x, int nparts, const void *const weights[2], int B, int S,
                   int rot, dash_rope_layout_t layout, dash_dtype_t dtype, dash_dtype_t wdtype,
                   const double *inv_freq, const void *positions, int positions64,
                   long long pos_stride_b, long long pos_stride_t, bool back) {
  if (!parts || !weights || (back && !x) || nparts < 1 || nparts > 3 || B <= 0 || S <= 0 ||
      rot <= 0 || (rot & 1))
    return DASH_ERR_INVALID;
  if (layout != DASH_ROPE_HALF && layout != DASH_ROPE_INTERLEAVED) return DASH_ERR_INVALID;
  if (dtype != DASH_BF16 && dtype != DASH_FP16 && dtype != DASH_FP32) return DASH_ERR_INVALID;
  if (wdtype != dtype && wdtype != DASH_FP32) return DASH_ERR_INVALID;
  if (!inv_freq || (reinterpret_cast<uintptr_t>(inv_freq) & 7)) return DASH_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(positions) & (positions64 ? 7 : 3)) return DASH_ERR_INVALID;
  const int size = dtype == DASH_FP32 ? 4 : 2, vec = 16 / size;
  const int wsize = wdtype == DASH_FP32 ? 4 : 2;
  wide = rot % (2 * vec) == 0;
  auto lies = [&](const void *at, const long long *stride, int heads, int D) {
    const long long count[3] = {B, S, heads};
    Bytes b = bytes_of(at, size, D);
    for (int k = 0; k < 3; ++k) b = along(b, size, stride[k], count[k]);
    return b;
  };
  auto lean = [&](const void *at, const long long *stride) {
    if (reinterpret_cast<uintptr_t>(at) & (size - 1)) return false;
    wide = wide && aligned16(at) && (stride[0] | stride[1] | stride[2]) % vec == 0;
    return true;
  };
  int turned = 0;
  for (int i = 0; i < nparts; ++i) {
    const dash_rope_part_t &q = parts[i];
    HeadPart &h = p.part[i];
    if (!q.in || !q.out || q.heads <= 0 || q.D <= 0 || (q.turn && (q.D < rot || turned == 2)))
      return DASH_ERR_INVALID;
    if (!lean(q.in, q.in_stride) || !lean(q.out, q.out_stride)) return DASH_ERR_INVALID;
    wide = wide && q.D % vec == 0;
    h.normed = q.turn != 0;
    h.heads = q.heads, h.D = q.D;
    h.out = q.out;
    h.ob = q.out_stride[0], h.ot = q.out_stride[1], h.oh = q.out_stride[2];
    // what is copied is read as x
    const dash_rope_part_t &from = back && q.turn ? x[turned] : q;
    if (back && q.turn) {
      if (!from.in || from.heads != q.heads || from.D != q.D || !lean(from.in, from.in_stride))
        return DASH_ERR_INVALID;
      h.dy = q.in;
      h.gb = q.in_stride[0], h.gt = q.in_stride[1], h.gh = q.in_stride[2];
      lay.dy[i] = lies(q.in, q.in_stride, q.heads, q.D);
    }
    h.x = from.in;
    h.xb = from.in_stride[0], h.xt = from.in_stride[1], h.xh = from.in_stride[2];
    lay.x[i] = lies(from.in, from.in_stride, q.heads, q.D);
    lay.out[i] = lies(q.out, q.out_stride, q.heads, q.D);
    if (q.turn) {
      h.w = weights[turned++];
      if (reinterpret_cast<uintptr_t>(h.w) & (wsize - 1)) return DASH_ERR_INVALID;
    }
    if (q.D > kMaxD) return DASH_ERR_UNSUPPORTED;
  }
  if (!turned) return DASH_ERR_INVALID;
  if ((long long)B * S >= (1LL << 31)) return DASH_ERR_UNSUPPORTED;
  for (int i = 0; i < nparts; ++i)
    if ((long long)parts[i].heads * parts[i].D >= (1LL << 28)) return DASH_ERR_UNSUPPORTED;
  // an output is its own input (the gradient), as it lies, or what nothing else is
  const int psize = positions64 ? 8 : 4;
  const Bytes rest[4] = {
      bytes_of(inv_freq, 8, rot / 2),
      along(along(bytes_of(positions, psize, 1), psize, pos_stride_t, S), psize, pos_stride_b, B),
      bytes_of(weights[0], wsize, weights[0] ? parts[0].D : 0),
      bytes_of(weights[1], wsize, weights[1] && nparts > 1 ? parts[1].D : 0)};
  for (int i = 0; i < nparts; ++i) {
    const dash_rope_part_t &q = parts[i];
    bool in_place = q.in == q.out;
    for (int k = 0; k < 3; ++k) in_place = in_place && q.in_stride[k] == q.out_stride[k];
    for (int k = 0; k < nparts; ++k) {
      const bool own = k == i && in_place;
      if (k < i && share(lay.out[i], lay.out[k])) return DASH_ERR_INVALID;
      if (share(lay.out[i], lay.x[k]) && !(own && !(back && q.turn))) return DASH_ERR_INVALID;
      if (share(lay.out[i], lay.dy[k]) && !own) return DASH_ERR_INVALID;
    }
    for (const Bytes &r : rest)
      if (share(lay.out[i], r)) return DASH_ERR_INVALID;
  }
  p.inv_freq = inv_freq;
  p.pos = positions;
  p.pos64 = positions64;
  p.pos_b = pos_stride_b, p.pos_t = pos_stride_t;
  p.tokens = (long long)B * S;
  p.S = S, p.rot = rot, p.nparts = nparts;
  p.wf32 = wdtype == DASH_FP32;
  deal(p, wide ? vec : 1, back);
  return DASH_OK;
}

cudaError_t launch_heads(const HeadParams &p, dash_dtype_t dtype, bool wide, bool half, bool back,
                         cudaStream_t s) {
  if (dtype == DASH_BF16) return launch_t<__nv_bfloat16>(p, wide, half, back, s);
  if (dtype == DASH_FP16) return launch_t<__half>(p, wide, half, back, s);
  return launch_t<float>(p, wide, half, back, s);
}

}  // namespace
}  // namespace dash

extern "C" {

dash_status_t dash_rope_norm_fwd(const dash_rope_part_t *parts, int nparts,
                                 const void *const weights[2], int B, int S, int rot,
                                 dash_rope_layout_t layout, dash_dtype_t dtype, dash_dtype_t wdtype,
                                 const double *inv_freq, float magnitude, float eps,
                                 const void *positions, int positions64, long long pos_stride_b,
                                 long long pos_stride_t, long long start, dash_stream_t stream) {
  using namespace dash;
  HeadParams p{};
  bool wide;
  Lay lay;
  dash_status_t st = fill(p, wide, lay, parts, nullptr, nparts, weights, B, S, rot, layout, dtype,
                          wdtype, inv_freq, positions, positions64, pos_stride_b, pos_stride_t,
                          false);
  if (st != DASH_OK) return st;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  p.magnitude = magnitude, p.eps = eps, p.start = start;
  return launch_heads(p, dtype, wide, layout == DASH_ROPE_HALF, false,
                      reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DASH_OK
             : DASH_ERR_CUDA;
}

size_t dash_rope_norm_bwd_workspace_bytes(int D) {
  return D > 0 && D <= dash::kMaxD ? (size_t)(dash::kSms * dash::kBackPerSm + 3) * D * 4 : 0;
}

dash_status_t dash_rope_norm_bwd(const dash_rope_part_t *parts, const dash_rope_part_t *x, int nparts,
                                 const void *const weights[2], void *const dweights[2], int B, int S,
                                 int rot, dash_rope_layout_t layout, dash_dtype_t dtype,
                                 dash_dtype_t wdtype, const double *inv_freq, float magnitude,
                                 float eps, const void *positions, int positions64,
                                 long long pos_stride_b, long long pos_stride_t, long long start,
                                 void *workspace, size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  HeadParams p{};
  bool wide;
  Lay lay;
  dash_status_t st = fill(p, wide, lay, parts, x, nparts, weights, B, S, rot, layout, dtype, wdtype,
                          inv_freq, positions, positions64, pos_stride_b, pos_stride_t, true);
  if (st != DASH_OK) return st;
  if (!dweights) return DASH_ERR_INVALID;
  HeadSums sums{};
  sums.f32 = p.wf32;
  float *at = static_cast<float *>(workspace);
  int turned = 0;
  size_t need = 0;
  bool any = false;
  const int wsize = wdtype == DASH_FP32 ? 4 : 2;
  Bytes dw[3];
  for (int i = 0; i < nparts; ++i) {
    HeadPart &h = p.part[i];
    if (!h.normed) continue;
    void *to = dweights[turned];
    if (reinterpret_cast<uintptr_t>(to) & (wsize - 1)) return DASH_ERR_INVALID;
    if (to) {
      if (any && h.D != sums.D) return DASH_ERR_UNSUPPORTED;  // heads of q and k are alike
      any = true;
      sums.D = h.D;
      sums.out[turned] = to;
      sums.ctas[turned] = h.ctas;
      sums.part[turned] = h.dw = at + need;
      dw[turned] = bytes_of(to, wsize, h.D);
      need += (size_t)h.ctas * h.D;
    }
    ++turned;
  }
  if (any && (!workspace || !aligned16(workspace) || workspace_bytes < need * 4))
    return DASH_ERR_WORKSPACE;
  dw[2] = bytes_of(any ? workspace : nullptr, 1, (long long)need * 4);
  for (int i = 0; i < 3; ++i) {
    for (int k = 0; k < nparts; ++k)
      if (share(dw[i], lay.x[k]) || share(dw[i], lay.dy[k]) || share(dw[i], lay.out[k]))
        return DASH_ERR_INVALID;
    for (int k = 0; k < i; ++k)
      if (share(dw[i], dw[k])) return DASH_ERR_INVALID;
    for (int k = 0; k < 2; ++k)
      if (share(dw[i], bytes_of(weights[k], wsize, weights[k] ? sums.D : 0)))
        return DASH_ERR_INVALID;
  }
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  p.magnitude = magnitude, p.eps = eps, p.start = start;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_heads(p, dtype, wide, layout == DASH_ROPE_HALF, true, s) != cudaSuccess)
    return DASH_ERR_CUDA;
  if (any) {
    const dim3 grid((sums.D + 31) / 32, 2);
    if (dtype == DASH_BF16)
      heads_sums_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(sums);
    else if (dtype == DASH_FP16)
      heads_sums_kernel<__half><<<grid, 256, 0, s>>>(sums);
    else
      heads_sums_kernel<float><<<grid, 256, 0, s>>>(sums);
  }
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
