// rope_norm.cu -- the norm of every head of q and k with the rotary turn behind it, and its gradient.
//   forward   x^ = x rstd(x),  rstd = (mean(x^2) + eps)^-1/2 over a head,  y = R(w x^)
//   backward  dz = R^T dy,  dx = rstd (w dz - x^ mean(w dz x^)),  dw = sum of dz x^ over all heads
// with R the turn of rope.cu (pairs of the first rot elements, magnitude included).
//
// Bound by memory: forward every element in and out once, backward dy and x in and dx out; rstd is
// formed again there (x is read anyway).  A group of lanes holds a head in registers, a lane two
// vectors: the two sides of its pairs, so that the turn needs no exchange, and the norm's sums (of
// x^2 and of w dz x, from which mean(w dz x^) follows) go through shuffles together.  The lane's
// cosines and sines stay in registers for the heads of a token, which the group goes through one by
// one, the weights in shared memory (registers decide how many warps there are); the next heads are
// on their way by asynchronous copies into rings of its threads' own.  A CTA takes heads of q, of k
// or of v only (v is copied), so that a thread has one set of sums of dw; the CTAs' sums are added in
// order by a second kernel, their number follows from the sizes.
//
// Measured on 2 x 8192 tokens of 32 + 8 + 8 heads of 128 in bf16: forward 69 us, 5.8 TB/s, 87 % of a
// plain copy's rate, backward 100 us, 5.7 TB/s; one token 3.9 and 6.2 us, launches.  Off 16 bytes 333 and
// 581 us: sizes, not places, decide which lane has an element, and with it the sums' order.
#include "angle.cuh"
#include "common.cuh"
#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxD = 512;
constexpr int kForwardPerSm = 6, kBackPerSm = 4;  // CTAs, for their registers

struct HeadPart {
  const void *x, *dy, *w;            // w null: ones
  void *out;
  float *dw;                         // [ctas][D] sums
  long long xb, xt, xh, gb, gt, gh;  // strides in elements: batch, token, head
  long long ob, ot, oh;
  int heads, D;
  int units, turn;  // pairs of vectors of a head, the ones that turn
  int lanes;        // of a group
  int across;       // groups of a warp that share a token
  int each, blocks; // steps through a token's heads that a warp takes at a time, times that
  int tokens, dt, dk;  // of a warp's blocks: groups of tokens, and how far on its next one is
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
// The values of a vector: pairs, or a single one.
template <int V>
using Values = std::conditional_t<V == 1, float, f2>;
using dash::f2_sum, dash::fma2, dash::mul2;  // of pairs, beside those of single values
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float f2_sum(float a) { return a; }
template <typename E>
__device__ __forceinline__ E both(float a);
template <>
__device__ __forceinline__ float both<float>(float a) { return a; }
template <>
__device__ __forceinline__ f2 both<f2>(float a) { return f2_of(a, a); }
__device__ __forceinline__ f2 swapped(f2 v) {
  float a, b;
  f2_to(v, a, b);
  return f2_of(b, a);
}
__device__ __forceinline__ float swapped(float v) { return v; }
template <int V>
__device__ __forceinline__ void values_of(const float (&f)[V], Values<V> (&v)[V == 1 ? 1 : V / 2]) {
  if constexpr (V == 1) {
    v[0] = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = f2_of(f[2 * i], f[2 * i + 1]);
  }
}
// A pair's frequency as the limbs 1 to 3 of the 128-bit fraction of a turn, and the magnitude (NaN for
// a frequency that is not finite).
__device__ __forceinline__ uint4 turns_in(const HeadParams &p, int i) {
  const double f = p.inv_freq[i];
  const u128 t = turns_of(f);
  return make_uint4((uint32_t)(t >> 32), (uint32_t)(t >> 64), (uint32_t)(t >> 96),
                    __float_as_uint(isfinite(f) ? p.magnitude : NAN));
}
// Cosine and sine, times the magnitude, of a position's turn.  Of the 192-bit product the bits 96 to
// 127 are the fraction of a turn; carries from below bit 96 are left out, two units of 2^-32 turns at
// most.  kShort: the hardware's sine, off by 2^-21, for types that round to 2^-12 and coarser.
template <bool kShort>
__device__ __forceinline__ void cos_sin(long long pos, const uint4 &t, float &c, float &s) {
  const unsigned long long m = pos < 0 ? 0ull - (unsigned long long)pos : (unsigned long long)pos;
  const uint32_t lo = (uint32_t)m, hi = (uint32_t)(m >> 32);
  uint32_t turn = lo * t.z + __umulhi(lo, t.y) + hi * t.y + __umulhi(hi, t.x);
  if (pos < 0) turn = 0u - turn;
  const float half_turns = (float)(int)turn * (1.0f / 2147483648.0f);
  if constexpr (kShort) {
    const float a = half_turns * 3.14159265358979f;
    c = __cosf(a), s = __sinf(a);
  } else {
    sincospif(half_turns, &s, &c);
  }
  const float by = __uint_as_float(t.w);
  c *= by, s *= by;
}
template <typename E>
__device__ __forceinline__ float value_of(const E *v, int e) {
  if constexpr (sizeof(E) == 4) {
    return v[e];
  } else {
    float x, y;
    f2_to(v[e >> 1], x, y);
    return e & 1 ? y : x;
  }
}

// What a turn multiplies a vector pair's values and their partners by: the partner of a value is the
// other vector's (half layout, single elements) or its neighbour.
template <int V>
struct Turn {
  static constexpr int C = V == 1 ? 1 : V / 2;
  Values<V> own0[C], other0[C], own1[C], other1[C];
};
template <int V, bool kAcross>
__device__ __forceinline__ void turn_by(const Turn<V> &t, Values<V> (&x)[Turn<V>::C],
                                        Values<V> (&y)[Turn<V>::C]) {
#pragma unroll
  for (int i = 0; i < Turn<V>::C; ++i) {
    const auto a = x[i], b = y[i];
    x[i] = fma2(kAcross ? b : swapped(a), t.other0[i], mul2(a, t.own0[i]));
    y[i] = fma2(kAcross ? a : swapped(b), t.other1[i], mul2(b, t.own1[i]));
  }
}

// Heads on their way to a group, in a ring of its own in shared memory (single elements are loaded
// when they are needed).  Of 2 x 8192 tokens the forward takes 69 us with 2 and 79 us with 3, the backward
// 102 us with 2, 100 with 3 and 106 with 4.
template <int V, int R, bool kBack>
constexpr int kRingStages = V == 1 ? 0 : kBack ? 3 : 2;
template <int V, int R, bool kBack>
constexpr int kRingBytes = kRingStages<V, R, kBack> * (kBack ? 4 : 2) * R * kThreads * 16;

// R pairs of vectors a lane.  Where tensors do not lie on 16 bytes (kLoose), a group's lanes bring their head
// into the ring, and take it out of it, element by element side by side in memory: every lane has the same
// elements as on 16 bytes, and every sum its order.
template <typename T, int V, int R, bool kHalf, bool kBack, bool kLoose>
__global__ void __launch_bounds__(kThreads, kBack ? kBackPerSm : kForwardPerSm)
    heads_kernel(const __grid_constant__ HeadParams p) {
  constexpr int N = kRingStages<V, R, kBack>, kVecs = (kBack ? 4 : 2) * R;
  extern __shared__ uint4 shared[];
  uint4 *ring = shared + threadIdx.x;                // [N][kVecs][kThreads]
  // what the lanes need for a token, by element of their vectors and then by lane, so that a warp's
  // reads meet no bank twice: frequencies of pairs, weights of both vectors
  uint4 *turns = shared + N * kVecs * kThreads;                   // [V][turning units]
  float *weights = reinterpret_cast<float *>(turns + p.rot / 2);  // [2][V / W][units][W]
  constexpr int W = V == 1 ? 1 : 4;
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
  // `across` groups of a warp take neighbouring heads of a token, the others the next tokens; step i
  // of block k moves them to heads (k each + i) across and behind.  The warps take blocks of tokens in
  // turn, so that what is under way at a time lies close together in memory.
  const int per_cta = kThreads / G, mine = (threadIdx.x & 31) / G, my_head = mine & (q.across - 1);
  const int my_token = mine / q.across, at_once = 32 / G / q.across;
  const int steps = q.heads / q.across;
  const long long xstep = q.xh * q.across, gstep = q.gh * q.across, ostep = q.oh * q.across;

  struct Place {
    const T *x, *dy;
    int t, k;  // group of tokens and block
    int left;  // steps
    int b, s, h;
    bool on;   // there is such a token
  };
  // (divisions would take longer than a head)
  auto place = [&](Place &at) {
    const uint32_t tok = (uint32_t)at.t * at_once + my_token;
    at.left = min(q.each, steps - at.k * q.each);
    at.on = at.t < q.tokens && tok < p.tokens;
    at.b = 0, at.s = at.on ? (int)tok : 0;
    if (at.s >= p.S) at.b = at.s / p.S, at.s -= at.b * p.S;
    at.h = at.on ? at.k * q.each * q.across + my_head : 0;
    at.x = static_cast<const T *>(q.x) + at.b * q.xb + at.s * q.xt + at.h * q.xh;
    if constexpr (kBack)
      at.dy = static_cast<const T *>(q.dy) + at.b * q.gb + at.s * q.gt + at.h * q.gh;
  };
  auto next_block = [&](Place &at) {
    at.t += q.dt, at.k += q.dk;
    if (at.k >= q.blocks) at.k -= q.blocks, ++at.t;
    place(at);
  };
  Place first{};
  first.t = (cta - q.cta0) * (kThreads / 32) + (threadIdx.x >> 5);
  first.k = first.t % q.blocks, first.t /= q.blocks;
  place(first);
  // where an element of the group's head lies in a slot of the ring
  auto place_of = [&](int slot, int which, int e) {
    const int vec = e / V;
    int u = vec >> 1, side = vec & 1;
    if (kHalf && vec < 2 * q.turn) side = vec >= q.turn, u = vec - side * q.turn;
    const int r = R == 1 ? 0 : u / 32;  // (more than one pair: a group is a warp)
    return reinterpret_cast<T *>(shared + (slot * kVecs + which * 2 * R + 2 * r + side) * kThreads +
                                 (threadIdx.x & ~(G - 1)) + (u & (G - 1))) +
           e % V;
  };
  // f(element, its value) for this lane's share of a head, eight on their way at once
  auto each_loose = [&](const T *src, bool on, auto &&f) {
    constexpr int kAtOnce = 8;
    for (int first = in_group; first < q.D; first += kAtOnce * G) {
      T v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int e = first + i * G;
        v[i] = on && e < q.D ? src[e] : from_f32<T>(0.f);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int e = first + i * G;
        if (e < q.D) f(e, v[i]);
      }
    }
  };
  auto bring_loose = [&](int slot, int which, const T *src, bool on) {
    each_loose(src, on, [&](int e, T v) { *place_of(slot, which, e) = v; });
  };
  // the head that is brought in next
  Place ahead = first;
  int filled = 0;  // the slot it goes to
  auto bring = [&] {
    if constexpr (N > 0) {
      const uint32_t at =
          (uint32_t)__cvta_generic_to_shared(ring + filled * kVecs * kThreads);
      if constexpr (kLoose)
        if (q.normed) {
          __syncwarp();  // what was there has been taken out
          bring_loose(filled, 0, ahead.x, ahead.on);
          if constexpr (kBack) bring_loose(filled, 1, ahead.dy, ahead.on);
        }
      filled = filled + 1 == N ? 0 : filled + 1;
      if constexpr (!kLoose)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        copy16(at + (2 * r) * kThreads * 16, ahead.x + e0[r], ahead.on && has0[r]);
        copy16(at + (2 * r + 1) * kThreads * 16, ahead.x + e1[r], ahead.on && has1[r]);
        if constexpr (kBack)
          if (q.normed) {
            copy16(at + (2 * R + 2 * r) * kThreads * 16, ahead.dy + e0[r], ahead.on && has0[r]);
            copy16(at + (2 * R + 2 * r + 1) * kThreads * 16, ahead.dy + e1[r], ahead.on && has1[r]);
          }
      }
      if constexpr (!kLoose) copies_end();
      ahead.x += xstep;
      if constexpr (kBack) ahead.dy += gstep;
      if (--ahead.left == 0) next_block(ahead);
    }
  };
#pragma unroll
  for (int i = 0; i < N - 1; ++i) bring();

  if (q.normed) {
    for (int i = threadIdx.x; i < p.rot / 2; i += kThreads)
      turns[i % V * q.turn + i / V] = turns_in(p, i);
    for (int i = threadIdx.x; i < 2 * V * q.units; i += kThreads) {
      const int part = i / (W * q.units), side = part / (V / W);
      const int u = i / W % q.units, e = part % (V / W) * W + i % W;
      const bool split = kHalf && u < q.turn;
      const int at = (split ? u * V + side * (p.rot / 2) : (2 * u + side) * V) + e;
      weights[i] = at >= q.D ? 0.f
                   : !q.w    ? 1.f
                   : p.wf32  ? static_cast<const float *>(q.w)[at]
                             : to_f32<T>(static_cast<const T *>(q.w)[at]);
    }
    __syncthreads();
  }
  constexpr int C = Turn<V>::C;
  constexpr bool kAcross = kHalf || V == 1;
  using E = Values<V>;
  // of a vector of unit u, which the lane may not have
  auto weights_of = [&](int side, int u, E (&w)[C]) {
    if constexpr (V == 1) {
      w[0] = u < q.units ? weights[side * q.units + u] : 0.f;
    } else {
      const uint4 *at = reinterpret_cast<const uint4 *>(weights) + side * (V / 4) * q.units +
                        (u < q.units ? u : 0);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const uint4 v = at[i * q.units];
        w[2 * i] = f2_of(v.x, v.y), w[2 * i + 1] = f2_of(v.z, v.w);
      }
    }
  };
  E s0[kBack ? R : 1][C] = {}, s1[kBack ? R : 1][C] = {};
  const float inv_d = 1.f / (float)q.D;
  int slot = 0;
  // forward R, backward R^T
  Turn<V> turn[R];
  for (Place at = first; at.t < q.tokens; next_block(at)) {
    T *row = static_cast<T *>(q.out) + at.b * q.ob + at.s * q.ot + at.h * q.oh;
    {
      if (q.normed) {
        long long pos = p.start + at.s;
        if (p.pos) {
          const long long i = at.b * p.pos_b + at.s * p.pos_t;
          pos = p.pos64 ? static_cast<const long long *>(p.pos)[i]
                        : (long long)static_cast<const int *>(p.pos)[i];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int u = in_group + r * G;
          float own[2][V], other[2][V];  // of the two vectors
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float c = 1.f, sn = 0.f;
            if (u < q.turn) {
              cos_sin<sizeof(T) == 2>(pos, turns[e * q.turn + u], c, sn);
              if (kBack) sn = -sn;
            }
            // pair e, elements a and b: (a, b) -> (c a - sn b, c b + sn a)
            const int va = kAcross || 2 * e < V ? 0 : 1, vb = kAcross ? 1 : va;
            const int a = kAcross ? e : (2 * e) % V, b = kAcross ? e : a + 1;
            own[va][a] = own[vb][b] = c;
            other[va][a] = -sn, other[vb][b] = sn;
          }
          values_of<V>(own[0], turn[r].own0);
          values_of<V>(own[1], turn[r].own1);
          values_of<V>(other[0], turn[r].other0);
          values_of<V>(other[1], turn[r].other1);
        }
      }
    }
    for (int left = at.left; left > 0; --left, row += ostep, at.x += xstep, at.dy += gstep) {
      E x0[R][C], x1[R][C], g0[kBack ? R : 1][C], g1[kBack ? R : 1][C];
      uint4 *v = nullptr;
      int now = 0;  // this head's slot
      if constexpr (N > 0) {
        bring();
        if constexpr (kLoose) {
          if (!q.normed) {
            if (at.on) each_loose(at.x, true, [&](int e, T v) { row[e] = v; });
            continue;
          }
          __syncwarp();
        } else {
          copies_wait<N - 1>();
        }
        v = ring + slot * kVecs * kThreads;
        now = slot;
        slot = slot + 1 == N ? 0 : slot + 1;
        if (!q.normed) {  // (a part's: the same for the whole CTA)
#pragma unroll
          for (int r = 0; r < R; ++r) {
            if (at.on && has0[r]) *reinterpret_cast<uint4 *>(row + e0[r]) = v[2 * r * kThreads];
            if (at.on && has1[r]) *reinterpret_cast<uint4 *>(row + e1[r]) = v[(2 * r + 1) * kThreads];
          }
          continue;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          // (copies leave zeros where a lane has no vector, elements nothing)
          const uint4 none = make_uint4(0, 0, 0, 0);
          const bool in0 = !kLoose || has0[r], in1 = !kLoose || has1[r];
          unpack2<T>(in0 ? v[2 * r * kThreads] : none, x0[r]);
          unpack2<T>(in1 ? v[(2 * r + 1) * kThreads] : none, x1[r]);
          if constexpr (kBack) {
            unpack2<T>(in0 ? v[(2 * R + 2 * r) * kThreads] : none, g0[r]);
            unpack2<T>(in1 ? v[(2 * R + 2 * r + 1) * kThreads] : none, g1[r]);
          }
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool on0 = at.on && has0[r], on1 = at.on && has1[r];
          if (!q.normed) {
            if (on0) row[e0[r]] = at.x[e0[r]];
            if (on1) row[e1[r]] = at.x[e1[r]];
            continue;
          }
          x0[r][0] = on0 ? to_f32<T>(at.x[e0[r]]) : 0.f;
          x1[r][0] = on1 ? to_f32<T>(at.x[e1[r]]) : 0.f;
          if constexpr (kBack) {
            g0[r][0] = on0 ? to_f32<T>(at.dy[e0[r]]) : 0.f;
            g1[r][0] = on1 ? to_f32<T>(at.dy[e1[r]]) : 0.f;
          }
        }
        if (!q.normed) continue;
      }
      E ss[2] = {both<E>(0.f), both<E>(0.f)}, sg[2] = {both<E>(0.f), both<E>(0.f)};
#pragma unroll
      for (int r = 0; r < R; ++r) {
        E w0[C], w1[C];
        if constexpr (kBack) {
          weights_of(0, in_group + r * G, w0), weights_of(1, in_group + r * G, w1);
          if (in_group + r * G < q.turn) turn_by<V, kAcross>(turn[r], g0[r], g1[r]);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          ss[0] = fma2(x0[r][i], x0[r][i], ss[0]);
          ss[1] = fma2(x1[r][i], x1[r][i], ss[1]);
          if constexpr (kBack) {
            sg[0] = fma2(mul2(g0[r][i], w0[i]), x0[r][i], sg[0]);
            sg[1] = fma2(mul2(g1[r][i], w1[i]), x1[r][i], sg[1]);
          }
        }
      }
      float sum = f2_sum(ss[0]) + f2_sum(ss[1]), sum_g = kBack ? f2_sum(sg[0]) + f2_sum(sg[1]) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < G) {
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if constexpr (kBack) sum_g += __shfl_xor_sync(0xffffffffu, sum_g, o);
        }
      const float rstd = at.on ? rsqrtf(fmaf(sum, inv_d, p.eps)) : 0.f;
      const E rs = both<E>(rstd);
      // -mean(w dz x^) rstd, x^ = x rstd
      const E mean = both<E>(-rstd * rstd * (sum_g * inv_d));
      auto store = [&](int vec, int e, const E (&f)[C], bool on) {
        if (!on) return;
        if constexpr (V == 1)
          row[e] = from_f32<T>(f[0]);
        else  // (into the slot that has been read)
          *(kLoose ? v + vec * kThreads : reinterpret_cast<uint4 *>(row + e)) = pack2<T>(f);
      };
#pragma unroll
      for (int r = 0; r < R; ++r) {
        E(&a)[C] = x0[r], (&b)[C] = x1[r], w0[C], w1[C];
        weights_of(0, in_group + r * G, w0), weights_of(1, in_group + r * G, w1);
        if constexpr (kBack) {
          E(&ga)[C] = g0[r], (&gb)[C] = g1[r];
#pragma unroll
          for (int i = 0; i < C; ++i) {
            s0[r][i] = fma2(ga[i], mul2(a[i], rs), s0[r][i]);
            s1[r][i] = fma2(gb[i], mul2(b[i], rs), s1[r][i]);
            ga[i] = mul2(rs, fma2(a[i], mean, mul2(ga[i], w0[i])));
            gb[i] = mul2(rs, fma2(b[i], mean, mul2(gb[i], w1[i])));
          }
          store(2 * r, e0[r], ga, at.on && has0[r]);
          store(2 * r + 1, e1[r], gb, at.on && has1[r]);
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i) {
            a[i] = mul2(mul2(a[i], rs), w0[i]);
            b[i] = mul2(mul2(b[i], rs), w1[i]);
          }
          if (in_group + r * G < q.turn) turn_by<V, kAcross>(turn[r], a, b);
          store(2 * r, e0[r], a, at.on && has0[r]);
          store(2 * r + 1, e1[r], b, at.on && has1[r]);
        }
      }
      if constexpr (kLoose) {
        __syncwarp();
        for (int e = in_group; at.on && e < q.D; e += G) row[e] = *place_of(now, 0, e);
      }
    }
  }
  if constexpr (kBack) {
    if constexpr (N > 0 && !kLoose) copies_wait<0>();
    if (!q.dw) return;
    // the groups' sums [group][D], added in order
    float *sums = reinterpret_cast<float *>(shared);
    __syncthreads();
    const int group = threadIdx.x / G;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (has0[r]) sums[group * q.D + e0[r] + e] = value_of(s0[r], e);
        if (has1[r]) sums[group * q.D + e1[r] + e] = value_of(s1[r], e);
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
// Shares out the CTAs among the parts, by the bytes that they move.
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
    long long share = kSms * (back ? kBackPerSm : kForwardPerSm) * cost(q) / all;
    if (share < 1) share = 1;
    const int per_warp = 32 / q.lanes, warps = kThreads / 32;
    // neighbouring heads side by side, as far as 8 steps through a token's heads are left: its cosines
    // and sines serve for them
    q.across = 1;
    while (2 * q.across <= per_warp && q.heads % (2 * q.across) == 0 && q.heads / (2 * q.across) >= 8)
      q.across *= 2;
    const int steps = q.heads / q.across, at_once = per_warp / q.across;
    const long long groups = (p.tokens + at_once - 1) / at_once;
    // as many of them at a time as leave every warp something, 16 at most
    long long each = groups * steps / (share * warps);
    each = each < 1 ? 1 : each > 16 ? 16 : each;
    if (each > steps) each = steps;
    q.blocks = (int)((steps + each - 1) / each);
    q.each = (int)((steps + q.blocks - 1) / q.blocks);
    const long long want = (groups * q.blocks + warps - 1) / warps;
    q.tokens = (int)groups;
    q.ctas = (int)(want < share ? want : share);
    q.dt = q.ctas * warps / q.blocks, q.dk = q.ctas * warps % q.blocks;
    q.cta0 = cta;
    cta += q.ctas;
  }
}
int ctas_of(const HeadParams &p) { return p.part[p.nparts - 1].cta0 + p.part[p.nparts - 1].ctas; }

template <typename T, int V, int R, bool kHalf, bool kBack, bool kLoose>
cudaError_t launch(const HeadParams &p, cudaStream_t s) {
  constexpr int kRing = kRingBytes<V, R, kBack>;
  int units = 0;
  for (int i = 0; i < p.nparts; ++i) units = p.part[i].units > units ? p.part[i].units : units;
  size_t smem = kRing + (size_t)p.rot / 2 * 16 + 2 * V * 4 * (size_t)units;
  if (kBack)
    for (int i = 0; i < p.nparts; ++i) {
      const size_t sums = (size_t)(kThreads / p.part[i].lanes) * p.part[i].D * 4;
      if (p.part[i].dw && sums > smem) smem = sums;
    }
  // (kMaxD / 2 pairs at most)
  const cudaError_t e =
      allow_smem<heads_kernel<T, V, R, kHalf, kBack, kLoose>>(kRing + kMaxD / 2 * 16 + 16384 + 8 * kMaxD);
  if (e != cudaSuccess) return e;
  heads_kernel<T, V, R, kHalf, kBack, kLoose><<<ctas_of(p), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <typename T, int V, int R, bool kLoose = false>
cudaError_t launch_v(const HeadParams &p, bool half, bool back, cudaStream_t s) {
  if (half)
    return back ? launch<T, V, R, true, true, kLoose>(p, s)
                : launch<T, V, R, true, false, kLoose>(p, s);
  return back ? launch<T, V, R, false, true, kLoose>(p, s)
              : launch<T, V, R, false, false, kLoose>(p, s);
}
// wide: the sizes are of whole vectors of 16 bytes; loose: they do not lie on 16 bytes
template <typename T>
cudaError_t launch_t(const HeadParams &p, bool wide, bool loose, bool half, bool back,
                     cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  int units = 0;
  for (int i = 0; i < p.nparts; ++i) units = p.part[i].units > units ? p.part[i].units : units;
  // sizes that 16-byte vectors do not fit, element by element: 2 x 8192 tokens of 32 + 8 + 8 heads of 126
  // take 376 us forward and 691 backward, of 128 69 and 100
  if (!wide)
    return units <= 32   ? launch_v<T, 1, 1>(p, half, back, s)
           : units <= 64 ? launch_v<T, 1, 2>(p, half, back, s)
                         : launch_v<T, 1, 8>(p, half, back, s);
  if constexpr (V == 4)
    if (units > 32)
      return loose ? launch_v<T, V, 2, true>(p, half, back, s) : launch_v<T, V, 2>(p, half, back, s);
  return loose ? launch_v<T, V, 1, true>(p, half, back, s) : launch_v<T, V, 1>(p, half, back, s);
}

struct Lay {
  Bytes x[3], dy[3], out[3];
  Bytes rest[4];  // frequencies, positions, weights
};

// Checks and fills everything but the addresses of partial sums.
dash_status_t fill(HeadParams &p, bool &wide, bool &loose, Lay &lay, const dash_rope_part_t *parts,
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
  loose = false;
  auto lies = [&](const void *at, const long long *stride, int heads, int D) {
    const long long count[3] = {B, S, heads};
    Bytes b = bytes_of(at, size, D);
    for (int k = 0; k < 3; ++k) b = along(b, size, stride[k], count[k]);
    return b;
  };
  auto lean = [&](const void *at, const long long *stride) {
    if (reinterpret_cast<uintptr_t>(at) & (size - 1)) return false;
    loose = loose || !aligned16(at) || (stride[0] | stride[1] | stride[2]) % vec != 0;
    return true;
  };
  int turned = 0, wsizes[2] = {};  // elements of the weights
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
      wsizes[turned] = q.D;
      h.w = weights[turned++];
      if (reinterpret_cast<uintptr_t>(h.w) & (wsize - 1)) return DASH_ERR_INVALID;
    }
    if (q.D > kMaxD) return DASH_ERR_UNSUPPORTED;
  }
  if (!turned) return DASH_ERR_INVALID;
  if ((long long)B * S >= (1LL << 31) - (1 << 16)) return DASH_ERR_UNSUPPORTED;
  for (int i = 0; i < nparts; ++i)
    if ((long long)parts[i].heads * parts[i].D >= (1LL << 28)) return DASH_ERR_UNSUPPORTED;
  // an output is its own input (the gradient), as it lies, or what nothing else is
  const int psize = positions64 ? 8 : 4;
  lay.rest[0] = bytes_of(inv_freq, 8, rot / 2);
  lay.rest[1] =
      along(along(bytes_of(positions, psize, 1), psize, pos_stride_t, S), psize, pos_stride_b, B);
  for (int i = 0; i < 2; ++i) lay.rest[2 + i] = bytes_of(weights[i], wsize, wsizes[i]);
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
    for (const Bytes &r : lay.rest)
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

cudaError_t launch_heads(const HeadParams &p, dash_dtype_t dtype, bool wide, bool loose, bool half,
                         bool back, cudaStream_t s) {
  if (dtype == DASH_BF16) return launch_t<__nv_bfloat16>(p, wide, loose, half, back, s);
  if (dtype == DASH_FP16) return launch_t<__half>(p, wide, loose, half, back, s);
  return launch_t<float>(p, wide, loose, half, back, s);
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
  bool wide, loose;
  Lay lay;
  dash_status_t st = fill(p, wide, loose, lay, parts, nullptr, nparts, weights, B, S, rot, layout, dtype,
                          wdtype, inv_freq, positions, positions64, pos_stride_b, pos_stride_t,
                          false);
  if (st != DASH_OK) return st;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  p.magnitude = magnitude, p.eps = eps, p.start = start;
  return launch_heads(p, dtype, wide, loose, layout == DASH_ROPE_HALF, false,
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
  bool wide, loose;
  Lay lay;
  dash_status_t st = fill(p, wide, loose, lay, parts, x, nparts, weights, B, S, rot, layout, dtype, wdtype,
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
    for (const Bytes &r : lay.rest)
      if (share(dw[i], r)) return DASH_ERR_INVALID;
  }
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  p.magnitude = magnitude, p.eps = eps, p.start = start;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_heads(p, dtype, wide, loose, layout == DASH_ROPE_HALF, true, s) != cudaSuccess)
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
