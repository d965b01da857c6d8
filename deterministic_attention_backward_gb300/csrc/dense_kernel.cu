// dense_kernel.cu -- the product kernel and the small kernels around it.
//
// Many rows: bound by the tensor core, and over more than a few milliseconds by the power limit.  A block
// of 64 contraction elements of a tile of 256 x 256 is 512 cycles of two SMs' tensor cores; measured 515
// to 520, the tensor pipe 94 to 96 % busy.  On the way there, 8192 x 4096 x 14336 in bf16:
//   one thread that brings in both operands                560 us  (85 cycles a box: 551 to 733 a block)
//   a converged warp for each operand, one lane issuing    487 us
//   groups of 16 rows of tiles (8: 567 under the power limit, 16: 556)
// cuBLAS takes 480 us, 535 to 550 under the power limit.  With gelu 570, gated forward 1160 (2 products),
// its backward 2500 (4 products, dz).  The epilogue runs beside the next tile's products; by rows through
// shared memory, so that a warp writes 64 bytes a row (a thread a row: 161 us at K = 512, now 110).
// Few rows: bound by the weights' bytes, see dense_few_kernel: 1 x 4096 x 14336 gated 37.3 us, 6.3 TB/s.
#include "dense.cuh"

#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"
#include "ptx.cuh"

namespace dash {
namespace {

constexpr int kStages = 6;
constexpr int kABytes = 128 * kDenseK * 2;  // one CTA's half of a tile's rows
constexpr int kStageBytes = 2 * kABytes;    // and its half of the columns (128 at most)
constexpr int kEpiWarps = 8;
constexpr int kThreads = (4 + kEpiWarps) * 32;
constexpr int kTurnBytes = 32 * 64;         // 32 rows of 32 two-byte elements
constexpr int kOffTurn = kStages * kStageBytes;  // two of them for each epilogue warp
constexpr int kOffBar = kOffTurn + 2 * kEpiWarps * kTurnBytes;
// full[], empty[], acc_full[2], acc_empty[2], drain
constexpr int kNumBars = 2 * kStages + 5;
constexpr int kOffMisc = kOffBar + kNumBars * 8;  // tmem address, abort flag
constexpr int kSmem = kOffMisc + 16;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kMnBox = kDenseK * 128;  // [64 x 64] box of an operand whose rows are contraction

// ------------------------------------------------------------------ pairs of CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (the aligned form wants whole warps: lanes that come out of a loop one by one meet first)
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The shared::cluster address of `p` in the CTA of rank 0.
__device__ __forceinline__ uint32_t in_leader(const void *p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Warp-wide wait (one answer for the whole warp); the limit runs from the 256th try on.  What is
// waited for comes from this CTA or its partners in the cluster, so that every wait runs out by itself:
// the status word is only written (its first CTA clears it, long before any limit).
template <bool kCluster>
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, const Abort &ab) {
  auto done = [&] {
    return __all_sync(0xffffffffu, kCluster ? try_wait_cluster(bar, parity)
                                            : mbar_try_wait(bar, parity));
  };
  if (done()) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (done()) return true;
    if ((it & 15u) == 0) {
      int stop = 0;
      if (lane_id() == 0) {
        if (ab.set()) {
          stop = 1;
        } else if ((it & 255u) == 0) {
          if (t0 == 0) t0 = globaltimer();
          if (globaltimer() - t0 > ab.limit_ns) {
            ab.raise(kErrMbarTimeout);
            stop = 1;
          }
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
  }
}
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, const Abort &ab) {
  return wait_for<true>(bar, parity, ab);
}
__device__ __forceinline__ bool wait_local(uint64_t *bar, uint32_t parity, const Abort &ab) {
  return wait_for<false>(bar, parity, ab);
}
// One box into this CTA's shared memory, its bytes counted on a barrier of either CTA; issued by the
// lane of a converged warp with `lead` set (a lane on its own takes 85 cycles a box).
__device__ __forceinline__ void load_box(uint32_t lead, uint32_t dst, const CUtensorMap *map,
                                         uint32_t bar, int c0, int c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void expect_l(uint32_t lead, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %2, 0;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
      "r"(bytes), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void alloc_pair(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(512u)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void dealloc_pair(uint32_t at) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(512u)
               : "memory");
}
// The same of a CTA alone.
__device__ __forceinline__ void load_box_alone(uint32_t lead, uint32_t dst, const CUtensorMap *map,
                                               uint32_t bar, int c0, int c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];\n\t}\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_alone(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit_alone(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::
          "r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// Adds the four values at shared address `at` of the cluster's CTAs, in order.
__device__ __forceinline__ void add_remote(float (&v)[4], uint32_t at, int ctas) {
  float r[8][4];
#pragma unroll
  for (int c = 0; c < 8; ++c)  // (all on their way before the first is needed)
    if (c < ctas) {
      uint32_t there;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(c));
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(r[c][0]), "=f"(r[c][1]), "=f"(r[c][2]), "=f"(r[c][3])
                   : "r"(there)
                   : "memory");
    }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    if (c < ctas)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] += r[c][k];
}
// D[tmem of both] (+)= A B^T, issued by the lane with `lead` set of the leader's warp.
__device__ __forceinline__ void mma_pair(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// One arrival on `bar` of both CTAs when the products issued so far are complete.
__device__ __forceinline__ void commit_pair(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "mov.b16 m, 3;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], m;\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// ------------------------------------------------------------------ activations
// 1 / (1 + e^-z), within a few units in the last place where it is not tiny: far below the rounding
// of the outputs to 16 bits.
__device__ __forceinline__ float sigmoid(float z) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2_approx(-kLog2e * z)));
  return r;
}
// z/2 (1 + tanh u) = z sigmoid(2u)
__device__ __forceinline__ float tanh_sigmoid(float z) {
  return sigmoid(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
}
template <int kAct>
__device__ __forceinline__ float activation(float z) {
  if constexpr (kAct == DASH_ACT_RELU) return z > 0.f || z != z ? z : 0.f;
  if constexpr (kAct == DASH_ACT_SILU) return z * sigmoid(z);
  if constexpr (kAct == DASH_ACT_GELU)
    return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  if constexpr (kAct == DASH_ACT_GELU_TANH) return z * tanh_sigmoid(z);
  return z;
}
// act(z) and its slope
template <int kAct>
__device__ __forceinline__ float activation(float z, float &slope) {
  if constexpr (kAct == DASH_ACT_RELU) {
    slope = z > 0.f ? 1.f : z != z ? z : 0.f;
    return activation<kAct>(z);
  }
  if constexpr (kAct == DASH_ACT_SILU) {
    const float s = sigmoid(z);
    slope = s * fmaf(z, 1.f - s, 1.f);
    return z * s;
  }
  if constexpr (kAct == DASH_ACT_GELU) {
    const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
    slope = fmaf(z, 0.39894228040143268f * ex2_approx(-0.5f * kLog2e * z * z), c);
    return z * c;
  }
  if constexpr (kAct == DASH_ACT_GELU_TANH) {
    const float s = tanh_sigmoid(z);
    const float t = s * (1.f - s);  // (0 at both ends, where what it multiplies may be infinite)
    slope = t > 0.f ? fmaf(t, 1.5957691216057308f * z * fmaf(0.134145f * z, z, 1.f), s) : s;
    return z * s;
  }
  slope = 1.f;
  return z;
}
template <int kAct, int C>
__device__ __forceinline__ void activate(float (&z)[C]) {
#pragma unroll
  for (int e = 0; e < C; ++e) z[e] = activation<kAct>(z[e]);
}
template <int C>
__device__ __forceinline__ void activate(int act, float (&z)[C]) {
  switch (act) {
    case DASH_ACT_RELU: return activate<DASH_ACT_RELU>(z);
    case DASH_ACT_GELU: return activate<DASH_ACT_GELU>(z);
    case DASH_ACT_GELU_TANH: return activate<DASH_ACT_GELU_TANH>(z);
    case DASH_ACT_SILU: return activate<DASH_ACT_SILU>(z);
    default: return;
  }
}

// Sets a word where one of the sums is infinite or NaN.
template <int C>
__device__ __forceinline__ void flag_special(uint32_t *set, const float (&v)[C]) {
  float zero[4] = {};  // (NaN from there on)
#pragma unroll
  for (int e = 0; e < C; ++e) zero[e & 3] = fmaf(v[e], 0.f, zero[e & 3]);
  if ((zero[0] + zero[1]) + (zero[2] + zero[3]) != 0.f) *set = 1;
}

// C values from column n of a row on, `left` of them inside it.
template <typename T, int C>
__device__ __forceinline__ void store_cols(void *base, long long at, const float (&v)[C], int left) {
  T *dst = static_cast<T *>(base) + at;
#pragma unroll
  for (int e = 0; e < C; ++e)
    if (e < left) dst[e] = from_f32<T>(v[e]);
}
template <typename T, int C>
__device__ __forceinline__ void add_cols(const void *base, long long at, float (&v)[C], int left) {
  const T *src = static_cast<const T *>(base) + at;
#pragma unroll
  for (int e = 0; e < C; ++e)
    if (e < left) v[e] += to_f32<T>(src[e]);
}
// Four values rounded to their upper 24 bits, to even between two (a NaN as it is: the addition would carry
// it over): two words of their upper halves and one of the bytes below.
__device__ __forceinline__ void split24(const float (&v)[4], uint32_t &h0, uint32_t &h1, uint32_t &l) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = __float_as_uint(v[i]);
    if (v[i] == v[i]) b[i] += 0x7fu + (b[i] >> 8 & 1u);
  }
  h0 = __byte_perm(b[0], b[1], 0x7632);
  h1 = __byte_perm(b[2], b[3], 0x7632);
  l = __byte_perm(__byte_perm(b[0], b[1], 0x0051), __byte_perm(b[2], b[3], 0x0051), 0x5410);
}
__device__ __forceinline__ float join24(uint32_t hi, uint32_t lo) {
  return __uint_as_float(hi << 16 | lo << 8);
}
// Four values of a row from column n on (rows have room for whole groups of four).
__device__ __forceinline__ void keep_cols(const DenseKept &k, long long stride, long long row, int n,
                                          const float (&v)[4]) {
  uint32_t h0, h1, l;
  split24(v, h0, h1, l);
  *reinterpret_cast<uint2 *>(k.hi + row * stride + n) = make_uint2(h0, h1);
  *reinterpret_cast<uint32_t *>(k.lo + row * stride + n) = l;
}

// A bias, the same for all rows of a warp.
template <typename T>
__device__ __forceinline__ void add_bias(const void *base, int n, float (&v)[32], int left, int lane) {
  const T *src = static_cast<const T *>(base) + n;
  if (left >= 32 && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[8];
      unpack<T, 8>(load_pack<T, 8>(src + 8 * i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] += f[e];
    }
  } else {  // a lane brings one column's and hands it round
    const float b = lane < left ? to_f32<T>(src[lane]) : 0.f;
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] += __shfl_sync(0xffffffffu, b, e);
  }
}

// ------------------------------------------------------------------ rows and columns change places
// A thread of the epilogue holds 32 columns of a row; memory wants the lanes of a warp along a
// row.  A turn buffer holds 32 rows of 64 bytes, the 16-byte pieces of a row permuted so that
// neither way meets a bank twice.
__device__ __forceinline__ uint8_t *turn_at(uint8_t *buf, int row, int piece) {
  return buf + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}
// This thread's row into the buffer, and what the buffer has of it added.
template <typename T>
__device__ __forceinline__ void turn_put(uint8_t *buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e];
    store_pack<T, 8>(reinterpret_cast<T *>(turn_at(buf, lane, i)), pack<T, 8>(f));
  }
}
template <typename T>
__device__ __forceinline__ void turn_add(uint8_t *buf, int lane, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
    unpack<T, 8>(load_pack<T, 8>(reinterpret_cast<const T *>(turn_at(buf, lane, i))), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[8 * i + e] += f[e];
  }
}
// The buffer to rows [row0, row0 + rows) of a tensor, columns [n, n + left): by 16-byte pieces, four
// lanes a row; a piece that ends behind the row by its elements.
template <typename T>
__device__ __forceinline__ void turn_store(uint8_t *buf, void *base, long long stride, long long row0,
                                           int rows, int n, int left, int lane) {
  T *dst = static_cast<T *>(base) + row0 * stride + n;
  const int c = lane & 3, in = left - 8 * c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (r >= rows) continue;
    const Pack<T, 8> v = load_pack<T, 8>(reinterpret_cast<const T *>(turn_at(buf, r, c)));
    T *to = dst + r * stride + 8 * c;
    if (in >= 8) {
      store_pack<T, 8>(to, v);
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < in) to[e] = v.e[e];
    }
  }
}
// The same pieces of a tensor that is read, and into the buffer.
template <typename T>
__device__ __forceinline__ void turn_fetch(uint4 (&v)[4], const void *base, long long stride,
                                           long long row0, int rows, int n, int left, int lane) {
  const T *src = static_cast<const T *>(base) + row0 * stride + n;
  const int c = lane & 3, in = left - 8 * c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= rows) continue;
    const T *from = src + r * stride + 8 * c;
    if (in >= 8) {
      v[i] = *reinterpret_cast<const uint4 *>(from);
    } else if (in > 0) {
      Pack<T, 8> p;
#pragma unroll
      for (int e = 0; e < 8; ++e) p.e[e] = e < in ? from[e] : from_f32<T>(0.f);
      v[i] = *reinterpret_cast<const uint4 *>(&p);
    }
  }
}
__device__ __forceinline__ void turn_fill(uint8_t *buf, const uint4 (&v)[4], int lane) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4 *>(turn_at(buf, 8 * i + (lane >> 2), lane & 3)) = v[i];
}

// 32 rows of 32 values, a thread a row, to rows [row0, row0 + rows) of what is kept, from column n on:
// the words through one buffer, the bytes (32 a row, in two pieces) through the other.
__device__ __forceinline__ void turn_keep(uint8_t *words, uint8_t *bytes, const DenseKept &k,
                                          long long stride, long long row0, int rows, int n, int lane,
                                          const float (&v)[32]) {
  uint32_t h[16], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f[4] = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    split24(f, h[2 * i], h[2 * i + 1], l[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4 *>(turn_at(words, lane, i)) =
        make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  auto byte_at = [&](int row, int piece) { return bytes + row * 32 + ((piece ^ (row >> 2 & 1)) << 4); };
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint4 *>(byte_at(lane, i)) =
        make_uint4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
  __syncwarp();
  const int c = lane & 3, room = (int)stride - n;  // (a multiple of 16)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + (lane >> 2);
    if (r < rows && 8 * c < room)
      *reinterpret_cast<uint4 *>(k.hi + (row0 + r) * stride + n + 8 * c) =
          *reinterpret_cast<const uint4 *>(turn_at(words, r, c));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 16 * i + (lane >> 1), d = lane & 1;
    if (r < rows && 16 * d < room)
      *reinterpret_cast<uint4 *>(k.lo + (row0 + r) * stride + n + 16 * d) =
          *reinterpret_cast<const uint4 *>(byte_at(r, d));
  }
  __syncwarp();
}

__device__ __forceinline__ void load32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
}

// Work items: the first `whole` tiles, then `splits` items for each of the others.  Tiles go in
// groups of `group` rows of tiles, so that those in flight share their operands in L2.
struct Item {
  int m, n, out, k0, k1;
  int cut;  // of a split tile: its place in the partial sums, else -1
};
__device__ __forceinline__ Item item_of(const DenseParams &p, int t) {
  Item w;
  w.cut = -1;
  w.k0 = 0, w.k1 = p.nk * p.parts;
  if (t >= p.whole) {
    const int j = t - p.whole, tile = j / p.splits;
    if (p.splits > 1 || p.stack) {
      w.cut = j;
      w.k0 = (j - tile * p.splits) * p.per;
      w.k1 = min(w.k0 + p.per, w.k1);
    }
    t = p.whole + tile;
  }
  const int tiles = p.mt * p.nt, r = t % tiles;
  w.out = t / tiles;
  const int per = p.group * p.nt, g = r / per, in = r - g * per;
  const int rows = min(p.group, p.mt - p.group * g);
  w.m = (p.group * g + in % rows) * kDenseM;
  w.n = in / rows;
  return w;
}

// ------------------------------------------------------------------ the product
// One pair of CTAs a tile of 256 rows and bn (256 or 128) columns, persistent over the work items.
// Each CTA brings in its half of the rows and of the columns; the leader's tensor core instruction
// reads both halves and leaves each CTA its 128 rows in its own TMEM, where two accumulators
// alternate so that a tile's epilogue runs beside the next one's products.
// Warps 0 and 3 TMA producers, 1 MMA issuer (leader), 2 TMEM, 4-11 epilogue (thread = row; the two
// warpgroups share the columns).
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap ta1,
                 const __grid_constant__ CUtensorMap tb0, const __grid_constant__ CUtensorMap tb1,
                 const __grid_constant__ DenseParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (p.clear && blockIdx.x == 0 && threadIdx.x < kStatusBytes / 4) p.status[threadIdx.x] = 0;
  // (the same for both CTAs, which leave together)
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrSmemAlign);
    return;
  }
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + kOffBar);
  uint64_t *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2;
  uint64_t *drain = acc_empty + 2;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + kOffMisc);
  int *s_abort = reinterpret_cast<int *>(smem + kOffMisc + 4);
  const Abort ab{s_abort, p.status, p.wait_ns};
  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  const int tiles = p.mt * p.nt * p.outs, items = p.whole + (tiles - p.whole) * p.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&ta0);
    tma_prefetch_desc(&tb0);
  }
  if (warp == 2) alloc_pair(s_tmem);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------------ TMA producers
    // Warp 0 brings in A, warp 3 B, so that neither's instructions hold up the tensor core.
    const bool isb = warp == 3;
    const int half = p.bn / 2;  // columns that this CTA brings in
    const bool mn = isb ? p.b_mn : p.a_mn;
    const int boxes = mn ? (isb ? half / 64 : 2) : 1;
    const uint32_t bytes = 2 * (isb ? half * kDenseK * 2 : kABytes);
    const uint32_t lead = elect_one(), base = smem_u32(smem) + (isb ? kABytes : 0);
    const uint32_t bar0 = in_leader(full), own0 = smem_u32(full), signals = leader ? lead : 0;
    bool ok = true;
    int it = 0, s = 0;
    uint32_t ph = 1;
    for (int t = first; ok && t < items; t += step) {
      const Item w = item_of(p, t);
      // gated: the leader brings w's columns of the tile, the other CTA w_gate's
      const int at = !isb         ? w.m + (int)rank * (p.stack ? p.a_low : 128)
                     : p.e.gated ? w.n * half
                                 : w.n * p.bn + (int)rank * half;
      const bool second = isb ? (w.out && p.b_out) || (p.e.gated && rank) : w.out && p.a_out;
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        if (it == p.withhold || !wait_pair(&empty[s], ph, ab)) {
          ok = false;
          break;
        }
        const int q = (k >= p.nk) + (k >= 2 * p.nk) + (k >= 3 * p.nk);
        const int term = p.pairs ? q >> 1 : q, kk = (k - q * p.nk) * kDenseK;
        const int low = term * (isb ? p.b_low : p.a_low);  // (0 where terms are stacked)
        const CUtensorMap *map =
            (p.pairs && (q & 1)) || second ? (isb ? &tb1 : &ta1) : (isb ? &tb0 : &ta0);
        const uint32_t bar = bar0 + 8 * s, dst = base + s * kStageBytes;
        expect_l(signals, own0 + 8 * s, bytes);
        if (mn) {
          load_box(lead, dst, map, bar, at, kk + low);
          if (boxes > 1) load_box(lead, dst + kMnBox, map, bar, at + 64, kk + low);
        } else {
          load_box(lead, dst, map, bar, kk, at + low);
        }
        if (++s == kStages) s = 0, ph ^= 1;
      }
    }
    // Leave no copy in flight into shared memory, whichever warp it was that gave up: both producers, as
    // one may be ahead of the other (the leader's barriers count the other CTA's copies too).
    if (leader)
      for (int j = max(0, it - kStages); j < it; ++j)
        mbar_wait_drain(&full[j % kStages], (j / kStages) & 1, 100000000ull);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (leader) {
      const uint32_t kind = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
      const uint32_t idesc = (1u << 4) | kind | ((uint32_t)p.a_mn << 15) |
                             ((uint32_t)p.b_mn << 16) | ((uint32_t)(p.bn >> 3) << 17) |
                             ((uint32_t)(kDenseM >> 4) << 24);
      // a step of 16 contraction elements: 32 bytes along a row, or 16 rows of 128 bytes
      const uint32_t astep = (p.a_mn ? 2048 : 32) >> 4, bstep = (p.b_mn ? 2048 : 32) >> 4;
      const uint32_t base = smem_u32(smem), lead = elect_one();
      bool ok = true;
      int it = 0, n = 0;
      for (int t = first; ok && t < items; t += step, ++n) {
        const Item w = item_of(p, t);
        ok = wait_pair(&acc_empty[n & 1], ((n >> 1) & 1) ^ 1, ab);
        tc_fence_after();
        const uint32_t d = tmem + (n & 1) * 256;
        for (int k = w.k0; ok && k < w.k1; ++k, ++it) {
          const int s = it % kStages;
          ok = wait_pair(&full[s], (it / kStages) & 1, ab);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = desc_lo(base + s * kStageBytes, p.a_mn ? kMnBox : 16);
          const uint32_t b = desc_lo(base + s * kStageBytes + kABytes, p.b_mn ? kMnBox : 16);
#pragma unroll
          for (int j = 0; j < kDenseK / 16; ++j)
            mma_pair(lead, d, desc_of(a + j * astep), desc_of(b + j * bstep), idesc,
                     (k > w.k0 || j > 0) ? 1u : 0u);
          commit_pair(lead, &empty[s]);
        }
        if (ok) commit_pair(lead, &acc_full[n & 1]);
      }
      commit_pair(lead, drain);
      mbar_wait_drain(drain, 0, 100000000ull);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3, wg = (warp - 4) >> 2;
    uint8_t *turn = smem + kOffTurn + (warp - 4) * 2 * kTurnBytes, *turn2 = turn + kTurnBytes;
    const DenseEpilogue &e = p.e;
    const int cols = e.gated ? p.bn / 2 : p.bn;  // output columns of a tile
    const int c0 = wg * (cols / 2), c1 = c0 + cols / 2;
    int n = 0;
    for (int t = first; t < items; t += step, ++n) {
      const Item w = item_of(p, t);
      const long long row0 = w.m + (p.stack ? 0 : (int)rank * 128) + quad * 32;
      const int rows = (int)max(0ll, min(32ll, p.M - row0));
      const int n0 = w.n * cols;
      // the residual's pieces are under way while the products are formed
      uint4 next[4];
      if (e.residual && w.cut < 0 && n0 + c0 < p.N)
        turn_fetch<T>(next, e.residual, e.rs, row0, rows, n0 + c0, p.N - n0 - c0, lane);
      if (!wait_pair(&acc_full[n & 1], (n >> 1) & 1, ab)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (n & 1) * 256;
      if (w.cut >= 0) {
        float *dst = p.part + (((long long)w.cut * 2 + rank) * 128 + quad * 32 + lane) * p.bn;
        for (int c = wg * (p.bn / 2); c < (wg + 1) * (p.bn / 2); c += 32) {
          float v[32];
          load32(acc + c, v);
          if (lane < rows) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4 *>(dst + c + 4 * i) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      } else {
        void *y = w.out ? p.y1 : e.y;
        const long long ys = w.out ? p.y1s : e.ys;
        for (int c = c0; c < c1; c += 32) {
          const int at = n0 + c, left = p.N - at;
          if (left <= 0) break;
          // (a barrier lies between a buffer's reads and its next filling)
          float z[32], g[32];
          load32(acc + c, z);
          if (e.gated) load32(acc + p.bn / 2 + c, g);
          if (p.special) flag_special(p.special, z);
          if (e.bias) add_bias<T>(e.bias, at, z, left, lane);
          if (e.z.hi) turn_keep(turn, turn2, e.z, e.ks, row0, rows, at, lane, z);
          if (e.gated) {
            if (e.bias_gate) add_bias<T>(e.bias_gate, at, g, left, lane);
            if (e.g.hi) turn_keep(turn, turn2, e.g, e.ks, row0, rows, at, lane, g);
          }
          activate(e.act, z);
          if (e.gated) {
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] *= g[i];
          }
          if (e.residual) {
            turn_fill(turn, next, lane);
            if (c + 32 < c1 && left > 32)
              turn_fetch<T>(next, e.residual, e.rs, row0, rows, at + 32, left - 32, lane);
            __syncwarp();
            turn_add<T>(turn, lane, z);
          }
          turn_put<T>(turn2, lane, z);
          __syncwarp();
          turn_store<T>(turn2, y, ys, row0, rows, at, left, lane);
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_cluster(in_leader(&acc_empty[n & 1]));
    }
  }

  tc_fence_before();
  __syncthreads();
  // the leader's last arrivals here come in before this CTA can end
  if (!leader && warp == 1) mbar_wait_drain(drain, 0, 100000000ull);
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    dealloc_pair(tmem);
  }
}

// The epilogue of 4 columns of a row.
template <typename T>
__device__ __forceinline__ void finish4(const DenseEpilogue &e, void *y, long long ys, long long row,
                                        int n, int N, float (&z)[4], float (&g)[4]) {
  const int left = N - n;
  if (e.bias) add_cols<T, 4>(e.bias, n, z, left);
  if (e.z.hi) keep_cols(e.z, e.ks, row, n, z);
  activate(e.act, z);
  if (e.gated) {
    if (e.bias_gate) add_cols<T, 4>(e.bias_gate, n, g, left);
    if (e.g.hi) keep_cols(e.g, e.ks, row, n, g);
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] *= g[k];
  }
  if (e.residual) add_cols<T, 4>(e.residual, row * e.rs + n, z, left);
  store_cols<T, 4>(y, row * ys + n, z, left);
}

// The splits' sums of the tiles that were split, added in order, and the epilogue; a thread takes 4
// columns of a row, a CTA's y one tile.
template <typename T>
__global__ void __launch_bounds__(256) dense_finish_kernel(const __grid_constant__ DenseParams p) {
  const DenseEpilogue &e = p.e;
  const int cols = e.gated ? p.bn / 2 : p.bn, groups = cols / 4;
  const int i = blockIdx.x * 256 + threadIdx.x, r = i / groups, c = (i - r * groups) * 4;
  const Item w = item_of(p, p.whole + blockIdx.y * p.splits);
  const long long row = w.m + r;
  const int n = w.n * cols + c;
  if (row >= p.M || n >= p.N) return;
  float z[4] = {}, g[4] = {};
  const long long stride = (long long)kDenseM * p.bn;
  const float *src = p.part + w.cut * stride + (long long)r * p.bn + c;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s, src += stride) {
    const float4 v = *reinterpret_cast<const float4 *>(src);
    z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
    if (e.gated || p.stack) {
      const float4 u = *reinterpret_cast<const float4 *>(src + (p.stack ? 128 * p.bn : p.bn / 2));
      g[0] += u.x, g[1] += u.y, g[2] += u.z, g[3] += u.w;
    }
  }
  if (p.stack)  // the second term
#pragma unroll
    for (int k = 0; k < 4; ++k) z[k] = isfinite(z[k]) ? z[k] + g[k] : z[k];
  else if (p.special)
    flag_special(p.special, z);
  finish4<T>(e, w.out ? p.y1 : e.y, w.out ? p.y1s : e.ys, row, n, p.N, z, g);
}

// ------------------------------------------------------------------ few rows
// Up to 64 rows of x: bound by the weights' way through the SMs (with the kernel above one row x 4096 x
// 14336 gated took 61 us, 17 x 14336 x 4096 31, now 37.3 and 22.4).  The weights are the rows of the tensor
// core's tile here (128 outputs), x its columns, so that nothing but x is read that is not needed.  A
// cluster shares a tile: every CTA forms the sums over its part of the contraction, leaves them in its
// shared memory, and finishes its share of the outputs from all CTAs' sums, added in order.
// 4 warps: 0 brings in the operands, 1 issues the products, 2 holds TMEM; all finish.
constexpr int kFewThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kFewThreads)
    dense_few_kernel(const __grid_constant__ CUtensorMap tw0, const __grid_constant__ CUtensorMap tw1,
                     const __grid_constant__ CUtensorMap tx, const __grid_constant__ DenseFewParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ uint64_t full[kFewStages], empty[kFewStages], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_rank();
  const int tile = blockIdx.x / p.split;
  if (blockIdx.x == 0 && threadIdx.x < kStatusBytes / 4) p.status[threadIdx.x] = 0;
  const Abort ab{&s_abort, p.status, p.wait_ns};
  const bool gated = p.e.gated;
  const int k0 = (int)rank * p.per, k1 = min(k0 + p.per, p.nk);
  const int n0 = tile * 128;
  const uint32_t base = smem_u32(smem), xoff = gated ? 2 * kABytes : kABytes;
  const bool aligned = (base & 1023u) == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done, 1);
    s_abort = aligned ? 0 : 1;
    if (!aligned) atomicOr(p.status, kErrSmemAlign);
    fence_mbar_init();
  }
  // the blocks of one filling of the ring are on their way before the others are ready to take them
  uint32_t lead = 0;
  auto bring = [&](int k, int s) {
    const uint32_t at = base + s * p.stage, bar = smem_u32(&full[s]);
    expect_l(lead, bar, xoff + p.cols * 128);
    for (int g = 0; g <= (int)gated; ++g) {
      const CUtensorMap *map = g ? &tw1 : &tw0;
      const uint32_t to = at + g * kABytes;
      if (p.w_mn) {
        load_box_alone(lead, to, map, bar, n0, k * kDenseK);
        load_box_alone(lead, to + kMnBox, map, bar, n0 + 64, k * kDenseK);
      } else {
        load_box_alone(lead, to, map, bar, k * kDenseK, n0);
      }
    }
    load_box_alone(lead, at + xoff, &tx, bar, k * kDenseK, 0);
  };
  int it = 0;
  const int wanted = p.withhold >= 0 && p.withhold < k1 - k0 ? p.withhold : k1 - k0;
  if (warp == 0 && aligned) {
    __syncwarp();
    lead = elect_one();
    for (; it < wanted && it < p.stages; ++it) bring(k0 + it, it);
  }
  if (warp == 2) {
    tmem_alloc(&s_tmem, p.tmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  bool ok = aligned;
  if (ok && warp == 0) {
    int s = it == p.stages ? 0 : it;
    uint32_t ph = 0;
    for (; it < wanted; ++it) {
      if (!wait_local(&empty[s], ph, ab)) {
        ok = false;
        break;
      }
      bring(k0 + it, s);
      if (++s == p.stages) s = 0, ph ^= 1;
    }
    // leave no copy in flight into shared memory, whichever warp it was that gave up
    for (int j = max(0, it - p.stages); j < it; ++j)
      mbar_wait_drain(&full[j % p.stages], (j / p.stages) & 1, 100000000ull);
  } else if (ok && warp == 1) {
    const uint32_t kind = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
    const uint32_t idesc = (1u << 4) | kind | ((uint32_t)p.w_mn << 15) |
                           ((uint32_t)(p.cols >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t wstep = (p.w_mn ? 2048 : 32) >> 4;
    lead = elect_one();
    int s = 0;
    uint32_t ph = 0;
    for (int k = k0; ok && k < k1; ++k) {
      ok = wait_local(&full[s], ph, ab);
      if (!ok) break;
      tc_fence_after();
      const uint32_t x = desc_lo(base + s * p.stage + xoff, 16);
      for (int g = 0; g <= (int)gated; ++g) {
        const uint32_t w = desc_lo(base + s * p.stage + g * kABytes, p.w_mn ? kMnBox : 16);
#pragma unroll
        for (int j = 0; j < kDenseK / 16; ++j)
          mma_alone(lead, tmem + g * p.cols, desc_of(w + j * wstep), desc_of(x + j * 2), idesc,
                    (k > k0 || j > 0) ? 1u : 0u);
      }
      commit_alone(lead, &empty[s]);
      if (++s == p.stages) s = 0, ph ^= 1;
    }
    commit_alone(lead, &done);
    mbar_wait_drain(&done, 0, 100000000ull);
  }
  __syncwarp();
  __syncthreads();  // all operands have been read: their place takes the sums
  tc_fence_after();
  const bool good = !s_abort;
  float *sums = reinterpret_cast<float *>(smem);  // [z, g][row][128]
  if (good) {
    const uint32_t acc = tmem + ((uint32_t)(warp * 32) << 16);
    for (int c = 0; c < (gated ? 2 : 1) * p.cols; c += 16) {
      uint32_t r[16];
      load16(acc + c, r);
#pragma unroll
      for (int e = 0; e < 16; ++e) sums[(c + e) * 128 + threadIdx.x] = __uint_as_float(r[e]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem);
  }
  cluster_sync();
  if (good) {
    // this CTA's groups of 4 outputs of a row
    const int groups = p.M * 32, each = (groups + p.split - 1) / p.split;
    const int end = min(groups, ((int)rank + 1) * each);
    for (int i = (int)rank * each + threadIdx.x; i < end; i += kFewThreads) {
      const int row = i >> 5, n = n0 + (i & 31) * 4;
      if (n >= p.N) continue;
      float z[4] = {}, g[4] = {};
      add_remote(z, base + i * 16, p.split);
      if (gated) add_remote(g, base + (p.cols * 32 + i) * 16, p.split);
      finish4<T>(p.e, p.e.y, p.e.ys, row, n, p.N, z, g);
    }
  }
  cluster_sync();  // the others have read what is here
}

// ------------------------------------------------------------------ infinities and NaN of two terms
// Ends at once where no product has set the word (the launch and the products' look at their sums take 2 to
// 5 us: dw of 8 x 14336 x 8192 97 -> 102; sums in accumulators apart, 128 columns a tile, 128).  Otherwise
// the tiles of 64 x 64 that have such an element are summed in fp32, 4 x 4 elements a thread, so that a step
// whose gradients are all NaN takes 28 ms at 8192 x 4096 x 4096 and no longer.
template <typename T>
__global__ void __launch_bounds__(256) dense_specials_kernel(const __grid_constant__ DenseSpecials p) {
  const DenseSpecial &q = p.s[blockIdx.y];
  if (!q.out || *p.set == 0) return;
  constexpr int kTileSide = 64, kDeep = 16;
  __shared__ float side[2][kDeep][kTileSide + 1];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long across = (q.cols + kTileSide - 1) / kTileSide;
  const long long tiles = (q.rows + kTileSide - 1) / kTileSide * across;
  auto at = [&](int r, int c) { return static_cast<T *>(q.out) + r * q.stride + c; };
  for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int r0 = (int)(tile / across) * kTileSide, c0 = (int)(tile % across) * kTileSide;
    uint32_t wanted = 0;
    for (int i = 0; i < 16; ++i) {
      const int r = r0 + ty + 16 * (i >> 2), c = c0 + tx + 16 * (i & 3);
      if (r < q.rows && c < q.cols && !isfinite(to_f32<T>(*at(r, c)))) wanted |= 1u << i;
    }
    if (!__syncthreads_or(wanted != 0)) continue;
    float sum[4][4] = {};
    for (int part = 0; part < q.parts; ++part)
      for (int k0 = 0; k0 < q.K; k0 += kDeep) {
        for (int which = 0; which < 2; ++which) {
          const DenseOperand &o = which ? q.b[part] : q.a[part];
          const int first = which ? c0 : r0, end = which ? q.cols : q.rows;
          for (int i = threadIdx.x; i < kDeep * kTileSide; i += 256) {  // along its contiguous dimension
            const int k = o.k == 1 ? i & (kDeep - 1) : i / kTileSide;
            const int r = o.k == 1 ? i / kDeep : i & (kTileSide - 1);
            side[which][k][r] =
                k0 + k < q.K && first + r < end
                    ? to_f32<T>(static_cast<const T *>(o.at)[(first + r) * o.row + (k0 + k) * o.k])
                    : 0.f;
          }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              sum[i][j] = fmaf(side[0][k][ty + 16 * i], side[1][k][tx + 16 * j], sum[i][j]);
        __syncthreads();
      }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (wanted >> i & 1) *at(r0 + ty + 16 * (i >> 2), c0 + tx + 16 * (i & 3)) = from_f32<T>(sum[i >> 2][i & 3]);
  }
}

// ------------------------------------------------------------------ dz, dgate and their sums
// 32 threads a strip of 256 columns, 8 rows at a time over a chunk of rows; the eight rows' sums are
// added in order through shared memory.  Bound by memory: 8192 x 14336 gated, 12 bytes an element, in
// 226 us, 6.2 TB/s.  Registers decide how much is on its way: without the sums 4 CTAs are on an SM (two rows
// at once, 153 registers: twice the time).
template <typename T, int kAct, bool kSums>
__global__ void __launch_bounds__(256, kSums ? 3 : 4)
    dense_grad_kernel(const __grid_constant__ DenseGradParams p) {
  constexpr int V = 8;
  const int lane = threadIdx.x & 31, by = threadIdx.x >> 5;
  const int n = (blockIdx.x * 32 + lane) * V;
  const int r1 = min(p.M, (int)(blockIdx.y + 1) * p.chunk);
  const bool whole = p.vec && n + V <= p.N;
  float sz[V] = {}, sg[V] = {};
  if (p.special && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.special = 0;
  auto kept = [&](const DenseKept &k, long long r, uint4 &h, uint2 &l) {
    h = *reinterpret_cast<const uint4 *>(k.hi + r * p.ks + n);
    l = *reinterpret_cast<const uint2 *>(k.lo + r * p.ks + n);
  };
  auto values = [](const uint4 &h, const uint2 &l, float (&f)[V]) {
    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[2] = {l.x, l.y};
#pragma unroll
    for (int e = 0; e < V; ++e)
      f[e] = join24(hw[e / 2] >> (16 * (e & 1)), (lw[e / 4] >> (8 * (e & 3))) & 0xffu);
  };
  if (n < p.N) {
    for (long long r = blockIdx.y * p.chunk + by; r < r1; r += 8) {
      float dy[V], z[V], g[V];
      uint4 zh, gh;
      uint2 zl, gl;
      Pack<T, V> d;
      const T *src = static_cast<const T *>(p.dy) + r * p.dys + n;
      if (whole) {
        d = load_pack<T, V>(src);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) d.e[e] = n + e < p.N ? src[e] : from_f32<T>(0.f);
      }
      if (p.z.hi) kept(p.z, r, zh, zl);
      if (p.g.hi) kept(p.g, r, gh, gl);
      unpack<T, V>(d, dy);
      if (p.z.hi) {
        values(zh, zl, z);
        if (p.g.hi) values(gh, gl, g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float slope;
          const float a = activation<kAct>(z[e], slope);
          z[e] = dy[e] * slope;
          if (p.g.hi) {
            z[e] *= g[e];
            g[e] = dy[e] * a;
          }
        }
        auto put = [&](void *base, const float(&f)[V]) {
          T *to = static_cast<T *>(base) + r * p.ds + n;
          const Pack<T, V> v = pack<T, V>(f);
          store_pack<T, V>(to, v);
          if (p.low) {
            float l[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              l[e] = f[e] - to_f32<T>(v.e[e]);
              if (!isfinite(l[e])) l[e] = 0.f;
            }
            store_pack<T, V>(to + (long long)p.M * p.ds, pack<T, V>(l));
          }
        };
        if (p.dz) put(p.dz, z);
        if (p.g.hi && p.dg) put(p.dg, g);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = dy[e];
      }
      if constexpr (kSums) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          sz[e] += z[e];
          if (p.g.hi) sg[e] += g[e];
        }
      }
    }
  }
  if constexpr (kSums) {
    __shared__ float sums[2][8][32 * V + 1];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sums[0][by][lane * V + e] = sz[e];
      sums[1][by][lane * V + e] = sg[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * V; i += 256) {
      const int which = i / (32 * V), c = i % (32 * V), col = blockIdx.x * 32 * V + c;
      float *dst = which ? p.part_gate : p.part;
      if (!dst || col >= p.N) continue;
      float s = 0.f;
#pragma unroll
      for (int b = 0; b < 8; ++b) s += sums[which][b][c];
      dst[(long long)blockIdx.y * p.N + col] = s;
    }
  }
}

// 8 runs of chunks for each of 32 columns, then the runs, in order.
template <typename T>
__global__ void __launch_bounds__(256) dense_sums_kernel(const float *part, const float *part_gate,
                                                         void *out, void *out_gate, int chunks,
                                                         int N) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, n = blockIdx.x * 32 + lane;
  const float *src = blockIdx.y ? part_gate : part;
  T *dst = static_cast<T *>(blockIdx.y ? out_gate : out);
  if (!src || !dst) return;
  const int per = (chunks + 7) / 8, end = min(chunks, (run + 1) * per);
  float s = 0.f;
  if (n < N)
#pragma unroll 8
    for (int c = run * per; c < end; ++c) s += src[(long long)c * N + n];
  sums[run][lane] = s;
  __syncthreads();
  if (run > 0 || n >= N) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) s += sums[r][lane];
  dst[n] = from_f32<T>(s);
}

// A thread writes 16 bytes; a row's reads, which lie on no boundary, meet in L1.
__global__ void __launch_bounds__(256) dense_copy_kernel(const __grid_constant__ DenseCopies p) {
  const DenseCopy &q = p.c[blockIdx.z];
  const int c = (blockIdx.x * 32 + (threadIdx.x & 31)) * 8;
  if (c >= q.cols) return;
  for (long long r = blockIdx.y * 8 + (threadIdx.x >> 5); r < q.rows; r += gridDim.y * 8) {
    const uint16_t *src = static_cast<const uint16_t *>(q.in) + r * q.is + c;
    Pack<uint16_t, 8> v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.e[e] = c + e < q.cols ? src[e] : (uint16_t)0;
    store_pack<uint16_t, 8>(static_cast<uint16_t *>(q.out) + r * q.os + c, v);
  }
}
__global__ void __launch_bounds__(256) dense_copy_out_kernel(const __grid_constant__ DenseCopies p) {
  const DenseCopy &q = p.c[blockIdx.z];
  const int c = blockIdx.x * 128 + (threadIdx.x & 31);
  for (long long r = blockIdx.y * 8 + (threadIdx.x >> 5); r < q.rows; r += gridDim.y * 8) {
    const uint16_t *src = static_cast<const uint16_t *>(q.in) + r * q.is + c;
    uint16_t *dst = static_cast<uint16_t *>(q.out) + r * q.os + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 32 * i < q.cols) dst[32 * i] = src[32 * i];
  }
}

template <typename T>
cudaError_t launch_t(const CUtensorMap (&ta)[2], const CUtensorMap (&tb)[2], const DenseParams &p,
                     int sms, cudaStream_t s) {
  const cudaError_t e = allow_smem<dense_kernel<T>>(kSmem);
  if (e != cudaSuccess) return e;
  const int rest = p.mt * p.nt * p.outs - p.whole, items = p.whole + rest * p.splits;
  const int pairs = items < sms / 2 ? items : sms / 2;
  dense_kernel<T><<<2 * pairs, kThreads, kSmem, s>>>(ta[0], ta[1], tb[0], tb[1], p);
  if (rest > 0 && (p.splits > 1 || p.stack)) {
    const int rows = p.M < kDenseM ? p.M : kDenseM, cols = p.e.gated ? p.bn / 2 : p.bn;
    dense_finish_kernel<T><<<dim3((rows * (cols / 4) + 255) / 256, rest), 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_few_t(const CUtensorMap &tw0, const CUtensorMap &tw1, const CUtensorMap &tx,
                         const DenseFewParams &p, cudaStream_t s) {
  const cudaError_t e = allow_smem<dense_few_kernel<T>>(kFewSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((p.N + 127) / 128 * p.split);
  c.blockDim = dim3(kFewThreads);
  c.dynamicSmemBytes = p.smem;
  c.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = p.split, a.val.clusterDim.y = a.val.clusterDim.z = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, dense_few_kernel<T>, tw0, tw1, tx, p);
}

template <typename T, int kAct>
void launch_grad_t(const DenseGradParams &p, int chunks, cudaStream_t s) {
  const dim3 grid((p.N + 255) / 256, chunks);
  if (p.part || p.part_gate)
    dense_grad_kernel<T, kAct, true><<<grid, 256, 0, s>>>(p);
  else
    dense_grad_kernel<T, kAct, false><<<grid, 256, 0, s>>>(p);
}
template <int kAct>
cudaError_t launch_grad(bool f16, const DenseGradParams &p, int chunks, cudaStream_t s) {
  f16 ? launch_grad_t<__half, kAct>(p, chunks, s) : launch_grad_t<__nv_bfloat16, kAct>(p, chunks, s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense(bool f16, const CUtensorMap (&ta)[2], const CUtensorMap (&tb)[2],
                         const DenseParams &p, int sms, cudaStream_t s) {
  return f16 ? launch_t<__half>(ta, tb, p, sms, s) : launch_t<__nv_bfloat16>(ta, tb, p, sms, s);
}

cudaError_t launch_dense_few(bool f16, const CUtensorMap &tw0, const CUtensorMap &tw1,
                             const CUtensorMap &tx, const DenseFewParams &p, cudaStream_t s) {
  return f16 ? launch_few_t<__half>(tw0, tw1, tx, p, s)
             : launch_few_t<__nv_bfloat16>(tw0, tw1, tx, p, s);
}

cudaError_t launch_dense_grad(bool f16, const DenseGradParams &p, int chunks, cudaStream_t s) {
  switch (p.act) {
    case DASH_ACT_RELU: return launch_grad<DASH_ACT_RELU>(f16, p, chunks, s);
    case DASH_ACT_GELU: return launch_grad<DASH_ACT_GELU>(f16, p, chunks, s);
    case DASH_ACT_GELU_TANH: return launch_grad<DASH_ACT_GELU_TANH>(f16, p, chunks, s);
    case DASH_ACT_SILU: return launch_grad<DASH_ACT_SILU>(f16, p, chunks, s);
    default: return launch_grad<DASH_ACT_NONE>(f16, p, chunks, s);
  }
}

cudaError_t launch_dense_specials(bool f16, const DenseSpecials &p, cudaStream_t s) {
  const dim3 grid(4 * 152, 3);
  if (f16)
    dense_specials_kernel<__half><<<grid, 256, 0, s>>>(p);
  else
    dense_specials_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dense_sums(bool f16, const float *part, const float *part_gate, void *out,
                              void *out_gate, int chunks, int N, cudaStream_t s) {
  const dim3 grid((N + 31) / 32, out_gate ? 2 : 1);
  if (f16)
    dense_sums_kernel<__half><<<grid, 256, 0, s>>>(part, part_gate, out, out_gate, chunks, N);
  else
    dense_sums_kernel<__nv_bfloat16>
        <<<grid, 256, 0, s>>>(part, part_gate, out, out_gate, chunks, N);
  return cudaGetLastError();
}

cudaError_t launch_dense_copies(const DenseCopies &c, bool out, cudaStream_t s) {
  int rows = 0, cols = 0;
  for (int i = 0; i < c.count; ++i) {
    rows = c.c[i].rows > rows ? c.c[i].rows : rows;
    cols = c.c[i].cols > cols ? c.c[i].cols : cols;
  }
  const int down = (rows + 7) / 8 < 16384 ? (rows + 7) / 8 : 16384;
  if (out)
    dense_copy_out_kernel<<<dim3((cols + 127) / 128, down, c.count), 256, 0, s>>>(c);
  else
    dense_copy_kernel<<<dim3((cols + 255) / 256, down, c.count), 256, 0, s>>>(c);
  return cudaGetLastError();
}

}  // namespace dash
