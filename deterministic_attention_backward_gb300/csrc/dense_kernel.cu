// dense_kernel.cu -- the product kernel and the small kernels around it.
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
constexpr int kOffBar = kStages * kStageBytes;
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
__device__ __forceinline__ void cluster_sync() {
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
// Warp-wide wait (one answer for the whole warp); the limit runs from the 256th try on.
__device__ __forceinline__ bool wait_pair(uint64_t *bar, uint32_t parity, const Abort &ab) {
  if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, try_wait_cluster(bar, parity))) return true;
    if ((it & 15u) == 0) {
      int stop = 0;
      if (lane_id() == 0) {
        if (ab.set()) {
          stop = 1;
        } else if ((it & 255u) == 0) {
          if (t0 == 0) t0 = globaltimer();
          if (ab.poll_global()) {
            stop = 1;
          } else if (globaltimer() - t0 > ab.limit_ns) {
            ab.raise(kErrMbarTimeout);
            stop = 1;
          }
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0)) return false;
    }
  }
}
// One box into this CTA's shared memory, its bytes counted on a barrier of either CTA.
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, uint32_t bar, int c0,
                                         int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
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
// act(z); the slope too where asked for.  expf, erff and tanhf are within a few units in the
// last place, far below the rounding of the outputs to 16 bits.
__device__ __forceinline__ float activation(float z, int act) {
  switch (act) {
    case DASH_ACT_RELU: return z > 0.f || z != z ? z : 0.f;
    case DASH_ACT_SILU: return z / (1.f + expf(-z));
    case DASH_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
    case DASH_ACT_GELU_TANH:
      return 0.5f * z * (1.f + tanhf(0.79788456080286536f * fmaf(0.044715f * z * z, z, z)));
    default: return z;
  }
}
__device__ __forceinline__ float activation(float z, int act, float &slope) {
  switch (act) {
    case DASH_ACT_RELU:
      slope = z > 0.f ? 1.f : z != z ? z : 0.f;
      return z > 0.f || z != z ? z : 0.f;
    case DASH_ACT_SILU: {
      const float s = 1.f / (1.f + expf(-z));
      slope = s * fmaf(z, 1.f - s, 1.f);
      return z * s;
    }
    case DASH_ACT_GELU: {
      const float c = 0.5f * (1.f + erff(z * 0.70710678118654752f));
      slope = fmaf(z, 0.39894228040143268f * expf(-0.5f * z * z), c);
      return z * c;
    }
    case DASH_ACT_GELU_TANH: {
      const float t = tanhf(0.79788456080286536f * fmaf(0.044715f * z * z, z, z));
      slope = fmaf(0.5f * z * (1.f - t * t), 0.79788456080286536f * fmaf(0.134145f * z, z, 1.f),
                   0.5f * (1.f + t));
      return 0.5f * z * (1.f + t);
    }
    default: slope = 1.f; return z;
  }
}

// C values of a row from element `at` on, `left` of them inside the row.
template <typename T, int C>
__device__ __forceinline__ void store_cols(void *base, long long at, const float (&v)[C], int left,
                                           bool vec) {
  T *dst = static_cast<T *>(base) + at;
  if (vec) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i)
      if (8 * i + 8 <= left) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[8 * i + e];
        store_pack<T, 8>(dst + 8 * i, pack<T, 8>(f));
      }
    if (left >= C) return;
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < left && e >= (left & ~7)) dst[e] = from_f32<T>(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < left) dst[e] = from_f32<T>(v[e]);
  }
}
template <typename T, int C>
__device__ __forceinline__ void add_cols(const void *base, long long at, float (&v)[C], int left,
                                         bool vec) {
  const T *src = static_cast<const T *>(base) + at;
  if (vec && left >= C) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      float f[8];
      unpack<T, 8>(load_pack<T, 8>(src + 8 * i), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] += f[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < left) v[e] += to_f32<T>(src[e]);
  }
}
// The epilogue of C columns of one row, from column n on.
template <typename T, int C>
__device__ __forceinline__ void finish(const DenseEpilogue &p, void *y, long long ys, long long row,
                                       int n, int N, float (&z)[C], float (&g)[C]) {
  const int left = N - n;
  const bool vec = p.vec;
  if (p.bias) add_cols<T, C>(p.bias, n, z, left, vec);
  if (p.z) store_cols<T, C>(p.z, row * p.zs + n, z, left, vec);
  if (p.act != DASH_ACT_NONE) {
#pragma unroll
    for (int e = 0; e < C; ++e) z[e] = activation(z[e], p.act);
  }
  if (p.gated) {
    if (p.bias_gate) add_cols<T, C>(p.bias_gate, n, g, left, vec);
    if (p.g) store_cols<T, C>(p.g, row * p.gs + n, g, left, vec);
#pragma unroll
    for (int e = 0; e < C; ++e) z[e] *= g[e];
  }
  if (p.residual) add_cols<T, C>(p.residual, row * p.rs + n, z, left, vec);
  store_cols<T, C>(y, row * ys + n, z, left, vec);
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

// Work items: (split, output, tile), tiles in groups of 8 rows of tiles, so that those in flight
// share their operands in L2.
struct Item {
  int m, n, out, split, k0, k1;
};
__device__ __forceinline__ Item item_of(const DenseParams &p, int t) {
  const int tiles = p.mt * p.nt, r = t % tiles, q = t / tiles;
  Item w;
  w.out = p.outs == 2 ? q & 1 : 0;
  w.split = p.outs == 2 ? q >> 1 : q;
  const int per = 8 * p.nt, g = r / per, in = r - g * per, rows = min(8, p.mt - 8 * g);
  w.m = (8 * g + in % rows) * kDenseM;
  w.n = in / rows;
  w.k0 = w.split * p.per;
  w.k1 = min(w.k0 + p.per, p.nk * p.parts);
  return w;
}

// ------------------------------------------------------------------ the product
// One pair of CTAs a tile of 256 rows and bn (256 or 128) columns, persistent over the work items.
// Each CTA brings in its half of the rows and of the columns; the leader's tensor core instruction
// reads both halves and leaves each CTA its 128 rows in its own TMEM, where two accumulators
// alternate so that a tile's epilogue runs beside the next one's products.
// Warp 0 TMA producer, 1 MMA issuer (leader), 2 TMEM, 4-11 epilogue (thread = row; the two
// warpgroups share the columns).
template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap ta1,
                 const __grid_constant__ CUtensorMap tb0, const __grid_constant__ CUtensorMap tb1,
                 const __grid_constant__ DenseParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
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
  const int items = p.mt * p.nt * p.outs * p.splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
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

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const int half = p.bn / 2;  // columns that this CTA brings in
      const uint32_t bytes = 2 * (kABytes + half * kDenseK * 2);
      bool ok = true;
      int it = 0;
      for (int t = first; ok && t < items; t += step) {
        const Item w = item_of(p, t);
        const int m = w.m + (int)rank * 128;
        // gated: the leader brings w's columns of the tile, the other CTA w_gate's
        const int n = p.e.gated ? w.n * half : w.n * p.bn + (int)rank * half;
        for (int k = w.k0; k < w.k1; ++k, ++it) {
          const int s = it % kStages;
          if (it == p.withhold || !mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, ab)) {
            ok = false;
            break;
          }
          const int part = k >= p.nk ? 1 : 0, kk = (k - part * p.nk) * kDenseK;
          const CUtensorMap *ma = part || (w.out && p.a_out) ? &ta1 : &ta0;
          const CUtensorMap *mb =
              part || (w.out && p.b_out) || (p.e.gated && rank) ? &tb1 : &tb0;
          const uint32_t bar = in_leader(&full[s]);
          if (leader) mbar_arrive_expect_tx(&full[s], bytes);
          uint8_t *sa = smem + s * kStageBytes, *sb = sa + kABytes;
          if (p.a_mn) {
            load_box(sa, ma, bar, m, kk);
            load_box(sa + kMnBox, ma, bar, m + 64, kk);
          } else {
            load_box(sa, ma, bar, kk, m);
          }
          if (p.b_mn) {
            load_box(sb, mb, bar, n, kk);
            if (half > 64) load_box(sb + kMnBox, mb, bar, n + 64, kk);
          } else {
            load_box(sb, mb, bar, kk, n);
          }
        }
      }
      if (!ok && leader)  // leave no copy in flight into shared memory
        for (int j = max(0, it - kStages); j < it; ++j)
          mbar_wait_drain(&full[j % kStages], (j / kStages) & 1, 100000000ull);
    }
    __syncwarp();
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
    const int r = quad * 32 + lane;
    const int cols = p.e.gated ? p.bn / 2 : p.bn;  // output columns of a tile
    int n = 0;
    for (int t = first; t < items; t += step, ++n) {
      const Item w = item_of(p, t);
      if (!wait_pair(&acc_full[n & 1], (n >> 1) & 1, ab)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (n & 1) * 256;
      const long long row = w.m + (int)rank * 128 + r;
      const bool in = row < p.M;
      if (p.splits > 1) {
        float *dst = p.part + ((long long)(w.split * p.outs + w.out) * p.M + row) * p.part_cols +
                     (long long)w.n * p.bn;
        for (int c = wg * (p.bn / 2); c < (wg + 1) * (p.bn / 2); c += 32) {
          float v[32];
          load32(acc + c, v);
          if (in) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<float4 *>(dst + c + 4 * e) =
                  make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        }
      } else {
        void *y = w.out ? p.y1 : p.e.y;
        const long long ys = w.out ? p.y1s : p.e.ys;
        const int n0 = w.n * cols;
        for (int c = wg * (cols / 2); c < (wg + 1) * (cols / 2); c += 32) {
          if (n0 + c >= p.N) break;
          float z[32], g[32];
          load32(acc + c, z);
          if (p.e.gated) load32(acc + p.bn / 2 + c, g);
          if (in) finish<T, 32>(p.e, y, ys, row, n0 + c, p.N, z, g);
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
  __syncwarp();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    dealloc_pair(tmem);
  }
}

// The splits' sums, added in order, and the epilogue; a thread takes 4 columns of a row.
template <typename T>
__global__ void __launch_bounds__(256) dense_finish_kernel(const __grid_constant__ DenseParams p) {
  const int groups = (p.N + 3) / 4;
  const long long i = blockIdx.x * 256ll + threadIdx.x;
  const long long row = i / groups;
  if (row >= p.M) return;
  const int n = (int)(i - row * groups) * 4, out = blockIdx.y;
  const int cols = p.e.gated ? p.bn / 2 : p.bn;
  const long long c = (long long)(n / cols) * p.bn + n % cols;
  float z[4] = {}, g[4] = {};
  const float *src = p.part + (out * (long long)p.M + row) * p.part_cols + c;
  const long long stride = (long long)p.outs * p.M * p.part_cols;
  for (int s = 0; s < p.splits; ++s, src += stride) {
    const float4 v = *reinterpret_cast<const float4 *>(src);
    z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
    if (p.e.gated) {
      const float4 u = *reinterpret_cast<const float4 *>(src + p.bn / 2);
      g[0] += u.x, g[1] += u.y, g[2] += u.z, g[3] += u.w;
    }
  }
  DenseEpilogue e = p.e;
  e.vec = 0;
  finish<T, 4>(e, out ? p.y1 : e.y, out ? p.y1s : e.ys, row, n, p.N, z, g);
}

// ------------------------------------------------------------------ dz, dgate and their sums
// 32 threads a strip of 32 V columns, 8 rows at a time over a chunk of rows; the eight rows'
// sums are added in order through shared memory.
template <typename T, int V>
__global__ void __launch_bounds__(256) dense_grad_kernel(const DenseGradParams p) {
  __shared__ float sums[2][8][32 * V + 1];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < kStatusBytes / 4)
    p.status[threadIdx.x] = 0;
  const int lane = threadIdx.x & 31, by = threadIdx.x >> 5;
  const int n = (blockIdx.x * 32 + lane) * V;
  const int r1 = min(p.M, (int)(blockIdx.y + 1) * p.chunk);
  float sz[V] = {}, sg[V] = {};
  if (n < p.N) {
    for (long long r = blockIdx.y * p.chunk + by; r < r1; r += 8) {
      float dy[V], z[V], g[V];
      unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.dy) + r * p.dys + n), dy);
      if (p.z) {
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.z) + r * p.zs + n), z);
        if (p.g) unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.g) + r * p.gs + n), g);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float slope;
          const float a = activation(z[e], p.act, slope);
          z[e] = dy[e] * slope;
          if (p.g) {
            z[e] *= g[e];
            g[e] = dy[e] * a;
          }
        }
        if (p.dz) store_pack<T, V>(static_cast<T *>(p.dz) + r * p.ds + n, pack<T, V>(z));
        if (p.g && p.dg) store_pack<T, V>(static_cast<T *>(p.dg) + r * p.ds + n, pack<T, V>(g));
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) z[e] = dy[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        sz[e] += z[e];
        if (p.g) sg[e] += g[e];
      }
    }
  }
  if (!p.part && !p.part_gate) return;
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

template <typename T>
__global__ void __launch_bounds__(128) dense_sums_kernel(const float *part, const float *part_gate,
                                                         void *out, void *out_gate, int chunks,
                                                         int N) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  const float *src = blockIdx.y ? part_gate : part;
  T *dst = static_cast<T *>(blockIdx.y ? out_gate : out);
  if (n >= N || !src || !dst) return;
  float s = 0.f;
  for (int c = 0; c < chunks; ++c) s += src[(long long)c * N + n];
  dst[n] = from_f32<T>(s);
}

__global__ void __launch_bounds__(256) dense_copy_kernel(const uint16_t *in, long long is,
                                                         uint16_t *out, long long os,
                                                         long long rows, int cols) {
  const long long stride = (long long)gridDim.x * 256, all = rows * os;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += stride) {
    const long long r = i / os, c = i - r * os;
    out[i] = c < cols ? in[r * is + c] : (uint16_t)0;
  }
}

template <typename T>
cudaError_t launch_t(const CUtensorMap (&ta)[2], const CUtensorMap (&tb)[2], const DenseParams &p,
                     int sms, cudaStream_t s) {
  const cudaError_t e = allow_smem<dense_kernel<T>>(kSmem);
  if (e != cudaSuccess) return e;
  const long long items = (long long)p.mt * p.nt * p.outs * p.splits;
  const int pairs = (int)(items < sms / 2 ? items : sms / 2);
  dense_kernel<T><<<2 * pairs, kThreads, kSmem, s>>>(ta[0], ta[1], tb[0], tb[1], p);
  if (p.splits > 1) {
    const long long threads = (long long)p.M * ((p.N + 3) / 4);
    dense_finish_kernel<T><<<dim3((unsigned)((threads + 255) / 256), p.outs), 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_dense(bool f16, const CUtensorMap (&ta)[2], const CUtensorMap (&tb)[2],
                         const DenseParams &p, int sms, cudaStream_t s) {
  return f16 ? launch_t<__half>(ta, tb, p, sms, s) : launch_t<__nv_bfloat16>(ta, tb, p, sms, s);
}

cudaError_t launch_dense_grad(bool f16, const DenseGradParams &p, int chunks, cudaStream_t s) {
  const int strip = 32 * (p.vec ? 8 : 1);
  const dim3 grid((p.N + strip - 1) / strip, chunks);
  if (f16)
    p.vec ? dense_grad_kernel<__half, 8><<<grid, 256, 0, s>>>(p)
          : dense_grad_kernel<__half, 1><<<grid, 256, 0, s>>>(p);
  else
    p.vec ? dense_grad_kernel<__nv_bfloat16, 8><<<grid, 256, 0, s>>>(p)
          : dense_grad_kernel<__nv_bfloat16, 1><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dense_sums(bool f16, const float *part, const float *part_gate, void *out,
                              void *out_gate, int chunks, int N, cudaStream_t s) {
  const dim3 grid((N + 127) / 128, out_gate ? 2 : 1);
  if (f16)
    dense_sums_kernel<__half><<<grid, 128, 0, s>>>(part, part_gate, out, out_gate, chunks, N);
  else
    dense_sums_kernel<__nv_bfloat16>
        <<<grid, 128, 0, s>>>(part, part_gate, out, out_gate, chunks, N);
  return cudaGetLastError();
}

cudaError_t launch_dense_copy(const void *in, long long is, void *out, long long os,
                              long long rows, int cols, cudaStream_t s) {
  const long long blocks = (rows * os + 255) / 256;
  dense_copy_kernel<<<(unsigned)(blocks < 8192 ? blocks : 8192), 256, 0, s>>>(
      static_cast<const uint16_t *>(in), is, static_cast<uint16_t *>(out), os, rows, cols);
  return cudaGetLastError();
}

}  // namespace dash
