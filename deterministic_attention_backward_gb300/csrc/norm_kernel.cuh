// norm_kernel.cuh -- root-mean-square norms of rows and the join of a residual stream with a
// branch, forward and backward.  With z = a rstd(a) (or z = a without a norm after the branch),
// rstd(v) = (mean(v^2) + eps)^-1/2:
//   forward    y = skip x + branch gate (z w_post)          h = y rstd(y) w_next
//   backward   q = y rstd_y, g = dh w_next:   Dy = dy + rstd_y (g - q mean(g q)),  dx = skip Dy
//              t = branch gate Dy, u = t w_post:  da = rstd_a (u - z mean(u z))    (da = t without)
//              dw_next = sum dh q     A = sum Dy z  ->  dgate = branch w_post A,
//                                                     dw_post = branch sum_groups gate A
// so one sum A serves the gate and the norm's weight.  A plain norm is the join without branch.
//
// Bound by memory: a row's values are read once into registers, stay there over both row
// sums, and leave once.  A group of kNT threads owns a row (a warp for short rows), kNV
// vectors of V elements each; the sums over a row are in fp32, by warp shuffles and one
// exchange through shared memory.  The weight gradients are sums over rows: each CTA walks
// over rows of one gate group with one fp32 sum per column in registers, writes its sums to
// `part`, and a second kernel adds the CTAs' sums in a fixed order -- no atomics, the same
// bits on every run.
//
// Measured in bf16 (of a plain copy's rate): the join of 16384 rows of 4096 forward 89 us, 6.0 TB/s
// (89 %); backward 162 us, 5.0 TB/s (73 %).  The backward is bound by latency: its factors and
// column sums fill the registers, so that two CTAs of 8 warps share an SM, 24 % of its warps, and
// they wait for the ring's rows and at the two sums of a row that depend on one another (issue slots
// 40 % busy; without its loads it takes 131 us).  Norms of 524288 heads of 128: forward 43 us,
// backward 68 us (88 %).  Rows off the 16-byte grid: 22324 of 1503 in bf16 the join forward 60 us,
// backward 128 us, 1.5 and 2.2 times a copy's time; of 1504 columns, on the grid, 50 and 102 us (188
// vectors leave a quarter of the lanes of their shape idle).
#pragma once
#include <type_traits>

#include "common.cuh"
#include "elem.cuh"
#include "host.cuh"
#include "norm.cuh"

namespace dash {
namespace norm {

// A weight vector in fp32; weights are of the rows' type or fp32 (uniform branch).
template <typename T, int V>
__device__ __forceinline__ void load_w(const void *w, long long at, int wf32, float (&f)[V]) {
  if (wf32) {
    if constexpr (V == 1) {
      f[0] = static_cast<const float *>(w)[at];
    } else {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 t =
            *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at + 4 * i);
        f[4 * i] = t.x, f[4 * i + 1] = t.y, f[4 * i + 2] = t.z, f[4 * i + 3] = t.w;
      }
    }
  } else {
    unpack<T, V>(load_pack<T, V>(static_cast<const T *>(w) + at), f);
  }
}
template <typename T>
__device__ __forceinline__ float load_w(const void *w, long long at, int wf32) {
  float f[1];
  load_w<T, 1>(w, at, wf32, f);
  return f[0];
}
template <typename T>
__device__ __forceinline__ void store_w(void *w, long long at, int wf32, float v) {
  if (wf32)
    static_cast<float *>(w)[at] = v;
  else
    static_cast<T *>(w)[at] = from_f32<T>(v);
}

// Sum over the kNT threads of a row (part of a warp, a warp, or a CTA), the same value in each.
// `red` holds two buffers of kNT / 32 floats used in turn, so one barrier per sum is enough.
template <int kNT>
struct RowSum {
  float *red;
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = (kNT < 32 ? kNT : 32) / 2; o > 0; o >>= 1)
      v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (kNT > 32) {
      float *r = red + turn * (kNT / 32);
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < kNT / 32; ++i) v += r[i];
    }
    return v;
  }
};

template <int kNT>
constexpr int kRowsPerCta = kNT == 32 ? 8 : 1;

// Rows element by element, in registers.
template <typename T, int kNT, int kNV, bool kJoin>
__global__ void __launch_bounds__(kNT * kRowsPerCta<kNT>) fwd_rows(const NormFwdParams p) {
  constexpr int kRows = kRowsPerCta<kNT>;
  __shared__ float red[2 * (kNT / 32)];
  RowSum<kNT> row_sum{red};
  const int lane = threadIdx.x % kNT;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kNT;
  if (row >= p.rows) return;  // whole rows: every thread of the row's sums, or none
  const float inv_c = 1.f / (float)p.C;
  const T *x = static_cast<const T *>(p.x) + row * p.xs;
  const T *a = static_cast<const T *>(p.a) + row * p.as;
  T px[kNV], pa[kNV];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = i * kNT + lane;
    if (c < p.C) {
      px[i] = x[c];
      if constexpr (kJoin) pa[i] = a[c];
    }
  }
  float rstd_a = 1.f;
  if constexpr (kJoin) {
    if (p.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kNV; ++i)
        if (i * kNT + lane < p.C) {
          const float v = to_f32<T>(pa[i]);
          ss = fmaf(v, v, ss);
        }
      rstd_a = rsqrtf(row_sum(ss) * inv_c + p.eps);
      if (lane == 0) p.rstd_a[row] = rstd_a;
    }
  }
  const long long grow = (row / p.gate_rows) * p.C;
  float y[kNV];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = i * kNT + lane;
    if (c < p.C) {
      y[i] = to_f32<T>(px[i]);
      if constexpr (kJoin) {
        float v = to_f32<T>(pa[i]) * (p.branch * rstd_a);
        if (p.w_post) v *= load_w<T>(p.w_post, c, p.wf32);
        if (p.gate) v *= load_w<T>(p.gate, grow + c, p.wf32);
        y[i] = fmaf(p.skip, y[i], v);
        static_cast<T *>(p.y)[row * p.ys + c] = from_f32<T>(y[i]);
      }
      ss = fmaf(y[i], y[i], ss);
    }
  }
  if (!p.w_next) return;
  // the norm takes the joined row before its rounding
  const float rstd = rsqrtf(row_sum(ss) * inv_c + p.eps);
  if (lane == 0) p.rstd_y[row] = rstd;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = i * kNT + lane;
    if (c < p.C)
      static_cast<T *>(p.h)[row * p.hs + c] =
          from_f32<T>(load_w<T>(p.w_next, c, p.wf32) * (y[i] * rstd));
  }
}

// Rows too long for registers: every pass reads the row again (it stays in the caches), the
// joined row is formed anew in the last one, so that y may be x itself.
template <typename T, int V, bool kJoin>
__global__ void __launch_bounds__(512) fwd_long(const NormFwdParams p) {
  __shared__ float red[2 * 16];
  RowSum<512> row_sum{red};
  const long long row = blockIdx.x;
  const T *x = static_cast<const T *>(p.x) + row * p.xs;
  const T *a = kJoin ? static_cast<const T *>(p.a) + row * p.as : nullptr;
  const float inv_c = 1.f / (float)p.C;
  const long long grow = (row / p.gate_rows) * p.C;
  float rstd_a = 1.f;
  if (kJoin && p.w_post) {
    float ss = 0.f;
    for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
      float v[V];
      unpack<T, V>(load_pack<T, V>(a + c), v);
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(v[e], v[e], ss);
    }
    rstd_a = rsqrtf(row_sum(ss) * inv_c + p.eps);
    if (threadIdx.x == 0) p.rstd_a[row] = rstd_a;
  }
  auto joined = [&](int c, float (&y)[V]) {
    unpack<T, V>(load_pack<T, V>(x + c), y);
    if constexpr (kJoin) {
      float v[V], w[V];
      unpack<T, V>(load_pack<T, V>(a + c), v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] *= p.branch * rstd_a;
      if (p.w_post) {
        load_w<T, V>(p.w_post, c, p.wf32, w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= w[e];
      }
      if (p.gate) {
        load_w<T, V>(p.gate, grow + c, p.wf32, w);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = fmaf(p.skip, y[e], v[e]);
    }
  };
  float rstd = 0.f;
  if (p.w_next) {
    float ss = 0.f;
    for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
      float y[V];
      joined(c, y);
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(y[e], y[e], ss);
    }
    rstd = rsqrtf(row_sum(ss) * inv_c + p.eps);
    if (threadIdx.x == 0) p.rstd_y[row] = rstd;
  }
  for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
    float y[V];
    joined(c, y);
    if constexpr (kJoin) store_pack<T, V>(static_cast<T *>(p.y) + row * p.ys + c, pack<T, V>(y));
    if (p.w_next) {
      float w[V];
      load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] *= y[e] * rstd;
      store_pack<T, V>(static_cast<T *>(p.h) + row * p.hs + c, pack<T, V>(w));
    }
  }
}

// ------------------------------------------------------------------------------- backward
// Rows element by element, in registers; kSmem: the column sums live in shared memory instead
// (long rows).
template <typename T, int kNT, int kNV, bool kJoin, bool kSmem>
__global__ void __launch_bounds__(kNT * kRowsPerCta<kNT>)
    bwd_rows(const NormBwdParams p) {
  constexpr int kRows = kRowsPerCta<kNT>;
  constexpr int kSums = kJoin ? 2 : 1;
  extern __shared__ float4 dyn4[];
  float *dyn = reinterpret_cast<float *>(dyn4);
  __shared__ float red[2 * (kNT / 32)];
  RowSum<kNT> row_sum{red};
  const int lane = threadIdx.x % kNT, sub = threadIdx.x / kNT;
  const int group = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas;
  const long long row0 = group * p.gate_rows, row1 = row0 + p.gate_rows;
  const float inv_c = 1.f / (float)p.C;
  float accN[kSmem ? 1 : kNV], accA[kSmem || !kJoin ? 1 : kNV];
  if constexpr (kSmem) {
    for (int c = threadIdx.x; c < kSums * p.C; c += kNT) dyn[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      accN[i] = 0.f;
      if constexpr (kJoin) accA[i] = 0.f;
    }
  }
  for (long long row = row0 + (long long)cta * kRows + sub; row < row1;
       row += (long long)p.ctas * kRows) {
    T pdh[kNV], py[kNV], pdy[kNV], pa[kNV];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = i * kNT + lane;
      if (c < p.C) {
        if (p.w_next) {
          pdh[i] = static_cast<const T *>(p.dh)[row * p.dhs + c];
          py[i] = static_cast<const T *>(p.y)[row * p.ys + c];
        }
        if (p.dy) pdy[i] = static_cast<const T *>(p.dy)[row * p.dys + c];
        if constexpr (kJoin) pa[i] = static_cast<const T *>(p.a)[row * p.as + c];
      }
    }
    const float rstd_y = p.w_next ? p.rstd_y[row] : 0.f;
    const float rstd_a = kJoin && p.w_post ? p.rstd_a[row] : 1.f;
    float c1 = 0.f;
    if (p.w_next) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = i * kNT + lane;
        if (c < p.C) {
          const float dq = to_f32<T>(pdh[i]) * (to_f32<T>(py[i]) * rstd_y);
          c1 = fmaf(dq, load_w<T>(p.w_next, c, p.wf32), c1);
          if constexpr (kSmem)
            dyn[c] += dq;
          else
            accN[i] += dq;
        }
      }
      c1 = row_sum(c1) * inv_c;
    }
    // Dy of one column
    auto joined = [&](int i, int c) {
      float D = p.dy ? to_f32<T>(pdy[i]) : 0.f;
      if (p.w_next)
        D = fmaf(rstd_y,
                 fmaf(-(to_f32<T>(py[i]) * rstd_y), c1,
                      to_f32<T>(pdh[i]) * load_w<T>(p.w_next, c, p.wf32)),
                 D);
      return D;
    };
    if constexpr (!kJoin) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = i * kNT + lane;
        if (c < p.C) static_cast<T *>(p.dx)[row * p.dxs + c] = from_f32<T>(joined(i, c));
      }
    } else {
      const long long grow = (p.row_gate ? row : group) * p.C;
      // t = branch gate Dy w_post of one column
      float c2 = 0.f;
      float t[kNV];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = i * kNT + lane;
        if (c < p.C) {
          const float D = joined(i, c), z = to_f32<T>(pa[i]) * rstd_a;
          static_cast<T *>(p.dx)[row * p.dxs + c] = from_f32<T>(D * p.skip);
          t[i] = D * p.branch;
          if (p.gate) t[i] *= load_w<T>(p.gate, grow + c, p.wf32);
          const float w = p.w_post ? load_w<T>(p.w_post, c, p.wf32) : 1.f;
          if (p.row_gate) store_w<T>(p.dgate, row * p.C + c, p.wf32, p.branch * D * w * z);
          const float A = (p.row_gate ? t[i] : D) * z;
          if constexpr (kSmem)
            dyn[p.C + c] += A;
          else
            accA[i] += A;
          t[i] *= w;
          c2 = fmaf(t[i], z, c2);
        }
      }
      if (p.w_post) c2 = row_sum(c2) * inv_c;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = i * kNT + lane;
        if (c < p.C) {
          if (p.w_post) t[i] = rstd_a * fmaf(-(to_f32<T>(pa[i]) * rstd_a), c2, t[i]);
          static_cast<T *>(p.da)[row * p.das + c] = from_f32<T>(t[i]);
        }
      }
    }
  }
  // this CTA's sums: the rows of a CTA added in order, one slot per CTA
  float *out = p.part + (size_t)blockIdx.x * kSums * p.C;
  if constexpr (kSmem) {
    __syncthreads();
    for (int c = threadIdx.x; c < kSums * p.C; c += kNT) out[c] = dyn[c];
  } else if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = i * kNT + lane;
      if (c < p.C) {
        out[c] = accN[i];
        if constexpr (kJoin) out[p.C + c] = accA[i];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = i * kNT + lane;
        if (c < p.C) dyn[sub * p.C + c] = k ? accA[kJoin ? i : 0] : accN[i];
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += kNT * kRows) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += dyn[r * p.C + c];
        out[k * p.C + c] = s;
      }
    }
  }
}

// ------------------------------------------------------------------------------- rings
// Rows of 16-byte vectors come in through a ring of shared memory that every thread fills and
// reads for itself (cp.async: no barrier, and a thread's loads for the next rows are in flight
// while it works on this one without holding registers).  Slot (stage, array, vector) of a
// thread is 16 bytes at thread * 16 of its own block of kThreads * 16.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

template <int kNT>
constexpr int kRingThreads = kNT < 256 ? (kNT > 32 ? kNT : 256) : kNT;

template <typename T, int kThreads, int kNV, int kArrays>
struct Ring {
  static constexpr int P = 8 / sizeof(T);  // pairs of a vector
  static constexpr uint32_t kStage = kArrays * kNV * kThreads * 16;
  uint32_t first;  // this thread's slots of stage 0; `at` below: those of a stage
  __device__ __forceinline__ explicit Ring(void *smem)
      : first(static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + threadIdx.x * 16) {}
  __device__ __forceinline__ void fetch(uint32_t at, int array, int i, const T *src) const {
    cp_async16(at + (array * kNV + i) * (kThreads * 16), src);
  }
  __device__ __forceinline__ void read(uint32_t at, int array, int i, f2 (&f)[P]) const {
    unpack2<T>(*static_cast<const uint4 *>(
                   __cvta_shared_to_generic(at + (array * kNV + i) * (kThreads * 16))),
               f);
  }
};
template <typename T>
__device__ __forceinline__ void put(T *dst, const f2 (&f)[8 / sizeof(T)]) {
  *reinterpret_cast<uint4 *>(dst) = pack2<T>(f);
}
// A weight vector in pairs (uniform branch on its type).
template <typename T>
__device__ __forceinline__ void load_w2(const void *w, long long at, int wf32,
                                        f2 (&f)[8 / sizeof(T)]) {
  if (sizeof(T) == 2 && wf32) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(w) + at);
#pragma unroll
    for (int i = 0; i < (int)(4 / sizeof(T)); ++i) {
      const uint4 v = q[i];
      f[2 * i] = f2_of(v.x, v.y);
      f[2 * i + 1] = f2_of(v.z, v.w);
    }
  } else {
    unpack2<T>(*reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + at), f);
  }
}
// Rows off the 16-byte grid.  Where all tensors lie on it in the same way, row r begins
// (off + r stride) mod V elements behind a boundary, the same for every `period`-th row: a CTA
// that takes such rows has its vectors at the same columns throughout, from `shift` columns before
// the row on, and works as with aligned rows, but for the ends, where a vector holds columns of
// the rows beside it: they count as zero and are not written.  (Each row read by itself, element
// by element, took 2 to 6 times as long.)
template <typename T>
__device__ __forceinline__ bool inside(int c, int C) {  // whether the whole vector is
  return c >= 0 && c + (int)(16 / sizeof(T)) <= C;
}
template <typename T>
__device__ __forceinline__ void zero_outside(f2 (&f)[8 / sizeof(T)], int c, int C) {
#pragma unroll
  for (int e = 0; e < (int)(8 / sizeof(T)); ++e) {
    float a, b;
    f2_to(f[e], a, b);
    f[e] = f2_of((unsigned)(c + 2 * e) < (unsigned)C ? a : 0.f,
                 (unsigned)(c + 2 * e + 1) < (unsigned)C ? b : 0.f);
  }
}
template <typename T, bool kShift>
__device__ __forceinline__ void put_at(T *row, int c, int C, const f2 (&f)[8 / sizeof(T)]) {
  if (!kShift || inside<T>(c, C)) {
    put<T>(row + c, f);
  } else {
#pragma unroll
    for (int e = 0; e < (int)(8 / sizeof(T)); ++e) {
      float a, b;
      f2_to(f[e], a, b);
      if ((unsigned)(c + 2 * e) < (unsigned)C) row[c + 2 * e] = from_f32<T>(a);
      if ((unsigned)(c + 2 * e + 1) < (unsigned)C) row[c + 2 * e + 1] = from_f32<T>(b);
    }
  }
}
// Columns c.. of the weights' row at `base`.
template <typename T, bool kShift>
__device__ __forceinline__ void weights_at(const void *w, long long base, int c, int C, int wf32,
                                           f2 (&f)[8 / sizeof(T)]) {
  if constexpr (!kShift) {
    load_w2<T>(w, base + c, wf32, f);
  } else {
#pragma unroll
    for (int e = 0; e < (int)(8 / sizeof(T)); ++e) {
      float v[2][1] = {{0.f}, {0.f}};
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if ((unsigned)(c + 2 * e + u) < (unsigned)C)
          load_w<T, 1>(w, base + c + 2 * e + u, wf32, v[u]);
      f[e] = f2_of(v[0][0], v[1][0]);
    }
  }
}
template <bool kShift, int P>
__device__ __forceinline__ void put_sums(float *out, int c, int C, const f2 (&acc)[P]) {
  if constexpr (!kShift) {
#pragma unroll
    for (int e = 0; e < P; e += 2)
      *reinterpret_cast<ulonglong2 *>(out + c + 2 * e) = make_ulonglong2(acc[e], acc[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      float a, b;
      f2_to(acc[e], a, b);
      if ((unsigned)(c + 2 * e) < (unsigned)C) out[c + 2 * e] = a;
      if ((unsigned)(c + 2 * e + 1) < (unsigned)C) out[c + 2 * e + 1] = b;
    }
  }
}
// branch_scale gate w_post of one vector (factors that are not there: 1); of the gate's row
// `grow`, in elements.
template <typename T, bool kShift, typename Params>
__device__ __forceinline__ void branch_factor(const Params &p, int c, long long grow,
                                              f2 (&f)[8 / sizeof(T)]) {
  constexpr int P = 8 / sizeof(T);
#pragma unroll
  for (int e = 0; e < P; ++e) f[e] = f2_of(p.branch, p.branch);
  if (p.w_post) {
    f2 w[P];
    weights_at<T, kShift>(p.w_post, 0, c, p.C, p.wf32, w);
#pragma unroll
    for (int e = 0; e < P; ++e) f[e] = mul2(f[e], w[e]);
  }
  if (p.gate) {
    f2 w[P];
    weights_at<T, kShift>(p.gate, grow, c, p.C, p.wf32, w);
#pragma unroll
    for (int e = 0; e < P; ++e) f[e] = mul2(f[e], w[e]);
  }
}

// Weights stay in registers over a CTA's rows (up to two vectors a thread): read again for
// every row they come from L2, whose latency then stands between the two sums of each row.
template <typename T, int kNT, int kNV, bool kJoin, int kDepth, bool kShift>
__global__ void __launch_bounds__(kRingThreads<kNT>) fwd_ring(const NormFwdParams p) {
  constexpr int V = 16 / sizeof(T), P = V / 2, kThreads = kRingThreads<kNT>;
  constexpr int kRows = kThreads / kNT;
  constexpr bool kKeep = kNV <= 2;
  extern __shared__ float4 dyn4[];
  __shared__ float red[2 * (kNT / 32 ? kNT / 32 : 1)];
  RowSum<kNT> row_sum{red};
  using R = Ring<T, kThreads, kNV, kJoin ? 2 : 1>;
  const R ring(dyn4);
  int stage = 0;
  const int lane = threadIdx.x % kNT;
  const int period = kShift ? p.period : 1, kind = kShift ? blockIdx.x % period : 0;
  const int shift = kShift ? (p.off + kind * p.stride_mod) & (V - 1) : 0;
  // consecutive rows (of a kind) for each CTA
  const int ctas = gridDim.x / period;  // of a kind
  const long long each = ((p.rows + period - 1) / period + ctas - 1) / ctas * period;
  const long long row0 = blockIdx.x / period * each + kind;
  const long long row1 = row0 + each < p.rows ? row0 + each : p.rows;
  const int step = kRows * period;
  long long row = row0 + (long long)(threadIdx.x / kNT) * period;
  const float inv_c = 1.f / (float)p.C;
  long long ahead = row;  // the row to fetch
  auto fetch = [&]() {
    const uint32_t at = ring.first + stage * R::kStage;
    if (ahead < row1) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (c < p.C) {
          if constexpr (kJoin)
            ring.fetch(at, 1, i, static_cast<const T *>(p.a) + ahead * p.as + c);
          ring.fetch(at, 0, i, static_cast<const T *>(p.x) + ahead * p.xs + c);
        }
      }
    }
    cp_async_commit();
    stage = stage + 1 == kDepth ? 0 : stage + 1;
    ahead += step;
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) fetch();
  f2 wn[kKeep ? kNV : 1][P], fac[kKeep && kJoin ? kNV : 1][P];
  long long held = -1;  // the gate row that `fac` holds
  if constexpr (kKeep) {
    if (p.w_next)
#pragma unroll
      for (int i = 0; i < kNV; ++i)
        if ((i * kNT + lane) * V - shift < p.C)
        weights_at<T, kShift>(p.w_next, 0, (i * kNT + lane) * V - shift, p.C, p.wf32, wn[i]);
  }
  const f2 skip = f2_of(p.skip, p.skip);
  auto read = [&](int array, int i, f2 (&f)[P]) {
    ring.read(ring.first + stage * R::kStage, array, i, f);
    const int c = (i * kNT + lane) * V - shift;
    if (kShift && !inside<T>(c, p.C)) zero_outside<T>(f, c, p.C);
  };
  // a warp stays until its last row is done: the sums of rows take part in full
  for (long long first = row - threadIdx.x % 32 / kNT * period; first < row1;
       first += step, row += step) {
    const bool in = row < row1;
    const long long gate = kJoin && p.gate && in ? (unsigned)row / (unsigned)p.gate_rows : 0;
    if (kKeep && kJoin && gate != held) {
      held = gate;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (c < p.C) branch_factor<T, kShift>(p, c, gate * p.C, fac[kJoin && kKeep ? i : 0]);
      }
    }
    cp_async_wait<kDepth - 1>();
    f2 y[kNV][P];  // the branch, then the joined row
    f2 ss2 = f2_of(0.f, 0.f);
    float rstd_a = 1.f;
    if constexpr (kJoin) {
#pragma unroll
      for (int i = 0; i < kNV; ++i)
        if (in && (i * kNT + lane) * V - shift < p.C) {
          read(1, i, y[i]);
#pragma unroll
          for (int e = 0; e < P; ++e) ss2 = fma2(y[i][e], y[i][e], ss2);
        }
      if (p.w_post) {
        rstd_a = rsqrtf(row_sum(f2_sum(ss2)) * inv_c + p.eps);
        if (lane == 0 && in) p.rstd_a[row] = rstd_a;
      }
      ss2 = f2_of(0.f, 0.f);
    }
    const f2 rstd_a2 = f2_of(rstd_a, rstd_a);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V - shift;
      if (in && c < p.C) {
        f2 x[P];
        read(0, i, x);
        if constexpr (kJoin) {
          f2 f[P];
          if constexpr (!kKeep) branch_factor<T, kShift>(p, c, gate * p.C, f);
#pragma unroll
          for (int e = 0; e < P; ++e)
            y[i][e] = fma2(mul2(y[i][e], rstd_a2), kKeep ? fac[kKeep ? i : 0][e] : f[e],
                           mul2(skip, x[e]));
          put_at<T, kShift>(static_cast<T *>(p.y) + row * p.ys, c, p.C, y[i]);
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) y[i][e] = x[e];
        }
#pragma unroll
        for (int e = 0; e < P; ++e) ss2 = fma2(y[i][e], y[i][e], ss2);
      }
    }
    fetch();  // everything of this stage has been read
    if (!p.w_next) continue;
    // the norm takes the joined row before its rounding
    const float rstd = rsqrtf(row_sum(f2_sum(ss2)) * inv_c + p.eps);
    if (lane == 0 && in) p.rstd_y[row] = rstd;
    const f2 rstd2 = f2_of(rstd, rstd);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V - shift;
      if (in && c < p.C) {
        f2 w[P];
        if constexpr (!kKeep) weights_at<T, kShift>(p.w_next, 0, c, p.C, p.wf32, w);
#pragma unroll
        for (int e = 0; e < P; ++e)
          w[e] = mul2(mul2(y[i][e], rstd2), kKeep ? wn[kKeep ? i : 0][e] : w[e]);
        put_at<T, kShift>(static_cast<T *>(p.h) + row * p.hs, c, p.C, w);
      }
    }
  }
}

template <typename T, int kNT, int kNV, bool kJoin, int kDepth, bool kShift>
__global__ void __launch_bounds__(kRingThreads<kNT>, kJoin ? 512 / kRingThreads<kNT>
                                                     : kNV == 1 ? 1024 / kRingThreads<kNT> : 1)
    bwd_ring(const NormBwdParams p) {
  constexpr int V = 16 / sizeof(T), P = V / 2, kThreads = kRingThreads<kNT>;
  constexpr int kRows = kThreads / kNT;
  constexpr int kSums = kJoin ? 2 : 1;
  constexpr bool kKeep = kNV <= 2;
  enum { kDh, kY, kDy, kA };
  extern __shared__ float4 dyn4[];
  __shared__ float red[2 * (kNT / 32 ? kNT / 32 : 1)];
  RowSum<kNT> row_sum{red};
  using R = Ring<T, kThreads, kNV, kJoin ? 4 : 3>;
  const R ring(dyn4);
  uint32_t at = ring.first;  // of the stage in turn
  const int lane = threadIdx.x % kNT, sub = threadIdx.x / kNT;
  const int group = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas;
  const int period = kShift ? p.period : 1, kind = kShift ? cta % period : 0;
  const int shift = kShift ? (p.off + kind * p.stride_mod) & (V - 1) : 0;
  const long long row0 = group * p.gate_rows;
  const long long row1 = row0 + p.gate_rows, step = (long long)p.ctas * kRows;
  long long row = row0 + ((long long)(cta / period) * kRows + sub) * period;
  if constexpr (kShift) row += ((kind - row0) % period + period) % period;  // the group's first
  const float inv_c = 1.f / (float)p.C;
  const f2 zero = f2_of(0.f, 0.f);
  f2 accN[kNV][P], accA[kJoin ? kNV : 1][P];
#pragma unroll
  for (int i = 0; i < kNV; ++i)
#pragma unroll
    for (int e = 0; e < P; ++e) {
      accN[i][e] = zero;
      if constexpr (kJoin) accA[i][e] = zero;
    }
  float next_y = 0.f, next_a = 1.f;  // rstd of the next row, a row ahead of their use
  auto stats = [&](long long r) {
    if (r < row1) {
      if (p.w_next) next_y = p.rstd_y[r];
      if (kJoin && p.w_post) next_a = p.rstd_a[r];
    }
  };
  long long ahead = row;  // the row to fetch
  auto fetch = [&]() {
    if (ahead < row1) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (c < p.C) {
          if (p.w_next) {
            ring.fetch(at, kDh, i, static_cast<const T *>(p.dh) + ahead * p.dhs + c);
            ring.fetch(at, kY, i, static_cast<const T *>(p.y) + ahead * p.ys + c);
          }
          if (p.dy) ring.fetch(at, kDy, i, static_cast<const T *>(p.dy) + ahead * p.dys + c);
          if constexpr (kJoin)
            ring.fetch(at, kA, i, static_cast<const T *>(p.a) + ahead * p.as + c);
        }
      }
    }
    cp_async_commit();
    at = at + R::kStage == ring.first + kDepth * R::kStage ? ring.first : at + R::kStage;
    ahead += step;
  };
#pragma unroll
  for (int s = 0; s < kDepth; ++s) fetch();
  f2 wn[kKeep ? kNV : 1][P], fac[kKeep && kJoin ? kNV : 1][P];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V - shift;
      if (c < p.C) {
        if (p.w_next) weights_at<T, kShift>(p.w_next, 0, c, p.C, p.wf32, wn[i]);
        if (kJoin && !p.row_gate)
          branch_factor<T, kShift>(p, c, (long long)group * p.C, fac[kJoin ? i : 0]);
      }
    }
  }
  stats(row);
  const f2 skip = f2_of(p.skip, p.skip), branch = f2_of(p.branch, p.branch);
  auto read = [&](int array, int i, f2 (&f)[P]) {
    ring.read(at, array, i, f);
    const int c = (i * kNT + lane) * V - shift;
    if (kShift && !inside<T>(c, p.C)) zero_outside<T>(f, c, p.C);
  };
  for (long long first = row - threadIdx.x % 32 / kNT * period; first < row1;
       first += step, row += step) {
    const bool in = row < row1;
    const float rstd_y = next_y, rstd_a = next_a;
    const f2 rstd_y2 = f2_of(rstd_y, rstd_y), rstd_a2 = f2_of(rstd_a, rstd_a);
    stats(row + step);
    cp_async_wait<kDepth - 1>();
    f2 D[kNV][P];  // dh w_next, then Dy, then branch gate Dy w_post
    float c1 = 0.f;
    if (p.w_next) {
      f2 c1_2 = zero;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (in && c < p.C) {
          f2 q[P], w[P];
          read(kDh, i, D[i]);
          read(kY, i, q);
          if constexpr (!kKeep) weights_at<T, kShift>(p.w_next, 0, c, p.C, p.wf32, w);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            q[e] = mul2(q[e], rstd_y2);
            accN[i][e] = fma2(D[i][e], q[e], accN[i][e]);
            D[i][e] = mul2(D[i][e], kKeep ? wn[kKeep ? i : 0][e] : w[e]);
            c1_2 = fma2(D[i][e], q[e], c1_2);
          }
        }
      }
      c1 = row_sum(f2_sum(c1_2)) * inv_c;
    }
    const float nc1 = -c1 * rstd_y;
    const f2 nc1_2 = f2_of(nc1, nc1);
    f2 c2_2 = zero;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V - shift;
      if (in && c < p.C) {
        f2 t[P];
        if (p.dy) {
          read(kDy, i, t);
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) t[e] = zero;
        }
        if (p.w_next) {
          f2 y[P];
          read(kY, i, y);
#pragma unroll
          for (int e = 0; e < P; ++e)
            D[i][e] = fma2(rstd_y2, fma2(y[e], nc1_2, D[i][e]), t[e]);
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) D[i][e] = t[e];
        }
        if constexpr (!kJoin) {
          put_at<T, kShift>(static_cast<T *>(p.dx) + row * p.dxs, c, p.C, D[i]);
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) t[e] = mul2(D[i][e], skip);
          put_at<T, kShift>(static_cast<T *>(p.dx) + row * p.dxs, c, p.C, t);
          f2 z[P], f[P];
          read(kA, i, z);
          if (!kKeep || p.row_gate)
            branch_factor<T, kShift>(p, c, (p.row_gate ? row : (long long)group) * p.C, f);
          else
#pragma unroll
            for (int e = 0; e < P; ++e) f[e] = fac[kKeep ? i : 0][e];
#pragma unroll
          for (int e = 0; e < P; ++e) {
            z[e] = mul2(z[e], rstd_a2);
            t[e] = mul2(D[i][e], z[e]);  // what A sums, or with the row's own gate below
            D[i][e] = mul2(D[i][e], f[e]);
            c2_2 = fma2(D[i][e], z[e], c2_2);
          }
          if (p.row_gate) {
            f2 g[P], w[P];
            weights_at<T, kShift>(p.gate, row * p.C, c, p.C, p.wf32, g);
#pragma unroll
            for (int e = 0; e < P; ++e) w[e] = f2_of(1.f, 1.f);
            if (p.w_post) weights_at<T, kShift>(p.w_post, 0, c, p.C, p.wf32, w);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              t[e] = mul2(t[e], branch);
              float d0, d1;
              f2_to(mul2(t[e], w[e]), d0, d1);
              if (!kShift || (unsigned)(c + 2 * e) < (unsigned)p.C)
                store_w<T>(p.dgate, row * p.C + c + 2 * e, p.wf32, d0);
              if (!kShift || (unsigned)(c + 2 * e + 1) < (unsigned)p.C)
                store_w<T>(p.dgate, row * p.C + c + 2 * e + 1, p.wf32, d1);
              t[e] = mul2(t[e], g[e]);
            }
          }
#pragma unroll
          for (int e = 0; e < P; ++e) accA[kJoin ? i : 0][e] = add2(accA[kJoin ? i : 0][e], t[e]);
        }
      }
    }
    if constexpr (kJoin) {
      const float c2 = p.w_post ? row_sum(f2_sum(c2_2)) * inv_c : 0.f;
      const float nc2 = -c2 * rstd_a;
      const f2 nc2_2 = f2_of(nc2, nc2);
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (in && c < p.C) {
          if (p.w_post) {
            f2 a[P];
            read(kA, i, a);
#pragma unroll
            for (int e = 0; e < P; ++e)
              D[i][e] = mul2(rstd_a2, fma2(a[e], nc2_2, D[i][e]));
          }
          put_at<T, kShift>(static_cast<T *>(p.da) + row * p.das, c, p.C, D[i]);
        }
      }
    }
    fetch();
  }
  // this CTA's sums, one slot per CTA: the rows of a thread added in order, then the row groups
  float *out = p.part + (size_t)blockIdx.x * kSums * p.C;
  if constexpr (kRows == 1) {
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V - shift;
      if (c < p.C) {
        put_sums<kShift>(out, c, p.C, accN[i]);
        if constexpr (kJoin) put_sums<kShift>(out + p.C, c, p.C, accA[i]);
      }
    }
  } else {
    float *dyn = reinterpret_cast<float *>(dyn4);
    cp_async_wait<0>();
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V - shift;
        if (c < p.C) put_sums<kShift>(dyn + sub * p.C, c, p.C, k ? accA[kJoin ? i : 0] : accN[i]);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < p.C; c += kThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int r = 0; r < kRows; ++r) s += dyn[r * p.C + c];
        out[k * p.C + c] = s;
      }
    }
  }
}

// Rows too long for registers and shared memory: passes over the row in the caches, the
// column sums in this CTA's slot of `part`, each column always by the same thread.
template <typename T, int V, bool kJoin>
__global__ void __launch_bounds__(512) bwd_long(const NormBwdParams p) {
  constexpr int kSums = kJoin ? 2 : 1;
  __shared__ float red[2 * 16];
  RowSum<512> row_sum{red};
  const int group = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas;
  const long long row0 = group * p.gate_rows, row1 = row0 + p.gate_rows;
  const float inv_c = 1.f / (float)p.C;
  float *sumN = p.part + (size_t)blockIdx.x * kSums * p.C, *sumA = sumN + p.C;
  for (int c = threadIdx.x * V; c < p.C; c += 512 * V)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      sumN[c + e] = 0.f;
      if constexpr (kJoin) sumA[c + e] = 0.f;
    }
  for (long long row = row0 + cta; row < row1; row += p.ctas) {
    const float rstd_y = p.w_next ? p.rstd_y[row] : 0.f;
    const float rstd_a = kJoin && p.w_post ? p.rstd_a[row] : 1.f;
    const long long grow = (p.row_gate ? row : group) * p.C;
    float c1 = 0.f;
    if (p.w_next) {
      for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
        float dh[V], q[V], w[V];
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.dh) + row * p.dhs + c), dh);
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.y) + row * p.ys + c), q);
        load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float dq = dh[e] * (q[e] * rstd_y);
          c1 = fmaf(dq, w[e], c1);
          sumN[c + e] += dq;
        }
      }
      c1 = row_sum(c1) * inv_c;
    }
    auto joined = [&](int c, float (&D)[V]) {
      if (p.dy)
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.dy) + row * p.dys + c), D);
      else
#pragma unroll
        for (int e = 0; e < V; ++e) D[e] = 0.f;
      if (p.w_next) {
        float dh[V], q[V], w[V];
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.dh) + row * p.dhs + c), dh);
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.y) + row * p.ys + c), q);
        load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
        for (int e = 0; e < V; ++e)
          D[e] = fmaf(rstd_y, fmaf(-(q[e] * rstd_y), c1, dh[e] * w[e]), D[e]);
      }
    };
    if constexpr (!kJoin) {
      for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
        float D[V];
        joined(c, D);
        store_pack<T, V>(static_cast<T *>(p.dx) + row * p.dxs + c, pack<T, V>(D));
      }
    } else {
      // Dy, z, t and w_post of one vector of columns
      auto cols = [&](int c, float (&D)[V], float (&z)[V], float (&t)[V], float (&w)[V]) {
        joined(c, D);
        unpack<T, V>(load_pack<T, V>(static_cast<const T *>(p.a) + row * p.as + c), z);
        float g[V];
        if (p.gate) {
          load_w<T, V>(p.gate, grow + c, p.wf32, g);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] = 1.f;
        }
        if (p.w_post) {
          load_w<T, V>(p.w_post, c, p.wf32, w);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) w[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          z[e] *= rstd_a;
          t[e] = D[e] * p.branch * g[e];
        }
      };
      float c2 = 0.f;
      for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
        float D[V], z[V], t[V], w[V];
        cols(c, D, z, t, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          c2 = fmaf(t[e] * w[e], z[e], c2);
          sumA[c + e] += (p.row_gate ? t[e] : D[e]) * z[e];
          if (p.row_gate)
            store_w<T>(p.dgate, row * p.C + c + e, p.wf32, p.branch * D[e] * w[e] * z[e]);
        }
      }
      if (p.w_post) c2 = row_sum(c2) * inv_c;
      for (int c = threadIdx.x * V; c < p.C; c += 512 * V) {
        float D[V], z[V], t[V], w[V];
        cols(c, D, z, t, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          t[e] *= w[e];
          if (p.w_post) t[e] = rstd_a * fmaf(-z[e], c2, t[e]);
          D[e] *= p.skip;
        }
        store_pack<T, V>(static_cast<T *>(p.dx) + row * p.dxs + c, pack<T, V>(D));
        store_pack<T, V>(static_cast<T *>(p.da) + row * p.das + c, pack<T, V>(t));
      }
    }
  }
}

// Adds the CTAs' sums in a fixed order: 32 columns a block, 32 lanes per column.  With fewer
// than 32 groups, 32 / groups lanes share a group's slots; otherwise each lane takes whole
// groups.  dw_next over all slots; A per group -> dgate, and dw_post over the groups.
template <typename T, bool kJoin>
__global__ void __launch_bounds__(1024) bwd_sums(const NormBwdParams p) {
  constexpr int kSums = kJoin ? 2 : 1;
  __shared__ float sN[32][33], sA[32][33];
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  int share = 32;  // lanes per group, a power of two
  while (share > 1 && p.groups * share > 32) share >>= 1;
  float n = 0.f, post = 0.f, A = 0.f;
  const int first = lane / share, step = 32 / share, sub = lane % share;
  if (c < p.C) {
    for (int g = first; g < p.groups; g += step) {
      A = 0.f;
      for (int k = sub; k < p.ctas; k += share) {
        const float *slot = p.part + ((size_t)g * p.ctas + k) * kSums * p.C + c;
        n += slot[0];
        if constexpr (kJoin) A += slot[p.C];
      }
      if (kJoin && share == 1) {  // a whole group's sum
        const long long at = (long long)g * p.C + c;
        float w = 1.f, gt = 1.f;
        if (p.w_post) w = p.wf32 ? static_cast<const float *>(p.w_post)[c]
                                 : to_f32<T>(static_cast<const T *>(p.w_post)[c]);
        if (p.gate && !p.row_gate)
          gt = p.wf32 ? static_cast<const float *>(p.gate)[at]
                      : to_f32<T>(static_cast<const T *>(p.gate)[at]);
        if (p.dgate && !p.row_gate) store_w<T>(p.dgate, at, p.wf32, p.branch * w * A);
        post += (p.row_gate ? 1.f : p.branch * gt) * A;
      }
    }
  }
  sN[lane][col] = n;
  if constexpr (kJoin) sA[lane][col] = share == 1 ? post : A;
  __syncthreads();
  if (lane != 0 || c >= p.C) return;
  float s = 0.f;
  for (int l = 0; l < 32; ++l) s += sN[l][col];
  if (p.dw_next) store_w<T>(p.dw_next, c, p.wf32, s);
  if constexpr (kJoin) {
    float dw = 0.f;
    if (share == 1) {
      for (int l = 0; l < 32; ++l) dw += sA[l][col];
    } else {
      for (int g = 0; g < p.groups; ++g) {
        float a = 0.f;
        for (int l = 0; l < share; ++l) a += sA[g * share + l][col];
        const long long at = (long long)g * p.C + c;
        float w = 1.f, gt = 1.f;
        if (p.w_post) w = p.wf32 ? static_cast<const float *>(p.w_post)[c]
                                 : to_f32<T>(static_cast<const T *>(p.w_post)[c]);
        if (p.gate && !p.row_gate)
          gt = p.wf32 ? static_cast<const float *>(p.gate)[at]
                      : to_f32<T>(static_cast<const T *>(p.gate)[at]);
        if (p.dgate && !p.row_gate) store_w<T>(p.dgate, at, p.wf32, p.branch * w * a);
        dw += (p.row_gate ? 1.f : p.branch * gt) * a;
      }
    }
    if (p.dw_post) store_w<T>(p.dw_post, c, p.wf32, dw);
  }
}

// ------------------------------------------------------------------------------- dispatch
// Rows of n 16-byte vectors: as few lanes as hold a row with one vector each up to a warp; then
// two vectors a thread, but one for a plain norm's backward.  Rows that only elements address
// (V = 1: tensors that lie on the grid of vectors in different ways, few rows of one alignment)
// take the register form, longer ones the long form.
template <int kNT, int kNV>
struct Shape {
  static constexpr int nt = kNT, nv = kNV;
};
template <bool kOne, typename F>
cudaError_t ring_shape(int n, F go) {
  if (n <= 4) return go(Shape<4, 1>());
  if (n <= 8) return go(Shape<8, 1>());
  if (n <= 16) return go(Shape<16, 1>());
  if (n <= 32) return go(Shape<32, 1>());
  if constexpr (kOne) {
    if (n <= 64) return go(Shape<64, 1>());
    if (n <= 128) return go(Shape<128, 1>());
    if (n <= 256) return go(Shape<256, 1>());
    if (n <= 512) return go(Shape<512, 1>());
  } else {
    if (n <= 64) return go(Shape<32, 2>());
    if (n <= 128) return go(Shape<64, 2>());
    if (n <= 256) return go(Shape<128, 2>());
    if (n <= 512) return go(Shape<256, 2>());
  }
  if (n <= 1024) return go(Shape<512, 2>());
  return go(Shape<512, 4>());
}

// A launch with `smem` bytes of dynamic shared memory.
constexpr int kMostSmem = 226 * 1024;
template <auto kKernel, typename Params>
cudaError_t launch_smem(unsigned grid, int threads, size_t smem, cudaStream_t s, const Params &p) {
  if (smem > 32 * 1024) {  // (48 KB less what is static)
    const cudaError_t e = allow_smem<kKernel>(kMostSmem);
    if (e != cudaSuccess) return e;
  }
  kKernel<<<grid, threads, smem, s>>>(p);
  return cudaGetLastError();
}

// CTAs of a kernel that the device holds at once (asked once: the same on every sm_103 device).
template <auto kKernel>
int resident(int threads, size_t smem) {
  int dev = 0, sms = 0, each = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || allow_smem<kKernel>(kMostSmem) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&each, kKernel, threads, smem) !=
          cudaSuccess ||
      each < 1)
    return 152;
  return sms * each;
}

template <typename T, int V, bool kJoin>
cudaError_t fwd(const NormFwdParams &p, cudaStream_t s) {
  // a shifted row covers V - 1 columns more at most
  const int n = (p.C + (p.period ? V - 1 : 0) + V - 1) / V;
  auto go = [&](auto kernel, int threads, int rows) {
    kernel<<<(unsigned)((p.rows + rows - 1) / rows), threads, 0, s>>>(p);
    return cudaGetLastError();
  };
  if (n > 2048) return go(fwd_long<T, V, kJoin>, 512, 1);
  if constexpr (V > 1) {
    return ring_shape<false>(n, [&](auto shape) {
      constexpr int kNT = decltype(shape)::nt, kNV = decltype(shape)::nv;
      constexpr int kThreads = kRingThreads<kNT>, kRows = kThreads / kNT;
      constexpr int kDepth = kNV == 4 ? 2 : 3;
      const size_t smem = (size_t)kDepth * (kJoin ? 2 : 1) * kNV * kThreads * 16;
      auto launch = [&](auto shifted) {
        constexpr bool kShift = decltype(shifted)::value;
        constexpr auto kKernel = fwd_ring<T, kNT, kNV, kJoin, kDepth, kShift>;
        static const int most = resident<kKernel>(kThreads, smem);
        const int kinds = kShift ? p.period : 1;
        const long long each = (p.rows + kinds - 1) / kinds, need = (each + kRows - 1) / kRows;
        // Several CTAs one after another in every place, as not all SMs reach memory equally fast:
        // dealt out once, 16384 rows of 4096 took 100 us, with 2, 4, 6 and 8 a place 95, 91, 88, 87
        // (rows of 8192 96, 92, 90, 91, 93).  Each loads the weights anew, so that it should have
        // some rows, and where that goes by elements of 16 bits one a place is faster (22324 rows
        // of 1503 62 us, with 6 72).
        const int once = most / kinds;
        long long ctas = kShift && sizeof(T) == 2 ? once : need / 8;
        ctas = ctas < once ? once : ctas < 6 * once ? ctas : 6 * once;
        return launch_smem<kKernel>((unsigned)((need < ctas ? need : ctas) * kinds), kThreads, smem,
                                    s, p);
      };
      return p.period ? launch(std::true_type()) : launch(std::false_type());
    });
  } else {
    if (n <= 128) return go(fwd_rows<T, 32, 4, kJoin>, 256, 8);
    if (n <= 512) return go(fwd_rows<T, 256, 2, kJoin>, 256, 1);
    return go(fwd_rows<T, 512, 4, kJoin>, 512, 1);
  }
}

template <typename T, int V, bool kJoin>
cudaError_t bwd(const NormBwdParams &p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.groups * p.ctas);
  constexpr int kSums = kJoin ? 2 : 1;
  const int n = (p.C + (p.period ? V - 1 : 0) + V - 1) / V;
  cudaError_t e;
  if (n > 2048) {
    e = launch_smem<bwd_long<T, V, kJoin>>(grid, 512, 0, s, p);
  } else if constexpr (V > 1) {
    e = ring_shape<!kJoin>(n, [&](auto shape) {
      constexpr int kNT = decltype(shape)::nt, kNV = decltype(shape)::nv;
      constexpr int kThreads = kRingThreads<kNT>;
      constexpr int kDepth = kNV == 4 ? 1 : 3;
      const size_t ring = (size_t)kDepth * (kJoin ? 4 : 3) * kNV * kThreads * 16;
      const size_t sums = kThreads > kNT ? (size_t)(kThreads / kNT) * p.C * 4 : 0;
      const size_t smem = ring > sums ? ring : sums;
      return p.period ? launch_smem<bwd_ring<T, kNT, kNV, kJoin, kDepth, true>>(grid, kThreads,
                                                                                smem, s, p)
                      : launch_smem<bwd_ring<T, kNT, kNV, kJoin, kDepth, false>>(grid, kThreads,
                                                                                 smem, s, p);
    });
  } else if (n <= 128) {
    e = launch_smem<bwd_rows<T, 32, 4, kJoin, false>>(grid, 256, (size_t)8 * p.C * 4, s, p);
  } else if (n <= 512) {
    e = launch_smem<bwd_rows<T, 256, 2, kJoin, false>>(grid, 256, 0, s, p);
  } else {
    e = launch_smem<bwd_rows<T, 512, 4, kJoin, true>>(grid, 512, (size_t)kSums * p.C * 4, s, p);
  }
  if (e != cudaSuccess) return e;
  bwd_sums<T, kJoin><<<(p.C + 31) / 32, 1024, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace norm
}  // namespace dash

// The launches of one element type (inside namespace dash); `wide`: rows, strides and addresses
// allow 16-byte vectors.
#define DASH_NORM_TYPE(T)                                                                       \
  template <>                                                                                   \
  cudaError_t launch_norm_fwd<T>(const NormFwdParams &p, bool join, bool wide, cudaStream_t s) { \
    constexpr int V = 16 / sizeof(T);                                                           \
    if (wide) return join ? norm::fwd<T, V, true>(p, s) : norm::fwd<T, V, false>(p, s);         \
    return join ? norm::fwd<T, 1, true>(p, s) : norm::fwd<T, 1, false>(p, s);                   \
  }                                                                                             \
  template <>                                                                                   \
  cudaError_t launch_norm_bwd<T>(const NormBwdParams &p, bool join, bool wide, cudaStream_t s) { \
    constexpr int V = 16 / sizeof(T);                                                           \
    if (wide) return join ? norm::bwd<T, V, true>(p, s) : norm::bwd<T, V, false>(p, s);         \
    return join ? norm::bwd<T, 1, true>(p, s) : norm::bwd<T, 1, false>(p, s);                   \
  }


