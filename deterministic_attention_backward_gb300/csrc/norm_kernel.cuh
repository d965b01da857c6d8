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
#pragma once
#include "common.cuh"
#include "elem.cuh"
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
        const float4 t = *reinterpret_cast<const float4 *>(static_cast<const float *>(w) + at + 4 * i);
        f[4 * i] = t.x, f[4 * i + 1] = t.y, f[4 * i + 2] = t.z, f[4 * i + 3] = t.w;
      }
    }
  } else {
    unpack<T, V>(load_pack<T, V>(static_cast<const T *>(w) + at), f);
  }
}
template <typename T>
__device__ __forceinline__ void store_w(void *w, long long at, int wf32, float v) {
  if (wf32)
    static_cast<float *>(w)[at] = v;
  else
    static_cast<T *>(w)[at] = from_f32<T>(v);
}

// Sum over the kNT threads of a row, the same value in each.  `red` holds two buffers of
// kNT / 32 floats used in turn, so one barrier per sum is enough.
template <int kNT>
struct RowSum {
  float *red;
  int turn = 0;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
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

template <typename T, int V, int kNT, int kNV, bool kJoin>
__global__ void __launch_bounds__(kNT * kRowsPerCta<kNT>) fwd_rows(const NormFwdParams p) {
  constexpr int kRows = kRowsPerCta<kNT>;
  __shared__ float red[2 * (kNT / 32)];
  RowSum<kNT> row_sum{red};
  const int lane = threadIdx.x % kNT;
  const long long row = (long long)blockIdx.x * kRows + threadIdx.x / kNT;
  if (row >= p.rows) return;  // whole rows: every thread of the row's sums, or none
  const float inv_c = 1.f / (float)p.C;
  const T *x = static_cast<const T *>(p.x) + row * p.xs;
  Pack<T, V> px[kNV], pa[kNV];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * kNT + lane) * V;
    if (c < p.C) {
      px[i] = load_pack<T, V>(x + c);
      if constexpr (kJoin) pa[i] = load_pack<T, V>(static_cast<const T *>(p.a) + row * p.as + c);
    }
  }
  float rstd_a = 1.f;
  if constexpr (kJoin) {
    if (p.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kNV; ++i)
        if ((i * kNT + lane) * V < p.C) {
          float a[V];
          unpack<T, V>(pa[i], a);
#pragma unroll
          for (int e = 0; e < V; ++e) ss = fmaf(a[e], a[e], ss);
        }
      rstd_a = rsqrtf(row_sum(ss) * inv_c + p.eps);
      if (lane == 0) p.rstd_a[row] = rstd_a;
    }
  }
  const long long grow = (row / p.gate_rows) * p.C;
  float y[kNV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * kNT + lane) * V;
    if (c < p.C) {
      unpack<T, V>(px[i], y[i]);
      if constexpr (kJoin) {
        float a[V], w[V];
        unpack<T, V>(pa[i], a);
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] *= p.branch * rstd_a;
        if (p.w_post) {
          load_w<T, V>(p.w_post, c, p.wf32, w);
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] *= w[e];
        }
        if (p.gate) {
          load_w<T, V>(p.gate, grow + c, p.wf32, w);
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) y[i][e] = fmaf(p.skip, y[i][e], a[e]);
        store_pack<T, V>(static_cast<T *>(p.y) + row * p.ys + c, pack<T, V>(y[i]));
      }
#pragma unroll
      for (int e = 0; e < V; ++e) ss = fmaf(y[i][e], y[i][e], ss);
    }
  }
  if (!p.w_next) return;
  // the norm takes the joined row before its rounding
  const float rstd = rsqrtf(row_sum(ss) * inv_c + p.eps);
  if (lane == 0) p.rstd_y[row] = rstd;
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * kNT + lane) * V;
    if (c < p.C) {
      float w[V];
      load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] *= y[i][e] * rstd;
      store_pack<T, V>(static_cast<T *>(p.h) + row * p.hs + c, pack<T, V>(w));
    }
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
// kSmem: the column sums live in shared memory instead of registers (long rows).
template <typename T, int V, int kNT, int kNV, bool kJoin, bool kSmem>
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
  float accN[kSmem ? 1 : kNV][V], accA[kSmem || !kJoin ? 1 : kNV][V];
  if constexpr (kSmem) {
    for (int c = threadIdx.x; c < kSums * p.C; c += kNT) dyn[c] = 0.f;
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        accN[i][e] = 0.f;
        if constexpr (kJoin) accA[i][e] = 0.f;
      }
  }
  for (long long row = row0 + (long long)cta * kRows + sub; row < row1;
       row += (long long)p.ctas * kRows) {
    Pack<T, V> pdh[kNV], py[kNV], pdy[kNV], pa[kNV];
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kNT + lane) * V;
      if (c < p.C) {
        if (p.w_next) {
          pdh[i] = load_pack<T, V>(static_cast<const T *>(p.dh) + row * p.dhs + c);
          py[i] = load_pack<T, V>(static_cast<const T *>(p.y) + row * p.ys + c);
        }
        if (p.dy) pdy[i] = load_pack<T, V>(static_cast<const T *>(p.dy) + row * p.dys + c);
        if constexpr (kJoin)
          pa[i] = load_pack<T, V>(static_cast<const T *>(p.a) + row * p.as + c);
      }
    }
    const float rstd_y = p.w_next ? p.rstd_y[row] : 0.f;
    const float rstd_a = kJoin && p.w_post ? p.rstd_a[row] : 1.f;
    float c1 = 0.f;
    if (p.w_next) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V;
        if (c < p.C) {
          float dh[V], q[V], w[V];
          unpack<T, V>(pdh[i], dh);
          unpack<T, V>(py[i], q);
          load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float dq = dh[e] * (q[e] * rstd_y);
            c1 = fmaf(dq, w[e], c1);
            if constexpr (kSmem)
              dyn[c + e] += dq;
            else
              accN[i][e] += dq;
          }
        }
      }
      c1 = row_sum(c1) * inv_c;
    }
    // Dy of one vector of columns
    auto joined = [&](int i, int c, float (&D)[V]) {
      if (p.dy)
        unpack<T, V>(pdy[i], D);
      else
#pragma unroll
        for (int e = 0; e < V; ++e) D[e] = 0.f;
      if (p.w_next) {
        float dh[V], q[V], w[V];
        unpack<T, V>(pdh[i], dh);
        unpack<T, V>(py[i], q);
        load_w<T, V>(p.w_next, c, p.wf32, w);
#pragma unroll
        for (int e = 0; e < V; ++e)
          D[e] = fmaf(rstd_y, fmaf(-(q[e] * rstd_y), c1, dh[e] * w[e]), D[e]);
      }
    };
    if constexpr (!kJoin) {
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V;
        if (c < p.C) {
          float D[V];
          joined(i, c, D);
          store_pack<T, V>(static_cast<T *>(p.dx) + row * p.dxs + c, pack<T, V>(D));
        }
      }
    } else {
      const long long grow = (p.row_gate ? row : group) * p.C;
      // t = branch gate Dy of one vector of columns (and the sums it feeds, the first time)
      float c2 = 0.f;
      float t[kNV][V];
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V;
        if (c < p.C) {
          float D[V], z[V], w[V];
          joined(i, c, D);
          unpack<T, V>(pa[i], z);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            z[e] *= rstd_a;
            t[i][e] = D[e] * p.skip;
          }
          store_pack<T, V>(static_cast<T *>(p.dx) + row * p.dxs + c, pack<T, V>(t[i]));
#pragma unroll
          for (int e = 0; e < V; ++e) t[i][e] = D[e] * p.branch;
          if (p.gate) {
            load_w<T, V>(p.gate, grow + c, p.wf32, w);
#pragma unroll
            for (int e = 0; e < V; ++e) t[i][e] *= w[e];
          }
          if (p.w_post) {
            load_w<T, V>(p.w_post, c, p.wf32, w);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] = 1.f;
          }
          if (p.row_gate)
#pragma unroll
            for (int e = 0; e < V; ++e)
              store_w<T>(p.dgate, row * p.C + c + e, p.wf32, p.branch * D[e] * w[e] * z[e]);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float A = (p.row_gate ? t[i][e] : D[e]) * z[e];
            if constexpr (kSmem)
              dyn[p.C + c + e] += A;
            else
              accA[i][e] += A;
            t[i][e] *= w[e];
            c2 = fmaf(t[i][e], z[e], c2);
          }
        }
      }
      if (p.w_post) c2 = row_sum(c2) * inv_c;
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V;
        if (c < p.C) {
          if (p.w_post) {
            float z[V];
            unpack<T, V>(pa[i], z);
#pragma unroll
            for (int e = 0; e < V; ++e)
              t[i][e] = rstd_a * fmaf(-(z[e] * rstd_a), c2, t[i][e]);
          }
          store_pack<T, V>(static_cast<T *>(p.da) + row * p.das + c, pack<T, V>(t[i]));
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
      const int c = (i * kNT + lane) * V;
      if (c < p.C)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          out[c + e] = accN[i][e];
          if constexpr (kJoin) out[p.C + c + e] = accA[i][e];
        }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kNT + lane) * V;
        if (c < p.C)
#pragma unroll
          for (int e = 0; e < V; ++e) dyn[sub * p.C + c + e] = k ? accA[kJoin ? i : 0][e] : accN[i][e];
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
// Threads per row and vectors per thread by the number of vectors in a row: a warp up to 128
// vectors (no exchange through shared memory), then as few threads as hold the row with at
// most two vectors each, so that several rows are in flight on an SM.
template <typename T, int V, bool kJoin>
cudaError_t fwd(const NormFwdParams &p, cudaStream_t s) {
  const int n = (p.C + V - 1) / V;
  auto go = [&](auto kernel, int threads, int rows) {
    kernel<<<(unsigned)((p.rows + rows - 1) / rows), threads, 0, s>>>(p);
    return cudaGetLastError();
  };
  if (n <= 32) return go(fwd_rows<T, V, 32, 1, kJoin>, 256, 8);
  if (n <= 64) return go(fwd_rows<T, V, 32, 2, kJoin>, 256, 8);
  if (n <= 128) return go(fwd_rows<T, V, 32, 4, kJoin>, 256, 8);
  if (n <= 256) return go(fwd_rows<T, V, 128, 2, kJoin>, 128, 1);
  if (n <= 512) return go(fwd_rows<T, V, 256, 2, kJoin>, 256, 1);
  if (n <= 1024) return go(fwd_rows<T, V, 512, 2, kJoin>, 512, 1);
  if (n <= 2048) return go(fwd_rows<T, V, 512, 4, kJoin>, 512, 1);
  return go(fwd_long<T, V, kJoin>, 512, 1);
}

// Shape of the backward for rows of n vectors: threads per row (0: the long form).
struct BwdShape {
  int nt, nv, smem;
};
inline BwdShape bwd_shape(int n) {
  if (n <= 32) return {32, 1, 0};
  if (n <= 64) return {32, 2, 0};
  if (n <= 128) return {32, 4, 0};
  if (n <= 256) return {128, 2, 0};
  if (n <= 512) return {256, 2, 0};
  if (n <= 1024) return {512, 2, 0};
  if (n <= 2048) return {512, 4, 1};
  return {0, 0, 0};
}

template <typename T, int V, bool kJoin>
cudaError_t bwd(const NormBwdParams &p, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.groups * p.ctas);
  constexpr int kSums = kJoin ? 2 : 1;
  auto go = [&](auto kernel, int threads, size_t smem) {
    if (smem > 48 * 1024) {
      const cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    kernel<<<grid, threads, smem, s>>>(p);
    return cudaGetLastError();
  };
  const int n = (p.C + V - 1) / V;
  const size_t warps = (size_t)8 * p.C * 4;  // the rows of a CTA side by side
  cudaError_t e;
  if (n <= 32)
    e = go(bwd_rows<T, V, 32, 1, kJoin, false>, 256, warps);
  else if (n <= 64)
    e = go(bwd_rows<T, V, 32, 2, kJoin, false>, 256, warps);
  else if (n <= 128)
    e = go(bwd_rows<T, V, 32, 4, kJoin, false>, 256, warps);
  else if (n <= 256)
    e = go(bwd_rows<T, V, 128, 2, kJoin, false>, 128, 0);
  else if (n <= 512)
    e = go(bwd_rows<T, V, 256, 2, kJoin, false>, 256, 0);
  else if (n <= 1024)
    e = go(bwd_rows<T, V, 512, 2, kJoin, false>, 512, 0);
  else if (n <= 2048)
    e = go(bwd_rows<T, V, 512, 4, kJoin, true>, 512, (size_t)kSums * p.C * 4);
  else
    e = go(bwd_long<T, V, kJoin>, 512, 0);
  if (e != cudaSuccess) return e;
  bwd_sums<T, kJoin><<<(p.C + 31) / 32, 1024, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace norm
}  // namespace dash

// The launches of one element type (inside namespace dash); `wide`: rows, strides and addresses allow 16-byte vectors.
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


