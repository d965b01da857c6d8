// grads.cu -- the norm over many gradients and clipping by it.
//   norm = sqrt(sum over all tensors of g^2),    g *= min(1, max_norm / (norm + eps))
//
// Bound by memory: the norm reads every gradient once, the scaling reads it again and writes it (in
// place and within the limit it does neither).  The tensors of a launch travel as its parameter; they
// are cut into chunks that the CTAs take in turn, and the scaling takes them in the opposite order, so
// that it begins with what the norm has left in L2.  A thread adds a chunk's squares in fp32, and what
// it has of all chunks in fp64; the CTAs' sums are added in a fixed order by whoever needs the norm,
// every CTA of the scaling for itself.  Which CTA takes a chunk, and which of its threads an element,
// follows from the sizes: the same bits on every run and wherever the tensors lie.
//
// Measured: 436 MB in bf16 clipped to other buffers 66 + 134 us, 6.6 TB/s, a copy's rate in both kernels
// (chunks taken in the same order by both: 2 us more); 3.5 GB in fp32 within the limit 490 us, 7.1 TB/s.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"
#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4 * 152;  // of a launch, GB300's SMs whatever GPU runs
constexpr int kMaxTensors = 512;
constexpr long long kMinChunk = 1 << 13, kMaxChunk = 1 << 16;  // elements

struct Grad {
  const void *in;
  void *out;
  long long n;
  int first;  // chunk
  int dtype;
};
template <int N>
struct GradTable {
  Grad t[N];
  int count, chunks, chunk;
};

// 16 bytes from `off` on of two neighbouring vectors.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, uint32_t off) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}, bits = 8 * (off & 3);
  uint32_t x[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    x[i] = off < 8 ? (off < 4 ? w[i] : w[i + 1]) : (off < 12 ? w[i + 2] : w[i + 3]);
  return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                    __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

// f(element, its place in its vector) for this thread's share of n elements: vectors of 16 bytes from the
// first element on, eight on their way at once, and single ones behind the last.  Which thread takes an
// element, and when, follows from its number alone: where the first does not lie on 16 bytes, a vector is
// put together from two that do (the first and the last from single elements, so that nothing beside the
// tensor is read; 2^28 elements in bf16 119 us there, on 16 bytes 108).
template <typename T, typename F>
__device__ __forceinline__ void each_element(const T *p, long long n, F &&f) {
  constexpr int V = 16 / sizeof(T), U = 8;
  const long long vecs = n / V;
  const uint32_t off = reinterpret_cast<uintptr_t>(p) & 15;
  const uint4 *v = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - off);
  auto take = [&](const uint4 &r) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int k = 0; k < V; ++k) f(to_f32<T>(e[k]), k);
  };
  long long i = threadIdx.x;
  if (off == 0) {
    for (; i + (U - 1) * kThreads < vecs; i += U * kThreads) {
      uint4 r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = v[i + u * kThreads];
#pragma unroll
      for (int u = 0; u < U; ++u) take(r[u]);
    }
    for (; i < vecs; i += kThreads) take(v[i]);
  } else {
    auto single = [&](long long i) {
#pragma unroll
      for (int k = 0; k < V; ++k) f(to_f32<T>(p[i * V + k]), k);
    };
    if (i == 0 && vecs > 0) single(0), i += kThreads;
    constexpr int H = U / 2;  // (two loads a vector)
    for (; i + (H - 1) * kThreads < vecs - 1; i += H * kThreads) {
      uint4 r[H], q[H];
#pragma unroll
      for (int u = 0; u < H; ++u) r[u] = v[i + u * kThreads], q[u] = v[i + u * kThreads + 1];
#pragma unroll
      for (int u = 0; u < H; ++u) take(shifted(r[u], q[u], off));
    }
    for (; i < vecs - 1; i += kThreads) take(shifted(v[i], v[i + 1], off));
    if (i == vecs - 1) single(i);
  }
  const long long rest = vecs * V + threadIdx.x;
  if (rest < n) f(to_f32<T>(p[rest]), 0);
}

// The sum of squares of a thread's elements.  Where fp32 has not held it, a value scaled by a power of
// two is squared instead: by 2^-70 behind an overflow (then a square of 2^120 at least is among them),
// by 2^96 where all are so small that squares may have been lost.  Zeros alone (rows of a table that a step
// has not met) are told by their bits and are not read again (2^28 fp32 zeros 185 us, as many values too,
// read twice 317).
template <typename T>
__device__ __forceinline__ double squares(const T *p, long long n) {
  float s[4] = {};
  uint32_t bits = 0;
  each_element<T>(p, n, [&](float x, int k) {
    s[k & 3] = fmaf(x, x, s[k & 3]);
    bits |= __float_as_uint(x);
  });
  float t = (s[0] + s[1]) + (s[2] + s[3]);
  if constexpr (std::is_same<T, __half>::value) return t;  // squares from 2^-48 to 2^32
  if ((t >= 0x1p-100f && t < INFINITY) || bits << 1 == 0) return t;
  const bool big = !(t < 1.f);
  const float by = big ? 0x1p-70f : 0x1p96f;
  float u[4] = {};
  each_element<T>(p, n, [&](float x, int k) { u[k & 3] = fmaf(x * by, x * by, u[k & 3]); });
  return (double)((u[0] + u[1]) + (u[2] + u[3])) * (big ? 0x1p140 : 0x1p-192);
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double sums[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) v += sums[i];
  return v;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ GradTable<N> g, double *part) {
  double s = 0.0;
  int t = 0;
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    while (t + 1 < g.count && g.t[t + 1].first <= c) ++t;
    const Grad &q = g.t[t];
    const long long at = (long long)(c - q.first) * g.chunk, n = min((long long)g.chunk, q.n - at);
    if (q.dtype == DASH_BF16)
      s += squares<__nv_bfloat16>(static_cast<const __nv_bfloat16 *>(q.in) + at, n);
    else if (q.dtype == DASH_FP16)
      s += squares<__half>(static_cast<const __half *>(q.in) + at, n);
    else
      s += squares<float>(static_cast<const float *>(q.in) + at, n);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The norm from the CTAs' sums, the same in every CTA that asks.
__device__ __forceinline__ float norm_of(const double *part, int parts) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return (float)sqrt(block_sum(s));
}
__global__ void __launch_bounds__(kThreads)
    grad_sum_kernel(const double *part, int parts, float *norm) {
  const float n = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = n;
}

template <typename T>
__device__ __forceinline__ void scale(const T *in, T *out, long long n, float by) {
  constexpr int V = 16 / sizeof(T), U = 4;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  long long skip = n;  // vectors where both lie alike
  if (((a ^ b) & 15) == 0) skip = min(n, (long long)((16 - (a & 15)) & 15) / (long long)sizeof(T));
  const long long vecs = (n - skip) / V;
  const uint4 *v = reinterpret_cast<const uint4 *>(in + skip);
  uint4 *w = reinterpret_cast<uint4 *>(out + skip);
  auto scaled = [&](uint4 r) {
    Pack<T, V> p;
    *reinterpret_cast<uint4 *>(&p) = r;
    float f[V];
    unpack<T, V>(p, f);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] *= by;
    p = pack<T, V>(f);
    return *reinterpret_cast<const uint4 *>(&p);
  };
  long long i = threadIdx.x;
  for (; i + (U - 1) * kThreads < vecs; i += U * kThreads) {
    uint4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = v[i + u * kThreads];
#pragma unroll
    for (int u = 0; u < U; ++u) w[i + u * kThreads] = scaled(r[u]);
  }
  for (; i < vecs; i += kThreads) w[i] = scaled(v[i]);
  for (long long e = threadIdx.x; e < skip; e += kThreads) out[e] = from_f32<T>(to_f32<T>(in[e]) * by);
  for (long long e = skip + vecs * V + threadIdx.x; e < n; e += kThreads)
    out[e] = from_f32<T>(to_f32<T>(in[e]) * by);
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_clip_kernel(const __grid_constant__ GradTable<N> g, const double *part, int parts,
                     const float *given, float *norm, float max_norm, float eps) {
  const float n = given ? *given : norm_of(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  float by = n == 0.f ? 1.f : max_norm / (n + eps);
  if (by > 1.f || (max_norm == INFINITY && n == n)) by = 1.f;  // (a NaN stays)
  int t = g.count - 1;
  // a CTA's last chunk first
  const int mine = (g.chunks - 1 - (int)blockIdx.x) / (int)gridDim.x;
  for (int i = mine; i >= 0; --i) {
    const int c = blockIdx.x + i * gridDim.x;
    while (g.t[t].first > c) --t;
    const Grad &q = g.t[t];
    if (by == 1.f && q.in == q.out) continue;
    const long long at = (long long)(c - q.first) * g.chunk, left = min((long long)g.chunk, q.n - at);
    if (q.dtype == DASH_BF16)
      scale(static_cast<const __nv_bfloat16 *>(q.in) + at, static_cast<__nv_bfloat16 *>(q.out) + at,
            left, by);
    else if (q.dtype == DASH_FP16)
      scale(static_cast<const __half *>(q.in) + at, static_cast<__half *>(q.out) + at, left, by);
    else
      scale(static_cast<const float *>(q.in) + at, static_cast<float *>(q.out) + at, left, by);
  }
}

// ------------------------------------------------------------------ host
int size_of(int dtype) { return dtype == DASH_FP32 ? 4 : 2; }

dash_status_t check(const dash_grad_t *g, int count, bool write) {
  if (count < 0 || (count > 0 && !g)) return DASH_ERR_INVALID;
  for (int i = 0; i < count; ++i) {
    const dash_grad_t &q = g[i];
    if (q.dtype != DASH_BF16 && q.dtype != DASH_FP16 && q.dtype != DASH_FP32) return DASH_ERR_INVALID;
    if (q.n < 0 || (q.n > 0 && !q.in) || (write && q.n > 0 && !q.out)) return DASH_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(q.in) | (write ? reinterpret_cast<uintptr_t>(q.out) : 0)) &
        (size_of(q.dtype) - 1))
      return DASH_ERR_INVALID;
    if (q.n >= (1LL << 46)) return DASH_ERR_UNSUPPORTED;
  }
  return DASH_OK;
}

struct Span {
  uintptr_t at, end;
  int tensor;
  bool out;
};
// Whether what is written meets nothing else, a tensor's own input in its place apart.
bool apart_from_all(const dash_grad_t *g, int count, const Bytes (&others)[2], const float *given) {
  std::vector<Span> all;
  all.reserve(2 * (size_t)count + 3);
  auto add = [&](const void *p, long long bytes, int tensor, bool out) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0 && p) all.push_back({at, at + (uintptr_t)bytes, tensor, out});
  };
  for (int i = 0; i < count; ++i) {
    const long long bytes = g[i].n * size_of(g[i].dtype);
    add(g[i].out, bytes, i, true);
    if (g[i].in != g[i].out) add(g[i].in, bytes, i, false);
  }
  for (const Bytes &o : others)
    if (o.run) all.push_back({o.at, o.at + (uintptr_t)o.run, -1, true});
  add(given, 4, -2, false);
  std::sort(all.begin(), all.end(), [](const Span &a, const Span &b) { return a.at < b.at; });
  uintptr_t end_out = 0, end_in = 0;  // how far what came before reaches
  for (const Span &s : all) {
    if (s.at < end_out || (s.out && s.at < end_in)) return false;
    uintptr_t &end = s.out ? end_out : end_in;
    if (s.end > end) end = s.end;
  }
  return true;
}

// Tensors [from, to) of at most N that are not empty; returns how far it came.
template <int N>
int fill(GradTable<N> &t, const dash_grad_t *g, int from, int count) {
  t.count = 0;
  long long all = 0;
  int to = from;
  for (int i = from, c = 0; i < count && c < N; to = ++i)
    if (g[i].n > 0) all += g[i].n, ++c;
  // a few chunks for every CTA, a whole number of vectors each
  long long chunk = (all / (4 * kCtas) + 63) / 64 * 64;
  chunk = chunk < kMinChunk ? kMinChunk : chunk > kMaxChunk ? kMaxChunk : chunk;
  while (all / chunk >= (1 << 30)) chunk *= 2;
  t.chunk = (int)chunk;
  long long first = 0;
  for (int i = from; i < to; ++i) {
    if (g[i].n <= 0) continue;
    t.t[t.count++] = {g[i].in, g[i].out, g[i].n, (int)first, g[i].dtype};
    first += (g[i].n + chunk - 1) / chunk;
  }
  t.chunks = (int)first;
  return to;
}

// Calls f(table, launch number) for the tensors of each launch.
template <typename F>
void launches(const dash_grad_t *g, int count, F &&f) {
  int used = 0;
  for (int i = 0; i < count; ++i) used += g[i].n > 0;
  if (used <= 64) {  // the smaller parameter is the quicker launch
    GradTable<64> t;
    if (used > 0) fill(t, g, 0, count), f(t, 0);
    return;
  }
  GradTable<kMaxTensors> t;
  for (int i = 0, k = 0; i < count; ++k) {
    i = fill(t, g, i, count);
    if (t.count > 0) f(t, k);
  }
}

template <int N>
int ctas(const GradTable<N> &t) { return t.chunks < kCtas ? t.chunks : kCtas; }

}  // namespace
}  // namespace dash

extern "C" {

size_t dash_grad_norm_workspace_bytes(int count) {
  using namespace dash;
  return count >= 0 ? (((size_t)count + kMaxTensors - 1) / kMaxTensors + 1) * kCtas * 8 : 0;
}

dash_status_t dash_grad_norm(const dash_grad_t *grads, int count, float *norm, void *workspace,
                             size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check(grads, count, false);
  if (st != DASH_OK) return st;
  if (!norm || !aligned4(norm)) return DASH_ERR_INVALID;
  const size_t need = dash_grad_norm_workspace_bytes(count);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need) return DASH_ERR_WORKSPACE;
  const Bytes own[2] = {bytes_of(norm, 4, 1), bytes_of(workspace, 1, (long long)need)};
  if (share(own[0], own[1])) return DASH_ERR_INVALID;
  for (int i = 0; i < count; ++i) {
    const Bytes g = bytes_of(grads[i].in, size_of(grads[i].dtype), grads[i].n);
    if (share(g, own[0]) || share(g, own[1])) return DASH_ERR_INVALID;
  }
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double *part = static_cast<double *>(workspace);
  int parts = 0;
  launches(grads, count, [&](const auto &t, int) {
    grad_norm_kernel<<<ctas(t), kThreads, 0, s>>>(t, part + parts);
    parts += ctas(t);
  });
  grad_sum_kernel<<<1, kThreads, 0, s>>>(part, parts, norm);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status_t dash_grad_clip(const dash_grad_t *grads, int count, float max_norm, float eps,
                             const float *given, float *norm, void *workspace,
                             size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check(grads, count, true);
  if (st != DASH_OK) return st;
  if (!(max_norm >= 0.f) || !(eps >= 0.f)) return DASH_ERR_INVALID;
  if ((!given && !norm) || !aligned4(norm) || !aligned4(given)) return DASH_ERR_INVALID;
  const size_t need = given ? 0 : dash_grad_norm_workspace_bytes(count);
  if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
    return DASH_ERR_WORKSPACE;
  const Bytes own[2] = {bytes_of(norm, 4, 1),
                        bytes_of(need ? workspace : nullptr, 1, (long long)need)};
  bool apart = false;
  try {
    apart = apart_from_all(grads, count, own, given);
  } catch (...) {  // no memory for the list
    return DASH_ERR_CUDA;
  }
  if (!apart) return DASH_ERR_INVALID;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double *part = static_cast<double *>(workspace);
  int parts = 0, left = 0;
  launches(grads, count, [&](const auto &t, int) {
    if (!given) grad_norm_kernel<<<ctas(t), kThreads, 0, s>>>(t, part + parts);
    parts += ctas(t), ++left;
  });
  if (left == 0 && norm) {  // nothing to clip: the norm of nothing, or the one given
    if (given)
      return cudaMemcpyAsync(norm, given, 4, cudaMemcpyDeviceToDevice, s) == cudaSuccess
                 ? DASH_OK
                 : DASH_ERR_CUDA;
    return cudaMemsetAsync(norm, 0, 4, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  }
  launches(grads, count, [&](const auto &t, int k) {
    grad_clip_kernel<<<ctas(t), kThreads, 0, s>>>(t, part, parts, given, k == 0 ? norm : nullptr,
                                                  max_norm, eps);
  });
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
