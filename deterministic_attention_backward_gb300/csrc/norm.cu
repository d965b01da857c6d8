// norm.cu -- the extern "C" entries of the row norms: argument checks, the partition of the
// rows among CTAs, the choice of vector width.
#include "norm.cuh"

#include "common.cuh"
#include "dash_attn.h"
#include "elem.cuh"
#include "host.cuh"

namespace dash {

// CTAs per gate group of the backward: in all as many as 152 SMs hold at once (by the ring's
// shared memory and the column sums' registers, see ring_shape), whatever the device, so that
// the order of the weight gradients' sums does not depend on it; never more than there are
// rows for.  Rows off the 16-byte grid: as many for each of `period` alignments.
int norm_bwd_ctas(long long rows, long long groups, int C, int elem_bytes, bool wide, int period,
                  bool join) {
  const int vec = 16 / elem_bytes;
  const int n = wide ? (C + (period ? vec - 1 : 0) + vec - 1) / vec : C;
  int sms_share = 2, at_once = 1;  // CTAs on an SM, rows of a CTA at once
  if (!wide) {
    if (n <= 128) at_once = 8;
  } else if (n <= 32) {
    at_once = n <= 4 ? 64 : n <= 8 ? 32 : n <= 16 ? 16 : 8;
    sms_share = join ? 2 : 4;
  } else if (n <= 64) {
    at_once = join ? 8 : 1;
    sms_share = join ? 2 : 16;
  } else if (n <= 512) {
    sms_share = n <= 128 ? 8 : n <= 256 ? 4 : 2;
  } else if (n <= 2048) {
    sms_share = 1;
  }
  const int kinds = period ? period : 1;
  const long long per = (rows / groups + kinds - 1) / kinds;
  const long long most = (per + at_once - 1) / at_once;
  const long long want = 152LL * sms_share / groups / kinds;
  return (int)(want < 1 ? 1 : want < most ? want : most) * kinds;
}

namespace {

bool elem_ok(int t) { return t == DASH_BF16 || t == DASH_FP16 || t == DASH_FP32; }
int elem_size(int t) { return t == DASH_FP32 ? 4 : 2; }

// Whether every pointer (null ones aside) is aligned to `size` bytes.
template <int N>
bool all_aligned(const void *const (&ptrs)[N], uintptr_t size) {
  uintptr_t any = 0;
  for (const void *q : ptrs) any |= reinterpret_cast<uintptr_t>(q);
  return (any & (size - 1)) == 0;
}

// Row tensors: outputs may each be an input as it lies, or what no other tensor of the call is.
struct Rows {
  const void *at;
  long long stride;
};
Bytes lies(const Rows &r, long long rows, int C, int size) {
  return along(bytes_of(r.at, size, C), size, r.stride, rows);
}
template <int N, int M, int K>
bool rows_apart(const Rows (&outs)[N], const Rows (&ins)[M], const Bytes (&others)[K],
                long long rows, int C, int size) {
  for (int i = 0; i < N; ++i) {
    const Bytes out = lies(outs[i], rows, C, size);
    for (int k = 0; k < i; ++k)
      if (share(out, lies(outs[k], rows, C, size))) return false;
    for (const Rows &r : ins)
      if (!(r.at == outs[i].at && r.stride == outs[i].stride) &&
          share(out, lies(r, rows, C, size)))
        return false;
    for (const Bytes &o : others)
      if (share(out, o)) return false;
  }
  return true;
}

dash_status_t check_rows(long long rows, int C, long long gate_rows, bool gate, int dtype,
                         int wdtype) {
  if (rows <= 0 || C <= 0 || !elem_ok(dtype) || (wdtype != dtype && wdtype != DASH_FP32))
    return DASH_ERR_INVALID;
  if (gate && (gate_rows <= 0 || rows % gate_rows)) return DASH_ERR_INVALID;
  if (rows >= (1LL << 31) || C > (1 << 24)) return DASH_ERR_UNSUPPORTED;
  return DASH_OK;
}

// How rows lie on the grid of 16-byte vectors: on it (wide, period 0), off it but in the same way
// in every tensor (wide, period the rows after which they lie the same again), or neither.
struct Lie {
  bool wide = false;
  int period = 0, off = 0, stride_mod = 0;
};
template <int N, int M>
Lie lie_of(const void *const (&ptrs)[N], const long long *strides, const void *const (&weights)[M],
           int C, int size, long long group_rows) {
  const int vec = 16 / size;
  Lie l;
  bool first = true, same = true;
  for (int i = 0; i < N; ++i) {
    if (!ptrs[i]) continue;
    const int off = (int)(reinterpret_cast<uintptr_t>(ptrs[i]) & 15) / size;
    const int mod = (int)(strides[i] & (vec - 1));
    if (first) l.off = off, l.stride_mod = mod;
    same = same && off == l.off && mod == l.stride_mod;
    first = false;
  }
  if (same && l.off == 0 && l.stride_mod == 0 && C % vec == 0 && all_aligned(weights, 16)) {
    l.wide = true;
    return l;
  }
  l.period = 1;
  while ((l.period * l.stride_mod) & (vec - 1)) l.period *= 2;
  // A CTA takes rows of one alignment: with few rows of each, or rows of a few vectors, it would
  // stand half empty, and element by element they take a launch's time as well.  At 22324 rows of
  // 1503 in bf16 the join takes 60 us forward, 128 backward (by elements 146, 212), at 124275 rows
  // of 270 98 and 200 (244, 599).  Rows beyond the ring's go element by element.
  l.wide = same && C >= 2 * vec && group_rows >= 8 * l.period && (C + 2 * vec - 2) / vec <= 2048;
  if (!l.wide) l.period = 0;
  return l;
}

struct Groups {
  int groups, ctas, row_gate;
  long long gate_rows;
};
Groups make_groups(long long rows, int C, long long gate_rows, bool gate, int dtype, bool wide,
                   int period, bool join) {
  Groups g{1, 1, gate && gate_rows == 1 && rows > 1, rows};
  if (gate && !g.row_gate) g.gate_rows = gate_rows;
  g.groups = (int)(rows / g.gate_rows);
  g.ctas = norm_bwd_ctas(rows, g.groups, C, elem_size(dtype), wide, period, join);
  return g;
}

}  // namespace
}  // namespace dash

extern "C" {

dash_status_t dash_join_fwd(const void *x, const void *a, const void *w_post, const void *gate,
                            const void *w_next, void *y, void *h, float *rstd_a, float *rstd_y,
                            long long rows, int C, long long gate_rows,
                            const long long strides[4], float skip_scale, float branch_scale,
                            float eps, dash_dtype_t dtype, dash_dtype_t wdtype,
                            dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_rows(rows, C, gate_rows, gate != nullptr, dtype, wdtype);
  if (st != DASH_OK) return st;
  const bool join = a != nullptr;
  if (!x || !strides || (join ? !y : !w_next || w_post || gate)) return DASH_ERR_INVALID;
  if ((w_next && (!h || !rstd_y)) || (w_post && !rstd_a)) return DASH_ERR_INVALID;
  const int size = elem_size(dtype);
  const void *rowp[] = {x, a, join ? y : nullptr, w_next ? h : nullptr};
  const void *wp[] = {w_post, gate, w_next};
  const void *fp[] = {rstd_a, rstd_y};
  if (!all_aligned(rowp, size) || !all_aligned(wp, elem_size(wdtype)) || !all_aligned(fp, 4))
    return DASH_ERR_INVALID;
  const int wsize = elem_size(wdtype);
  const Bytes stats[] = {bytes_of(w_post ? rstd_a : nullptr, 4, rows),
                         bytes_of(w_next ? rstd_y : nullptr, 4, rows)};
  const Bytes weights[] = {bytes_of(w_post, wsize, C),
                           bytes_of(gate, wsize, gate ? rows / gate_rows * C : 0),
                           bytes_of(w_next, wsize, C)};
  const Rows outs[] = {{rowp[2], strides[2]}, {rowp[3], strides[3]}};
  const Rows ins[] = {{x, strides[0]}, {a, strides[1]}};
  const Bytes beside[] = {weights[0], weights[1], weights[2], stats[0], stats[1]};
  const Bytes reads[] = {lies(ins[0], rows, C, size), lies(ins[1], rows, C, size),
                         weights[0], weights[1], weights[2]};
  if (!rows_apart(outs, ins, beside, rows, C, size) || !apart(stats, reads))
    return DASH_ERR_INVALID;
  const Lie lie = lie_of(rowp, strides, wp, C, size, rows);
  const bool wide = lie.wide;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  NormFwdParams p{};
  p.x = x, p.a = a, p.w_post = w_post, p.gate = gate, p.w_next = w_next;
  p.y = y, p.h = h, p.rstd_a = rstd_a, p.rstd_y = rstd_y;
  p.xs = strides[0], p.as = strides[1], p.ys = strides[2], p.hs = strides[3];
  p.rows = rows;
  p.gate_rows = gate ? gate_rows : rows;
  p.C = C;
  p.wf32 = wdtype == DASH_FP32 && dtype != DASH_FP32;
  p.period = lie.period, p.off = lie.off, p.stride_mod = lie.stride_mod;
  p.skip = skip_scale, p.branch = branch_scale, p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DASH_BF16   ? launch_norm_fwd<__nv_bfloat16>(p, join, wide, s)
                        : dtype == DASH_FP16 ? launch_norm_fwd<__half>(p, join, wide, s)
                                             : launch_norm_fwd<float>(p, join, wide, s);
  return e == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

size_t dash_join_bwd_workspace_bytes(long long rows, int C, long long gate_rows, int join,
                                     dash_dtype_t dtype) {
  using namespace dash;
  if (check_rows(rows, C, gate_rows, gate_rows > 0, dtype, dtype) != DASH_OK) return 0;
  size_t most = 0;
  for (int form = 0; form < 6; ++form) {  // by elements, on the grid, off it in 1 to 8 ways
    const int period = form < 2 ? 0 : 1 << (form - 2);
    const Groups g = make_groups(rows, C, gate_rows, gate_rows > 0, dtype, form > 0, period, join);
    if (period && g.gate_rows < 8 * period) break;
    const size_t n = align256((size_t)g.groups * g.ctas * (join ? 2 : 1) * C * sizeof(float));
    most = n > most ? n : most;
  }
  return most;
}

dash_status_t dash_join_bwd(const void *dy, const void *dh, const void *y, const void *a,
                            const void *w_post, const void *gate, const void *w_next,
                            const float *rstd_a, const float *rstd_y, void *dx, void *da,
                            void *dw_post, void *dgate, void *dw_next, long long rows, int C,
                            long long gate_rows, const long long strides[6], float skip_scale,
                            float branch_scale, dash_dtype_t dtype, dash_dtype_t wdtype,
                            void *workspace, size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  dash_status_t st = check_rows(rows, C, gate_rows, gate != nullptr, dtype, wdtype);
  if (st != DASH_OK) return st;
  const bool join = a != nullptr;
  if (!dx || !strides || (join ? !da || (!dy && !w_next) : !w_next || w_post || gate))
    return DASH_ERR_INVALID;
  if (w_next && (!dh || !y || !rstd_y || !dw_next)) return DASH_ERR_INVALID;
  if ((w_post && (!rstd_a || !dw_post)) || (gate && !dgate)) return DASH_ERR_INVALID;
  const int size = elem_size(dtype);
  const void *rowp[] = {dy, w_next ? dh : nullptr, w_next ? y : nullptr, a, dx,
                        join ? da : nullptr};
  const void *wp[] = {w_post, gate, w_next};
  const void *dwp[] = {w_post ? dw_post : nullptr, gate ? dgate : nullptr,
                       w_next ? dw_next : nullptr};
  const void *fp[] = {rstd_a, rstd_y};
  if (!all_aligned(rowp, size) || !all_aligned(wp, elem_size(wdtype)) ||
      !all_aligned(dwp, elem_size(wdtype)) || !all_aligned(fp, 4))
    return DASH_ERR_INVALID;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < dash_join_bwd_workspace_bytes(rows, C, gate ? gate_rows : 0, join, dtype))
    return DASH_ERR_WORKSPACE;
  const int wsize = elem_size(wdtype);
  const long long gates = gate ? rows / gate_rows * C : 0;
  const Bytes sums[] = {bytes_of(dwp[0], wsize, C), bytes_of(dwp[1], wsize, gates),
                        bytes_of(dwp[2], wsize, C),
                        bytes_of(workspace, 1,
                                 dash_join_bwd_workspace_bytes(rows, C, gate ? gate_rows : 0, join,
                                                               dtype))};
  const Bytes weights[] = {bytes_of(w_post, wsize, C), bytes_of(gate, wsize, gates),
                           bytes_of(w_next, wsize, C), bytes_of(w_post ? rstd_a : nullptr, 4, rows),
                           bytes_of(w_next ? rstd_y : nullptr, 4, rows)};
  const Rows outs[] = {{dx, strides[4]}, {rowp[5], strides[5]}};
  const Rows ins[] = {{rowp[0], strides[0]}, {rowp[1], strides[1]}, {rowp[2], strides[2]},
                      {a, strides[3]}};
  const Bytes beside[] = {weights[0], weights[1], weights[2], weights[3], weights[4],
                          sums[0],    sums[1],    sums[2],    sums[3]};
  const Bytes reads[] = {weights[0], weights[1], weights[2], weights[3], weights[4],
                         lies(ins[0], rows, C, size), lies(ins[1], rows, C, size),
                         lies(ins[2], rows, C, size), lies(ins[3], rows, C, size)};
  if (!rows_apart(outs, ins, beside, rows, C, size) || !apart(sums, reads))
    return DASH_ERR_INVALID;
  const bool own_gates = gate && gate_rows == 1 && rows > 1;
  const Lie lie = lie_of(rowp, strides, wp, C, size, gate && !own_gates ? gate_rows : rows);
  const bool wide = lie.wide;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  const Groups g =
      make_groups(rows, C, gate_rows, gate != nullptr, dtype, wide, lie.period, join);
  NormBwdParams p{};
  p.dy = dy, p.dh = dh, p.y = y, p.a = a;
  p.w_post = w_post, p.gate = gate, p.w_next = w_next;
  p.rstd_a = rstd_a, p.rstd_y = rstd_y;
  p.dx = dx, p.da = da;
  p.dw_post = w_post ? dw_post : nullptr;
  p.dgate = gate ? dgate : nullptr;
  p.dw_next = w_next ? dw_next : nullptr;
  p.part = static_cast<float *>(workspace);
  p.dys = strides[0], p.dhs = strides[1], p.ys = strides[2], p.as = strides[3];
  p.dxs = strides[4], p.das = strides[5];
  p.rows = rows;
  p.gate_rows = g.gate_rows;
  p.groups = g.groups, p.ctas = g.ctas, p.row_gate = g.row_gate;
  p.C = C;
  p.wf32 = wdtype == DASH_FP32 && dtype != DASH_FP32;
  p.period = lie.period, p.off = lie.off, p.stride_mod = lie.stride_mod;
  p.skip = skip_scale, p.branch = branch_scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == DASH_BF16   ? launch_norm_bwd<__nv_bfloat16>(p, join, wide, s)
                        : dtype == DASH_FP16 ? launch_norm_bwd<__half>(p, join, wide, s)
                                             : launch_norm_bwd<float>(p, join, wide, s);
  return e == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
