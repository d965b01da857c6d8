// norm.cuh -- parameters and launch interface of the row norms (norm_kernel.cuh).
#pragma once
#include <cuda_runtime.h>

namespace dash {

// Rows of C elements; a row stride of its own for every tensor.  Weights and gates are of the
// rows' type, or fp32 where wf32.
struct NormFwdParams {
  const void *x, *a;                     // residual stream, branch (join only)
  const void *w_post, *gate, *w_next;    // each may be null (join); w_next is there for a norm
  void *y, *h;                           // joined stream (join only), normed rows (null: none)
  float *rstd_a, *rstd_y;
  long long xs, as, ys, hs;
  long long rows, gate_rows;             // gate row of row r: r / gate_rows
  int C, wf32;
  int period, off, stride_mod;           // rows off the 16-byte grid (period 0: on it)
  float skip, branch, eps;
};
struct NormBwdParams {
  const void *dy, *dh, *y, *a;           // dy: gradient of the joined stream, may be null
  const void *w_post, *gate, *w_next;
  const float *rstd_a, *rstd_y;
  void *dx, *da, *dw_post, *dgate, *dw_next;
  float *part;                           // [groups * ctas][2][C] partial sums
  long long dys, dhs, ys, as, dxs, das;
  long long rows, gate_rows;             // rows of a group: groups * gate_rows = rows
  int groups, ctas;                      // CTAs per group
  int row_gate;                          // every row has a gate row of its own
  int C, wf32;
  int period, off, stride_mod;
  float skip, branch;
};

int norm_bwd_ctas(long long rows, long long groups, int C, int elem_bytes, bool wide, int period,
                  bool join);

template <typename T>
cudaError_t launch_norm_fwd(const NormFwdParams &p, bool join, bool wide, cudaStream_t s);
template <typename T>
cudaError_t launch_norm_bwd(const NormBwdParams &p, bool join, bool wide, cudaStream_t s);

}  // namespace dash
