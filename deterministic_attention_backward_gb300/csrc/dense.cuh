// dense.cuh -- products with their epilogue: parameters and launch interface of the kernels.
//
//   C[m, n] = sum over parts p, sum over k:  A_p[m, k] B_p[n, k]
// with either dimension of an operand contiguous.  Forward, dx and dw are this one product with
// other operands:
//   forward  A = x, B = w^T; gated: B tiles of w and of w_gate side by side in one accumulator
//   dx       A = dz (and dgate as second part), B = w (and w_gate)
//   dw       A = x^T, B = dz^T (and dgate^T for a second output); w stored [N, K]: A and B change
//            places
#pragma once
#include "common.cuh"

namespace dash {

constexpr int kDenseM = 256;   // rows of a tile, of a pair of CTAs
constexpr int kDenseK = 64;    // contraction elements of a stage

// What the backward needs of z and g is kept in three bytes an element, the fp32 value rounded to its upper
// 24 bits: with 16 bits their rounding would make a third and more of the gradients' squared error.  Rows of
// `stride` (N rounded up to 16) 16-bit words, then as many rows of bytes.
struct DenseKept {
  uint16_t *hi;  // null: not kept
  uint8_t *lo;
};
inline long long kept_stride(long long N) { return (N + 15) / 16 * 16; }
inline DenseKept kept_at(void *p, long long M, long long N) {
  return {static_cast<uint16_t *>(p),
          p ? static_cast<uint8_t *>(p) + 2 * M * kept_stride(N) : nullptr};
}

// What follows the product: y = residual + act(z) * g, with z = product + bias (and g likewise,
// gated); z and g kept where asked for.
struct DenseEpilogue {
  void *y;
  DenseKept z, g;
  const void *bias, *bias_gate, *residual;
  long long ys, ks, rs;  // row strides in elements; the product kernel wants 16-byte steps
  int act, gated;
};
struct DenseParams {
  DenseEpilogue e;
  void *y1;                  // the second output (outs == 2)
  long long y1s;
  float *part;               // fp32 sums of the split tiles: [tile][split][256][bn]
  uint32_t *status;
  uint32_t *special;         // set where a sum is infinite or NaN; null: not asked
  int clear;                 // the status block (the first product of a call does)
  unsigned long long wait_ns;
  int M, N;
  int group;                 // rows of tiles that are worked through together
  int mt, nt, bn;            // tiles; bn columns of a tile's accumulator (gated: half z, half g)
  int nk, parts, outs;       // blocks of kDenseK of a part; parts, terms counted too
  int pairs;                 // parts go by pairs of operands (a gated dx): the first pair, the second
  int stack;                 // A's second term in rows 128 on of the (only) tile's, added behind to sums
                             // that are finite (see DenseSpecials)
  int a_low, b_low;          // rows behind which an operand's second term begins (0: it has the same)
  int whole, splits, per;    // tiles that are whole; splits of each other tile, blocks of a split
  int a_mn, b_mn;            // the contiguous dimension is M (N), not the contraction
  int a_out, b_out;          // the second output takes the second A (B)
  int withhold;              // block at which a CTA's loads end, else -1
};

// A forward of few rows (outputs as in the epilogue above).
constexpr int kFewRows = 64, kFewStages = 12, kFewSmem = 224 * 1024;
struct DenseFewParams {
  DenseEpilogue e;
  uint32_t *status;
  unsigned long long wait_ns;
  int M, N, nk;
  int cols;            // M rounded up to 16
  int split, per;      // CTAs of a cluster, blocks of kDenseK of each
  int stages, stage;   // their number and bytes
  int smem, tmem;
  int w_mn;            // the weights' rows are the contraction
  int withhold;
};

// dz = dy g act'(z), dgate = dy act(z) and their sums over rows.
struct DenseGradParams {
  const void *dy;
  DenseKept z, g;            // no z: dz = dy (and is not written); no g: not gated
  void *dz, *dg;             // null where only the sums are wanted
  int low;                   // what dz and dg lose by rounding follows them, M rows on
  uint32_t *special;         // cleared (DenseParams), null: there is none
  float *part, *part_gate;   // [chunks][N]; null where the sums are not wanted
  long long dys, ks, ds;
  int M, N, act, chunk;      // rows of a chunk
  int vec;                   // dy lies on 16 bytes
};

// A second term of dz is added to the first one's sums in one accumulator.  An infinity in x or a weight is
// multiplied by both: infinity times a second term that is 0, or of the other sign, would make NaN of what
// is infinite.  Such elements are formed again from the first term alone, out[r, c] = sum over parts and k
// of a[r, k] b[c, k], as a call of one term has them.
struct DenseOperand {
  const void *at;
  long long row, k;          // strides in elements
};
struct DenseSpecial {
  void *out;                 // null: nothing to do
  long long stride;
  int rows, cols, K, parts;
  DenseOperand a[2], b[2];
};
struct DenseSpecials {
  DenseSpecial s[3];
  const uint32_t *set;
};

cudaError_t launch_dense(bool f16, const CUtensorMap (&ta)[2], const CUtensorMap (&tb)[2],
                         const DenseParams &p, int sms, cudaStream_t s);
cudaError_t launch_dense_few(bool f16, const CUtensorMap &tw0, const CUtensorMap &tw1,
                             const CUtensorMap &tx, const DenseFewParams &p, cudaStream_t s);
cudaError_t launch_dense_grad(bool f16, const DenseGradParams &p, int chunks, cudaStream_t s);
cudaError_t launch_dense_specials(bool f16, const DenseSpecials &p, cudaStream_t s);
// out[n] = sum over chunks, in order (gate: a second row of sums and its output)
cudaError_t launch_dense_sums(bool f16, const float *part, const float *part_gate, void *out,
                              void *out_gate, int chunks, int N, cudaStream_t s);
// Up to four copies of rows of cols elements of two bytes in one launch: to rows on 16 bytes, the last
// vector filled up with zeros, or (out) from there to rows anywhere.
struct DenseCopy {
  const void *in;
  void *out;
  long long is, os;
  int rows, cols;
};
struct DenseCopies {
  DenseCopy c[4];
  int count;
};
cudaError_t launch_dense_copies(const DenseCopies &c, bool out, cudaStream_t s);

}  // namespace dash
