// dense.cu -- the extern "C" entries of products with their epilogue: argument checks, the choice
// of tiles and splits, workspace carving, tensor maps, launches.
#include "dense.cuh"

#include "dash_attn.h"
#include "host.cuh"

namespace dash {
namespace {

std::atomic<int> g_dense_withhold{-1};

constexpr int kMaxSize = 1 << 30;  // coordinates and row numbers are 32-bit
bool aligned2(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
long long up(long long n, long long to) { return (n + to - 1) / to * to; }
int ceil_div(long long n, long long d) { return (int)((n + d - 1) / d); }

// An operand as rows of `cols` contiguous elements; `pad`: copied to an aligned place first.
struct Rows {
  const void *at = nullptr;
  long long stride = 0;
  int rows = 0, cols = 0;
  bool pad = false;
  Rows() = default;
  Rows(const void *at, long long stride, int rows, int cols)
      : at(at), stride(rows > 1 ? stride : up(cols, 8)), rows(rows), cols(cols) {
    pad = at && (!aligned16(at) || this->stride % 8 || this->stride < cols);
  }
  size_t bytes() const { return pad ? align256((size_t)rows * up(cols, 8) * 2) : 0; }
  Bytes lies() const { return along(bytes_of(at, 2, cols), 2, stride, rows); }
};

// A tensor map over rows: boxes of 64 contiguous elements x `box` rows.
bool make_rows_map(CUtensorMap *m, const Rows &r, int box, bool f16) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)r.cols, (cuuint64_t)r.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)r.stride * 2};
  const cuuint32_t boxes[2] = {(cuuint32_t)kDenseK, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
             const_cast<void *>(r.at), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One product: its sizes, and the tiles and splits chosen for them.
struct Product {
  int M, N, K, parts, outs;
  bool gated;
  bool stack = false;  // A's second term in the tile's other 128 rows
  int bn = 256, whole = 0, splits = 1, per = 0;
  double cost = 0;
  int cols() const { return gated ? bn / 2 : bn; }
  int mt() const { return ceil_div(M, kDenseM); }
  int nt() const { return ceil_div(N, cols()); }
  int nk() const { return ceil_div(K, kDenseK); }
  long long tiles() const { return (long long)mt() * nt() * outs; }
  size_t part_bytes() const {
    return splits > 1 || stack ? (size_t)(tiles() - whole) * splits * kDenseM * bn * 4 : 0;
  }
};

// The choice follows from the sizes alone, as the order of the sums does (the pairs of SMs are those of
// a GB300, not of the GPU that runs).  Tiles that fill whole rounds of the pairs stay whole; the rest,
// which would leave pairs idle, are split along the contraction where that is shorter, or, of a few
// rounds, all of them.  Time is counted in blocks of 64 of a 256-column tile (0.27 us): a block of 128
// columns costs 0.62 (19456 x 4096 x 4096 402 us against 325; 1237 x 4096 x 4096, where it fills the
// pairs better, 39 against 40), an item 3 beside its blocks, the kernel that adds the splits 10 and the
// partial sums their way to memory.
constexpr int kPairs = 76, kMaxSplits = 64;
Product plan(int M, int N, int K, int parts, int outs, bool gated, bool stack = false) {
  Product best;
  for (int bn = 256; bn >= 128; bn -= 128) {
    Product p{M, N, K, parts, outs, gated, stack, bn};
    const long long tiles = p.tiles(), rounds = tiles / kPairs;
    if (tiles >= (1LL << 28)) continue;
    const int blocks = p.nk() * parts;
    const double block = bn == 256 ? 1.0 : 0.62;
    // whole rounds stay whole, or (a few rounds; two terms, which are added behind) every tile is split
    for (int all = stack; all <= (stack || (rounds > 0 && rounds < 4)); ++all) {
      p.whole = all ? 0 : (int)(rounds * kPairs);
      const long long cut = tiles - p.whole;
      for (int s = 1; s <= kMaxSplits && s <= blocks; ++s) {
        p.per = ceil_div(blocks, s);
        if (ceil_div(blocks, p.per) != s) continue;  // no split is empty
        if (s > 1 && (cut == 0 || cut * s > 8 * kPairs)) break;
        double t = (double)(p.whole / kPairs) * (blocks * block + 3);
        t += (double)((cut * s + kPairs - 1) / kPairs) * (p.per * block + 3);
        if (s > 1 || stack) t += 10 + 8.0 * cut * s * (M < kDenseM ? M : kDenseM) * bn / 1.8e6;
        if (best.cost == 0 || t < 0.98 * best.cost) {
          best = p;
          best.splits = s;
          best.cost = t;
        }
      }
    }
  }
  return best;
}

// How a forward of few rows goes: tiles of 128 outputs, each shared by a cluster.  Counted in blocks of
// an SM's share: the memory's pace (what the busiest SM would have if all had the same), or what the
// busiest SM has at the pace of one SM, 1.4 times its share of the memory's (112 SMs reach 6.2 TB/s);
// 3 for a round of CTAs, 1 for each that an SM holds at once, 2 for sums through a cluster.  Measured, one
// row x 4096 x 14336 gated: 112 CTAs alone 38 us, 224 in pairs 39, 448 in fours 42 to 55, in eights 71;
// 17 x 14336 x 4096: 32 CTAs 58, 64 in pairs 32, 128 in fours 23, 256 in eights 22.  At 64 rows x 4096 x
// 14336 27 us, with the other kernel 65 rows take 27.5.
constexpr int kMaxCluster = 8;
// CTAs that a GB300 holds at once, 1 to 4 on an SM, in clusters of 1, 2, 4 and 8
// (cudaOccupancyMaxActiveClusters): clusters do not fill every group of SMs.
constexpr int kFewSlots[4][4] = {
    {152, 152, 144, 120}, {304, 304, 296, 288}, {456, 456, 440, 408}, {608, 608, 592, 592}};
struct Few {
  int split = 0, per, stages, stage, smem, tmem, cols;
};
Few plan_few(int M, int N, int K, bool gated) {
  Few best;
  const int nk = ceil_div(K, kDenseK), tiles = ceil_div(N, 128);
  Few f;
  f.cols = (int)up(M, 16);
  f.stage = (gated ? 2 : 1) * 128 * kDenseK * 2 + f.cols * 128;
  f.tmem = 32;
  while (f.tmem < (gated ? 2 : 1) * f.cols) f.tmem *= 2;
  const int sums = (gated ? 2 : 1) * f.cols * 512;
  double least = 0;
  for (int i = 0; 1 << i <= kMaxCluster && 1 << i <= nk; ++i) {
    f.split = 1 << i;
    f.per = ceil_div(nk, f.split);
    if (ceil_div(nk, f.per) != f.split) continue;  // every CTA has a part
    const long long ctas = (long long)tiles * f.split;
    for (int at_once = 1; at_once <= 4 && at_once * f.tmem <= 512; ++at_once) {
      const int room = 224 * 1024 / at_once - 1536;
      f.stages = room / f.stage < kFewStages ? room / f.stage : kFewStages;
      f.smem = f.stages * f.stage > sums ? f.stages * f.stage : sums;
      if (f.stages < 2 || f.smem > room) break;
      const long long rounds = (ctas + kFewSlots[at_once - 1][i] - 1) / kFewSlots[at_once - 1][i];
      const double all = (double)tiles * nk / kFewSlots[0][0], one = rounds * at_once * f.per / 1.4;
      const double t = (all > one ? all : one) + 3.0 * rounds + at_once + (i > 0 ? 2 : 0);
      if (least == 0 || t < least) least = t, best = f;
    }
  }
  return best;
}

bool sizes_ok(const Product &p) { return p.per > 0; }

struct Arena {
  char *base;
  size_t off = kStatusBytes;
  explicit Arena(void *ws) : base(static_cast<char *>(ws)) {}
  void *take(size_t bytes) {
    void *p = bytes ? base + off : nullptr;
    off += align256(bytes);
    return p;
  }
};

// Copies that wait for their launch.
struct Copies {
  DenseCopies list{};
  bool out;
  explicit Copies(bool out) : out(out) {}
  void add(const void *in, long long is, void *to, long long os, int rows, int cols) {
    list.c[list.count++] = {in, to, is, os, rows, cols};
  }
  bool run(cudaStream_t s) const {
    return list.count == 0 || launch_dense_copies(list, out, s) == cudaSuccess;
  }
};

// Gives an operand that TMA cannot read where it lies a place in the workspace.
void place(Rows &r, Arena &arena, Copies &copies) {
  if (!r.pad) return;
  const long long stride = up(r.cols, 8);
  void *to = arena.take(r.bytes());
  copies.add(r.at, r.stride, to, stride, r.rows, r.cols);
  r = Rows(to, stride, r.rows, r.cols);
}

// An output that does not lie on 16 bytes is formed in the workspace and copied to its place.
struct Out {
  void *to = nullptr, *at = nullptr;
  long long to_stride = 0, stride = 0;
  int rows = 0, cols = 0;
  Out() = default;
  Out(void *p, long long s, int rows, int cols)
      : to(p), at(p), to_stride(s), stride(rows > 1 ? s : up(cols, 8)), rows(rows), cols(cols) {}
  bool pad() const { return to && (!aligned16(to) || stride % 8); }
  size_t bytes() const { return pad() ? align256((size_t)rows * up(cols, 8) * 2) : 0; }
  void place(Arena &arena) {
    if (!pad()) return;
    const size_t n = bytes();
    stride = up(cols, 8);
    at = arena.take(n);
  }
  void finish(Copies &copies) const {
    if (at != to) copies.add(at, stride, to, to_stride, rows, cols);
  }
};

// The limit of a wait.  A kernel's first CTA clears the status word that a wait which runs out sets: a
// millisecond at least lies between.
unsigned long long wait_limit_ns() {
  const unsigned long long ns = g_wait_ns.load();
  return ns > 1000000ull ? ns : 1000000ull;
}

// Launches a product of rows a[0..1], b[0..1] (the second ones where `pairs`, a second output or a gate
// ask for them, otherwise empty).
dash_status_t launch(const Product &p, const Rows (&a)[2], const Rows (&b)[2], bool a_mn, bool b_mn,
                     bool a_out, bool b_out, bool pairs, int a_low, int b_low,
                     const DenseEpilogue &e, void *y1, long long y1s, float *part, void *workspace,
                     bool clear, bool f16, int sms, cudaStream_t s, uint32_t *special = nullptr) {
  CUtensorMap ta[2], tb[2];
  for (int i = 0; i < 2; ++i)
    if (!make_rows_map(&ta[i], a[i].at ? a[i] : a[0], a_mn ? 64 : 128, f16) ||
        !make_rows_map(&tb[i], b[i].at ? b[i] : b[0], b_mn ? 64 : p.bn / 2, f16))
      return DASH_ERR_CUDA;
  DenseParams d{};
  d.e = e;
  d.y1 = y1, d.y1s = y1s;
  d.part = part;
  d.status = static_cast<uint32_t *>(workspace);
  d.special = special;
  d.clear = clear;
  d.wait_ns = wait_limit_ns();
  d.M = p.M, d.N = p.N;
  d.mt = p.mt(), d.nt = p.nt(), d.bn = p.bn;
  // 16 rows of tiles while A's part of them stays in L2 beside the rest (8192 x 4096 x 14336 567 -> 556 us
  // under the power limit; 4 and 32 rows 590), otherwise 8
  d.group = 16LL * kDenseM * p.K * p.parts * 2 <= (36LL << 20) ? 16 : 8;
  d.nk = p.nk(), d.parts = p.parts, d.outs = p.outs;
  d.whole = p.whole, d.splits = p.splits, d.per = p.per;
  d.a_mn = a_mn, d.b_mn = b_mn, d.a_out = a_out, d.b_out = b_out;
  d.pairs = pairs, d.stack = p.stack, d.a_low = a_low, d.b_low = b_low;
  d.withhold = g_dense_withhold.load();
  return launch_dense(f16, ta, tb, d, sms, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

// ------------------------------------------------------------------ forward
struct Fwd {
  Product p;
  Few few;
  Rows x, w[2], res;
  Out y;
  size_t need;
};
dash_status_t check_fwd(const dash_dense_fwd_t *a, Fwd &f) {
  if (!a || !a->x || !a->w || !a->y || a->M <= 0 || a->K <= 0 || a->N <= 0) return DASH_ERR_INVALID;
  if (a->order != DASH_DENSE_KN && a->order != DASH_DENSE_NK) return DASH_ERR_INVALID;
  if (a->act < DASH_ACT_NONE || a->act > DASH_ACT_SILU) return DASH_ERR_INVALID;
  if (a->dtype != DASH_BF16 && a->dtype != DASH_FP16)
    return a->dtype == DASH_FP32 ? DASH_ERR_UNSUPPORTED : DASH_ERR_INVALID;
  const void *all[] = {a->x, a->w, a->w_gate, a->bias, a->bias_gate, a->residual, a->y};
  for (const void *t : all)
    if (!aligned2(t)) return DASH_ERR_INVALID;
  if (!aligned16(a->z) || !aligned16(a->gate)) return DASH_ERR_INVALID;
  if ((a->bias_gate || a->gate) && !a->w_gate) return DASH_ERR_INVALID;
  if (a->M > 1 && a->y_stride < a->N) return DASH_ERR_INVALID;
  const bool kn = a->order == DASH_DENSE_KN;
  if (a->M > kMaxSize || a->K > kMaxSize || a->N > kMaxSize) return DASH_ERR_UNSUPPORTED;
  const bool gated = a->w_gate != nullptr;
  f.p = Product{a->M, a->N, a->K, 1, 1, gated};
  if (a->M <= kFewRows) {
    f.few = plan_few(a->M, a->N, a->K, gated);
  } else {
    f.p = plan(a->M, a->N, a->K, 1, 1, gated);
    if (!sizes_ok(f.p)) return DASH_ERR_UNSUPPORTED;
  }
  f.x = Rows(a->x, a->x_stride, a->M, a->K);
  f.w[0] = Rows(a->w, a->w_stride, kn ? a->K : a->N, kn ? a->N : a->K);
  f.w[1] = Rows(a->w_gate, a->w_gate_stride, f.w[0].rows, f.w[0].cols);
  f.res = Rows(a->residual, a->residual_stride, a->M, a->N);
  f.y = Out(a->y, a->y_stride, a->M, a->N);
  f.need = kStatusBytes + f.x.bytes() + f.w[0].bytes() + f.w[1].bytes();
  if (!f.few.split)  // (few rows need no more room)
    f.need += f.p.part_bytes() + f.res.bytes() + f.y.bytes();
  return DASH_OK;
}

// ------------------------------------------------------------------ backward
// dz is rounded for the tensor core, which is off by as much as the rounding of dx and dw: 1.4 times that
// in all.  Of few elements it may come out well above that, and what the rounding lost is multiplied as
// well there, unless the caller says otherwise (it doubles the products: 8192 x 4096 x 4096 345 us, 591 with
// it).
constexpr long long kTwoTerms = 1 << 16;  // elements of dz
// dx: a second term is another part of the contraction, or, of up to 128 rows, takes the tile's other half,
// which is empty: every block of the weights is read and multiplied once for both (8 x 8192 x 8192 46 us,
// without a second term 44, as another part 60).  That writes all tiles' sums to the workspace (no more of
// them than a split would), so short contractions go the other way (128 x 4096 x 512 22 us, stacked 25).
Product plan_dx(int M, int N, int K, int parts, int terms) {
  const Product p = plan(M, N, K, parts * terms, 1, false);
  if (terms == 1 || M > kDenseM / 2 || ceil_div(N, 256) > 8 * kPairs) return p;
  const Product q = plan(M, N, K, parts, 1, false, true);
  return q.per > 0 && q.cost < p.cost ? q : p;
}
struct Bwd {
  Product dx, dw;
  int terms;
  Rows dy, x, w[2];
  Out out[3];          // dx, dw, dw_gate
  bool grads, pad_dy;  // dz (and dgate) are formed; dy is copied
  int chunks, chunk;
  size_t dz_bytes, sum_bytes, part_bytes, need;
  size_t special_bytes() const { return terms == 2 ? kStatusBytes : 0; }
};
dash_status_t check_bwd(const dash_dense_bwd_t *a, int terms, Bwd &b) {
  if (terms < 0 || terms > 2) return DASH_ERR_INVALID;
  if (!a || !a->dy || a->M < 0 || a->K <= 0 || a->N <= 0) return DASH_ERR_INVALID;
  if (a->order != DASH_DENSE_KN && a->order != DASH_DENSE_NK) return DASH_ERR_INVALID;
  if (a->act < DASH_ACT_NONE || a->act > DASH_ACT_SILU) return DASH_ERR_INVALID;
  if (a->dtype != DASH_BF16 && a->dtype != DASH_FP16)
    return a->dtype == DASH_FP32 ? DASH_ERR_UNSUPPORTED : DASH_ERR_INVALID;
  const void *all[] = {a->dy, a->x, a->w, a->w_gate, a->dx, a->dw, a->dw_gate, a->dbias,
                       a->dbias_gate};
  for (const void *t : all)
    if (!aligned2(t)) return DASH_ERR_INVALID;
  if (!aligned16(a->z) || !aligned16(a->gate)) return DASH_ERR_INVALID;
  const bool kn = a->order == DASH_DENSE_KN, gated = a->gate != nullptr;
  b.grads = a->act != DASH_ACT_NONE || gated;
  if (b.grads && !a->z) return DASH_ERR_INVALID;
  if ((a->dx && !a->w) || (a->dw && !a->x)) return DASH_ERR_INVALID;
  if (gated ? (a->dx && !a->w_gate) || !a->dw != !a->dw_gate : a->dw_gate || a->dbias_gate)
    return DASH_ERR_INVALID;
  const int wr = kn ? a->K : a->N, wc = kn ? a->N : a->K;
  if ((a->dx && a->M > 1 && a->dx_stride < a->K) ||
      (a->dw && wr > 1 && (a->dw_stride < wc || (gated && a->dw_gate_stride < wc))))
    return DASH_ERR_INVALID;
  b.dy = Rows(a->dy, a->dy_stride, a->M, a->N);
  b.x = Rows(a->dw ? a->x : nullptr, a->x_stride, a->M, a->K);
  b.w[0] = Rows(a->dx ? a->w : nullptr, a->w_stride, wr, wc);
  b.w[1] = Rows(a->dx && gated ? a->w_gate : nullptr, a->w_gate_stride, wr, wc);
  if (a->M > kMaxSize || a->K > kMaxSize || a->N > kMaxSize) return DASH_ERR_UNSUPPORTED;
  const int M = a->M ? a->M : 1;
  b.terms = !b.grads ? 1 : terms ? terms : (long long)M * a->N <= kTwoTerms ? 2 : 1;
  if (b.terms == 2 && M > kMaxSize / 2) return DASH_ERR_UNSUPPORTED;
  b.dx = plan_dx(M, a->K, a->N, gated ? 2 : 1, b.terms);
  b.dw = kn ? plan(a->K, a->N, M, b.terms, gated ? 2 : 1, false)
            : plan(a->N, a->K, M, b.terms, gated ? 2 : 1, false);
  if (!sizes_ok(b.dx) || !sizes_ok(b.dw)) return DASH_ERR_UNSUPPORTED;
  // rows of a chunk: four rounds of CTAs or so, 32 rows at least
  const int strips = ceil_div(a->N, 256);
  b.chunk = ceil_div(M, ceil_div(4 * 4 * 152, strips));
  b.chunk = (int)up(b.chunk < 32 ? 32 : b.chunk, 8);
  b.chunks = ceil_div(M, b.chunk);
  b.dz_bytes = b.grads && (a->dx || a->dw) ? align256((size_t)b.terms * M * up(a->N, 8) * 2) : 0;
  b.sum_bytes = align256((size_t)b.chunks * a->N * 4);
  b.part_bytes = 0;
  if (a->dx) b.part_bytes = b.dx.part_bytes();
  if (a->dw && b.dw.part_bytes() > b.part_bytes) b.part_bytes = b.dw.part_bytes();
  b.pad_dy = !b.grads && (a->dx || a->dw) && b.dy.pad;
  b.out[0] = Out(a->dx, a->dx_stride, a->M, a->K);
  b.out[1] = Out(a->dw, a->dw_stride, wr, wc);
  b.out[2] = Out(a->dw_gate, a->dw_gate_stride, wr, wc);
  b.need = kStatusBytes + b.out[0].bytes() + b.out[1].bytes() + b.out[2].bytes() +
           (gated ? 2 : 1) * b.dz_bytes + (a->dbias ? b.sum_bytes : 0) +
           (a->dbias_gate ? b.sum_bytes : 0) + b.special_bytes() + b.part_bytes + (b.pad_dy ? b.dy.bytes() : 0) +
           b.x.bytes() + b.w[0].bytes() + b.w[1].bytes();
  return DASH_OK;
}

}  // namespace
}  // namespace dash

extern "C" {

dash_status_t dash_dense_withhold(int block) {
  dash::g_dense_withhold.store(block < 0 ? -1 : block);
  return DASH_OK;
}

size_t dash_dense_fwd_workspace_bytes(const dash_dense_fwd_t *args) {
  dash::Fwd f;
  return dash::check_fwd(args, f) == DASH_OK ? f.need : 0;
}

dash_status_t dash_dense_fwd(const dash_dense_fwd_t *a, void *workspace, size_t workspace_bytes,
                             dash_stream_t stream) {
  using namespace dash;
  Fwd f;
  dash_status_t st = check_fwd(a, f);
  if (st != DASH_OK) return st;
  if (!workspace || !aligned16(workspace) || workspace_bytes < f.need) return DASH_ERR_WORKSPACE;
  const Rows y(a->y, a->y_stride, a->M, a->N);
  const long long kept = 3LL * a->M * kept_stride(a->N);
  const Bytes outs[] = {y.lies(), bytes_of(a->z, 1, kept), bytes_of(a->gate, 1, kept),
                        bytes_of(workspace, 1, (long long)f.need)};
  const Bytes reads[] = {f.x.lies(), f.w[0].lies(), f.w[1].lies(), bytes_of(a->bias, 2, a->N),
                         bytes_of(a->bias_gate, 2, a->N)};
  if (!apart(outs, reads)) return DASH_ERR_INVALID;
  const bool in_place = a->y == a->residual && (a->M == 1 || a->y_stride == a->residual_stride);
  for (int i = in_place ? 1 : 0; i < 4; ++i)
    if (share(outs[i], f.res.lies())) return DASH_ERR_INVALID;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  const bool f16 = a->dtype == DASH_FP16, kn = a->order == DASH_DENSE_KN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Arena arena(workspace);
  Copies in(false), out(true);
  for (Rows *r : {&f.x, &f.w[0], &f.w[1]}) place(*r, arena, in);
  DenseEpilogue e{};
  e.bias = a->bias, e.bias_gate = a->bias_gate;
  e.act = a->act, e.gated = f.p.gated;
  e.z = kept_at(a->z, a->M, a->N), e.g = kept_at(a->gate, a->M, a->N);
  e.ks = kept_stride(a->N);
  if (f.few.split) {
    if (!in.run(s)) return DASH_ERR_CUDA;
    e.y = a->y, e.residual = a->residual;
    e.ys = a->y_stride, e.rs = a->residual_stride;
    CUtensorMap tw[2], tx;
    for (int i = 0; i < 2; ++i)
      if (!make_rows_map(&tw[i], f.w[i].at ? f.w[i] : f.w[0], kn ? 64 : 128, f16))
        return DASH_ERR_CUDA;
    if (!make_rows_map(&tx, f.x, f.few.cols, f16)) return DASH_ERR_CUDA;
    DenseFewParams d{};
    d.e = e;
    d.status = static_cast<uint32_t *>(workspace);
    d.wait_ns = wait_limit_ns();
    d.M = f.p.M, d.N = f.p.N, d.nk = f.p.nk();
    d.cols = f.few.cols, d.split = f.few.split, d.per = f.few.per;
    d.stages = f.few.stages, d.stage = f.few.stage, d.smem = f.few.smem, d.tmem = f.few.tmem;
    d.w_mn = kn;
    d.withhold = g_dense_withhold.load();
    return launch_dense_few(f16, tw[0], tw[1], tx, d, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  }
  float *part = static_cast<float *>(arena.take(f.p.part_bytes()));
  place(f.res, arena, in);
  f.y.place(arena);
  if (!in.run(s)) return DASH_ERR_CUDA;
  e.y = f.y.at, e.residual = f.res.at;
  e.ys = f.y.stride, e.rs = f.res.stride;
  const Rows x[2] = {f.x, Rows()};
  st = launch(f.p, x, f.w, false, kn, false, false, false, 0, 0, e, nullptr, 0, part, workspace, true,
              f16, dev.sms, s);
  if (st != DASH_OK) return st;
  f.y.finish(out);
  return out.run(s) ? DASH_OK : DASH_ERR_CUDA;
}

size_t dash_dense_bwd_workspace_bytes(const dash_dense_bwd_t *args) {
  return dash_dense_bwd_terms_workspace_bytes(args, 0);
}

dash_status_t dash_dense_bwd(const dash_dense_bwd_t *args, void *workspace, size_t workspace_bytes,
                             dash_stream_t stream) {
  return dash_dense_bwd_terms(args, 0, workspace, workspace_bytes, stream);
}

size_t dash_dense_bwd_terms_workspace_bytes(const dash_dense_bwd_t *args, int terms) {
  dash::Bwd b;
  return dash::check_bwd(args, terms, b) == DASH_OK ? b.need : 0;
}

dash_status_t dash_dense_bwd_terms(const dash_dense_bwd_t *a, int terms, void *workspace,
                                   size_t workspace_bytes, dash_stream_t stream) {
  using namespace dash;
  Bwd b;
  dash_status_t st = check_bwd(a, terms, b);
  if (st != DASH_OK) return st;
  if (!workspace || !aligned16(workspace) || workspace_bytes < b.need) return DASH_ERR_WORKSPACE;
  const bool kn = a->order == DASH_DENSE_KN, gated = a->gate != nullptr,
             f16 = a->dtype == DASH_FP16;
  const int wr = kn ? a->K : a->N, wc = kn ? a->N : a->K;
  const long long kept = 3LL * a->M * kept_stride(a->N);
  const Rows dw(a->dw, a->dw_stride, wr, wc), dwg(a->dw_gate, a->dw_gate_stride, wr, wc);
  const Bytes outs[] = {Rows(a->dx, a->dx_stride, a->M, a->K).lies(), dw.lies(), dwg.lies(),
                        bytes_of(a->dbias, 2, a->N), bytes_of(a->dbias_gate, 2, a->N),
                        bytes_of(workspace, 1, (long long)b.need)};
  const Bytes reads[] = {b.dy.lies(), Rows(a->x, a->x_stride, a->M, a->K).lies(),
                         Rows(a->w, a->w_stride, wr, wc).lies(),
                         Rows(a->w_gate, a->w_gate_stride, wr, wc).lies(),
                         bytes_of(a->z, 1, kept), bytes_of(a->gate, 1, kept)};
  if (!apart(outs, reads)) return DASH_ERR_INVALID;
  DevInfo dev;
  if ((st = device_info(&dev)) != DASH_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a->M == 0) {
    const Rows *const w[2] = {&dw, &dwg};
    for (const Rows *r : w)
      if (r->at && cudaMemset2DAsync(const_cast<void *>(r->at), r->stride * 2, 0, (size_t)wc * 2,
                                     wr, s) != cudaSuccess)
        return DASH_ERR_CUDA;
    for (void *d : {a->dbias, a->dbias_gate})
      if (d && cudaMemsetAsync(d, 0, (size_t)a->N * 2, s) != cudaSuccess) return DASH_ERR_CUDA;
    return cudaMemsetAsync(workspace, 0, kStatusBytes, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  }
  Arena arena(workspace);
  Rows dz[2] = {b.dy, Rows()};
  void *dz_at = arena.take(b.dz_bytes), *dg_at = gated ? arena.take(b.dz_bytes) : nullptr;
  float *sum = static_cast<float *>(arena.take(a->dbias ? b.sum_bytes : 0));
  float *sum_gate = static_cast<float *>(arena.take(a->dbias_gate ? b.sum_bytes : 0));
  uint32_t *special = static_cast<uint32_t *>(arena.take(b.special_bytes()));
  float *part = static_cast<float *>(arena.take(b.part_bytes));
  if (b.grads || a->dbias) {
    DenseGradParams g{};
    g.dy = a->dy;
    if (b.grads)
      g.z = kept_at(const_cast<void *>(a->z), a->M, a->N),
      g.g = kept_at(const_cast<void *>(a->gate), a->M, a->N);
    g.dz = dz_at, g.dg = dg_at;
    g.low = b.terms == 2;
    g.special = special;
    g.part = sum, g.part_gate = sum_gate;
    g.dys = b.dy.stride, g.ks = kept_stride(a->N), g.ds = up(a->N, 8);
    g.M = a->M, g.N = a->N, g.act = a->act, g.chunk = b.chunk;
    g.vec = aligned16(a->dy) && b.dy.stride % 8 == 0;
    if (launch_dense_grad(f16, g, b.chunks, s) != cudaSuccess) return DASH_ERR_CUDA;
    if ((sum || sum_gate) && launch_dense_sums(f16, sum, sum_gate, a->dbias, a->dbias_gate,
                                               b.chunks, a->N, s) != cudaSuccess)
      return DASH_ERR_CUDA;
    if (b.grads) {
      dz[0] = Rows(dz_at, g.ds, b.terms * a->M, a->N);
      dz[1] = Rows(dg_at, g.ds, b.terms * a->M, a->N);
    }
  }
  if (!a->dx && !a->dw)  // no product clears the status block
    return cudaMemsetAsync(workspace, 0, kStatusBytes, s) == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  Copies in(false), out(true);
  for (Rows *r : {&dz[0], &b.x, &b.w[0], &b.w[1]}) place(*r, arena, in);
  if (!in.run(s)) return DASH_ERR_CUDA;
  for (Out &o : b.out) o.place(arena);
  const int low = b.terms == 2 ? a->M : 0;  // (rows of x behind the last are zeros there)
  if (a->dx) {
    DenseEpilogue e{};
    e.y = b.out[0].at, e.ys = b.out[0].stride;
    st = launch(b.dx, dz, b.w, false, !kn, false, false, gated, low, 0, e, nullptr, 0, part,
                workspace, true, f16, dev.sms, s, b.dx.stack ? nullptr : special);
    if (st != DASH_OK) return st;
  }
  if (a->dw) {
    DenseEpilogue e{};
    e.y = b.out[1].at, e.ys = b.out[1].stride;
    const Rows x[2] = {b.x, Rows()};
    st = kn ? launch(b.dw, x, dz, true, true, false, gated, false, 0, low, e, b.out[2].at,
                     b.out[2].stride, part, workspace, !a->dx, f16, dev.sms, s, special)
            : launch(b.dw, dz, x, true, true, gated, false, false, low, 0, e, b.out[2].at,
                     b.out[2].stride, part, workspace, !a->dx, f16, dev.sms, s, special);
    if (st != DASH_OK) return st;
  }
  if (special && (a->dw || !b.dx.stack)) {
    DenseSpecials sp{};
    sp.set = special;
    auto along_row = [](const Rows &r) { return DenseOperand{r.at, r.stride, 1}; };
    auto along_column = [](const Rows &r) { return DenseOperand{r.at, 1, r.stride}; };
    if (a->dx && !b.dx.stack) {
      DenseSpecial &q = sp.s[0];
      q = {b.out[0].at, b.out[0].stride, a->M, a->K, a->N, gated ? 2 : 1};
      for (int i = 0; i < q.parts; ++i) {
        q.a[i] = along_row(dz[i]);
        q.b[i] = kn ? along_row(b.w[i]) : along_column(b.w[i]);
      }
    }
    for (int i = 0; a->dw && i <= (int)gated; ++i) {
      DenseSpecial &q = sp.s[1 + i];
      q = {b.out[1 + i].at, b.out[1 + i].stride, wr, wc, a->M, 1};
      q.a[0] = along_column(kn ? b.x : dz[i]);
      q.b[0] = along_column(kn ? dz[i] : b.x);
    }
    if (launch_dense_specials(f16, sp, s) != cudaSuccess) return DASH_ERR_CUDA;
  }
  for (const Out &o : b.out) o.finish(out);
  return out.run(s) ? DASH_OK : DASH_ERR_CUDA;
}

}  // extern "C"
