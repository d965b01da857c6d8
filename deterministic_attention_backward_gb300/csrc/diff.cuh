// diff.cuh -- differential attention: parameters, launch interface and the small device
// helpers its kernels share.
//
//   O = P1 V - lam P2 V,   Pm = softmax(c Qm Km^T + mask)
// Head pair h holds the query maps 2h and 2h+1 (d elements each, neighbours in memory), the key
// maps of its KV head likewise, and a value head of dv = 2d: every operand is a [B, S, heads,
// 2d] tensor of the plain attention, so the same TMA boxes bring it in, and map m is columns
// [m d, (m+1) d) of a Q or K tile.
#pragma once
#include "common.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"

namespace dash {

struct DiffFwdParams {
  __nv_bfloat16 *o, *o2;  // [B,S,H,2d]
  __nv_bfloat16 *rest;    // [2,B,S,H,2d], what o and o2 lose by their rounding (may be null)
  float *lse;             // [B,2H,S]
  const void *lam;        // [H] or [B,S,H], bf16 or fp32
  uint32_t *status;
  uint32_t *taken;        // tiles that CTAs have taken beside their first (cleared)
  int B, S, H, Hkv, G, N, causal;
  int lam_f32, lam_token;
  int withhold;           // block at which a CTA's loads end (dash_diff_withhold), else -1
  unsigned long long wait_ns;
  float scale_log2;       // softmax scale * log2(e)
};

// Row vectors of the backward, per half tile (64 rows) of a (batch, head pair) kRowVecs arrays
// of 64 floats, each negated for the fused multiply-adds that take them:
//   -LSE1 log2e, -LSE2 log2e, -D1, -D2, -lam       (Dm = dO . Om)
// Rows past S hold -inf, -inf, 0, 0, 0, which give them no weight.
constexpr int kRowVecs = 5;
// Where vector 0 of row r of `tile` lies; vector k follows 64 k further on.
__host__ __device__ __forceinline__ size_t rowv_at(size_t tile, int r) {
  return (tile * 2 + (r >> 6)) * (kRowVecs * 64) + (r & 63);
}
struct DiffBwdParams {
  const __nv_bfloat16 *o, *o2, *dout;
  const __nv_bfloat16 *rest;  // the forward's, may be null
  const float *lse;
  const void *lam;
  float *rowv;            // [B,H,N][2][kRowVecs][64]
  float *dlam_part;       // [B,H,N] (weights per head only)
  uint32_t *status;
  __nv_bfloat16 *dq, *dk, *dv;
  void *dlam;             // [H] or [B,S,H], lam's type
  int B, S, H, Hkv, G, N, causal;
  int lam_f32, lam_token;
  int withhold_dq, withhold_dkv;  // as in the forward
  unsigned long long wait_ns;
  float scale_log2, scale;
  // dK/dV's kernel: the first kv_whole tiles are a CTA each, the others kv_pieces CTAs each,
  // whose fp32 sums [piece][4d/4][128][4] of kv_part diff_join_kernel adds
  int kv_whole, kv_pieces;
  float *kv_part;
};

cudaError_t launch_diff_fwd(int d, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const DiffFwdParams &p, int sms,
                            cudaStream_t s);
cudaError_t launch_diff_bwd(int d, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tdo,
                            const DiffBwdParams &p, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ float lam_at(const void *lam, int f32, size_t at) {
  return f32 ? static_cast<const float *>(lam)[at]
             : __bfloat162float(static_cast<const __nv_bfloat16 *>(lam)[at]);
}

// mbar_wait_warp without a read of the global timer on the way of a wait that is short: the
// read takes longer than most of these waits last.  The limit runs from the first look at the
// timer, after 256 tries.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, const Abort &ab) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
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

// tcgen05.wait::ld that the loaded registers depend on, so that no use moves above it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// 16 lanes x 16 columns as matrix fragments: thread t holds of 8-column group g, in r[4g..4g+3],
// columns 8g + 2 (t % 4) and the next one of lanes t / 4 and t / 4 + 8.  Four rows and four
// columns a thread over the warp's 32 lanes (two such loads), so that what goes by column is
// read once for four rows.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr));
}
// The fragments' pairs rounded to bf16: 16 lanes x 8 columns of two values each; v[2g] the
// pair of group g of lane t / 4, v[2g+1] of lane t / 4 + 8.
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ f2 ex2_2(f2 v) {
  float a, b;
  f2_to(v, a, b);
  return f2_of(ex2_approx(a), ex2_approx(b));
}
__device__ __forceinline__ uint32_t pack_bf16(f2 v) {
  float a, b;
  f2_to(v, a, b);
  return pack_bf16(a, b);
}

// tcgen05.mma and commit for a converged warp whose lane with `lead` set issues (elect_one(),
// asked once: electing anew for every instruction costs a third of the issue rate; measured
// 12.6 against 21 cycles an instruction, 18 against 32 beside busy warps).
__device__ __forceinline__ void mma_ss_l(uint32_t lead, uint32_t d_tmem, uint64_t adesc,
                                         uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts_l(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem,
                                         uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred e, p;\n\t"
      "setp.ne.b32 e, %5, 0;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit_l(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "setp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::
          "r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// Byte offset of element column `col` (a multiple of 16) of row 0 in a [128 x 2d] operand tile
// of 64-column boxes.
__device__ __forceinline__ constexpr uint32_t col_bytes(int col) {
  return (uint32_t)(col >> 6) * kBoxBytes + (uint32_t)(col & 63) * 2;
}

// What an fp32 value loses when it is rounded to bf16.
__device__ __forceinline__ uint32_t rest_of(uint32_t v) {
  const float x = __uint_as_float(v);
  return __float_as_uint(x - __bfloat162float(__float2bfloat16_rn(x)));
}

// C fp32 columns of this thread's row, scaled, as C bf16 at dst (16-byte aligned).
template <int C>
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const uint32_t (&v)[C],
                                          float scale) {
  uint32_t pk[C / 2];
#pragma unroll
  for (int i = 0; i < C / 2; ++i)
    pk[i] = pack_bf16(__uint_as_float(v[2 * i]) * scale, __uint_as_float(v[2 * i + 1]) * scale);
  uint4 *d4 = reinterpret_cast<uint4 *>(dst);
#pragma unroll
  for (int i = 0; i < C / 8; ++i)
    d4[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
}
#endif

}  // namespace dash
