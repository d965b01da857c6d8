// diff_bwd.cu -- differential attention backward, deterministic without any ordering between
// CTAs: one kernel stationary in queries accumulates dQ, one stationary in keys accumulates
// dK and dV, each on chip in the order of its own loop.
//
// With dP = dO V^T (both maps share it), Dm = dO . Om, and ~ for the rounding to bf16 that the
// tensor core asks for:
//   dS1 = P1 (dP - D1)       dS2 = -lam P2 (dP - D2)        dlam_i = - sum_j P2 dP
//   dQm = c ~dSm Km          dKm = c ~dSm^T Qm              dV = ~(P1 - lam P2)^T dO
// Two passes form S1, S2, dP and both maps' exponentials twice (512 of then 1792 flops a pair at
// d = 64), so that no sum leaves the chip and nothing waits for another CTA.  One pass would be
// stationary in keys and add 64 KB of fp32 dQ partials a tile pair in global memory in a fixed
// order, as this library's main backward does at D = 128 with the same products: that reaches 1216
// TFLOP/s full and 937 to 975 causal at 8192, these two 959 and 872 of the same useful flops.  So
// one pass is the faster form as far as products and partials go; the two exponentials a pair in
// place of its one have not been weighed.
#include "diff.cuh"

#include "dash_attn.h"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kStatusWords = kStatusBytes / 4;
constexpr int kWarps = 16;                   // warps of elementwise work: four warpgroups
constexpr int kThreads = (kWarps + 2) * 32;  // and the TMA producer, the MMA issuer

// -------------------------------------------------------------------- row vectors
// One CTA per tile of a (batch, head pair); DV / 8 lanes per row.  Bound by memory: 8 sequences of
// 2048, 32 heads of 128, 66 us for 403 MB, 6.1 TB/s.  kRest: with what the outputs lost by
// rounding, 17 us more at 8192 tokens of 32 heads.
template <int d, bool kRest>
__global__ void __launch_bounds__(256) diff_rows_kernel(const DiffBwdParams p) {
  constexpr int DV = 2 * d, kLanes = DV / 8, kRows = 256 / kLanes;
  __shared__ float s_d[2][kTile];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int tile = blockIdx.x, i = tile % p.N, h = (tile / p.N) % p.H, b = tile / p.N / p.H;
  if (tile == 0 && threadIdx.x < kStatusWords) p.status[threadIdx.x] = 0;  // for what follows
#pragma unroll 4
  for (int r = sub; r < kTile; r += kRows) {
    const int row = i * kTile + r;
    float d1 = 0.f, d2 = 0.f;
    if (row < p.S) {
      const size_t off = (((size_t)b * p.S + row) * p.H + h) * DV + lane * 8;
      const uint4 g = *reinterpret_cast<const uint4 *>(p.dout + off);
      const uint4 x = *reinterpret_cast<const uint4 *>(p.o + off);
      const uint4 y = *reinterpret_cast<const uint4 *>(p.o2 + off);
      const __nv_bfloat162 *g2 = reinterpret_cast<const __nv_bfloat162 *>(&g);
      const __nv_bfloat162 *x2 = reinterpret_cast<const __nv_bfloat162 *>(&x);
      const __nv_bfloat162 *y2 = reinterpret_cast<const __nv_bfloat162 *>(&y);
      uint4 xr, yr;
      if constexpr (kRest) {
        xr = *reinterpret_cast<const uint4 *>(p.rest + off);
        yr = *reinterpret_cast<const uint4 *>(p.rest + (size_t)p.B * p.S * p.H * DV + off);
      }
      const __nv_bfloat162 *xr2 = reinterpret_cast<const __nv_bfloat162 *>(&xr);
      const __nv_bfloat162 *yr2 = reinterpret_cast<const __nv_bfloat162 *>(&yr);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = __bfloat1622float2(g2[e]);
        float2 u = __bfloat1622float2(x2[e]), w = __bfloat1622float2(y2[e]);
        if constexpr (kRest) {
          const float2 ur = __bfloat1622float2(xr2[e]), wr = __bfloat1622float2(yr2[e]);
          u.x += ur.x, u.y += ur.y, w.x += wr.x, w.y += wr.y;
        }
        d1 = fmaf(a.x, u.x, fmaf(a.y, u.y, d1));
        d2 = fmaf(a.x, w.x, fmaf(a.y, w.y, d2));
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      d1 += __shfl_xor_sync(0xffffffffu, d1, o);
      d2 += __shfl_xor_sync(0xffffffffu, d2, o);
    }
    if (lane == 0) s_d[0][r] = d1, s_d[1][r] = d2;
  }
  __syncthreads();
  const int r = threadIdx.x;
  if (r >= kTile) return;
  const int row = i * kTile + r;
  float v[kRowVecs] = {-INFINITY, -INFINITY, 0.f, 0.f, 0.f};
  if (row < p.S) {
    const size_t at = ((size_t)b * p.S + row) * p.H + h;
    const float lam = lam_at(p.lam, p.lam_f32, p.lam_token ? at : (size_t)h);
    const size_t l = ((size_t)b * 2 * p.H + 2 * h) * p.S + row;
    v[0] = -p.lse[l] * kLog2e;
    v[1] = -p.lse[l + p.S] * kLog2e;
    v[2] = -fmaf(lam, s_d[1][r], s_d[0][r]);  // O1 = O + lam O2
    v[3] = -s_d[1][r];
    v[4] = -lam;
  }
#pragma unroll
  for (int k = 0; k < kRowVecs; ++k) p.rowv[rowv_at(tile, r) + k * 64] = v[k];
}

// -------------------------------------------------------------------- dQ
// CTA: a 128-row query tile of one head pair, over its 128-key blocks.  All four warpgroups
// work on one map at a time (thread = query row, 32 keys each), so that the tensor core has the
// other map's products to run meanwhile:
//   elementwise   S1, dP -> dS1 |          S2, dP (kept) -> dS2      | ...
//   tensor core   dP of the next block, dQ2 += , next S2 | dQ1 +=, next S1 | ...
//   S1 [0,128) S2 [128,256) dP [256,384) dQ1 [384,384+d) dQ2 [448,448+d)
// dS goes back as bf16 over the columns that the thread itself has read (the first 16 of every
// 32); a product's 16-key steps address them one by one.  All products have 128 columns or take
// A from TMEM: with both operands in shared memory, 64 columns would read 6 KB for 32 cycles of
// tensor work, more than its 128 bytes a cycle.
// D for dS comes from the outputs, rounded or with what they lost added (rest); the exact sums
// over j of Pm dP fall out of this pass and replace it for dK, and give dlam.  Of its norm dQ is
// off by, at queries of spread 1, 2, 4, 8 (the more peaked the maps, the more dP - D cancels): with
// rest 2.4e-3, 2.5e-3, 3.0e-3, 3.0e-3, from rounded outputs 2.5e-3, 2.9e-3, 4.7e-3, 7.5e-3.  The
// rounding of dQ alone is 1.7e-3, with that of dS 2.4e-3; what is left with rest is P's in the
// forward.  dS as two bf16 terms took a tenth off, for a kernel 1.3 times as long.
// Measured at 8192 tokens, 32 head pairs of 64 with 8 KV heads: causal 633 us, full 1200 us.  A
// block's products take 1570 cycles of the tensor core, a block 2650: the wait for a product, the
// 64 exponentials a thread and the stores follow one another, 4 warps a scheduler cover them in
// part.  CTAs that stay for further tiles (as in the forward) were 4 % slower here.
template <int d>
struct DqL {
  static constexpr int DV = 2 * d;
  // K is read until a block's last product, V only by its dP, one block ahead of the others
  static constexpr int kK = 3, kV = 2;
  static constexpr int kTileBytes = DV * kTile * 2;
  static constexpr int kBoxes = DV / kBoxCols;
  static constexpr int offQ = 0, offDO = kTileBytes;
  static constexpr int offK = 2 * kTileBytes, offV = offK + kK * kTileBytes;
  static constexpr int offAlong = offK;  // float [2][4][128], once K has been used
  static constexpr int offBar = offV + kV * kTileBytes;
  // q_full, k_full[], k_empty[], v_full[], v_empty[], s_full[2], dp_full, dp_free, ds_full[2],
  // acc_full, drain
  static constexpr int kNumBars = 1 + 2 * (kK + kV) + 8;
  static constexpr int offMisc = offBar + kNumBars * 8;  // tmem address, abort flag, 4 floats
  static constexpr int kBytes = offMisc + 32;
  static constexpr uint32_t tP = 256, tAcc = 384, kTmemCols = 512;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int d>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_do, const DiffBwdParams p) {
  using L = DqL<d>;
  constexpr int DV = L::DV;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrSmemAlign);
    return;
  }
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::offBar);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + L::kK;
  uint64_t *v_full = k_empty + L::kK, *v_empty = v_full + L::kV;
  uint64_t *s_full = v_empty + L::kV, *dp_full = s_full + 2, *dp_free = s_full + 3;
  uint64_t *ds_full = s_full + 4, *acc_full = s_full + 6, *drain = s_full + 7;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::offMisc);
  int *s_abort = reinterpret_cast<int *>(smem + L::offMisc + 4);
  float *s_part = reinterpret_cast<float *>(smem + L::offMisc + 16);
  float *s_along = reinterpret_cast<float *>(smem + L::offAlong);
  const Abort ab{s_abort, p.status, p.wait_ns};
  const int warp = warp_id(), lane = lane_id();

  const int i = p.N - 1 - (int)(blockIdx.x % p.N);  // heaviest causal tiles first
  const int bh = blockIdx.x / p.N;
  const int h = bh % p.H, b = bh / p.H;
  const int hkv = h / p.G;
  const int nkv = p.causal ? i + 1 : p.N;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < L::kK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < L::kV; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&ds_full[m], kWarps);
    }
    mbar_init(dp_full, 1);
    mbar_init(dp_free, kWarps);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
  }
  if (warp == kWarps + 1) {
    tmem_alloc(s_tmem, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kWarps && lane == 0) {
    // ------------------------------------------------------------------ TMA producer
    bool ok = true;
    int nk = 0, nv = 0;  // blocks brought in
    mbar_arrive_expect_tx(q_full, 2 * L::kTileBytes);
    for (int bx = 0; bx < 2 * L::kBoxes; ++bx) {  // boxes of Q and dO are half tiles
      const int at = bx * (kBoxBytes / 2), col = (bx >> 1) * kBoxCols;
      const int row = i * kTile + (bx & 1) * (kTile / 2);
      tma_load_4d(smem + L::offQ + at, &tm_q, q_full, col, h, row, b);
      tma_load_4d(smem + L::offDO + at, &tm_do, q_full, col, h, row, b);
    }
    for (int j = 0; j < nkv; ++j) {
      const int sk = j % L::kK, sv = j % L::kV;
      if (j == p.withhold_dq || !mbar_wait(&v_empty[sv], ((j / L::kV) & 1) ^ 1, ab)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&v_full[sv], L::kTileBytes);
      for (int bx = 0; bx < L::kBoxes; ++bx)
        tma_load_4d(smem + L::offV + sv * L::kTileBytes + bx * kBoxBytes, &tm_v, &v_full[sv],
                    bx * kBoxCols, hkv, j * kTile, b);
      ++nv;
      if (!mbar_wait(&k_empty[sk], ((j / L::kK) & 1) ^ 1, ab)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&k_full[sk], L::kTileBytes);
      for (int bx = 0; bx < L::kBoxes; ++bx)
        tma_load_4d(smem + L::offK + sk * L::kTileBytes + bx * kBoxBytes, &tm_k, &k_full[sk],
                    bx * kBoxCols, hkv, j * kTile, b);
      ++nk;
    }
    if (!ok) {  // leave no copy in flight into shared memory
      mbar_wait_drain(q_full, 0, 100000000ull);
      for (int j = max(0, nv - L::kV); j < nv; ++j)
        mbar_wait_drain(&v_full[j % L::kV], (j / L::kV) & 1, 100000000ull);
      for (int j = max(0, nk - L::kK); j < nk; ++j)
        mbar_wait_drain(&k_full[j % L::kK], (j / L::kK) & 1, 100000000ull);
    }
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, so that descriptors and control flow stay warp-uniform;
    // one elected lane issues (one lane alone forms every descriptor in vector registers and
    // moves it over, which bounds short products).
    constexpr uint32_t kIdescIn = make_idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdescQ = make_idesc_bf16(128, d, false, true);
    const uint32_t sbase = smem_u32(smem), lead = elect_one();
    const uint32_t loQ = desc_lo(sbase + L::offQ, 16), loDO = desc_lo(sbase + L::offDO, 16);
    auto k_at = [&](int j) { return sbase + L::offK + (j % L::kK) * L::kTileBytes; };
    auto issue_s = [&](int j, int m) {
      const uint32_t loK = desc_lo(k_at(j), 16);
#pragma unroll
      for (int k = 0; k < d / 16; ++k) {
        const uint32_t off = col_bytes(m * d + 16 * k) >> 4;
        mma_ss_l(lead, tmem + m * 128, desc_of(loQ + off), desc_of(loK + off), kIdescIn, k > 0);
      }
      mma_commit_l(lead, &s_full[m]);
    };
    auto issue_dp = [&](int j) {
      const uint32_t loV = desc_lo(sbase + L::offV + (j % L::kV) * L::kTileBytes, 16);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k) {
        const uint32_t off = col_bytes(16 * k) >> 4;
        mma_ss_l(lead, tmem + L::tP, desc_of(loDO + off), desc_of(loV + off), kIdescIn, k > 0);
      }
      mma_commit_l(lead, dp_full);
      mma_commit_l(lead, &v_empty[j % L::kV]);
    };
    auto k_there = [&](int j) { return wait_warp(&k_full[j % L::kK], (j / L::kK) & 1, ab); };
    auto v_there = [&](int j) { return wait_warp(&v_full[j % L::kV], (j / L::kV) & 1, ab); };
    bool ok = wait_warp(q_full, 0, ab) && k_there(0) && v_there(0);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      issue_dp(0);
      issue_s(0, 1);
    }
    for (int j = 0; ok && j < nkv; ++j) {
      const bool more = j + 1 < nkv;
      if (!wait_warp(dp_free, j & 1, ab) || (more && !v_there(j + 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (more) issue_dp(j + 1);
      const uint32_t loK = desc_lo(k_at(j), kBoxBytes);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (ok && !wait_warp(&ds_full[m], j & 1, ab)) ok = false;
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          mma_ts_l(lead, tmem + L::tAcc + m * 64, tmem + m * 128 + 32 * (k >> 1) + 8 * (k & 1),
                   desc_of(loK + ((col_bytes(m * d) + k * 2048) >> 4)), kIdescQ,
                   (j > 0 || k > 0) ? 1u : 0u);
        if (m == 1) mma_commit_l(lead, &k_empty[j % L::kK]);
        if (more) {
          if (m == 0 && !k_there(j + 1)) {
            ok = false;
            break;
          }
          issue_s(j + 1, m);
        }
      }
    }
    if (ok) mma_commit_l(lead, acc_full);
    mma_commit_l(lead, drain);
    mbar_wait_drain(drain, 0, 100000000ull);
  } else if (warp < kWarps) {
    // ------------------------------------------------------------------ dS
    const int wg = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // query row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int row = i * kTile + r;
    const bool row_ok = row < p.S;
    float *rowv = p.rowv + rowv_at(((size_t)b * p.H + h) * p.N + i, r);
    const f2 c2 = f2_of(p.scale_log2, p.scale_log2);
    float nl[2], nD[2];
    f2 along[2];  // sum_j Pm dP of this row, even and odd keys
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      nl[m] = rowv[m * 64];
      nD[m] = rowv[(2 + m) * 64];
      along[m] = f2_of(0.f, 0.f);
    }
    const uint32_t t0 = tmem + lane_off + 32 * wg;
    bool ok = true;
    for (int j = 0; ok && j < nkv; ++j) {
      // of this thread's 32 keys, those that the row sees
      const int limit = min(p.S, p.causal ? row + 1 : p.S) - j * kTile - 32 * wg;
      const bool cut = __any_sync(0xffffffffu, limit < 32);
      uint32_t g[32];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t s[32];
        if (ok) ok = wait_warp(&s_full[m], j & 1, ab) &&
                     (m == 1 || wait_warp(dp_full, j & 1, ab));
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(t0 + m * 128, s);
        if (m == 0) tmem_ld32(t0 + L::tP, g);
        tmem_ld_wait_for(s);
        if (m == 0) {
          tmem_ld_wait_for(g);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_free);
        }
        if (cut) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (e >= limit) s[e] = __float_as_uint(-INFINITY), g[e] = 0u;
        }
        const f2 nl2 = f2_of(nl[m], nl[m]), nD2 = f2_of(nD[m], nD[m]);
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const f2 P = ex2_2(fma2(f2_of(s[2 * e], s[2 * e + 1]), c2, nl2));
          const f2 dP = f2_of(g[2 * e], g[2 * e + 1]);
          along[m] = fma2(P, dP, along[m]);
          pk[e] = pack_bf16(mul2(P, add2(dP, nD2)));
        }
        tmem_st16(t0 + m * 128, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ds_full[m]);
      }
    }
    // ------------------------------------------------------------------ epilogue
    ok = ok && wait_warp(acc_full, 0, ab);  // every product has run: K's memory is free
    if (!ok) mbar_wait_drain(drain, 0, 100000000ull);
    tc_fence_after();
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float even, odd;
      f2_to(along[m], even, odd);
      s_along[(m * 4 + wg) * kTile + r] = even + odd;
    }
    named_bar_sync(1, kWarps * 32);
    if (wg < 2) {
      const float *al = s_along + wg * 4 * kTile + r;
      const float D = (al[0] + al[kTile]) + (al[2 * kTile] + al[3 * kTile]);
      if (row_ok) rowv[(2 + wg) * 64] = -D;
      if (wg == 1) {
        if (p.lam_token) {
          const size_t at = ((size_t)b * p.S + row) * p.H + h;
          if (row_ok) {
            if (p.lam_f32)
              static_cast<float *>(p.dlam)[at] = -D;
            else
              static_cast<__nv_bfloat16 *>(p.dlam)[at] = __float2bfloat16_rn(-D);
          }
        } else {
          float sum = row_ok ? D : 0.f;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == 0) s_part[quad] = sum;
          named_bar_sync(2, 128);
          if (quad == 0 && lane == 0)
            p.dlam_part[((size_t)b * p.H + h) * p.N + i] =
                -((s_part[0] + s_part[1]) + (s_part[2] + s_part[3]));
        }
      }
    }
    if (ok) {
      // half of dQm's columns; dS2 was formed without its weight, a factor of the row
      const int m = wg >> 1, half = (wg & 1) * (d / 2);
      const float by = m ? rowv[4 * 64] * p.scale : p.scale;
      __nv_bfloat16 *out = p.dq + (((size_t)b * p.S + row) * 2 * p.H + 2 * h + m) * d + half;
      uint32_t v[d / 2];
      if constexpr (d == 64)
        tmem_ld32(tmem + lane_off + L::tAcc + m * 64 + half, v);
      else
        tmem_ld16(tmem + lane_off + L::tAcc + m * 64 + half, v);
      tmem_ld_wait_for(v);
      if (row_ok) store_row(out, v, by);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Weights per head: the tiles' sums of head h, added in a fixed order by one warp.
__device__ __forceinline__ void sum_dlam(const DiffBwdParams &p, int h, int lane) {
  float v = 0.f;
#pragma unroll 4
  for (int k = lane; k < p.B * p.N; k += 32)
    v += p.dlam_part[((size_t)(k / p.N) * p.H + h) * p.N + k % p.N];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane > 0) return;
  if (p.lam_f32)
    static_cast<float *>(p.dlam)[h] = v;
  else
    static_cast<__nv_bfloat16 *>(p.dlam)[h] = __float2bfloat16_rn(v);
}

// -------------------------------------------------------------------- dK, dV
// CTA: a 128-key block of one KV head, over the query heads of its group and their tiles in
// ascending order, everything transposed (TMEM lane = key row, so that the bf16 operands P^T
// and dS^T go back to TMEM where their rows are), in steps of 64 queries, 16 a warpgroup:
//   A   S1, dP -> P1 and dP kept in registers, dS1 over S1
//   B   S2 -> w = -lam P2, P = P1 + w and dS2 over S2
// The accumulators (dV [0,dv), dK1 [128,+d), dK2 [192,+d)) leave four slots of 64 columns from
// 256 on, which the steps pass around so that a step's inputs are formed beside the elementwise
// work of the one before:
//   dP(t)   slot 1, free again once A(t) has read it
//   S1(t)   slots 0, 3, 2, 0, ...: that of S2(t-2), read for the last time by dV, dK2 of t-2
//   S2(t)   slots 2, 0, 3, 2, ...: that of S1(t-1), read for the last time by dK1 of t-1
// Q, dO and the row vectors come in by half tiles, a step each, in a ring of four.
// Measured at 8192 tokens, 32 head pairs of 64 with 8 KV heads: causal 903 us, full 1600 us.  Bound
// by the tensor core's pipe, 80 % busy: a step's products take 1310 cycles of 1650, 780 of them the
// 64-column products with both operands in shared memory, which need 49 cycles for 33 of work.
constexpr int kStep = 64;

template <int d>
struct DkvL {
  static constexpr int DV = 2 * d;
  static constexpr int kStages = 4;  // half tiles
  static constexpr int kTileBytes = DV * kTile * 2;
  static constexpr int kHalfBytes = kTileBytes / 2, kHalfBox = kBoxBytes / 2;
  static constexpr int kBoxes = DV / kBoxCols;
  static constexpr int kRowBytes = kRowVecs * kStep * 4;
  static constexpr int offK = 0, offV = kTileBytes;
  static constexpr int offStage = 2 * kTileBytes;  // per stage Q, dO
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int offRow = offStage + kStages * kStageBytes;  // per stage row vectors
  static constexpr int offBar = offRow + kStages * kRowBytes;
  // kv_full, q_full[], q_empty[], a_full, dp_free, ds1_full, s2_full, out_full, acc_full, drain
  static constexpr int kNumBars = 1 + 2 * kStages + 7;
  static constexpr int offMisc = offBar + kNumBars * 8;
  static constexpr int kBytes = offMisc + 16;
  static constexpr uint32_t tV = 0, tK = 128, tSlots = 256, kTmemCols = 512;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int d>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dkv_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ CUtensorMap tm_do, const DiffBwdParams p) {
  using L = DkvL<d>;
  constexpr int DV = L::DV;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrSmemAlign);
    return;
  }
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + L::offBar);
  uint64_t *q_full = kv_full + 1, *q_empty = q_full + L::kStages;
  uint64_t *a_full = q_empty + L::kStages, *dp_free = a_full + 1, *ds1_full = a_full + 2;
  uint64_t *s2_full = a_full + 3, *out_full = a_full + 4, *acc_full = a_full + 5;
  uint64_t *drain = a_full + 6;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::offMisc);
  int *s_abort = reinterpret_cast<int *>(smem + L::offMisc + 4);
  const Abort ab{s_abort, p.status, p.wait_ns};
  const int warp = warp_id(), lane = lane_id();

  const int heads = p.B * p.Hkv;
  int tile = blockIdx.x, part = -1;  // part: where a piece's sums go
  if (tile >= p.kv_whole) {
    part = tile - p.kv_whole;
    tile = p.kv_whole + part / p.kv_pieces;
  }
  const int j = tile / heads;  // causal: block 0 meets the most queries, first
  const int bh = tile % heads;
  const int hkv = bh % p.Hkv, b = bh / p.Hkv;
  const int i0 = p.causal ? j : 0, tiles = p.N - i0;
  int first_step = 0, steps = 2 * p.G * tiles;  // of the tile, and how many from there
  if (part >= 0) {
    const int piece = part % p.kv_pieces, all = steps;
    first_step = all * piece / p.kv_pieces;
    steps = all * (piece + 1) / p.kv_pieces - first_step;
  }
  auto heads_dlam = [&]() {  // by the producer's warp, behind its work
    if (!p.lam_token)
      for (int h = blockIdx.x; h < p.H; h += gridDim.x) sum_dlam(p, h, lane);
  };
  if (steps == 0) {  // (diff_join_kernel leaves such a piece out)
    if (warp == kWarps) heads_dlam();
    return;
  }

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], kWarps + 1);  // the products' commit, the readers of row vectors
    }
    mbar_init(a_full, 1);
    mbar_init(dp_free, kWarps);
    mbar_init(ds1_full, kWarps);
    mbar_init(s2_full, 1);
    mbar_init(out_full, kWarps);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
  }
  if (warp == kWarps + 1) {
    tmem_alloc(s_tmem, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kWarps) {
    if (lane == 0) {
      // ------------------------------------------------------------------ TMA producer
      int last[L::kStages];
      for (int s = 0; s < L::kStages; ++s) last[s] = -1;
      bool ok = true;
      mbar_arrive_expect_tx(kv_full, 2 * L::kTileBytes);
      for (int bx = 0; bx < L::kBoxes; ++bx) {
        tma_load_4d(smem + L::offK + bx * kBoxBytes, &tm_k, kv_full, bx * kBoxCols, hkv, j * kTile,
                    b);
        tma_load_4d(smem + L::offV + bx * kBoxBytes, &tm_v, kv_full, bx * kBoxCols, hkv, j * kTile,
                    b);
      }
      for (int n = 0; n < steps; ++n) {
        const int s = n % L::kStages;
        const uint32_t ph = (n / L::kStages) & 1;
        if (n == p.withhold_dkv || !mbar_wait(&q_empty[s], ph ^ 1, ab)) {
          ok = false;
          break;
        }
        const int at = first_step + n;
        const int h = hkv * p.G + (at >> 1) / tiles, i = i0 + (at >> 1) % tiles, u = at & 1;
        mbar_arrive_expect_tx(&q_full[s], L::kStageBytes + L::kRowBytes);
        uint8_t *sq = smem + L::offStage + s * L::kStageBytes;
        for (int bx = 0; bx < L::kBoxes; ++bx) {
          tma_load_4d(sq + bx * L::kHalfBox, &tm_q, &q_full[s], bx * kBoxCols, h,
                      i * kTile + u * kStep, b);
          tma_load_4d(sq + L::kHalfBytes + bx * L::kHalfBox, &tm_do, &q_full[s], bx * kBoxCols, h,
                      i * kTile + u * kStep, b);
        }
        bulk_load(smem + L::offRow + s * L::kRowBytes,
                  p.rowv + rowv_at(((size_t)b * p.H + h) * p.N + i, u * kStep), L::kRowBytes,
                  &q_full[s]);
        last[s] = (int)ph;
      }
      if (!ok) {
        mbar_wait_drain(kv_full, 0, 100000000ull);
        for (int s = 0; s < L::kStages; ++s)
          if (last[s] >= 0) mbar_wait_drain(&q_full[s], (uint32_t)last[s], 100000000ull);
      }
    }
    __syncwarp();
    heads_dlam();
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ MMA issuer
    // (a converged warp, one elected lane issues)
    constexpr uint32_t kIdescIn = make_idesc_bf16(128, kStep, false, false);
    constexpr uint32_t kIdescV = make_idesc_bf16(128, DV, false, true);
    constexpr uint32_t kIdescK = make_idesc_bf16(128, d, false, true);
    const uint32_t sbase = smem_u32(smem), lead = elect_one();
    const uint32_t loK = desc_lo(sbase + L::offK, 16), loV = desc_lo(sbase + L::offV, 16);
    auto q_at = [&](int n) {  // Q of step n; dO lies kHalfBytes on
      return sbase + L::offStage + (n % L::kStages) * L::kStageBytes;
    };
    auto half_bytes = [](int col) {  // col_bytes in a half tile's boxes
      return (uint32_t)(col >> 6) * L::kHalfBox + (uint32_t)(col & 63) * 2;
    };
    auto q_there = [&](int n) {
      return wait_warp(&q_full[n % L::kStages], (n / L::kStages) & 1, ab);
    };
    auto issue_s = [&](int n, int m, uint32_t to) {  // Sm^T -> slot `to`
      const uint32_t loQ = desc_lo(q_at(n), 16);
#pragma unroll
      for (int k = 0; k < d / 16; ++k) {
        const int col = m * d + 16 * k;
        mma_ss_l(lead, to, desc_of(loK + (col_bytes(col) >> 4)),
                 desc_of(loQ + (half_bytes(col) >> 4)), kIdescIn, k > 0);
      }
    };
    auto issue_dp = [&](int n) {  // dP^T -> slot 1
      const uint32_t loO = desc_lo(q_at(n) + L::kHalfBytes, 16);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ss_l(lead, tmem + L::tSlots + 64, desc_of(loV + (col_bytes(16 * k) >> 4)),
                 desc_of(loO + (half_bytes(16 * k) >> 4)), kIdescIn, k > 0);
    };
    // slots of S1 and S2 of this step, and of the next step's S1 (its S2 takes S1's of this)
    uint32_t slot1 = tmem + L::tSlots, slot2 = slot1 + 128, spare = slot1 + 192;
    bool ok = wait_warp(kv_full, 0, ab) && q_there(0);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0, slot1);
      issue_dp(0);
      mma_commit_l(lead, a_full);
      issue_s(0, 1, slot2);
      mma_commit_l(lead, s2_full);
    }
    // A barrier's phase n + 1 must not complete before every waiter has seen its phase n, so the
    // commits that let the elementwise warps go on stand behind the waits for what they did
    // before: a_full(n+1) behind ds1_full(n), s2_full(n+1) behind out_full(n).
    for (int n = 0; ok && n < steps; ++n) {
      const bool more = n + 1 < steps;
      const uint32_t ph = n & 1, first = n > 0 ? 1u : 0u;
      const uint32_t loQ = desc_lo(q_at(n), L::kHalfBox);
      const uint32_t loO = desc_lo(q_at(n) + L::kHalfBytes, L::kHalfBox);
      if (more) {
        if (!q_there(n + 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_s(n + 1, 0, spare);
        if (!wait_warp(dp_free, ph, ab)) {
          ok = false;
          break;
        }
        tc_fence_after();
        issue_dp(n + 1);
      }
      if (!wait_warp(ds1_full, ph, ab)) {
        ok = false;
        break;
      }
      if (more) mma_commit_l(lead, a_full);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        mma_ts_l(lead, tmem + L::tK, slot1 + 16 * k, desc_of(loQ + ((k * 2048) >> 4)), kIdescK,
                 k > 0 ? 1u : first);
      if (more) issue_s(n + 1, 1, slot1);
      if (!wait_warp(out_full, ph, ab)) {
        ok = false;
        break;
      }
      if (more) mma_commit_l(lead, s2_full);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        mma_ts_l(lead, tmem + L::tV, slot2 + 16 * k, desc_of(loO + ((k * 2048) >> 4)), kIdescV,
                 k > 0 ? 1u : first);
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        mma_ts_l(lead, tmem + L::tK + 64, slot2 + 8 + 16 * k,
                 desc_of(loQ + ((half_bytes(d) + k * 2048) >> 4)), kIdescK, k > 0 ? 1u : first);
      mma_commit_l(lead, &q_empty[n % L::kStages]);
      const uint32_t was2 = slot2;
      slot2 = slot1;
      slot1 = spare;
      spare = was2;
    }
    if (ok) mma_commit_l(lead, acc_full);
    mma_commit_l(lead, drain);
    mbar_wait_drain(drain, 0, 100000000ull);
  } else if (warp < kWarps) {
    // ------------------------------------------------------------------ P, dS (transposed)
    // In fragments (tmem_ld_frag): the row vectors go by query, a column here; read for every
    // element they would cost 40 broadcast loads of 16 bytes a warp and tile on the memory that
    // feeds the tensor core, in fragments 20 of 8 bytes.
    const int wg = warp >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // key row of the epilogue = TMEM lane
    const int q0 = 16 * wg;          // this warpgroup's queries within a step
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t t0 = tmem + lane_off + L::tSlots + q0;
    constexpr uint32_t kLanes16 = 16u << 16;
    const int key = j * kTile + r;
    const f2 c2 = f2_of(p.scale_log2, p.scale_log2);
    const float *rowv = reinterpret_cast<const float *>(smem + L::offRow) + q0 + 2 * (lane & 3);
    auto vec = [&](int n, int k, int g) {  // vector k of this thread's columns of group g, step n
      return *reinterpret_cast<const f2 *>(rowv + (n % L::kStages) * (L::kRowBytes / 4) +
                                           k * kStep + 8 * g);
    };
    // On the diagonal tile, queries before the key see nothing of it.  Key of fragment row 0
    // less the query of its column 0, of the tile's first step:
    const int ahead = quad * 32 + lane / 4 - (q0 + 2 * (lane & 3));
    auto hide = [&](uint32_t (&x)[8], int n, int half, uint32_t with) {
#pragma unroll
      for (int e = 0; e < 8; ++e)  // key - query of the element
        if (ahead - kStep * ((first_step + n) & 1) + 16 * half + 8 * ((e >> 1) & 1) - 8 * (e >> 2) - (e & 1) > 0)
          x[e] = with;
    };
    auto diagonal = [&](int n) { return p.causal && ((first_step + n) >> 1) % tiles == 0; };
    uint32_t slot1 = t0, slot2 = t0 + 128, spare = t0 + 192;
    bool ok = true;
    for (int n = 0; n < steps; ++n) {
      const uint32_t ph = n & 1;
      const bool cut = diagonal(n);
      // [half of the lanes][2 * group + row]
      f2 P1[2][4], dP[2][4];
      // A
      if (!wait_warp(&q_full[n % L::kStages], (n / L::kStages) & 1, ab) ||
          !wait_warp(a_full, ph, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      {
        uint32_t x[2][8], y[2][8];
        tmem_ld_frag(slot1, x[0]);
        tmem_ld_frag(slot1 + kLanes16, x[1]);
        tmem_ld_frag(t0 + 64, y[0]);
        tmem_ld_frag(t0 + 64 + kLanes16, y[1]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_ld_wait_for(x[half]);
          tmem_ld_wait_for(y[half]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(dp_free);
        if (cut) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            hide(x[half], n, half, __float_as_uint(-INFINITY));
            hide(y[half], n, half, 0u);
          }
        }
        uint32_t pk[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f2 nl = vec(n, 0, g), nD = vec(n, 2, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int half = e >> 1, at = 2 * g + (e & 1);
            P1[half][at] = ex2_2(fma2(f2_of(x[half][2 * at], x[half][2 * at + 1]), c2, nl));
            dP[half][at] = f2_of(y[half][2 * at], y[half][2 * at + 1]);
            pk[half][at] = pack_bf16(mul2(P1[half][at], add2(dP[half][at], nD)));
          }
        }
        tmem_st_frag(slot1, pk[0]);
        tmem_st_frag(slot1 + kLanes16, pk[1]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds1_full);
      // B
      if (!wait_warp(s2_full, ph, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      {
        uint32_t x[2][8], pP[2][4], pk[2][4];
        tmem_ld_frag(slot2, x[0]);
        tmem_ld_frag(slot2 + kLanes16, x[1]);
        tmem_ld_wait_for(x[0]);
        tmem_ld_wait_for(x[1]);
        if (cut) {
          hide(x[0], n, 0, __float_as_uint(-INFINITY));
          hide(x[1], n, 1, __float_as_uint(-INFINITY));
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f2 nl = vec(n, 1, g), nD = vec(n, 3, g), nlam = vec(n, 4, g);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int half = e >> 1, at = 2 * g + (e & 1);
            const f2 w =
                mul2(ex2_2(fma2(f2_of(x[half][2 * at], x[half][2 * at + 1]), c2, nl)), nlam);
            pP[half][at] = pack_bf16(add2(P1[half][at], w));
            pk[half][at] = pack_bf16(mul2(w, add2(dP[half][at], nD)));
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          tmem_st_frag(slot2 + half * kLanes16, pP[half]);
          tmem_st_frag(slot2 + 8 + half * kLanes16, pk[half]);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(out_full);
        mbar_arrive(&q_empty[n % L::kStages]);
      }
      const uint32_t was2 = slot2;
      slot2 = slot1;
      slot1 = spare;
      spare = was2;
    }
    if (ok && wait_warp(acc_full, 0, ab)) {
      tc_fence_after();
      // one of dK1, dK2 and the halves of dV
      const size_t at = (size_t)b * p.S + key;
      __nv_bfloat16 *out = wg < 2 ? p.dk + (at * 2 * p.Hkv + 2 * hkv + wg) * d
                                  : p.dv + (at * p.Hkv + hkv) * DV + (wg - 2) * d;
      const uint32_t from = tmem + lane_off + (wg < 2 ? L::tK + 64 * wg : L::tV + (wg - 2) * d);
#pragma unroll 1
      for (int c = 0; c < d / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(from + 32 * c, v);
        tmem_ld_wait_for(v);
        if (part >= 0) {  // dK1, dK2, dV side by side
          float4 *sum = reinterpret_cast<float4 *>(p.kv_part) +
                        ((size_t)part * d + wg * (d / 4) + 8 * c) * kTile + r;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sum[e * kTile] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                         __uint_as_float(v[4 * e + 2]),
                                         __uint_as_float(v[4 * e + 3]));
        } else if (key < p.S) {
          store_row(out + 32 * c, v, wg < 2 ? p.scale : 1.f);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// dK and dV of the tiles that were cut: their pieces' sums, added in order.  One CTA per tile and
// 8 columns, thread = key row.
template <int d>
__global__ void __launch_bounds__(kTile) diff_join_kernel(const DiffBwdParams p) {
  const int heads = p.B * p.Hkv, tile = p.kv_whole + blockIdx.x, c8 = blockIdx.y;
  const int j = tile / heads, bh = tile % heads, hkv = bh % p.Hkv, b = bh / p.Hkv;
  const int all = 2 * p.G * (p.N - (p.causal ? j : 0));
  const int key = j * kTile + threadIdx.x;
  const float4 *part = reinterpret_cast<const float4 *>(p.kv_part) +
                       ((size_t)blockIdx.x * p.kv_pieces * d + 2 * c8) * kTile + threadIdx.x;
  float v[8] = {};
#pragma unroll 4
  for (int k = 0; k < p.kv_pieces; ++k) {
    if (all * k / p.kv_pieces == all * (k + 1) / p.kv_pieces) continue;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float4 x = part[((size_t)k * d + u) * kTile];
      v[4 * u] += x.x, v[4 * u + 1] += x.y, v[4 * u + 2] += x.z, v[4 * u + 3] += x.w;
    }
  }
  if (key >= p.S) return;
  const int col = 8 * c8, m = col / d;  // dK1, dK2 and the halves of dV
  const size_t at = (size_t)b * p.S + key;
  __nv_bfloat16 *out = m < 2 ? p.dk + (at * 2 * p.Hkv + 2 * hkv) * d + col
                             : p.dv + (at * p.Hkv + hkv) * 2 * d + (col - 2 * d);
  uint32_t bits[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bits[e] = __float_as_uint(v[e]);
  store_row(out, bits, m < 2 ? p.scale : 1.f);
}

template <int d>
cudaError_t launch_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const CUtensorMap &tdo,
                     const DiffBwdParams &p, cudaStream_t s) {
  using LQ = DqL<d>;
  using LK = DkvL<d>;
  cudaError_t e = allow_smem<diff_dq_kernel<d>>(LQ::kBytes);
  if (e == cudaSuccess) e = allow_smem<diff_dkv_kernel<d>>(LK::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)p.B * p.H * p.N;
  if (p.rest)
    diff_rows_kernel<d, true><<<tiles, 256, 0, s>>>(p);
  else
    diff_rows_kernel<d, false><<<tiles, 256, 0, s>>>(p);
  diff_dq_kernel<d><<<tiles, kThreads, LQ::kBytes, s>>>(tq, tk, tv, tdo, p);
  const unsigned cut = (unsigned)p.B * p.Hkv * p.N - p.kv_whole;  // tiles in pieces
  diff_dkv_kernel<d><<<p.kv_whole + cut * p.kv_pieces, kThreads, LK::kBytes, s>>>(tq, tk, tv,
                                                                                  tdo, p);
  if (cut) diff_join_kernel<d><<<dim3(cut, d / 2), kTile, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_bwd(int d, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tdo,
                            const DiffBwdParams &p, cudaStream_t s) {
  return d == 32 ? launch_t<32>(tq, tk, tv, tdo, p, s) : launch_t<64>(tq, tk, tv, tdo, p, s);
}

}  // namespace dash
