// diff_fwd.cu -- differential attention forward: O, O2 = P2 V (the backward's second row
// product and the weight's gradient need it) and both maps' LSE.
//
// Persistent CTAs, one on an SM, over the 128-row query tiles of every (batch, head pair): a
// tile's first scores are formed beside the epilogue of the one before.  The next tile is the
// next that no CTA has taken (a counter in the status block; which CTA forms a tile changes
// nothing in it): unlike a fixed deal this keeps causal tiles of one head, which read the same
// keys, near each other in time, and evens out their lengths.  The two maps are two independent
// online softmaxes over the same KV blocks, two warpgroups each (thread = query row, 64 keys of
// a block; they exchange their halves of the row's maximum through shared memory), so that while
// one map's scores become probabilities the tensor core runs the other's products:
//   Sm = Qm Km^T -> max, exp2, sum -> Pm (bf16, in TMEM over Sm) -> Om += Pm V
// The running maximum of a row is only raised when a block exceeds it by 2^8 (the row's Om
// and sum are then rescaled in place; no product on Om is in flight, the next Sm follows Pm V
// in issue order).  P is rounded to bf16 for the tensor core, relative error 2^-8 at most per
// entry; sums, maxima and accumulators are fp32.
//
// Measured at 8192 tokens, 32 head pairs of 64 with 8 KV heads: causal 628 us, 1313 TFLOP/s; full
// 1120 us, 1475 TFLOP/s (78 % of cuBLAS's bf16 rate).  A block's products take 1560 cycles of the
// tensor core and its 32768 exponentials 1024 cycles; a block takes 2450, as each map's softmax
// (wait, maximum, exchange, exponentials, stores) is a chain that the other map's products hide in
// part only: tensor pipe 61 % busy.  16 sequences of 1024, full: 390 us (442 us with a CTA a tile).
// With the outputs' rest 661 us causal, 1220 us full: two more bf16 stores an output element.
//
// TMEM columns: S1 [0,128), S2 [128,256), O1 [256, 256+dv), O2 [256+dv, 256+2dv); P over the
// first half of the columns that its warpgroup reads.
// Warps 0-7 map 1, 8-15 map 2, 16 TMA producer, 17 MMA issuer.
#include "diff.cuh"

#include "dash_attn.h"
#include "host.cuh"

namespace dash {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = (kWarps + 2) * 32;
constexpr float kRaise = 8.f;  // log2 of how far a row's scores may pass its running maximum

template <int d>
struct FwdL {
  static constexpr int DV = 2 * d;
  static constexpr int kStages = 2;
  static constexpr int kTileBytes = DV * kTile * 2;
  static constexpr int kBoxes = DV / kBoxCols;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K then V
  static constexpr int offQ = 0;
  static constexpr int offStage = kTileBytes;
  static constexpr int offSum = offStage + kStages * kStageBytes;  // float [2][2][2][128]
  static constexpr int offMax = offSum + 8 * kTile * 4;            // float [2][2][2][128]
  static constexpr int offBar = offMax + 8 * kTile * 4;
  // q_full, q_empty, k_full[], k_empty[], v_full[], v_empty[], s_full[2], p_full[2][2], o_full,
  // o_free, t_full, t_empty, drain
  static constexpr int kNumBars = 2 + 4 * kStages + 6 + 5;
  static constexpr int offMisc = offBar + kNumBars * 8;
  // tmem address, abort flag, next tile, -, failed [2]
  static constexpr int kBytes = offMisc + 32;
  static constexpr uint32_t tS = 0, tO = 256, kTmemCols = 512;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int d>
__global__ void __launch_bounds__(kThreads, 1)
    diff_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const DiffFwdParams p) {
  using L = FwdL<d>;
  constexpr int DV = L::DV;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrSmemAlign);
    return;
  }
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + L::offBar);
  uint64_t *q_empty = q_full + 1, *k_full = q_full + 2, *k_empty = k_full + L::kStages;
  uint64_t *v_full = k_empty + L::kStages, *v_empty = v_full + L::kStages;
  uint64_t *s_full = v_empty + L::kStages, *p_full = s_full + 2, *o_full = p_full + 4;
  uint64_t *o_free = o_full + 1, *t_full = o_full + 2, *t_empty = o_full + 3;
  uint64_t *drain = o_full + 4;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::offMisc);
  int *s_abort = reinterpret_cast<int *>(smem + L::offMisc + 4);
  volatile int *s_next = reinterpret_cast<int *>(smem + L::offMisc + 8);
  volatile int *s_failed = reinterpret_cast<int *>(smem + L::offMisc + 16);
  const Abort ab{s_abort, p.status, p.wait_ns};
  const int warp = warp_id(), lane = lane_id();

  // tile -> query tile (a head's heaviest causal one first), head pair, batch, key blocks
  auto tile_i = [&](int tile) { return p.N - 1 - tile % p.N; };
  auto blocks = [&](int i) { return p.causal ? i + 1 : p.N; };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&p_full[2 * m], kWarps / 2);
      mbar_init(&p_full[2 * m + 1], kWarps / 2);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, kWarps);
    mbar_init(t_full, 1);
    mbar_init(t_empty, kWarps + 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    s_failed[0] = s_failed[1] = 0;
    fence_mbar_init();
  }
  if (warp == kWarps && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
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
    // K is free again once S2 of its block is formed, long before V.  Counters of what was
    // brought in run over all tiles, as do the rings.
    bool ok = true;
    int nq = 0, nk = 0, nv = 0;
    for (int tile = blockIdx.x; ok && tile >= 0;) {
      const int i = tile_i(tile), bh = tile / p.N, h = bh % p.H, b = bh / p.H, hkv = h / p.G;
      const int nkv = blocks(i);
      int next = 0;
      for (int j = 0; j < nkv; ++j) {
        // taken late, so that tiles go to the CTAs that will be free first
        if (j + 1 == nkv) next = (int)gridDim.x + (int)atomicAdd(p.taken, 1u);
        const int s = nk % L::kStages;
        const uint32_t ph = (nk / L::kStages) & 1;
        uint8_t *sk = smem + L::offStage + s * L::kStageBytes;
        if (nk == p.withhold || !mbar_wait(&k_empty[s], ph ^ 1, ab)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&k_full[s], L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sk + bx * kBoxBytes, &tm_k, &k_full[s], bx * kBoxCols, hkv, j * kTile, b);
        ++nk;
        if (j == 0) {
          if (nq > 0 && !mbar_wait(q_empty, (nq - 1) & 1, ab)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(q_full, L::kTileBytes);
          for (int bx = 0; bx < L::kBoxes; ++bx)
            tma_load_4d(smem + L::offQ + bx * kBoxBytes, &tm_q, q_full, bx * kBoxCols, h,
                        i * kTile, b);
          ++nq;
        }
        if (!mbar_wait(&v_empty[s], ph ^ 1, ab)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&v_full[s], L::kTileBytes);
        for (int bx = 0; bx < L::kBoxes; ++bx)
          tma_load_4d(sk + L::kTileBytes + bx * kBoxBytes, &tm_v, &v_full[s], bx * kBoxCols, hkv,
                      j * kTile, b);
        ++nv;
      }
      // every reader has taken the tile before
      if (ok && nq > 1 && !mbar_wait(t_empty, nq & 1, ab)) ok = false;
      if (!ok) break;
      if (next >= p.B * p.H * p.N) next = -1;
      *s_next = next;
      mbar_arrive(t_full);
      tile = next;
    }
    if (!ok) {  // leave no copy in flight into shared memory
      if (nq > 0) mbar_wait_drain(q_full, (nq - 1) & 1, 100000000ull);
      for (int j = max(0, nk - L::kStages); j < nk; ++j)
        mbar_wait_drain(&k_full[j % L::kStages], (j / L::kStages) & 1, 100000000ull);
      for (int j = max(0, nv - L::kStages); j < nv; ++j)
        mbar_wait_drain(&v_full[j % L::kStages], (j / L::kStages) & 1, 100000000ull);
    }
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, so that descriptors and control flow stay warp-uniform;
    // one elected lane issues.
    constexpr uint32_t kIdescS = make_idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdescO = make_idesc_bf16(128, DV, false, true);
    const uint32_t sbase = smem_u32(smem), lead = elect_one();
    const uint32_t loQ = desc_lo(sbase + L::offQ, 16);
    // g counts key blocks over all tiles
    auto issue_s = [&](int g, int m) {
      const uint32_t loK = desc_lo(sbase + L::offStage + (g % L::kStages) * L::kStageBytes, 16);
#pragma unroll
      for (int k = 0; k < d / 16; ++k) {
        const uint32_t off = col_bytes(m * d + 16 * k) >> 4;
        mma_ss_l(lead, tmem + L::tS + m * 128, desc_of(loQ + off), desc_of(loK + off), kIdescS,
                 k > 0);
      }
      mma_commit_l(lead, &s_full[m]);
      if (m == 1) mma_commit_l(lead, &k_empty[g % L::kStages]);
    };
    auto k_there = [&](int g) {
      return wait_warp(&k_full[g % L::kStages], (g / L::kStages) & 1, ab);
    };
    bool ok = true;
    int g = 0, tile = blockIdx.x;
    for (int n = 0; ok; ++n) {  // tiles
      const int nkv = blocks(tile_i(tile));
      // S1 and S2 were read for the last time by the tile before's last products
      ok = wait_warp(q_full, n & 1, ab) && k_there(g);
      if (!ok) break;
      tc_fence_after();
      issue_s(g, 0);
      issue_s(g, 1);
      if (nkv == 1) mma_commit_l(lead, q_empty);
      // its first product overwrites what the tile before's epilogue reads
      if (n > 0) ok = wait_warp(o_free, (n - 1) & 1, ab);
      for (int j = 0; ok && j < nkv; ++j, ++g) {
        const int s = g % L::kStages, j1 = j + 1;
        const uint32_t loV =
            desc_lo(sbase + L::offStage + s * L::kStageBytes + L::kTileBytes, kBoxBytes);
        // what the products read first: it is there long before the probabilities
        ok = wait_warp(&v_full[s], (g / L::kStages) & 1, ab) && (j1 == nkv || k_there(g + 1));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          // the first 32 keys of both warpgroups as soon as they are there, then the others
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (ok) ok = wait_warp(&p_full[2 * m + c], g & 1, ab);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = 4 * (e >> 1) + 2 * c + (e & 1);
              mma_ts_l(lead, tmem + L::tO + m * DV,
                       tmem + L::tS + m * 128 + 64 * (k >> 2) + 8 * (k & 3),
                       desc_of(loV + ((k * 2048) >> 4)), kIdescO,
                       (j > 0 || c > 0 || e > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          if (j1 < nkv) issue_s(g + 1, m);
          if (m == 1) mma_commit_l(lead, &v_empty[s]);
        }
        if (ok && j + 2 == nkv) mma_commit_l(lead, q_empty);  // the tile's last S2 is formed
      }
      if (!ok) break;
      mma_commit_l(lead, o_full);
      ok = wait_warp(t_full, n & 1, ab);
      tile = *s_next;
      __syncwarp();
      if (lane == 0) mbar_arrive(t_empty);
      if (tile < 0) break;
    }
    mma_commit_l(lead, drain);
    mbar_wait_drain(drain, 0, 100000000ull);
  } else if (warp < kWarps) {
    // ------------------------------------------------------------------ softmax of map m
    const int wg = warp >> 2, m = wg >> 1, half = wg & 1;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // query row within the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + L::tS + m * 128 + 64 * half;
    const uint32_t tO = tmem + lane_off + L::tO + m * DV + half * d;  // this warpgroup's columns
    float *s_max = reinterpret_cast<float *>(smem + L::offMax) + m * 4 * kTile + r;
    const f2 c2 = f2_of(p.scale_log2, p.scale_log2);
    // A wait that gives up must not part warps that meet at a barrier: the warp goes on through
    // its tile without waiting, and all leave together behind it.
    uint32_t ph = 0;  // parity of the key blocks so far, and (bit 1) of the tiles
    for (int tile = blockIdx.x; tile >= 0; ph ^= 2) {
      const int nkv = blocks(tile_i(tile));
      float ref = -INFINITY;                         // running maximum (log2 units)
      f2 l[2] = {f2_of(0.f, 0.f), f2_of(0.f, 0.f)};  // sum over this warpgroup's keys
      bool ok = true;
      // of this thread's 64 keys of the block, those that the row sees
      int limit = (p.causal ? min(p.S, tile_i(tile) * kTile + r + 1) : p.S) - 64 * half;
      for (int left = nkv; left > 0; --left, limit -= kTile, ph ^= 1) {
        if (ok) ok = wait_warp(&s_full[m], ph & 1, ab);
        tc_fence_after();
        const bool cut = __any_sync(0xffffffffu, limit < 64);
        // The scores are read twice, by 32 columns: once for the maximum, once for the
        // probabilities (held between, they would not fit the registers of 18 warps).
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t s[32];
          tmem_ld32(tS + 32 * c, s);
          tmem_ld_wait_for(s);
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= limit) s[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(s[e]));
        }
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
        s_max[((ph & 1) * 2 + half) * kTile] = top;
        named_bar_sync(1 + m, kWarps * 16);
        top = fmaxf(top, s_max[((ph & 1) * 2 + (half ^ 1)) * kTile]);
        if (left == nkv) {
          ref = top;
        } else if (__any_sync(0xffffffffu, top > ref + kRaise)) {
          // (both warpgroups of a map take the same decision from the same values)
          top = fmaxf(ref, top);
          const float by = ex2_approx(ref - top);
          const f2 by2 = f2_of(by, by);
          ref = top;
          l[0] = mul2(l[0], by2);
          l[1] = mul2(l[1], by2);
#pragma unroll 1
          for (int c = 0; c < d / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait_for(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
            tmem_st32(tO + 32 * c, o);
          }
          tmem_st_wait();
        }
        const f2 nref2 = f2_of(-ref, -ref);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t s[32], pk[16];
          tmem_ld32(tS + 32 * c, s);
          tmem_ld_wait_for(s);
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= limit) s[e] = __float_as_uint(-INFINITY);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const f2 P = ex2_2(fma2(f2_of(s[2 * e], s[2 * e + 1]), c2, nref2));
            l[e & 1] = add2(l[e & 1], P);
            pk[e] = pack_bf16(P);
          }
          tmem_st16(tS + 16 * c, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * m + c]);
        }
      }
      // ------------------------------------------------------------------ epilogue
      const int bh = tile / p.N, h = bh % p.H, b = bh / p.H;
      const int row = tile_i(tile) * kTile + r;
      const bool row_ok = row < p.S;
      float *s_sum = reinterpret_cast<float *>(smem + L::offSum) + (ph >> 1) * 4 * kTile + r;
      s_sum[(m * 2 + half) * kTile] = f2_sum(add2(l[0], l[1]));
      ok = ok && wait_warp(o_full, ph >> 1, ab) && wait_warp(t_full, ph >> 1, ab);
      tile = *s_next;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(t_empty);
        if (!ok) s_failed[ph >> 1] = 1;
      }
      named_bar_sync(3, kWarps * 32);
      if (s_failed[ph >> 1]) break;
      const float l1 = s_sum[0] + s_sum[kTile], l2 = s_sum[2 * kTile] + s_sum[3 * kTile];
      if (row_ok && half == 0)
        p.lse[((size_t)b * 2 * p.H + 2 * h + m) * p.S + row] = (ref + log2f(m ? l2 : l1)) * kLn2;
      tc_fence_after();
      // this warpgroup's quarter of the columns of both accumulators
      const float n1 = 1.f / l1, n2 = 1.f / l2;
      const size_t at = (size_t)b * p.S + row;
      const float lam =
          row_ok ? lam_at(p.lam, p.lam_f32, p.lam_token ? at * p.H + h : (size_t)h) : 0.f;
      const uint32_t t1 = tmem + lane_off + L::tO + wg * (d / 2);
      const size_t out = (at * p.H + h) * DV + wg * (d / 2);
      uint32_t o1[d / 2], o2[d / 2];
      if constexpr (d == 64) {
        tmem_ld32(t1, o1);
        tmem_ld32(t1 + DV, o2);
      } else {
        tmem_ld16(t1, o1);
        tmem_ld16(t1 + DV, o2);
      }
      tmem_ld_wait_for(o1);
      tmem_ld_wait_for(o2);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
#pragma unroll
      for (int e = 0; e < d / 2; ++e) {
        const float z = __uint_as_float(o2[e]) * n2;
        o2[e] = __float_as_uint(z);
        o1[e] = __float_as_uint(fmaf(-lam, z, __uint_as_float(o1[e]) * n1));
      }
      if (row_ok) {
        store_row(p.o + out, o1, 1.f);
        store_row(p.o2 + out, o2, 1.f);
        if (p.rest) {
#pragma unroll
          for (int e = 0; e < d / 2; ++e) o1[e] = rest_of(o1[e]), o2[e] = rest_of(o2[e]);
          store_row(p.rest + out, o1, 1.f);
          store_row(p.rest + (size_t)p.B * p.S * p.H * DV + out, o2, 1.f);
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

template <int d>
cudaError_t launch_t(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     const DiffFwdParams &p, int sms, cudaStream_t s) {
  using L = FwdL<d>;
  const cudaError_t e = allow_smem<diff_fwd_kernel<d>>(L::kBytes);
  if (e != cudaSuccess) return e;
  const int tiles = p.B * p.H * p.N;
  diff_fwd_kernel<d><<<tiles < sms ? tiles : sms, kThreads, L::kBytes, s>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_fwd(int d, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const DiffFwdParams &p, int sms,
                            cudaStream_t s) {
  return d == 32 ? launch_t<32>(tq, tk, tv, p, sms, s) : launch_t<64>(tq, tk, tv, p, sms, s);
}

}  // namespace dash
