// diff_bwd.cu -- differential attention backward, deterministic without any ordering between
// CTAs: one kernel stationary in queries accumulates dQ, one stationary in keys accumulates
// dK and dV, each on chip in the order of its own loop.
//
// With dP = dO V^T (both maps share it), Dm = dO . Om, and ~ for the rounding to bf16 that the
// tensor core asks for:
//   dS1 = P1 (dP - D1)       dS2 = -lam P2 (dP - D2)        dlam_i = - sum_j P2 dP
//   dQm = c ~dSm Km          dKm = c ~dSm^T Qm              dV = ~(P1 - lam P2)^T dO
// Splitting the pass recomputes S1, S2 and dP (512 of then 1792 flops a pair at d = 64), and
// avoids what a single key-stationary kernel pays on this GPU: fp32 dQ partials pushed into L2
// at 16-20 bytes a cycle and SM, 64 KB a tile pair, longer than all of a tile pair's products,
// and their ordering.
#include "diff.cuh"

namespace dash {
namespace {

constexpr int kWarps = 16;                   // warps of elementwise work: four warpgroups
constexpr int kThreads = (kWarps + 2) * 32;  // and the TMA producer, the MMA issuer

// -------------------------------------------------------------------- row vectors
// One CTA per tile of a (batch, head pair); DV / 8 lanes per row.
template <int d>
__global__ void __launch_bounds__(256) diff_rows_kernel(const DiffBwdParams p) {
  constexpr int DV = 2 * d, kLanes = DV / 8, kRows = 256 / kLanes;
  __shared__ float s_d[2][kTile];
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int tile = blockIdx.x, i = tile % p.N, h = (tile / p.N) % p.H, b = tile / p.N / p.H;
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
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = __bfloat1622float2(g2[e]), u = __bfloat1622float2(x2[e]),
                     w = __bfloat1622float2(y2[e]);
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
  for (int k = 0; k < kRowVecs; ++k) p.rowv[((size_t)tile * kRowVecs + k) * kTile + r] = v[k];
}

// -------------------------------------------------------------------- dQ
// CTA: a 128-row query tile of one head pair; steps of 64 keys.  The stationary operands Q1, Q2
// and dO live in TMEM as the A operands: a product of 64 columns with both operands in shared
// memory reads 6 KB for 32 cycles of tensor work, more than the 128 bytes a cycle that shared
// memory gives; with A in TMEM it reads 2 KB.  A step's S1, S2, dP go to registers at once,
// which frees their columns for the next step's products while dS is formed.
//   S1 [0,64) S2 [64,128) dP [128,192)   dS1 [192,224) dS2 [224,256)  (bf16)
//   dQ1 [256,256+d) dQ2 [320,320+d)      Q1 [384,+d/2) Q2 [416,+d/2) dO [448,+d)  (bf16)
// Warpgroup w: map w / 2, keys 32 (w % 2) on of the step; thread = query row.
// D for dS comes from the rounded outputs; the exact sums over j of Pm dP fall out of this pass
// and replace it for dK, and give dlam.
constexpr int kKeys = 64;  // keys of a step

template <int d>
struct DqL {
  static constexpr int DV = 2 * d;
  static constexpr int kStages = 3;
  static constexpr int kTileBytes = DV * kTile * 2;
  static constexpr int kBoxes = DV / kBoxCols;
  static constexpr int kStageBytes = 2 * kTileBytes;  // K then V, 128 keys
  static constexpr int offStage = 0;
  static constexpr int offAlong = kStages * kStageBytes;  // float [4][128]
  static constexpr int offBar = offAlong + 4 * kTile * 4;
  // kv_full[], kv_empty[], in_full, in_free, out_full, out_free, drain
  static constexpr int kNumBars = 2 * kStages + 5;
  static constexpr int offMisc = offBar + kNumBars * 8;  // tmem address, abort flag, 4 floats
  static constexpr int kBytes = offMisc + 32;
  static constexpr uint32_t tOut = 192, tAcc = 256, tQ = 384, tDO = 448, kTmemCols = 512;
  static_assert(kBytes <= 232448, "shared memory budget");
};

template <int d>
__global__ void __launch_bounds__(kThreads, 1)
    diff_dq_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __nv_bfloat16 *q,
                   const DiffBwdParams p) {
  using L = DqL<d>;
  constexpr int DV = L::DV;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, kErrSmemAlign);
    return;
  }
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(smem + L::offBar);
  uint64_t *kv_empty = kv_full + L::kStages, *in_full = kv_empty + L::kStages;
  uint64_t *in_free = in_full + 1, *out_full = in_full + 2, *out_free = in_full + 3;
  uint64_t *drain = in_full + 4;
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
  const int keys = p.causal ? min(p.S, (i + 1) * kTile) : p.S;
  const int steps = (keys + kKeys - 1) / kKeys, stages = (steps + 1) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(in_full, 1);
    mbar_init(in_free, kWarps);
    mbar_init(out_full, kWarps);
    mbar_init(out_free, 1);
    mbar_init(drain, 1);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarps && lane == 0) {
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
  const int wg = warp >> 2, quad = warp & 3;
  const int r = quad * 32 + lane;  // query row within the tile = TMEM lane
  const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
  const int row = i * kTile + r;
  const bool row_ok = row < p.S;
  if (warp < kWarps) {
    // A quarter of this row's Q1 | Q2 | dO (both of d / 2 words, the latter in two parts) into
    // TMEM, whose columns hold the row's memory words; rows past S are zeros.
    const size_t at = (size_t)b * p.S + row;
    const __nv_bfloat16 *src = (wg < 2 ? q : p.dout) + (at * p.H + h) * DV + (wg & 1) * d;
    const uint32_t to = tmem + lane_off + (wg < 2 ? L::tQ + wg * 32 : L::tDO + (wg & 1) * (d / 2));
#pragma unroll
    for (int c = 0; c < d / 32; ++c) {
      uint32_t v[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 x = row_ok ? reinterpret_cast<const uint4 *>(src)[4 * c + e]
                               : make_uint4(0u, 0u, 0u, 0u);
        v[4 * e] = x.x, v[4 * e + 1] = x.y, v[4 * e + 2] = x.z, v[4 * e + 3] = x.w;
      }
      tmem_st16(to + 16 * c, v);
    }
    tmem_st_wait();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == kWarps && lane == 0) {
    // ------------------------------------------------------------------ TMA producer
    int last[L::kStages];
    for (int s = 0; s < L::kStages; ++s) last[s] = -1;
    bool ok = true;
    for (int j = 0; j < stages; ++j) {
      const int s = j % L::kStages;
      const uint32_t ph = (j / L::kStages) & 1;
      if (!mbar_wait(&kv_empty[s], ph ^ 1, ab)) {
        ok = false;
        break;
      }
      mbar_arrive_expect_tx(&kv_full[s], L::kStageBytes);
      uint8_t *sk = smem + L::offStage + s * L::kStageBytes;
      for (int bx = 0; bx < L::kBoxes; ++bx) {
        tma_load_4d(sk + bx * kBoxBytes, &tm_k, &kv_full[s], bx * kBoxCols, hkv, j * kTile, b);
        tma_load_4d(sk + L::kTileBytes + bx * kBoxBytes, &tm_v, &kv_full[s], bx * kBoxCols, hkv,
                    j * kTile, b);
      }
      last[s] = (int)ph;
    }
    if (!ok)
      for (int s = 0; s < L::kStages; ++s)
        if (last[s] >= 0) mbar_wait_drain(&kv_full[s], (uint32_t)last[s], 100000000ull);
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, so that descriptors and control flow stay warp-uniform;
    // one elected lane issues (one lane alone forms every descriptor in vector registers and
    // moves it over: the issue then bounds these short products).
    constexpr uint32_t kIdescIn = make_idesc_bf16(128, kKeys, false, false);
    constexpr uint32_t kIdescQ = make_idesc_bf16(128, d, false, true);
    const uint32_t sbase = smem_u32(smem);
    auto step_at = [&](int t) {  // K rows of step t
      return sbase + L::offStage + ((t >> 1) % L::kStages) * L::kStageBytes +
             (t & 1) * (kKeys * 128);
    };
    // S1, S2 and dP of step t; keys (t & 1) * 64 on of its stage
    auto issue_in = [&](int t) -> bool {
      if (!(t & 1) && !mbar_wait_warp(&kv_full[(t >> 1) % L::kStages],
                                      ((t >> 1) / L::kStages) & 1, ab))
        return false;
      tc_fence_after();
      const uint32_t loK = desc_lo(step_at(t), 16), loV = desc_lo(step_at(t) + L::kTileBytes, 16);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < d / 16; ++k)
          mma_ts_e(tmem + m * 64, tmem + L::tQ + m * 32 + 8 * k,
                   desc_of(loK + (col_bytes(m * d + 16 * k) >> 4)), kIdescIn, k > 0);
#pragma unroll
      for (int k = 0; k < DV / 16; ++k)
        mma_ts_e(tmem + 128, tmem + L::tDO + 8 * k, desc_of(loV + (col_bytes(16 * k) >> 4)),
                 kIdescIn, k > 0);
      mma_commit_e(in_full);
      return true;
    };
    bool ok = issue_in(0);
    for (int t = 0; ok && t < steps; ++t) {
      if (t + 1 < steps && !(mbar_wait_warp(in_free, t & 1, ab) && issue_in(t + 1))) {
        ok = false;
        break;
      }
      if (!mbar_wait_warp(out_full, t & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t loK = desc_lo(step_at(t), kBoxBytes);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts_e(tmem + L::tAcc + m * 64, tmem + L::tOut + m * 32 + 8 * k,
                   desc_of(loK + ((col_bytes(m * d) + k * 2048) >> 4)), kIdescQ,
                   (t > 0 || k > 0) ? 1u : 0u);
      mma_commit_e(out_free);
      if (t & 1) mma_commit_e(&kv_empty[(t >> 1) % L::kStages]);
    }
    mma_commit_e(drain);
    mbar_wait_drain(drain, 0, 100000000ull);
  } else if (warp < kWarps) {
    // ------------------------------------------------------------------ dS of map m
    const int m = wg >> 1, k0 = 32 * (wg & 1);
    float *rowv = p.rowv + (((size_t)b * p.H + h) * p.N + i) * (kRowVecs * kTile) + r;
    const float nlse = rowv[m * kTile], nD = rowv[(2 + m) * kTile];
    const f2 c2 = f2_of(p.scale_log2, p.scale_log2), nl2 = f2_of(nlse, nlse), nD2 = f2_of(nD, nD);
    f2 along2 = f2_of(0.f, 0.f);  // sum_j Pm dP of this row, even and odd keys
    const uint32_t tS = tmem + lane_off + m * 64 + k0, tP = tmem + lane_off + 128 + k0;
    const uint32_t tO = tmem + lane_off + L::tOut + m * 32 + k0 / 2;
    bool ok = true;
    for (int t = 0; t < steps; ++t) {
      if (!mbar_wait_warp(in_full, t & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s[32], g[32];
      tmem_ld32(tS, s);
      tmem_ld32(tP, g);
      tmem_ld_wait_for(s);
      tmem_ld_wait_for(g);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(in_free);
      // of these 32 keys, those that the row sees
      const int limit = min(p.S, p.causal ? row + 1 : p.S) - t * kKeys - k0;
      if (__any_sync(0xffffffffu, limit < 32)) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (e >= limit) s[e] = __float_as_uint(-INFINITY), g[e] = 0u;
      }
      uint32_t pk[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const f2 P = ex2_2(fma2(f2_of(s[2 * e], s[2 * e + 1]), c2, nl2));
        const f2 dP = f2_of(g[2 * e], g[2 * e + 1]);
        along2 = fma2(P, dP, along2);
        pk[e] = pack_bf16(mul2(P, add2(dP, nD2)));
      }
      if (t > 0 && !mbar_wait_warp(out_free, (t - 1) & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_st16(tO, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(out_full);
    }
    // ------------------------------------------------------------------ epilogue
    float along, odd;
    f2_to(along2, along, odd);
    s_along[wg * kTile + r] = along + odd;
    named_bar_sync(1, kWarps * 32);
    const float D = s_along[2 * m * kTile + r] + s_along[(2 * m + 1) * kTile + r];
    if (wg & 1) {
      if (row_ok) rowv[(2 + m) * kTile] = -D;
    } else if (m == 1) {
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
    if (ok && mbar_wait_warp(out_free, (steps - 1) & 1, ab)) {
      tc_fence_after();
      // half of dQm's columns; dS2 was formed without its weight, a factor of the row
      const float by = m ? rowv[4 * kTile] * p.scale : p.scale;
      __nv_bfloat16 *out =
          p.dq + (((size_t)b * p.S + row) * 2 * p.H + 2 * h + m) * d + (wg & 1) * (d / 2);
      uint32_t v[d / 2];
      if constexpr (d == 64)
        tmem_ld32(tmem + lane_off + L::tAcc + m * 64 + (wg & 1) * 32, v);
      else
        tmem_ld16(tmem + lane_off + L::tAcc + m * 64 + (wg & 1) * 16, v);
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

// Weights per head: the tiles' sums of one head, added in a fixed order.
__global__ void __launch_bounds__(256) diff_dlam_kernel(const DiffBwdParams p) {
  __shared__ float s[8];
  const int h = blockIdx.x;
  float v = 0.f;
  for (int k = threadIdx.x; k < p.B * p.N; k += 256)
    v += p.dlam_part[((size_t)(k / p.N) * p.H + h) * p.N + k % p.N];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.f;
    for (int k = 0; k < 8; ++k) v += s[k];
    if (p.lam_f32)
      static_cast<float *>(p.dlam)[h] = v;
    else
      static_cast<__nv_bfloat16 *>(p.dlam)[h] = __float2bfloat16_rn(v);
  }
}

// -------------------------------------------------------------------- dK, dV
// CTA: a 128-key block of one KV head, over the query heads of its group and their tiles in
// ascending order, in steps of 64 queries with everything transposed (thread = key row, so
// the bf16 operands P^T, dS1^T go back to TMEM where their rows are):
//   dV [0,dv)  dK1 [128,128+d) dK2 [192,192+d)
//   in: S1^T [256,320) S2^T [320,384) dP^T [384,448)   out: P^T [448,480) dS1^T [480,512)
// The step's inputs go to registers at once, which frees their columns for the next step's
// products; dS2^T finds no room in TMEM and goes through shared memory.  The four warpgroups
// share a step's queries (16 each).
constexpr int kQueries = 64;

template <int d>
struct DkvL {
  static constexpr int DV = 2 * d;
  static constexpr int kStages = 2;
  static constexpr int kTileBytes = DV * kTile * 2;
  static constexpr int kBoxes = DV / kBoxCols;
  static constexpr int kRowBytes = kRowVecs * kTile * 4;
  static constexpr int offK = 0, offV = kTileBytes;
  static constexpr int offStage = 2 * kTileBytes;  // per stage Q, dO
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int offDS = offStage + kStages * kStageBytes;  // dS2^T, one box
  static constexpr int offRow = offDS + kBoxBytes;                // per stage row vectors
  static constexpr int offBar = offRow + kStages * kRowBytes;
  // kv_full, q_full[2], q_empty[2], in_full, in_free, out_full, out_free, acc_full, drain
  static constexpr int kNumBars = 1 + 2 * kStages + 6;
  static constexpr int offMisc = offBar + kNumBars * 8;
  static constexpr int kBytes = offMisc + 16;
  static constexpr uint32_t tV = 0, tK = 128, tIn = 256, tP = 448, tDS = 480, kTmemCols = 512;
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
  uint64_t *in_full = q_empty + L::kStages, *in_free = in_full + 1, *out_full = in_full + 2;
  uint64_t *out_free = in_full + 3, *acc_full = in_full + 4, *drain = in_full + 5;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + L::offMisc);
  int *s_abort = reinterpret_cast<int *>(smem + L::offMisc + 4);
  const Abort ab{s_abort, p.status, p.wait_ns};
  const int warp = warp_id(), lane = lane_id();

  const int heads = p.B * p.Hkv;
  const int j = blockIdx.x / heads;  // causal: block 0 meets the most queries, first
  const int bh = blockIdx.x % heads;
  const int hkv = bh % p.Hkv, b = bh / p.Hkv;
  const int i0 = p.causal ? j : 0, tiles = p.N - i0;
  const int stages = p.G * tiles;
  // the last tile has one step where S ends in its first half
  const int last_steps = p.S - (p.N - 1) * kTile > kQueries ? 2 : 1;
  const int steps = p.G * (2 * (tiles - 1) + last_steps);
  // advances (tile, half) to the next step; true where a new stage begins
  auto next = [&](int &i, int &u) {
    if (++u < (i == p.N - 1 ? last_steps : 2)) return false;
    u = 0;
    if (++i == p.N) i = i0;
    return true;
  };

  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], kWarps + 1);  // the products' commit, the readers of row vectors
    }
    mbar_init(in_full, 1);
    mbar_init(in_free, kWarps);
    mbar_init(out_full, kWarps);
    mbar_init(out_free, 1);
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
    for (int n = 0; n < stages; ++n) {
      const int s = n % L::kStages;
      const uint32_t ph = (n / L::kStages) & 1;
      if (!mbar_wait(&q_empty[s], ph ^ 1, ab)) {
        ok = false;
        break;
      }
      const int h = hkv * p.G + n / tiles, i = i0 + n % tiles;
      mbar_arrive_expect_tx(&q_full[s], L::kStageBytes + L::kRowBytes);
      uint8_t *sq = smem + L::offStage + s * L::kStageBytes;
      for (int bx = 0; bx < L::kBoxes; ++bx) {
        tma_load_4d(sq + bx * kBoxBytes, &tm_q, &q_full[s], bx * kBoxCols, h, i * kTile, b);
        tma_load_4d(sq + L::kTileBytes + bx * kBoxBytes, &tm_do, &q_full[s], bx * kBoxCols, h,
                    i * kTile, b);
      }
      bulk_load(smem + L::offRow + s * L::kRowBytes,
                p.rowv + (((size_t)b * p.H + h) * p.N + i) * (kRowVecs * kTile), L::kRowBytes,
                &q_full[s]);
      last[s] = (int)ph;
    }
    if (!ok) {
      mbar_wait_drain(kv_full, 0, 100000000ull);
      for (int s = 0; s < L::kStages; ++s)
        if (last[s] >= 0) mbar_wait_drain(&q_full[s], (uint32_t)last[s], 100000000ull);
    }
  } else if (warp == kWarps + 1) {
    // ------------------------------------------------------------------ MMA issuer
    // (a converged warp, one elected lane issues)
    constexpr uint32_t kIdescIn = make_idesc_bf16(128, kQueries, false, false);
    constexpr uint32_t kIdescV = make_idesc_bf16(128, DV, false, true);
    constexpr uint32_t kIdescK = make_idesc_bf16(128, d, false, true);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t loK = desc_lo(sbase + L::offK, 16), loV = desc_lo(sbase + L::offV, 16);
    const uint32_t loDS = desc_lo(sbase + L::offDS, 16);
    auto step_at = [&](int n, int u) {  // Q rows of half u of stage n
      return sbase + L::offStage + (n % L::kStages) * L::kStageBytes + u * (kQueries * 128);
    };
    // S1^T, S2^T and dP^T of half u of stage n
    auto issue_in = [&](int n, int u) -> bool {
      if (u == 0 && !mbar_wait_warp(&q_full[n % L::kStages], (n / L::kStages) & 1, ab))
        return false;
      tc_fence_after();
      const uint32_t loQ = desc_lo(step_at(n, u), 16);
      const uint32_t loO = desc_lo(step_at(n, u) + L::kTileBytes, 16);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int k = 0; k < d / 16; ++k) {
          const uint32_t off = col_bytes(m * d + 16 * k) >> 4;
          mma_ss_e(tmem + L::tIn + m * 64, desc_of(loK + off), desc_of(loQ + off), kIdescIn, k > 0);
        }
#pragma unroll
      for (int k = 0; k < DV / 16; ++k) {
        const uint32_t off = col_bytes(16 * k) >> 4;
        mma_ss_e(tmem + L::tIn + 128, desc_of(loV + off), desc_of(loO + off), kIdescIn, k > 0);
      }
      mma_commit_e(in_full);
      return true;
    };
    bool ok = mbar_wait_warp(kv_full, 0, ab) && issue_in(0, 0);
    int i = i0, u = 0, n = 0;     // step t
    int i1 = i0, u1 = 0, n1 = 0;  // step t + 1
    if (next(i1, u1)) ++n1;
    for (int t = 0; ok && t < steps; ++t) {
      if (t + 1 < steps && !(mbar_wait_warp(in_free, t & 1, ab) && issue_in(n1, u1))) {
        ok = false;
        break;
      }
      if (!mbar_wait_warp(out_full, t & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t loQ = desc_lo(step_at(n, u), kBoxBytes);
      const uint32_t loO = desc_lo(step_at(n, u) + L::kTileBytes, kBoxBytes);
      const uint32_t first = t > 0 ? 1u : 0u;
#pragma unroll
      for (int k = 0; k < kQueries / 16; ++k)
        mma_ts_e(tmem + L::tV, tmem + L::tP + 8 * k, desc_of(loO + ((k * 2048) >> 4)), kIdescV,
                 k > 0 ? 1u : first);
#pragma unroll
      for (int k = 0; k < kQueries / 16; ++k)
        mma_ts_e(tmem + L::tK, tmem + L::tDS + 8 * k, desc_of(loQ + ((k * 2048) >> 4)), kIdescK,
                 k > 0 ? 1u : first);
#pragma unroll
      for (int k = 0; k < kQueries / 16; ++k)
        mma_ss_e(tmem + L::tK + 64, desc_of(loDS + ((k * 32) >> 4)),
                 desc_of(loQ + ((col_bytes(d) + k * 2048) >> 4)), kIdescK, k > 0 ? 1u : first);
      mma_commit_e(out_free);
      const int s = n % L::kStages;
      if (next(i, u)) {
        ++n;
        mma_commit_e(&q_empty[s]);
      }
      if (next(i1, u1)) ++n1;
    }
    if (ok) mma_commit_e(acc_full);
    mma_commit_e(drain);
    mbar_wait_drain(drain, 0, 100000000ull);
  } else if (warp < kWarps) {
    // ------------------------------------------------------------------ P, dS (transposed)
    const int wg = warp >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // key row within the block = TMEM lane
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tI = tmem + lane_off + L::tIn + 16 * wg;
    const int key = j * kTile + r;
    uint8_t *ds_row = smem + L::offDS + r * 128;
    const f2 c2 = f2_of(p.scale_log2, p.scale_log2);
    bool ok = true;
    int i = i0, u = 0, n = 0;
    for (int t = 0; t < steps; ++t) {
      if (!mbar_wait_warp(in_full, t & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t s1[16], s2[16], g[16];
      tmem_ld16(tI, s1);
      tmem_ld16(tI + 64, s2);
      tmem_ld16(tI + 128, g);
      tmem_ld_wait_for(s1);
      tmem_ld_wait_for(s2);
      tmem_ld_wait_for(g);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(in_free);
      const int s = n % L::kStages;
      const int q0 = u * kQueries + 16 * wg;  // first query within the tile
      const float *rv = reinterpret_cast<const float *>(smem + L::offRow + s * L::kRowBytes) + q0;
      // queries before this key see nothing of it
      const int from = p.causal && i == j ? r - q0 : 0;
      if (__any_sync(0xffffffffu, from > 0)) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (e < from) s1[e] = s2[e] = __float_as_uint(-INFINITY), g[e] = 0u;
      }
      uint32_t pP[8], p1[8], p2[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // row vectors of four queries, the same for every lane
        ulonglong2 v[kRowVecs];
#pragma unroll
        for (int k = 0; k < kRowVecs; ++k)
          v[k] = *reinterpret_cast<const ulonglong2 *>(rv + k * kTile + 4 * e);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int c = 4 * e + 2 * z;
          auto at = [&](int k) { return z ? v[k].y : v[k].x; };
          const f2 P1 = ex2_2(fma2(f2_of(s1[c], s1[c + 1]), c2, at(0)));
          const f2 w = mul2(ex2_2(fma2(f2_of(s2[c], s2[c + 1]), c2, at(1))), at(4));  // -lam P2
          const f2 dP = f2_of(g[c], g[c + 1]);
          pP[2 * e + z] = pack_bf16(add2(P1, w));
          p1[2 * e + z] = pack_bf16(mul2(P1, add2(dP, at(2))));
          p2[2 * e + z] = pack_bf16(mul2(w, add2(dP, at(3))));
        }
      }
      if (t > 0 && !mbar_wait_warp(out_free, (t - 1) & 1, ab)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_st8(tmem + lane_off + L::tP + 8 * wg, pP);
      tmem_st8(tmem + lane_off + L::tDS + 8 * wg, p1);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4 *>(ds_row + (((2 * wg + c) ^ (r & 7)) << 4)) =
            make_uint4(p2[4 * c], p2[4 * c + 1], p2[4 * c + 2], p2[4 * c + 3]);
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(out_full);
      if (next(i, u)) {
        ++n;
        if (lane == 0) mbar_arrive(&q_empty[s]);
      }
    }
    if (ok && mbar_wait_warp(acc_full, 0, ab)) {
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
        if (key < p.S) store_row(out + 32 * c, v, wg < 2 ? p.scale : 1.f);
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
                     const CUtensorMap &tdo, const __nv_bfloat16 *q,
                     const DiffBwdParams &p, cudaStream_t s) {
  using LQ = DqL<d>;
  using LK = DkvL<d>;
  cudaError_t e = cudaFuncSetAttribute(diff_dq_kernel<d>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, LQ::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(diff_dkv_kernel<d>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             LK::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned tiles = (unsigned)p.B * p.H * p.N;
  diff_rows_kernel<d><<<tiles, 256, 0, s>>>(p);
  diff_dq_kernel<d><<<tiles, kThreads, LQ::kBytes, s>>>(tk, tv, q, p);
  if (!p.lam_token) diff_dlam_kernel<<<p.H, 256, 0, s>>>(p);
  diff_dkv_kernel<d>
      <<<(unsigned)p.B * p.Hkv * p.N, kThreads, LK::kBytes, s>>>(tq, tk, tv, tdo, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_bwd(int d, const CUtensorMap &tq, const CUtensorMap &tk,
                            const CUtensorMap &tv, const CUtensorMap &tdo, const __nv_bfloat16 *q,
                            const DiffBwdParams &p, cudaStream_t s) {
  return d == 32 ? launch_t<32>(tq, tk, tv, tdo, q, p, s) : launch_t<64>(tq, tk, tv, tdo, q, p, s);
}

}  // namespace dash
