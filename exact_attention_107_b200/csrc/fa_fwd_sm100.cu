// fa_fwd_sm100.cu -- bf16 / fp16 attention forward on the sm_100a tensor cores.
//
// Computes O = softmax(scale * Q K^T [causal]) V and lse = ln(sum_j exp(scale * q.k_j))
// with the tiled, online-softmax scheme of "LLM paper notes #8: FlashAttention"
// (adg.csdn.net), sections "tiling" and "online softmax", and of "CUDA-kernel-level
// optimisation: why Flash Attention is 5-10x faster than native PyTorch"
// (guanweilu.cn), section "three tricks": Q/K/V tiles are staged on chip, each
// query row keeps a running max m and sum l, the output accumulated so far is
// rescaled when m grows, and it is normalised once at the end.  No N x N matrix
// ever reaches device memory.
//
// B200 mapping (one CTA per SM, 384 threads, 2 query tiles of 128 rows per CTA):
//   warp 0      TMA producer: Q tiles once, then K_j / V_j through a shared-memory ring
//   warp 1      MMA issuer (one thread): S_t = Q_t K_j^T into tensor memory, then
//               O_t += P_t V_j with P_t read straight from tensor memory
//   warps 4-7   softmax for query tile 0 (thread r owns query row r = TMEM lane r)
//   warps 8-11  softmax for query tile 1
// The MMA thread interleaves the two tiles (S_0, S_1, PV_0, S_0', PV_1, S_1', ...)
// so one tile's softmax overlaps the other tile's matrix products.
//
// Tensor memory (512 columns): S_0 [0,128), S_1 [128,256), O_0 [256,256+D),
// O_1 [256+D, 256+2D).  P_t (16-bit, two per 32-bit column) overwrites the first 64
// columns of S_t once the scores have been read into registers.  P_t takes the
// element type of the inputs (bf16, or fp16 when F16), as the tensor-core operands
// of one MMA share one type.  It is written and announced in two halves of 64 keys,
// and the MMA thread issues the first half's P V products while the softmax computes
// the second half.
//
// Online-softmax detail: the running max used for the exponentials is only raised
// when a new row max exceeds it by more than 2^8 (in exp2 units).  Numerator and
// denominator then share the same, possibly stale, reference, so the normalised
// result is unchanged while most O rescales (a TMEM round trip) are skipped; the
// un-normalised probabilities stay below 2^8.
#include <cstdint>
#include <math_constants.h>

#include "fa_internal.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;            // query rows per tile (= TMEM lanes)
constexpr int kBN = 128;            // keys per tile
constexpr int kThreads = 384;
constexpr float kRescaleThreshold = 8.0f;
// All exponentials of the forward go to the MUFU unit: with two softmax warps per SMSP
// the FMA-pipe polynomial (exp2_poly2) gave no measurable gain here (it does in the
// backward, whose phases run four warps per SMSP).
template <int D>
__device__ __forceinline__ bool poly_pair(int) { return false; }
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

template <int D>
struct FwdSmem {
  static constexpr int kStages = (D == 128) ? 2 : 4;
  static constexpr int kBox = 128 * 64 * 2;      // 128 rows x 64 16-bit values: one 128-byte swizzle span
  static constexpr int kNBox = D / 64;
  static constexpr int kTile = kBox * kNBox;     // one 128-row tile of Q, K, V (or O staging)
  static constexpr int kOffQ = 0;                // 2 query tiles (reused to stage O)
  static constexpr int kOffK = kOffQ + 2 * kTile;
  static constexpr int kOffV = kOffK + kStages * kTile;
  static constexpr int kOffBar = kOffV + kStages * kTile;
  static constexpr int kBarQFull = 0;
  static constexpr int kBarKFull = 1;
  static constexpr int kBarKEmpty = kBarKFull + kStages;
  static constexpr int kBarVFull = kBarKEmpty + kStages;
  static constexpr int kBarVEmpty = kBarVFull + kStages;
  static constexpr int kBarSFull = kBarVEmpty + kStages;  // [2]
  static constexpr int kBarPFull = kBarSFull + 2;         // [half][tile]: P of keys [64h, 64h+64)
  static constexpr int kBarOFull = kBarPFull + 4;         // [2]
  static constexpr int kBarMmaDone = kBarOFull + 2;
  static constexpr int kNumBars = kBarMmaDone + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kNumBars;  // TMEM base address, then abort flag
  // + slack for 1024-byte alignment; at least 120 KB so that only one CTA (which
  // holds all 512 tensor-memory columns) is ever resident per SM.
  static constexpr int kBytes = (kOffSlot + 16 + 1024) > 122880 ? (kOffSlot + 16 + 1024) : 122880;
  static_assert(kBytes <= 232448, "shared memory budget");
};

// The score-modified instances (MOD) run the same pipeline with, per batch element, query rows
// that see an interval of keys each (a mask plan, or full / causal), key-value heads shared by
// H / Hkv query heads, and optionally
//   CAP    x = cap tanh(s / cap), s = scale q.k.  The score registers are replaced by the tanh and
//          the softmax runs on cap log2e tanh.  Two MUFU operations a score for an accurate tanh
//          next to the exponential's one made the MUFU unit the limit (B1 H8 N16384 D128 causal:
//          1176 us against 483 without a cap); scores up to 0.75 cap, as nearly all are, take a
//          polynomial on the FMA pipe instead (a warp's choice for its 32 rows of a tile).
//   ALIBI  x -= slope_h |i - j|, in fp32, joined to the exponent.
// At that size 469 us plain, 647 capped, 638 with a bias, 875 with both.  The capped instances spill
// 28 bytes of the 168 registers a thread, those with a bias too 80 to 84.
// Rows that see nothing get O = 0 and lse = -inf.
template <int D, bool CAUSAL, bool F16, bool MOD, bool CAP, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                    float* __restrict__ lse, int N, int BH, int nqb, int hg, float scale_log2, int* status,
                    const __grid_constant__ ScoreMods mods) {
  using L = FwdSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8 * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Work item: 256 query rows (two tiles) of one (batch, head).  Causal work grows
  // with the query index, so the heaviest blocks are handed out first.
  int qblk, bh;
  {
    const WorkItem wi = grouped_order(static_cast<int>(blockIdx.x), BH, nqb, hg);
    bh = wi.bh;
    qblk = (CAUSAL || MOD) ? nqb - 1 - wi.tile : wi.tile;
  }
  const int nkv_all = (N + kBN - 1) / kBN;
  // Query tile t meets the key tiles j0 + [ka[t], ka[t] + nkv[t]); j0 is the first key tile that
  // either meets, 0 without a mask plan.
  int q0[2], ka[2] = {0, 0}, nkv[2], j0 = 0;
  int kv_bh = bh, batch = 0;
  if constexpr (MOD) {
    batch = bh / mods.H;
    if (mods.plan != nullptr)
      qblk = mask_plan_view(mods.plan, BH / mods.H, N).order[static_cast<size_t>(batch) * nkv_all + (nqb - 1 - qblk)].y;
    kv_bh = batch * mods.Hkv + (bh - batch * mods.H) / (mods.H / mods.Hkv);
  }
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    q0[t] = qblk * 2 * kBM + t * kBM;
    const bool causal = MOD ? mods.causal != 0 : CAUSAL;
    nkv[t] = (q0[t] >= N) ? 0 : (causal ? min(nkv_all, q0[t] / kBN + 1) : nkv_all);
    if constexpr (MOD) {
      if (mods.plan != nullptr && q0[t] < N) {
        const int4 tl = mask_plan_view(mods.plan, BH / mods.H, N).tiles[static_cast<size_t>(batch) * nkv_all + q0[t] / kBM];
        ka[t] = tl.x;
        nkv[t] = tl.y - tl.x;
      }
    }
  }
  int nkv_max = max(nkv[0], nkv[1]);
  if constexpr (MOD) {
    j0 = nkv[0] == 0 ? ka[1] : (nkv[1] == 0 ? ka[0] : min(ka[0], ka[1]));
#pragma unroll
    for (int t = 0; t < 2; ++t) ka[t] = nkv[t] == 0 ? 0 : ka[t] - j0;
    nkv_max = max(ka[0] + nkv[0], ka[1] + nkv[1]);
  }

  if (threadIdx.x == 0) {
    mbar_init(bar(L::kBarQFull), 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarKFull + s), 1);
      mbar_init(bar(L::kBarKEmpty + s), 1);
      mbar_init(bar(L::kBarVFull + s), 1);
      mbar_init(bar(L::kBarVEmpty + s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(L::kBarSFull + t), 1);
      mbar_init(bar(L::kBarPFull + t), kBM);
      mbar_init(bar(L::kBarPFull + 2 + t), kBM);
      mbar_init(bar(L::kBarOFull + t), 1);
    }
    mbar_init(bar(L::kBarMmaDone), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    FA_CONVERGED(status);
    tmem_alloc(smem_u32(slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *slot;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmO);
      uint32_t qbytes = 0;
      for (int t = 0; t < 2; ++t)
        if (nkv[t] > 0) qbytes += L::kTile;
      mbar_arrive_expect_tx(bar(L::kBarQFull), qbytes);
      for (int t = 0; t < 2; ++t)
        if (nkv[t] > 0)
          for (int c = 0; c < L::kNBox; ++c)
            tma_load_3d(sb + L::kOffQ + t * L::kTile + c * L::kBox, &tmQ, bar(L::kBarQFull), c * 64, q0[t], bh);
      int nk = 0, nv = 0;
      bool ok = true;
      for (int j = 0; j < nkv_max; ++j) {
        const int s = j % L::kStages;
        const uint32_t ph = (j / L::kStages) & 1;
        if (!(ok = mbar_wait(bar(L::kBarKEmpty + s), ph ^ 1, abort_flag))) break;
        mbar_arrive_expect_tx(bar(L::kBarKFull + s), L::kTile);
        for (int c = 0; c < L::kNBox; ++c)
          tma_load_3d(sb + L::kOffK + s * L::kTile + c * L::kBox, &tmK, bar(L::kBarKFull + s), c * 64, (j0 + j) * kBN, kv_bh);
        ++nk;
        if (!(ok = mbar_wait(bar(L::kBarVEmpty + s), ph ^ 1, abort_flag))) break;
        mbar_arrive_expect_tx(bar(L::kBarVFull + s), L::kTile);
        for (int c = 0; c < L::kNBox; ++c)
          tma_load_3d(sb + L::kOffV + s * L::kTile + c * L::kBox, &tmV, bar(L::kBarVFull + s), c * 64, (j0 + j) * kBN, kv_bh);
        ++nv;
      }
      if (!ok) raise_error(status, abort_flag, kStatusTimeout);
      // Never leave with copies in flight: wait for the last load of every stage.
      mbar_wait_drain(bar(L::kBarQFull), 0);
      for (int j = max(0, nk - L::kStages); j < nk; ++j)
        mbar_wait_drain(bar(L::kBarKFull + j % L::kStages), (j / L::kStages) & 1);
      for (int j = max(0, nv - L::kStages); j < nv; ++j)
        mbar_wait_drain(bar(L::kBarVFull + j % L::kStages), (j / L::kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_16(kBM, kBN, false, false, F16);  // Q, K both K-major
      constexpr uint32_t kIdO = idesc_16(kBM, D, false, true, F16);    // P from TMEM, V MN-major
      // Each 64-column box of Q_t and K_j holds four K-steps of 16 (32 bytes apart).
      auto issue_s = [&](int t, int j) {
        const uint32_t qa = sb + L::kOffQ + t * L::kTile;
        const uint32_t kb = sb + L::kOffK + (j % L::kStages) * L::kTile;
#pragma unroll
        for (int c = 0; c < L::kNBox; ++c)
          mma_ss_x4<2, 4, 6, 2, 4, 6>(tmem + t * 128, sdesc_sw128(qa + c * L::kBox, 16, 1024),
                                      sdesc_sw128(kb + c * L::kBox, 16, 1024), kIdS, c > 0 ? 1u : 0u);
        tc_commit(bar(L::kBarSFull + t));
      };
      // O_t += P_t V_j over keys [64h, 64h+64): K-steps 4h .. 4h+3, each 8 packed P columns
      // and 16 V rows (2048 bytes) further on.
      auto issue_pv = [&](int t, int j, int h) {
        const uint32_t vb = sb + L::kOffV + (j % L::kStages) * L::kTile;
        mma_ts_x4<8, 16, 24, 128, 256, 384>(tmem + 256 + t * D, tmem + t * 128 + 32 * h,
                                            sdesc_sw128(vb + h * 4 * 2048, L::kBox, 1024), kIdO,
                                            (j > ka[t] || h > 0) ? 1u : 0u);
      };
      bool ok = mbar_wait_spin(bar(L::kBarQFull), 0, abort_flag);
      if (ok && nkv_max > 0) {
        ok = mbar_wait_spin(bar(L::kBarKFull), 0, abort_flag);
        if (ok) {
          tc_fence_after();
          for (int t = 0; t < 2; ++t)
            if (nkv[t] > 0 && ka[t] == 0) issue_s(t, 0);
          tc_commit(bar(L::kBarKEmpty));
        }
      }
      for (int j = 0; ok && j < nkv_max; ++j) {
        const int s = j % L::kStages;
        if (!(ok = mbar_wait_spin(bar(L::kBarVFull + s), (j / L::kStages) & 1, abort_flag))) break;
        tc_fence_after();
        bool k_next = false;
        for (int t = 0; t < 2; ++t) {
          if (j >= ka[t] + nkv[t]) continue;
          if (!MOD || j >= ka[t]) {
            // P_t arrives in two halves; the first half's products start while the
            // softmax still computes the second.
            const uint32_t ph = static_cast<uint32_t>(j - ka[t]) & 1u;
            if (!(ok = mbar_wait_spin(bar(L::kBarPFull + t), ph, abort_flag))) break;
            tc_fence_after();
            issue_pv(t, j, 0);
            if (!(ok = mbar_wait_spin(bar(L::kBarPFull + 2 + t), ph, abort_flag))) break;
            tc_fence_after();
            issue_pv(t, j, 1);
            if (j == ka[t] + nkv[t] - 1) tc_commit(bar(L::kBarOFull + t));
          }
          if (j + 1 < ka[t] + nkv[t] && (!MOD || j + 1 >= ka[t])) {
            if (!k_next) {
              const int jn = j + 1;
              if (!(ok = mbar_wait_spin(bar(L::kBarKFull + jn % L::kStages), (jn / L::kStages) & 1, abort_flag)))
                break;
              tc_fence_after();
              k_next = true;
            }
            issue_s(t, j + 1);
          }
        }
        if (!ok) break;
        if constexpr (MOD) {
          // Neither tile meets key tile j + 1 (a gap between their ranges): release it unread.
          if (!k_next && j + 1 < nkv_max) {
            const int jn = j + 1;
            if (!(ok = mbar_wait_spin(bar(L::kBarKFull + jn % L::kStages), (jn / L::kStages) & 1, abort_flag))) break;
            k_next = true;
          }
        }
        tc_commit(bar(L::kBarVEmpty + s));
        if (k_next) tc_commit(bar(L::kBarKEmpty + (j + 1) % L::kStages));
      }
      if (!ok) raise_error(status, abort_flag, kStatusTimeout);
      // Every MMA this thread issued has finished before tensor memory is released.
      tc_commit(bar(L::kBarMmaDone));
      mbar_wait_drain(bar(L::kBarMmaDone), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax + epilogue
    const int t = (warp - 4) >> 2;
    const int r = threadIdx.x - kBM * (t + 1);                  // row in tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128;
    const uint32_t tO = tmem + lane_off + 256 + t * D;
    const int qrow = q0[t] + r;
    float m = -CUDART_INF_F, l = 0.f;
    // MOD: the keys [lo, hi) that this row sees (none for rows past N).
    int lo = 0, hi = 0;
    float slope2 = 0.f, cap_in = 0.f;                     // slope * log2e; scale / cap
    float softmax_scale = scale_log2;                     // multiplies the score registers in the exponent
    if constexpr (MOD) {
      if (qrow < N) {
        hi = mods.causal ? qrow + 1 : N;
        if (mods.plan != nullptr) {
          const int2 iv = mask_plan_view(mods.plan, BH / mods.H, N).rows[static_cast<size_t>(batch) * nkv_all * kBN + qrow];
          lo = iv.x;
          hi = iv.y;
        }
      }
      if (CAP) {
        cap_in = scale_log2 * kLn2 / mods.softcap;
        softmax_scale = mods.softcap * kLog2e;
      }
      if (ALIBI) slope2 = mods.slopes[bh - batch * mods.H] * kLog2e;
    }
    bool ok = true;
    for (int j = 0; j < nkv[t]; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSFull + t), j & 1, abort_flag));
      if (!ok) break;
      FA_CONVERGED(status);                                     // warp-collective TMEM loads follow
      tc_fence_after();
      uint32_t sr[4][32];
      tmem_ld32(tS, sr[0]);
      tmem_ld32(tS + 32, sr[1]);
      tmem_ld32(tS + 64, sr[2]);
      tmem_ld32(tS + 96, sr[3]);
      tmem_ld_wait();
      reg_fence(sr[0]);
      reg_fence(sr[1]);
      reg_fence(sr[2]);
      reg_fence(sr[3]);
      const int kv0 = MOD ? (j0 + ka[t] + j) * kBN : j * kBN;
      const bool diag = CAUSAL && (kv0 + kBN - 1 > q0[t]);
      // The score registers stay raw (masked ones -inf): the maximum is found on them, and the
      // exponentials' arguments are formed on the fly.
      if constexpr (CAP) {
        float most[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kBN; c += 2)
          most[(c >> 1) & 1] = fmax3_abs(most[(c >> 1) & 1], __uint_as_float(sr[c >> 5][c & 31]),
                                         __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]));
        if (!__all_sync(0xffffffffu, fmaxf(most[0], most[1]) <= mods.poly_limit)) {
          // Rare, and so a loop through tensor memory that costs the other tiles no register: scores
          // beyond the polynomial's range become those for which it gives their tanh.
          FA_CONVERGED(status);
          const float out_in = cap_in > 0.f ? 1.f / cap_in : 0.f;
#pragma unroll 1
          for (int c = 0; c < kBN; c += 16) {
            uint32_t x[16];
            tmem_ld16(tS + c, x);
            tmem_ld_wait();
            reg_fence(x);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float z = __uint_as_float(x[e]) * cap_in, th = tanh_any(z), far = quartic_inverse(fabsf(th)) * out_in;
              x[e] = mods.poly_limit < 0.f ? __float_as_uint(th)
                     : fabsf(z) <= kTanhPolyLimit ? x[e] : __float_as_uint(copysignf(far, z));
            }
            tmem_st16(tS + c, x);
          }
          tmem_st_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, sr[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) reg_fence(sr[q]);
        }
      }
      // ALIBI: the bias is linear in the column where every visible key of the tile lies on one side
      // of the warp's rows: growing by s2 a column, slope2 to the left and -slope2 to the right.
      bool one_side = true;
      float s2 = 0.f;
      if constexpr (ALIBI) {
        const bool right = kv0 >= qrow - lane + 31;
        one_side = right || __all_sync(0xffffffffu, kv0 + kBN - 1 <= qrow || hi <= qrow + 1);
        s2 = right ? -slope2 : slope2;
        if (!CAP && !one_side) {
          // Keys to both sides (around the diagonal, without a causal mask): the scores to the right
          // take the difference to the left side's bias, in a loop through tensor memory as above.
          FA_CONVERGED(status);
          const float per = -2.f * slope2 / softmax_scale;
#pragma unroll 1
          for (int c = 0; c < kBN; c += 16) {
            uint32_t x[16];
            tmem_ld16(tS + c, x);
            tmem_ld_wait();
            reg_fence(x);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = __float_as_uint(fmaf(per, static_cast<float>(max(kv0 + c + e - qrow, 0)), __uint_as_float(x[e])));
            tmem_st16(tS + c, x);
          }
          tmem_st_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, sr[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 4; ++q) reg_fence(sr[q]);
          one_side = true;
        }
      }
      if constexpr (MOD) {
        if (!__all_sync(0xffffffffu, lo <= kv0 && hi >= kv0 + kBN)) {
          const int first = lo - kv0;
          const unsigned width = static_cast<unsigned>(hi - lo);          // keep first <= c < first + width
#pragma unroll
          for (int c = 0; c < kBN; ++c)
            if (static_cast<unsigned>(c - first) >= width) sr[c >> 5][c & 31] = 0xff800000u;   // -inf
        }
      } else if (diag || kv0 + kBN > N) {
        const int lim = min(CAUSAL ? qrow - kv0 : kBN - 1, N - 1 - kv0);   // keep columns c <= lim
#pragma unroll
        for (int c = 0; c < kBN; ++c)
          if (c > lim) sr[c >> 5][c & 31] = 0xff800000u;                  // -inf
      }
      // log2e cap tanh(score / cap) or log2e score, of a pair
      auto scaled = [&](float2 v) {
        if constexpr (CAP) return __fmul2_rn(v, quartic2(v, mods.poly));
        return make_float2(v.x * softmax_scale, v.y * softmax_scale);
      };
      float m_tile, slack = 0.f;                         // the tile's maximum is at most `slack` above m_tile
      if constexpr (ALIBI) {
        // After its first tile a row's reference needs no exact maximum, only one that is not above it
        // (that would cost P bits) nor far below: of eight columns the largest score and the greatest
        // bias against it, at most `slack` too low.  The first reference is exact, so that a row of one
        // key has P = 1.  Slopes for which the slack is more than the rescaling threshold go column by
        // column throughout.
        const float d0 = static_cast<float>(qrow - kv0);
        float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
        bool exact = !one_side || fabsf(slope2) * 7.f > kRescaleThreshold;
        if (!exact) {
          slack = fabsf(slope2) * 7.f;
          const float base = fmaf(-s2, d0, s2 < 0.f ? 7.f * s2 : 0.f);
#pragma unroll
          for (int c = 0; c < kBN; c += 8) {
            const int q = c >> 5, e = c & 31;
            float v = fmax3(__uint_as_float(sr[q][e]), __uint_as_float(sr[q][e + 1]), __uint_as_float(sr[q][e + 2]));
            v = fmax3(v, __uint_as_float(sr[q][e + 3]), __uint_as_float(sr[q][e + 4]));
            v = fmax3(v, __uint_as_float(sr[q][e + 5]), fmaxf(__uint_as_float(sr[q][e + 6]), __uint_as_float(sr[q][e + 7])));
            const float bias = fmaf(s2, static_cast<float>(c), base);
            top[(c >> 3) & 1] = fmaxf(top[(c >> 3) & 1], (CAP ? scaled(make_float2(v, v)).x : v * softmax_scale) + bias);
          }
          exact = __any_sync(0xffffffffu, m == -CUDART_INF_F && fmaxf(top[0], top[1]) > -CUDART_INF_F);
        }
        if (exact) {
          slack = 0.f;
          top[0] = top[1] = -CUDART_INF_F;
#pragma unroll
          for (int c = 0; c < kBN; c += 2) {
            const float2 v = scaled(make_float2(__uint_as_float(sr[c >> 5][c & 31]),
                                                __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31])));
            const float e = d0 - static_cast<float>(c);
            top[0] = fmaxf(top[0], one_side ? fmaf(-s2, e, v.x) : fmaf(-slope2, fabsf(e), v.x));
            top[1] = fmaxf(top[1], one_side ? fmaf(-s2, e - 1.f, v.y) : fmaf(-slope2, fabsf(e - 1.f), v.y));
          }
        }
        m_tile = fmaxf(top[0], top[1]);
      } else {
        float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int c = 0; c < kBN; c += 2)
          mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(sr[c >> 5][c & 31]),
                                   __uint_as_float(sr[(c + 1) >> 5][(c + 1) & 31]));
        const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        m_tile = CAP ? scaled(make_float2(most, most)).x : most * scale_log2;
      }
      const float m_new = fmaxf(m, m_tile);
      const bool need = m_new + slack > m + kRescaleThreshold;             // always true at j == 0
      const float m_use = need ? m_new : m;
      const float alpha = need ? ex2_approx(m - m_new) : 1.f;
      const float neg = (m_use == -CUDART_INF_F) ? 0.f : -m_use;
      // P = exp2(s * scale * log2 e - m) in two halves of 64 keys; each half is stored as
      // packed 16-bit pairs over the first 32 + 32 columns of S_t (already read) and
      // announced on its own barrier, so the P V products of the first half overlap the
      // exponentials of the second.
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      // arg(c, s): the exponents of columns 2c and 2c + 1, whose scores are s
      auto exponentials = [&](auto arg) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // P of keys [64h, 64h+64) as packed pairs, stored 16 (CAP: 8) pairs at a time (nothing reads
          // them before this half's barrier arrival below), to keep the registers for S.
          constexpr int kPk = CAP ? 8 : 16;
#pragma unroll
          for (int hh = 0; hh < 32 / kPk; ++hh) {
            uint32_t pk[kPk];
#pragma unroll
            for (int c2 = 0; c2 < kPk; ++c2) {
              const int c = 32 * h + kPk * hh + c2;          // pair index: columns 2c, 2c + 1
              const float2 sv = make_float2(__uint_as_float(sr[(2 * c) >> 5][(2 * c) & 31]),
                                            __uint_as_float(sr[(2 * c + 1) >> 5][(2 * c + 1) & 31]));
              const float2 p = exp2_pair(arg(c, sv), poly_pair<D>(c));
              sum[c & 1] = __fadd2_rn(sum[c & 1], p);
              pk[c2] = pack16<F16>(p.x, p.y);
            }
            if constexpr (CAP) tmem_st8(tS + 32 * h + kPk * hh, pk);
            else tmem_st16(tS + 32 * h + kPk * hh, pk);
          }
          if (h == 0 && j > 0 && __any_sync(0xffffffffu, need)) {
            FA_CONVERGED(status);
            // Rescale O_t before any of this step's P V products lands in it (after the
            // first half's exponentials, whose scores no longer occupy registers).  O_t was
            // finished by the PV MMAs of step j-1: the commit that announced S_t(j) also
            // covers every earlier MMA of this thread, including those.
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                            make_float2(alpha, alpha));
                o[i] = __float_as_uint(v.x);
                o[i + 1] = __float_as_uint(v.y);
              }
              tmem_st32(tO + cc * 32, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(L::kBarPFull + 2 * h + t));
        }
      };
      const float2 sl2 = make_float2(softmax_scale, softmax_scale), neg2 = make_float2(neg, neg);
      if constexpr (!CAP && !ALIBI) {
        exponentials([&](int, float2 sv) { return __ffma2_rn(sv, sl2, neg2); });
      } else {
        auto exponent = [&](float2 sv, float2 add) {
          return __ffma2_rn(sv, CAP ? quartic2(sv, mods.poly) : sl2, add);
        };
        if constexpr (!ALIBI) {
          exponentials([&](int, float2 sv) { return exponent(sv, neg2); });
        } else {
          // bias - m: linear in the column, 16 columns by additions from a product (CAP, whose scores
          // cannot carry a bias: or |i - j| around the diagonal)
          const float d0 = static_cast<float>(qrow - kv0);
          if (!CAP || one_side) {
            float2 bias = make_float2(0.f, 0.f);
            exponentials([&](int c, float2 sv) {
              if (c % 8 == 0) {
                const float b0 = fmaf(s2, static_cast<float>(2 * c) - d0, neg);
                bias = make_float2(b0, b0 + s2);
              } else {
                bias = __fadd2_rn(bias, make_float2(2.f * s2, 2.f * s2));
              }
              return exponent(sv, bias);
            });
          } else {
            exponentials([&](int c, float2 sv) {
              const float e = d0 - static_cast<float>(2 * c);
              return exponent(sv, make_float2(fmaf(-slope2, fabsf(e), neg), fmaf(-slope2, fabsf(e - 1.f), neg)));
            });
          }
        }
      }
      l = l * alpha + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
      m = m_use;
    }
    if (ok && nkv[t] > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull + t), 0, abort_flag));
    if (!ok) {
      raise_error(status, abort_flag, kStatusTimeout);
    } else if (nkv[t] > 0 || (MOD && q0[t] < N)) {
      FA_CONVERGED(status);
      tc_fence_after();
      // Epilogue: O / l -> bf16 / fp16 into this warp's 32 rows of the (now idle) Q_t tile,
      // in the 128-byte-swizzled layout the O tensor map expects, then one TMA store
      // per warp (rows past N are clipped by the hardware).
      const float inv_l = (MOD && l == 0.f) ? 0.f : 1.f / l;      // a row that sees no key: O = 0
      uint8_t* stage = smem + L::kOffQ + t * L::kTile;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        if (!MOD || nkv[t] > 0) {
          tmem_ld32(tO + cc * 32, o);
          tmem_ld_wait();
          reg_fence(o);
        } else {                                                  // no product was ever added
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        const int box = cc >> 1;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int chunk = (cc & 1) * 4 + q4;
          uint4 v;
          v.x = pack16<F16>(__uint_as_float(o[8 * q4 + 0]) * inv_l, __uint_as_float(o[8 * q4 + 1]) * inv_l);
          v.y = pack16<F16>(__uint_as_float(o[8 * q4 + 2]) * inv_l, __uint_as_float(o[8 * q4 + 3]) * inv_l);
          v.z = pack16<F16>(__uint_as_float(o[8 * q4 + 4]) * inv_l, __uint_as_float(o[8 * q4 + 5]) * inv_l);
          v.w = pack16<F16>(__uint_as_float(o[8 * q4 + 6]) * inv_l, __uint_as_float(o[8 * q4 + 7]) * inv_l);
          *reinterpret_cast<uint4*>(stage + box * L::kBox + r * 128 + ((chunk ^ (r & 7)) << 4)) = v;
        }
      }
      fence_async_smem();
      __syncwarp();
      const int wrow = (warp & 3) * 32;
      if (lane == 0 && q0[t] + wrow < N) {
        for (int c = 0; c < L::kNBox; ++c)
          tma_store_3d(&tmO, sb + L::kOffQ + t * L::kTile + c * L::kBox + wrow * 128, c * 64, q0[t] + wrow, bh);
        bulk_commit();
        bulk_wait_read0();
      }
      if (qrow < N && FA_BOUNDS(static_cast<size_t>(bh) < static_cast<size_t>(BH), status))
        lse[static_cast<size_t>(bh) * N + qrow] = m * kLn2 + logf(l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    FA_CONVERGED(status);
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool CAUSAL, bool F16, bool MOD, bool CAP, bool ALIBI>
cudaError_t launch_impl(const FwdLaunch& a, const ScoreMods& m, cudaStream_t stream) {
  using L = FwdSmem<D>;
  auto kern = fwd_kernel<D, CAUSAL, F16, MOD, CAP, ALIBI>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int nqb = (a.N + 2 * kBM - 1) / (2 * kBM);
  const unsigned grid = static_cast<unsigned>(nqb) * static_cast<unsigned>(a.BH);
  const float scale_log2 = a.scale * 1.44269504088896340736f;
  kern<<<grid, kThreads, L::kBytes, stream>>>(a.tmQ, a.tmK, a.tmV, a.tmO, a.lse, a.N, a.BH, nqb, a.hg, scale_log2,
                                               a.status, m);
  return cudaGetLastError();
}

template <bool F16>
cudaError_t launch_typed(const FwdLaunch& a, cudaStream_t stream) {
  // Head dims 32 and 96 run the 64- and 128-column kernels: the tensor maps describe
  // the caller's D, so the TMA fills the missing columns of every loaded tile with
  // zeros (which add nothing to Q K^T and give zero columns of P V) and clips them
  // from every store.
  const ScoreMods none{};
  if (a.D <= 64)
    return a.causal ? launch_impl<64, true, F16, false, false, false>(a, none, stream)
                    : launch_impl<64, false, F16, false, false, false>(a, none, stream);
  return a.causal ? launch_impl<128, true, F16, false, false, false>(a, none, stream)
                  : launch_impl<128, false, F16, false, false, false>(a, none, stream);
}

template <int D, bool F16>
cudaError_t launch_mod_typed(const FwdLaunch& a, const ScoreMods& m, cudaStream_t stream) {
  const bool cap = m.softcap != 0.f, alibi = m.slopes != nullptr;
  if (cap)
    return alibi ? launch_impl<D, false, F16, true, true, true>(a, m, stream)
                 : launch_impl<D, false, F16, true, true, false>(a, m, stream);
  return alibi ? launch_impl<D, false, F16, true, false, true>(a, m, stream)
               : launch_impl<D, false, F16, true, false, false>(a, m, stream);
}

}  // namespace

cudaError_t launch_fwd_16(const FwdLaunch& a, cudaStream_t stream) {
  return a.f16 ? launch_typed<true>(a, stream) : launch_typed<false>(a, stream);
}

cudaError_t launch_fwd_mod(const FwdLaunch& a, const ScoreMods& mods, cudaStream_t stream) {
  ScoreMods m = mods;
  if (m.softcap != 0.f)
    set_cap_poly(&m, static_cast<double>(a.scale) / m.softcap, static_cast<double>(m.softcap) * kLog2e,
                 {kTanhC0, kTanhC1, kTanhC2, kTanhC3, kTanhC4}, kTanhPolyLimit);
  if (a.D <= 64) return a.f16 ? launch_mod_typed<64, true>(a, m, stream) : launch_mod_typed<64, false>(a, m, stream);
  return a.f16 ? launch_mod_typed<128, true>(a, m, stream) : launch_mod_typed<128, false>(a, m, stream);
}

}  // namespace fa
