// fa_bwd_fused_sm100.cu -- the attention backward in one pass over the key tiles: dK, dV and dQ.
//
// The backward recomputes P from the saved logsumexp instead of storing it ("LLM paper
// notes #8: FlashAttention", adg.csdn.net, section "recomputation"; "CUDA-kernel-level
// optimisation: why Flash Attention is 5-10x faster than native PyTorch", guanweilu.cn,
// section "three tricks").  With s = scale * q.k and P_ij = exp(s_ij - lse_i):
//     dV = P^T dO,  dP = dO V^T,  dS = P * (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
//
// One CTA per 128-key tile j (K_j, V_j resident in shared memory) walks the query tiles i,
// streaming Q_i and dO_i through two rings, and per tile pair issues five tcgen05 GEMMs:
//   S^T  = K_j Q_i^T        dP^T = V_j dO_i^T        (M = 128 keys, N = 128 queries)
//   dV_j += P^T dO_i        dK_j += dS^T Q_i          (A = packed 16-bit P^T / dS^T in tensor memory)
//   dQ_i  = dS_i K_j                                  (A = dS^T staged in shared memory, read MN-major)
// 512 threads (four warpgroups, 32 query columns each) turn S^T into P^T and dP^T into
// dS^T, and drain each dQ_i from tensor memory into an fp32 accumulator in device memory
// with vector reductions performed in L2 (red.global.add.v4.f32).  dq_finish then scales
// the accumulator and rounds it to the 16-bit output.  Against the three-stage path
// (fa_bwd_sm100.cu) this drops the separate dQ pass and its recomputed S and dP: five
// GEMMs per tile pair instead of seven.  The reduction order of dQ varies from run to
// run, so dQ is reproducible to rounding, not bit for bit; dK and dV are deterministic.
//
// Tensor memory (512 columns, lanes = the 128 keys of the tile; lanes = queries for dQ):
//   S^T / P^T [0,128)   dP^T / dS^T [128,256)   dV [256,256+D)   dK [256+D,256+2D)
//   dQ_i: D = 128: [128,256), over dP^T once dS^T has been read (dP^T of the next tile
//         waits until dQ_i has been drained);  D = 64: its own columns [384,448).
// Order of the MMAs per query tile i (each waits only for what it reads or overwrites):
//   dK(i), dQ(i), dV(i+1), dP^T(i+1), S^T(i+2)
// and of the element-wise warps: dS(i), P(i+1), drain dQ(i); so the tensor pipe works on
// dK/dQ while P(i+1) is computed and on dV(i+1) while dQ(i) is drained.
#include <climits>
#include <cstdint>
#include <math_constants.h>
#include <type_traits>

#include "bwd_common.cuh"
#include "fa_internal.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

template <int D>
struct FusedSmem {
  using T = Tile<D, 128>;
  static constexpr int kStages = (D == 128) ? 2 : 4;
  static constexpr int kOffK = 0;                                 // K_j (later dK staging)
  static constexpr int kOffV = kOffK + T::kBytes;                 // V_j (later dV staging)
  static constexpr int kOffQ = kOffV + T::kBytes;                 // [stage] Q_i
  static constexpr int kOffdO = kOffQ + kStages * T::kBytes;      // [stage] dO_i
  static constexpr int kDSBox = 128 * 128;                        // 128 keys x 64 queries x 2 bytes
  static constexpr int kOffDS = kOffdO + kStages * T::kBytes;     // dS^T: 128 keys x 128 queries, 2 boxes
  static constexpr int kOffStat = kOffDS + 2 * kDSBox;            // [stage] nl[128], delta[128]
  static constexpr int kStatBytes = 2 * 128 * 4;
  static constexpr int kOffBar = kOffStat + kStages * kStatBytes;
  static constexpr int kBarKV = 0;
  static constexpr int kBarQFull = 1;
  static constexpr int kBarQEmpty = kBarQFull + kStages;
  static constexpr int kBarOFull = kBarQEmpty + kStages;
  static constexpr int kBarOEmpty = kBarOFull + kStages;
  static constexpr int kBarS = kBarOEmpty + kStages;
  static constexpr int kBarDP = kBarS + 1;
  static constexpr int kBarP = kBarDP + 1;
  static constexpr int kBarDS = kBarP + 1;
  static constexpr int kBarDQFull = kBarDS + 1;
  static constexpr int kBarDQEmpty = kBarDQFull + 1;
  static constexpr int kBarAcc = kBarDQEmpty + 1;
  static constexpr int kBarMmaDone = kBarAcc + 1;
  static constexpr int kNumBars = kBarMmaDone + 1;
  static constexpr int kOffSlot = kOffBar + 8 * kNumBars;
  // No slack for aligning the base: the kernel checks that the dynamic shared memory starts
  // on a 1024-byte boundary (the 128-byte swizzle atom) and reports FA_ERR_LAUNCH otherwise.
  static constexpr int kBytes = kOffSlot + 16;
  static_assert(kOffDS % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(kBytes <= 232448, "shared memory budget");
  static_assert(kBytes > 116 * 1024, "one CTA per SM (each CTA allocates all 512 TMEM columns)");
};

// The score-modified instances (MOD, see the forward) walk, per key tile of one key-value head, the
// query tiles that meet it in each of the H / Hkv query heads that share that head, one head after
// the other: dK_j and dV_j stay in tensor memory over all of them.  Where that leaves few and long
// work items, two CTAs (a cluster) take half of the heads each and join their halves at the end.  With CAP the score gradient
// carries the factor 1 - tanh^2, folded into the copy of P that dS is formed from.  That copy (`pw`)
// is kept apart from the operand of dV: as fp16 times 2^12 where the operand is bf16, so that dS
// gets P to 11 bits and loses only its own rounding (scores that weigh below 2^-26 keep fewer bits,
// and matter less).  Where it is 0, as it is for masked pairs, so is dS (2% of a backward over packed
// documents).
template <int D, bool CAUSAL, bool F16, bool MOD, bool CAP, bool ALIBI>
__global__ void __launch_bounds__(kThreads, 1)
    bwd_fused_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                     const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
                     const float* __restrict__ ws_nl, const float* __restrict__ ws_delta, float* __restrict__ ws_dq,
                     int N, int Npad, int BH, int nkt, int hg, float scale, int* status,
                     const __grid_constant__ ScoreMods mods) {
  using L = FusedSmem<D>;
  using T = Tile<D, 128>;
  extern __shared__ uint8_t smem[];   // alignment checked below, not assumed
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {   // uniform over the CTA: nothing has been touched yet
    if (threadIdx.x == 0) atomicCAS(status, 0, kStatusLaunch);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sb + L::kOffBar + 8 * i; };
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::kOffSlot);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Work item: key tile kt of head bh (causal: tile 0, which meets every query tile, first).
  const int pair = MOD ? static_cast<int>(cluster_size()) : 1;   // CTAs that share a work item: 1 or 2
  const int rank = MOD ? static_cast<int>(cluster_rank()) : 0;
  const WorkItem wi = grouped_order(static_cast<int>(blockIdx.x) / pair, BH, nkt, hg);
  const int bh = wi.bh;                   // MOD: a key-value head
  int kt = wi.tile;
  int kv0 = kt * 128;
  int it0 = CAUSAL ? kt : 0;              // first query tile
  int nq = nkt - it0;                     // query tiles of one query head that meet this key tile
  int n = nq;                             // query tiles visited (>= 1; MOD: >= 0, over all heads)
  int batch = 0, qh0 = bh;                // first query head
  if constexpr (MOD) {
    const int group = mods.H / mods.Hkv;
    batch = bh / mods.Hkv;
    qh0 = batch * mods.H + (bh - batch * mods.Hkv) * group + rank * (group / pair);
    if (mods.plan != nullptr) {
      const MaskPlan plan = mask_plan_view(mods.plan, BH / mods.Hkv, N);
      kt = plan.order[static_cast<size_t>(batch) * nkt + kt].x;
      kv0 = kt * 128;
      const int4 tl = plan.tiles[static_cast<size_t>(batch) * nkt + kt];
      it0 = tl.z;
      nq = tl.w - tl.z;
    } else {
      it0 = mods.causal ? kt : 0;
      nq = nkt - it0;
    }
    n = nq * (group / pair);
  }

  if (threadIdx.x == 0) {
    mbar_init(bar(L::kBarKV), 1);
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarQFull + s), 1);
      mbar_init(bar(L::kBarQEmpty + s), 1);
      mbar_init(bar(L::kBarOFull + s), 1);
      mbar_init(bar(L::kBarOEmpty + s), 1);
    }
    mbar_init(bar(L::kBarS), 1);
    mbar_init(bar(L::kBarDP), 1);
    mbar_init(bar(L::kBarP), 512);
    mbar_init(bar(L::kBarDS), 512);
    mbar_init(bar(L::kBarDQFull), 1);
    mbar_init(bar(L::kBarDQEmpty), 512);
    mbar_init(bar(L::kBarAcc), 1);
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
  constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 256 + D;
  constexpr uint32_t kColDQ = (D == 128) ? 128u : 384u;

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmdO);
      mbar_arrive_expect_tx(bar(L::kBarKV), 2 * T::kBytes);
      for (int c = 0; c < T::kNBox; ++c) {
        tma_load_3d(sb + L::kOffK + c * T::kBox, &tmK, bar(L::kBarKV), c * 64, kv0, bh);
        tma_load_3d(sb + L::kOffV + c * T::kBox, &tmV, bar(L::kBarKV), c * 64, kv0, bh);
      }
      int nql = 0, no = 0;
      bool ok = true;
      int qt = it0, qh = qh0;             // query tile and head of step i
      for (int i = 0; i < n; ++i) {
        const int s = i % L::kStages;
        const uint32_t ph = ((i / L::kStages) & 1) ^ 1;
        const int q0 = qt * 128, bhq = qh;
        if (++qt == it0 + nq) {
          qt = it0;
          ++qh;
        }
        if (!(ok = mbar_wait(bar(L::kBarQEmpty + s), ph, abort_flag))) break;
        const uint32_t qf = bar(L::kBarQFull + s);
        const size_t srow = static_cast<size_t>(bhq) * Npad + q0;     // padded rows: always in bounds
        const bool stats_in = FA_BOUNDS(srow + 128 <= static_cast<size_t>(MOD ? BH / mods.Hkv * mods.H : BH) * Npad, status);
        mbar_arrive_expect_tx(qf, T::kBytes + (stats_in ? L::kStatBytes : 0));
        for (int c = 0; c < T::kNBox; ++c)
          tma_load_3d(sb + L::kOffQ + s * T::kBytes + c * T::kBox, &tmQ, qf, c * 64, q0, bhq);
        if (stats_in) {
          bulk_load(sb + L::kOffStat + s * L::kStatBytes, ws_nl + srow, 128 * 4, qf);
          bulk_load(sb + L::kOffStat + s * L::kStatBytes + 128 * 4, ws_delta + srow, 128 * 4, qf);
        }
        ++nql;
        if (!(ok = mbar_wait(bar(L::kBarOEmpty + s), ph, abort_flag))) break;
        const uint32_t of = bar(L::kBarOFull + s);
        mbar_arrive_expect_tx(of, T::kBytes);
        for (int c = 0; c < T::kNBox; ++c)
          tma_load_3d(sb + L::kOffdO + s * T::kBytes + c * T::kBox, &tmdO, of, c * 64, q0, bhq);
        ++no;
      }
      if (!ok) raise_error(status, abort_flag, kStatusTimeout);
      mbar_wait_drain(bar(L::kBarKV), 0);
      for (int i = max(0, nql - L::kStages); i < nql; ++i)
        mbar_wait_drain(bar(L::kBarQFull + i % L::kStages), (i / L::kStages) & 1);
      for (int i = max(0, no - L::kStages); i < no; ++i)
        mbar_wait_drain(bar(L::kBarOFull + i % L::kStages), (i / L::kStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_16(128, 128, false, false, F16);  // S^T, dP^T: K-major A and B
      constexpr uint32_t kIdAcc = idesc_16(128, D, false, true, F16);   // dV, dK: A in TMEM, B MN-major
      constexpr uint32_t kIdDQ = idesc_16(128, D, true, true, F16);     // dQ: A (dS) and B (K_j) MN-major
      const uint32_t sK = sb + L::kOffK, sV = sb + L::kOffV, sDS = sb + L::kOffDS;
      auto sQ = [&](int i) { return sb + L::kOffQ + (i % L::kStages) * T::kBytes; };
      auto sdO = [&](int i) { return sb + L::kOffdO + (i % L::kStages) * T::kBytes; };
      auto phase = [&](int i) { return static_cast<uint32_t>((i / L::kStages) & 1); };
      // K-major operands: four K-steps of 16 per 64-column box, 32 bytes apart.  MN-major
      // operands: one K-step per 16 rows (2048 bytes).  Packed 16-bit A operands in tensor
      // memory: K-steps at columns +0, +8, +32, +40 (see packed_col), then the next 64.
      auto issue_st = [&](int i) {      // S^T = K_j Q_i^T
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          mma_ss_x4<2, 4, 6, 2, 4, 6>(tmem + kColS, sdesc_sw128(sK + c * T::kBox, 16, 1024),
                                      sdesc_sw128(sQ(i) + c * T::kBox, 16, 1024), kIdS, c > 0 ? 1u : 0u);
        tc_commit(bar(L::kBarS));
      };
      auto issue_dpt = [&](int i) {     // dP^T = V_j dO_i^T
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          mma_ss_x4<2, 4, 6, 2, 4, 6>(tmem + kColDP, sdesc_sw128(sV + c * T::kBox, 16, 1024),
                                      sdesc_sw128(sdO(i) + c * T::kBox, 16, 1024), kIdS, c > 0 ? 1u : 0u);
        tc_commit(bar(L::kBarDP));
      };
      // acc (+)= A_tmem (packed 16-bit, 128 queries) * B_smem (128 queries x D, MN-major)
      auto issue_acc = [&](uint32_t dcol, uint32_t abase, uint32_t b_tile, bool first) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
          mma_ts_x4<8, 32, 40, 128, 256, 384>(tmem + dcol, tmem + packed_col(abase, 4 * g),
                                              sdesc_sw128(b_tile + g * 4 * 2048, T::kBox, 1024), kIdAcc,
                                              (!first || g > 0) ? 1u : 0u);
      };
      auto issue_dq = [&]() {           // dQ_i = dS_i K_j: 128 queries x D over the 128 keys
#pragma unroll
        for (int g = 0; g < 2; ++g)
          mma_ss_x4<128, 256, 384, 128, 256, 384>(tmem + kColDQ, sdesc_sw128(sDS + g * 4 * 2048, L::kDSBox, 1024),
                                                  sdesc_sw128(sK + g * 4 * 2048, T::kBox, 1024), kIdDQ,
                                                  g > 0 ? 1u : 0u);
        tc_commit(bar(L::kBarDQFull));
      };
      bool ok = mbar_wait_spin(bar(L::kBarKV), 0, abort_flag);
      const bool any = !MOD || n > 0;
      if (any) ok = ok && mbar_wait_spin(bar(L::kBarQFull), 0, abort_flag) && mbar_wait_spin(bar(L::kBarOFull), 0, abort_flag);
      if (ok && any) {
        tc_fence_after();
        issue_st(0);
        issue_dpt(0);
        ok = mbar_wait_spin(bar(L::kBarP), 0, abort_flag);
      }
      if (ok && any) {
        tc_fence_after();
        issue_acc(kColDV, kColS, sdO(0), true);                                   // dV = P^T dO_0
        tc_commit(bar(L::kBarOEmpty));
        if (n > 1 && (ok = mbar_wait_spin(bar(L::kBarQFull + 1), 0, abort_flag))) {
          tc_fence_after();
          issue_st(1);                                                            // over P^T_0 (read above)
        }
      }
      for (int i = 0; ok && i < n; ++i) {
        if (!(ok = mbar_wait_spin(bar(L::kBarDS), i & 1, abort_flag))) break;
        tc_fence_after();
        issue_acc(kColDK, kColDP, sQ(i), i == 0);                                 // dK += dS^T Q_i
        tc_commit(bar(L::kBarQEmpty + i % L::kStages));
        if (D != 128 && i > 0) {                                                  // own columns: dQ_{i-1} drained
          if (!(ok = mbar_wait_spin(bar(L::kBarDQEmpty), (i - 1) & 1, abort_flag))) break;
          tc_fence_after();
        }
        issue_dq();                                                               // dQ_i = dS_i K_j
        if (i + 1 < n) {
          const int j = i + 1;
          if (!(ok = mbar_wait_spin(bar(L::kBarP), j & 1, abort_flag))) break;
          if (!(ok = mbar_wait_spin(bar(L::kBarOFull + j % L::kStages), phase(j), abort_flag))) break;
          tc_fence_after();
          issue_acc(kColDV, kColS, sdO(j), false);                                // dV += P^T dO_{i+1}
          if (D == 128) {                                                         // dP^T over dQ_i: drained
            if (!(ok = mbar_wait_spin(bar(L::kBarDQEmpty), i & 1, abort_flag))) break;
            tc_fence_after();
          }
          issue_dpt(j);
          tc_commit(bar(L::kBarOEmpty + j % L::kStages));
        }
        if (i + 2 < n) {
          const int j = i + 2;
          if (!(ok = mbar_wait_spin(bar(L::kBarQFull + j % L::kStages), phase(j), abort_flag))) break;
          tc_fence_after();
          issue_st(j);                                                            // over P^T_{i+1} (read above)
        }
      }
      if (!ok) raise_error(status, abort_flag, kStatusTimeout);
      tc_commit(bar(L::kBarAcc));
      tc_commit(bar(L::kBarMmaDone));
      mbar_wait_drain(bar(L::kBarMmaDone), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ P^T, dS^T, dQ drain, epilogue
    const int g = (warp - 4) >> 2;                       // query columns [32g, 32g+32) of S^T / dP^T
    const int r = threadIdx.x - 128 * (1 + g);           // TMEM lane: key row of S^T, query row of dQ
    const uint32_t tb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int key = kv0 + r;
    const bool key_oob = key >= N;                       // padding rows of the last key tile
    const bool tail = __any_sync(0xffffffffu, key_oob);  // warp-uniform
    const float scale_log2 = scale * kLog2e;
    const float x_scale = CAP ? mods.softcap * kLog2e : scale_log2;   // CAP: of tanh(s / cap)
    const float cap_in = CAP ? scale / mods.softcap : 0.f;
    const float2 sl2 = make_float2(x_scale, x_scale);
    const int2* rows = nullptr;                          // MOD: the plan's intervals of this batch element
    if (MOD && mods.plan != nullptr) rows = mask_plan_view(mods.plan, BH / mods.Hkv, N).rows + static_cast<size_t>(batch) * Npad;
    int pqt = it0, pqh = 0;                              // MOD: query tile and head (within the group) of p_tile's next step
    int dqt = it0, dqh = 0;                              // and of drain's
    // Row r of the dS^T tile (box g/2 holds queries [64(g/2), 64(g/2)+64)); chunk c of a row sits at c ^ (r % 8).
    uint8_t* ds_row = smem + L::kOffDS + (g >> 1) * L::kDSBox + r * 128;
    const int sw = r & 7;
    float* dq_head = ws_dq + static_cast<size_t>(qh0) * Npad * D;
    uint32_t pk[16];                                     // packed P^T of the current tile
    constexpr bool kWide = MOD && !F16;                  // pw holds fp16 of 2^12 P
    constexpr bool kOwnW = CAP || kWide;                 // pw differs from pk
    constexpr float kWScale = kWide ? 4096.f : 1.f, kWBack = 1.f / kWScale;
    uint32_t pw[kOwnW ? 16 : 1];                         // packed P^T (1 - tanh^2) for dS
    // dQ of the previous query tile (this thread: query row r, D/4 columns), held in registers
    // from its drain out of tensor memory until its 16-byte reductions are issued, a few at a
    // time, between the next tile's dS^T and P^T arithmetic.  Each SM can send only about
    // 32 bytes per clock towards L2, so the 64 KB of a tile's dQ take ~2000 clocks to leave:
    // spread over the tile's work they overlap it, issued in one burst they would stall the
    // warps for that long.
    constexpr int kCols = D / 4;
    constexpr int kReds = kCols / 4;                     // reductions per thread per tile: 8 or 4
    uint32_t held[kCols];
    float* held_acc = dq_head + 4 * r;
    const float* const acc_end = ws_dq + static_cast<size_t>(MOD ? BH / mods.Hkv * mods.H : BH) * Npad * D;   // end of the accumulator
    (void)acc_end;
    auto red_held = [&](int q) {
      float* a = held_acc + (kReds * g + q) * 512;
      if (FA_BOUNDS(a >= ws_dq && a + 4 <= acc_end, status)) red_add_f32x4(a, held[4 * q], held[4 * q + 1], held[4 * q + 2], held[4 * q + 3]);
    };

    // P^T[r][c] = exp2(s * scale * log2e + nl_c), zero where key > query or key >= N; with
    // `reds`, issues the held reductions kReds/2 .. kReds-1 along the way.
    auto p_tile = [&](int i, bool reds) -> bool {
      int mod_qc0 = 0;
      int2 iv = make_int2(0, INT_MAX);                   // MOD: the keys that query mod_qc0 + lane sees
      float slope2 = 0.f;
      if constexpr (MOD) {
        // read before the wait for the scores; padding queries (P = 0 by their statistics) bound nothing
        mod_qc0 = pqt * 128 + 32 * g;
        const int row = mod_qc0 + lane;
        if (row < N) iv = mods.plan != nullptr ? rows[row] : make_int2(0, mods.causal ? row + 1 : N);
        if (ALIBI) slope2 = mods.slopes[qh0 - batch * mods.H + pqh] * kLog2e;
        if (++pqt == it0 + nq) {
          pqt = it0;
          ++pqh;
        }
      }
      const int s = i % L::kStages;
      bool ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarQFull + s), (i / L::kStages) & 1, abort_flag));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarS), i & 1, abort_flag));
      if (!ok) return false;
      FA_CONVERGED(status);                              // warp-collective TMEM loads follow
      tc_fence_after();
      const float4* st = reinterpret_cast<const float4*>(smem + L::kOffStat + s * L::kStatBytes) + 8 * g;
      const int qc0 = MOD ? mod_qc0 : (it0 + i) * 128 + 32 * g;   // query of this thread's column 0
      bool edge = tail || (CAUSAL && __any_sync(0xffffffffu, qc0 < key + 32));   // warp-uniform
      uint32_t seen = 0xffffffffu;                       // MOD: bit c: this key is seen by query qc0 + c
      if constexpr (MOD) {
        edge = !__all_sync(0xffffffffu, iv.x <= kv0 && iv.y >= kv0 + 128);
        if (edge) {
          // lane c: which of the warp's keys query c sees; turned around, which queries see this key
          const int w0 = key - lane;
          const int from = min(max(iv.x - w0, 0), 32), to = min(max(iv.y - w0, 0), 32);
          uint32_t word = to > from ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) {
            const uint32_t low = d == 16 ? 0x0000ffffu : d == 8 ? 0x00ff00ffu : d == 4 ? 0x0f0f0f0fu : d == 2 ? 0x33333333u : 0x55555555u;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, word, d);
            word = (lane & d) ? (word & ~low) | ((other >> d) & low) : (word & low) | ((other << d) & ~low);
          }
          seen = word;
        }
      }
      // two halves of 16 columns (one TMEM load each), to keep the held dQ values in registers
      auto p_phase = [&](auto masked) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t sr[16];
          tmem_ld16(tb + kColS + 32 * g + 16 * hf, sr);
          tmem_ld_wait();
          reg_fence(sr);
          if constexpr (CAP) {                           // scores -> tanh(s / cap), as in the forward
            float most = 0.f;
#pragma unroll
            for (int c = 0; c < 16; c += 2) most = fmax3_abs_nan(most, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            if (__all_sync(0xffffffffu, most <= mods.poly_limit)) {
#pragma unroll
              for (int c = 0; c < 16; c += 2) {
                const float2 sv = make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                const float2 th = __fmul2_rn(sv, quartic2(sv, mods.poly));
                sr[c] = __float_as_uint(th.x);
                sr[c + 1] = __float_as_uint(th.y);
              }
            } else {
#pragma unroll
              for (int c = 0; c < 16; ++c)      // NaN becomes finite (see dS): where it counts, lse holds one too
                sr[c] = __float_as_uint(tanh_any(fminf(fmaxf(__uint_as_float(sr[c]) * cap_in, -20.f), 20.f)));
            }
          }
#pragma unroll
          for (int c4 = 4 * hf; c4 < 4 * hf + 4; ++c4) {
            const float4 nl = st[c4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c2 = 2 * c4 + h, c = 2 * c2, cl = c - 16 * hf;
              const float2 nlp = h ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y);
              float2 sv = make_float2(__uint_as_float(sr[cl]), __uint_as_float(sr[cl + 1]));
              float2 add = nlp;
              if constexpr (ALIBI) {
                const float d0 = static_cast<float>(qc0 + c - key);
                add.x = fmaf(-slope2, fabsf(d0), add.x);
                add.y = fmaf(-slope2, fabsf(d0 + 1.f), add.y);
              }
              float2 p = exp2_pair(__ffma2_rn(sv, sl2, add), poly_pair(c2));
              if (decltype(masked)::value) {
                if constexpr (MOD) {
                  if (!((seen >> c) & 1u)) p.x = 0.f;
                  if (!((seen >> (c + 1)) & 1u)) p.y = 0.f;
                } else {
                  if (key_oob || (CAUSAL && key > qc0 + c)) p.x = 0.f;
                  if (key_oob || (CAUSAL && key > qc0 + c + 1)) p.y = 0.f;
                }
              }
              pk[c2] = pack16<F16>(p.x, p.y);
              if constexpr (kOwnW) {
                float2 w = __fmul2_rn(p, make_float2(kWScale, kWScale));
                if constexpr (CAP) w = __fmul2_rn(w, __ffma2_rn(sv, make_float2(-sv.x, -sv.y), make_float2(1.f, 1.f)));
                pw[c2] = kWide ? pack16<true>(w.x, w.y) : pack16<F16>(w.x, w.y);
              }
            }
            if (reds && kReds == 8 && (c4 & 1)) red_held(4 + (c4 >> 1));         // reductions 4..7
            if (reds && kReds == 4 && (c4 & 3) == 3) red_held(2 + (c4 >> 2));    // reductions 2, 3
          }
        }
      };
      if (edge) p_phase(std::true_type{});
      else p_phase(std::false_type{});
      tmem_st16(tb + kColS + 32 * g, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kBarP));
      return true;
    };

    // dS^T[r][c] = P^T[r][c] * (dP^T[r][c] - delta_c), in two halves of 16 columns: packed into
    // tensor memory (for dK) and into the swizzled shared-memory tile (for dQ).
    auto ds_tile = [&](int i) -> bool {
      const int s = i % L::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kBarDP), i & 1, abort_flag))) return false;
      FA_CONVERGED(status);
      tc_fence_after();
      const float4* st = reinterpret_cast<const float4*>(smem + L::kOffStat + s * L::kStatBytes + 512) + 8 * g;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t dp[16], dsk[8];
        tmem_ld16(tb + kColDP + 32 * g + 16 * hf, dp);
        tmem_ld_wait();
        reg_fence(dp);
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          const float4 dl = st[4 * hf + c4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c2 = 2 * c4 + h, c = 2 * c2;
            const float2 dlp = h ? make_float2(dl.z, dl.w) : make_float2(dl.x, dl.y);
            const float2 dpv = make_float2(__uint_as_float(dp[c]), __uint_as_float(dp[c + 1]));
            const uint32_t pp = kOwnW ? pw[(8 * hf + c2) & (kOwnW ? 15 : 0)] : pk[8 * hf + c2];
            constexpr bool kHalfP = F16 || kWide;
            const float2 ds = __fmul2_rn(make_float2(unpack16_lo<kHalfP>(pp), unpack16_hi<kHalfP>(pp)),
                                         __ffma2_rn(dlp, make_float2(-kWBack, -kWBack),
                                                    kWide ? __fmul2_rn(dpv, make_float2(kWBack, kWBack)) : dpv));
            dsk[c2] = pack16<F16>(ds.x, ds.y);
            // P = 0 makes dS = 0 also where the products of masked rows have left the fp32 range.
            if constexpr (MOD) dsk[c2] &= nonzero_f16x2(pp);   // pp is fp16 in either case
          }
        }
        // packed columns [8 hf, 8 hf + 8) of this warpgroup's range (already read: half 0 read
        // columns [0, 16)) and 16-byte chunks 2 hf, 2 hf + 1 of its 64-byte part of row r
        tmem_st8(tb + kColDP + 32 * g + 8 * hf, dsk);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (FA_BOUNDS(ds_row + ((((g & 1) * 4 + 2 * hf + q) ^ sw) << 4) + 16 <= smem + L::kOffDS + 2 * L::kDSBox, status))
          *reinterpret_cast<uint4*>(ds_row + ((((g & 1) * 4 + 2 * hf + q) ^ sw) << 4)) =
              make_uint4(dsk[4 * q], dsk[4 * q + 1], dsk[4 * q + 2], dsk[4 * q + 3]);
      }
      fence_async_smem();
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(L::kBarDS));
      return true;
    };

    // dQ_i out of tensor memory into `held`; the columns are released at once (the next dP^T
    // may overwrite them) and the first half of the reductions into the accumulator tile of
    // query tile i (laid out [D/4][128 rows][4 floats], so that a warp's reduction covers 512
    // contiguous bytes) is issued while the MMAs compute dV and that dP^T, which the next
    // dS^T waits for; the second half goes out during the next P^T.
    auto drain = [&](int i) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(bar(L::kBarDQFull), i & 1, abort_flag))) return false;
      FA_CONVERGED(status);
      tc_fence_after();
      if constexpr (kCols == 32) tmem_ld32(tb + kColDQ + 32 * g, held);
      else tmem_ld16(tb + kColDQ + 16 * g, held);
      tmem_ld_wait();
      reg_fence(held);
      tc_fence_before();
      mbar_arrive(bar(L::kBarDQEmpty));
      if constexpr (MOD) {
        held_acc = dq_head + (static_cast<size_t>(dqh) * Npad + static_cast<size_t>(dqt) * 128) * D + 4 * r;
        if (++dqt == it0 + nq) {
          dqt = it0;
          ++dqh;
        }
      } else {
        held_acc = dq_head + static_cast<size_t>(it0 + i) * 128 * D + 4 * r;
      }
#pragma unroll
      for (int q = 0; q < kReds / 2; ++q) red_held(q);
      return true;
    };

    bool ok = (MOD && n == 0) || p_tile(0, false);
    for (int i = 0; ok && i < n; ++i) {
      ok = ds_tile(i);
      if (ok && i + 1 < n) {
        ok = p_tile(i + 1, i > 0);                       // + second half of dQ_{i-1}'s reductions
      } else if (ok && i > 0) {
#pragma unroll
        for (int q = kReds / 2; q < kReds; ++q) red_held(q);
      }
      if (ok) ok = drain(i);                             // + first half of dQ_i's
    }
    if (ok && (!MOD || n > 0)) {
#pragma unroll
      for (int q = kReds / 2; q < kReds; ++q) red_held(q);   // the last tile's second half
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarAcc), 0, abort_flag));
    if (!ok) {
      raise_error(status, abort_flag, kStatusTimeout);
    } else {
      // One 64-column box per warpgroup: dV boxes into the V tile, dK boxes into the K tile
      // (the K tile is free: the last dQ product, which reads it, completed before kBarAcc).
      FA_CONVERGED(status);
      tc_fence_after();
      const int wrow = (warp & 3) * 32;
      const int nbox = T::kNBox;                          // 1 (D=64) or 2 (D=128)
      if (pair == 1 && g < 2 * nbox) {
        const bool is_dv = g < nbox;
        const int box = is_dv ? g : g - nbox;
        uint8_t* stage = smem + (is_dv ? L::kOffV : L::kOffK);
        if (!MOD || n > 0) {
          stage_box_16<D, F16>(tb + (is_dv ? kColDV : kColDK), box, is_dv ? 1.f : scale, stage, r);
        } else {                                          // no query sees these keys
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(stage + box * T::kBox + r * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        store_warp_box<D>(is_dv ? &tmdV : &tmdK, sb + (is_dv ? L::kOffV : L::kOffK), box, wrow, kv0, bh, lane, N);
      }
    }
  }

  if constexpr (MOD) {
    if (pair == 2) {
      // Each CTA holds dK and dV of half of the group's query heads: CTA 0 finishes dV, CTA 1 dK,
      // each with the other's fp32 half out of its shared memory ([16-byte chunk][row], over the K
      // and V tiles).  Both barriers are reached by every thread, in a failing CTA too.
      constexpr int kC = D / 4;                           // columns a thread
      const int g = (warp - 4) >> 2, r = (warp & 3) * 32 + lane;
      const uint32_t tb = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      auto load = [&](uint32_t col, uint32_t (&o)[kC]) {
        if (n > 0) {
#pragma unroll
          for (int c = 0; c < kC; c += 16)
            tmem_ld16(tb + col + g * kC + c, reinterpret_cast<uint32_t(&)[16]>(o[c]));
          tmem_ld_wait();
          reg_fence(o);
        } else {                                          // no query sees these keys
#pragma unroll
          for (int c = 0; c < kC; ++c) o[c] = 0u;
        }
      };
      __syncthreads();
      tc_fence_after();
      if (warp >= 4) {
        FA_CONVERGED(status);
        uint32_t o[kC];
        load(rank == 0 ? kColDK : kColDV, o);
#pragma unroll
        for (int c = 0; c < kC; c += 4)
          *reinterpret_cast<uint4*>(smem + ((g * kC + c) / 4 * 128 + r) * 16) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
      }
      cluster_sync();
      if (warp >= 4) {
        FA_CONVERGED(status);
        uint32_t o[kC];
        load(rank == 0 ? kColDV : kColDK, o);
        const float mul = rank == 0 ? 1.f : scale;
#pragma unroll
        for (int c = 0; c < kC; c += 8) {
          const float4 x = ld_cluster_f32x4(sb + ((g * kC + c) / 4 * 128 + r) * 16, rank ^ 1);
          const float4 y = ld_cluster_f32x4(sb + ((g * kC + c + 4) / 4 * 128 + r) * 16, rank ^ 1);
          auto sum = [&](int e, float p) { return (__uint_as_float(o[c + e]) + p) * mul; };
          const int col = g * kC + c;                     // chunk col / 8 % 8 of box col / 64
          *reinterpret_cast<uint4*>(smem + L::kOffQ + (col >> 6) * T::kBox + r * 128 + ((((col >> 3) & 7) ^ (r & 7)) << 4)) =
              make_uint4(pack16<F16>(sum(0, x.x), sum(1, x.y)), pack16<F16>(sum(2, x.z), sum(3, x.w)),
                         pack16<F16>(sum(4, y.x), sum(5, y.y)), pack16<F16>(sum(6, y.z), sum(7, y.w)));
        }
        fence_async_smem();
      }
      __syncthreads();
      if (warp >= 4 && g < T::kNBox && *abort_flag == 0)
        store_warp_box<D>(rank == 0 ? &tmdV : &tmdK, sb + L::kOffQ, g, (warp & 3) * 32, kv0, bh, lane, N);
      cluster_sync();
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

// dQ = scale * accumulator, rounded to the 16-bit type, for 64 query rows per CTA: the
// tile layout [DK/4][128][4] is read with consecutive threads on consecutive rows, turned
// around in shared memory and written as whole rows of the caller's (B,H,N,D) dQ.
template <int DK, bool F16>
__global__ void __launch_bounds__(256) bwd_dq_finish_kernel(const float* __restrict__ acc, uint16_t* __restrict__ dq,
                                                            int N, int Npad, int D, float scale, int* status) {
  constexpr int kStride = DK / 4 + 1;                     // float4 per staged row (one of padding)
  __shared__ float4 stage[64 * kStride];
  const long long blk = blockIdx.x;
  const int halves = Npad / 64;
  const long long bh = blk / halves;
  const int half = static_cast<int>(blk % halves);
  const int qt = half >> 1, h = half & 1;
  const float4* src = reinterpret_cast<const float4*>(acc + (bh * Npad + static_cast<long long>(qt) * 128) * DK);
  for (int f = threadIdx.x; f < (DK / 4) * 64; f += 256) {
    const int c4 = f >> 6, rr = f & 63;
    const float4* sp = src + c4 * 128 + 64 * h + rr;
    stage[rr * kStride + c4] =
        FA_BOUNDS(sp + 1 <= reinterpret_cast<const float4*>(acc) + static_cast<long long>(gridDim.x) * 64 * DK / 4, status)
            ? *sp : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  const int row0 = qt * 128 + 64 * h;
  const int rows = min(64, N - row0);
  for (int f = threadIdx.x; f < 64 * (DK / 8); f += 256) {
    const int rr = f / (DK / 8), c8 = f % (DK / 8);
    if (rr >= rows || 8 * c8 >= D) continue;
    const float4 a = stage[rr * kStride + 2 * c8], b = stage[rr * kStride + 2 * c8 + 1];
    uint4 o;
    o.x = pack16<F16>(a.x * scale, a.y * scale);
    o.y = pack16<F16>(a.z * scale, a.w * scale);
    o.z = pack16<F16>(b.x * scale, b.y * scale);
    o.w = pack16<F16>(b.z * scale, b.w * scale);
    const long long di = (bh * N + row0 + rr) * D + 8 * c8;
    if (FA_BOUNDS(di + 8 <= static_cast<long long>(gridDim.x) / (Npad / 64) * N * D, status))
      *reinterpret_cast<uint4*>(dq + di) = o;
  }
}

// Whether pairs of CTAs share the work items of a score-modified call: where the items are few, the
// longest of them (all query tiles of all heads of a group) decide.  Measured, one CTA an item
// against a pair: D = 128, H / Hkv = 4: N = 4096 causal 64 items 434 / 238 us, packed documents of
// N = 16384 256 items 626 / 491 us, 256 items (B2 H32 N4096) 1075 / 811 us, 1024 items 1582 / 1587 us;
// D = 64, whose items are shorter against the joining: 16 items 58 / 40 us, 256 items 201 / 215 us,
// 1024 items 692 / 756 us.
template <int D>
bool pair_items(long long items, const ScoreMods& m, int num_sms) {
  return m.H / m.Hkv % 2 == 0 && items < (D == 128 ? 4LL : 1LL) * num_sms;
}

template <int D, bool CAUSAL, bool F16, bool MOD, bool CAP, bool ALIBI>
cudaError_t fused_impl(const BwdLaunch& a, const ScoreMods& m, cudaStream_t stream) {
  using L = FusedSmem<D>;
  auto kern = bwd_fused_kernel<D, CAUSAL, F16, MOD, CAP, ALIBI>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int nkt = (a.N + 127) / 128;
  const int BH = MOD ? a.BH / m.H * m.Hkv : a.BH;     // one CTA (or pair) per key tile of a key-value head
  const long long items = static_cast<long long>(nkt) * BH;
  const unsigned pair = MOD && pair_items<D>(items, m, a.num_sms) ? 2 : 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(items) * pair);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pair;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kern, a.tmQ, a.tmK, a.tmV, a.tmdO, a.tmdK, a.tmdV, a.ws_nl, a.ws_delta, a.ws_dq, a.N,
                         a.Npad, BH, nkt, a.hg, a.scale, a.status, m);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <bool F16>
cudaError_t fused_typed(const BwdLaunch& a, cudaStream_t stream) {
  // Head dims 32 and 96 run the 64- and 128-column kernels on zero-filled tile columns.
  const ScoreMods none{};
  if (a.DK == 64)
    return a.causal ? fused_impl<64, true, F16, false, false, false>(a, none, stream)
                    : fused_impl<64, false, F16, false, false, false>(a, none, stream);
  return a.causal ? fused_impl<128, true, F16, false, false, false>(a, none, stream)
                  : fused_impl<128, false, F16, false, false, false>(a, none, stream);
}

template <int D, bool F16>
cudaError_t fused_mod_typed(const BwdLaunch& a, const ScoreMods& m, cudaStream_t stream) {
  const bool cap = m.softcap != 0.f, alibi = m.slopes != nullptr;
  if (cap)
    return alibi ? fused_impl<D, false, F16, true, true, true>(a, m, stream)
                 : fused_impl<D, false, F16, true, true, false>(a, m, stream);
  return alibi ? fused_impl<D, false, F16, true, false, true>(a, m, stream)
               : fused_impl<D, false, F16, true, false, false>(a, m, stream);
}

template <int DK, bool F16>
cudaError_t finish_impl(const BwdLaunch& a, void* dq, cudaStream_t stream) {
  const long long blocks = static_cast<long long>(a.BH) * (a.Npad / 64);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  bwd_dq_finish_kernel<DK, F16><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
      a.ws_dq, static_cast<uint16_t*>(dq), a.N, a.Npad, a.D, a.scale, a.status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_fused(const BwdLaunch& a, cudaStream_t stream) {
  if (a.DK != 64 && a.DK != 128) return cudaErrorInvalidValue;
  return a.f16 ? fused_typed<true>(a, stream) : fused_typed<false>(a, stream);
}

cudaError_t launch_bwd_fused_mod(const BwdLaunch& a, const ScoreMods& mods, cudaStream_t stream) {
  ScoreMods m = mods;
  if (m.softcap != 0.f)
    set_cap_poly(&m, static_cast<double>(a.scale) / m.softcap, 1.0, {kTanhC0, kTanhC1, kTanhC2, kTanhC3, kTanhC4},
                 kTanhPolyLimit);
  if (a.DK == 64) return a.f16 ? fused_mod_typed<64, true>(a, m, stream) : fused_mod_typed<64, false>(a, m, stream);
  if (a.DK == 128) return a.f16 ? fused_mod_typed<128, true>(a, m, stream) : fused_mod_typed<128, false>(a, m, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_bwd_dq_finish(const BwdLaunch& a, void* dq, cudaStream_t stream) {
  if (a.DK == 64) return a.f16 ? finish_impl<64, true>(a, dq, stream) : finish_impl<64, false>(a, dq, stream);
  if (a.DK == 128) return a.f16 ? finish_impl<128, true>(a, dq, stream) : finish_impl<128, false>(a, dq, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
