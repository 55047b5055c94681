// fa_paged.cu -- attention of a few new tokens a sequence over a paged key-value cache.
//
// The M = (H / Hkv) T query rows that share a key-value head are one group of up to R rows (R = 16,
// 32 or 64); a unit is (sequence, key-value head, group).  Per tile of 128 cached positions
//     S^T = K Q^T     tcgen05.mma, M = 128 keys, N = R rows, K = D
//     x   = scale s (capped, biased), m = max(m, max x), p = 2^(x log2e - m)
//     O^T += V^T P^T  tcgen05.mma, M = D (two of 128 at D = 256), N = R rows, K = 128 keys
// with the running maximum and sum of the softmax in fp32 and P rounded once to the inputs' type
// (the tensor core's operand), unnormalised; O is divided by the fp32 sum at the end.  The key is
// the accumulator's lane, so 128 threads share the element-wise work however few rows there are,
// and a row's maximum is a warp reduction and four values in shared memory.
//
// Bound by memory: K and V of the visible positions are read once, 4 D bytes a position and head,
// against 4 M D operations.  So the loads never pause: K and V have a warp each, which looks up pages
// (each lane one page of the tile, the next tile's while this one waits for room) and issues one TMA
// box per page and 64 columns into its own ring of tile slots, 128 to 192 KB a CTA for both; the
// 128-byte swizzle makes the boxes of a tile's pages one operand tile.  The MMA warp runs one tile of
// S^T ahead of the softmax.
//
// The work is split over the caches' length, evenly and whatever their lengths: all units' tiles
// form one line, sequence after sequence, and each of the CTAs (one per SM) takes an equal piece of
// it.  Every CTA finds its piece by itself from the lengths, which the host does not know.  A unit
// that lies in one piece is finished there; of one that crosses pieces each CTA leaves O, m and the
// sum in fp32 in the workspace, and a second kernel, resident before the first one ends
// (programmatic dependent launch), joins them in the pieces' order, so results do not vary.
//
// Measured (one B200, whole call): 48 sequences of up to 8192, 32 heads on 8, D = 128, pages of 16:
// 162 us, 5.5 TB/s; one sequence of 262144, 16 heads on 2: 52 us, 5.1 TB/s; 17 sequences of up to
// 6000, 5 new tokens, D = 256, window 4096: 55 us, 4.3 TB/s; one sequence of 500: 9.5 us.  Not bound
// by memory where a tile is small (16 sequences of 4096, 32 heads: D = 64 146 us, 3.7 TB/s, and D = 32
// as long; there the thread that issues both products is busy throughout) or R is 64 (16 sequences of
// 8192, 8 key-value heads of D = 128: 122 us with 16 rows, 130 with 32, 185 or 2.9 TB/s with 64: the
// exponentials, of 64 rows in 255 registers with 48 to 64 bytes spilled).  Two
// softmax warpgroups with a piece each, and a warp for either product, were built and measured: a few
// percent faster at D <= 64, up to a third slower at R = 32 and D = 256 (168 registers a thread).
//
// Positions that no row may see (behind the length, before the window, on a page outside the pool)
// have p = 0 and their V rows are zeroed in shared memory, as 0 times a NaN would not be 0.
#include <climits>
#include <cstdint>
#include <math_constants.h>

#include "fa_internal.h"
#include "paged_index.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 224;        // warps 0-3: softmax; 4: Q and K loads; 5: MMA; 6: V loads
constexpr int kTile = 128;           // positions a tile
constexpr int kBox = kTile * 128;    // bytes of 64 columns of a tile
constexpr int kMaxCtas = 148;
// The maximum that the exponents refer to follows the running one only when that has grown by a
// factor of 2^8: P stays below 2^8, and O^T is hardly ever rescaled.
constexpr float kRescale = 8.f;

constexpr int tile_dim(int D) { return D <= 64 ? 64 : (D <= 128 ? 128 : 256); }

template <int D, int R>
struct Smem {
  static constexpr int kDP = tile_dim(D);
  static constexpr int kNBox = kDP / 64;                            // 64-column boxes of a tile
  static constexpr int kParts = kDP == 256 ? 2 : 1;                 // a tile's slots: up to 128 columns each
  static constexpr int kPartBoxes = kNBox / kParts;
  static constexpr int kSlot = kPartBoxes * kBox;
  static constexpr int kQ = kNBox * R * 128;
  static constexpr int kP = 2 * R * 128;
  static constexpr int kBufs = (kDP == 256 && R > 16) ? 1 : 2;     // Q and P buffers
  static constexpr int kRing = 227 * 1024 - 4096 - kBufs * (kQ + kP);
  static constexpr int kSlots = kRing / kSlot < 12 ? kRing / kSlot : 12;
  // K and V have a ring each, with one warp that fills it in order and the MMA warp that empties it
  // in order: every parity is then waited for at most one phase ahead.
  static constexpr int kKSlots = (kSlots + 1) / 2, kVSlots = kSlots / 2;
  static constexpr int kOffV = kKSlots * kSlot;
  static constexpr int kOffQ = kSlots * kSlot;
  static constexpr int kOffP = kOffQ + kBufs * kQ;
  static constexpr int kOffRows = kOffP + kBufs * kP;               // int4 (position, first, slope2, -) per row
  static constexpr int kOffMax = kOffRows + R * 16;                 // float [2][R][4]: the warps' maxima
  static constexpr int kOffRef = kOffMax + 2 * R * 16;              // float [R] reference maximum, [R] factor
  static constexpr int kOffFlags = kOffRef + 2 * R * 4;             // int [2][4]
  static constexpr int kOffSum = kOffFlags + 32;                    // float [R][4]: the warps' sums
  static constexpr int kOffBar = kOffSum + R * 16;
  static constexpr int kBarKFull = 0, kBarKEmpty = kKSlots, kBarVFull = 2 * kKSlots, kBarVEmpty = kBarVFull + kVSlots;
  static constexpr int kBarQFull = 2 * kSlots, kBarQEmpty = kBarQFull + 2;
  static constexpr int kBarSFull = kBarQEmpty + 2, kBarSEmpty = kBarSFull + 2;
  static constexpr int kBarPFull = kBarSEmpty + 2, kBarPEmpty = kBarPFull + 2, kBarDone = kBarPEmpty + 2,
                       kBarSync = kBarDone + 1;
  static constexpr int kOffMisc = kOffBar + (kBarSync + 1) * 8;      // TMEM address, abort flag, scan
  // One 64-column tile is read as 128 rows of V^T (rows past 64 are not used): what follows the
  // last slot is inside the buffer.
  static constexpr int kEnd = kOffMisc + 128;
  static constexpr int kBytes = (kEnd > kOffQ + kBox ? kEnd : kOffQ + kBox) + 1024;
  static constexpr int kTmemCols = 2 * R + R * (kDP == 256 ? 2 : 1) <= 64 ? 64 : (R <= 32 ? 128 : 256);
  static_assert(kVSlots >= 2 && kVSlots >= kParts && kBytes <= 227 * 1024, "shared memory");
};

// The call's shape as the kernels use it.
struct Geometry {
  int M, groups, units;     // query rows of a key-value head; groups of R; units of a sequence
};

__device__ __forceinline__ Span span_of(const PagedLaunch& a, int b) {
  return fa::span_of(a.seq_lens[b], a.table_width << a.page_shift, a.T, a.window, kTile);
}

// A CTA's piece of the line of tiles, unit by unit; each role walks it by itself.
struct Walk {
  long long left;           // tiles of the piece from here on
  int b, unit, tile;        // sequence, unit in it, tile in the unit
  Span s;
  __device__ __forceinline__ bool more() const { return left > 0; }
  // tiles of this unit in the piece
  __device__ __forceinline__ int count() const { return static_cast<int>(min(left, static_cast<long long>(s.ntiles - tile))); }
  __device__ __forceinline__ void next(const PagedLaunch& a, int units) {
    left -= count();
    tile = 0;
    if (left <= 0) return;
    if (++unit == units) {
      unit = 0;
      do s = span_of(a, ++b);
      while (s.ntiles == 0);
    }
  }
};

__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// What a CTA leaves for the joining kernel: the unit that begins in its piece and goes on.
struct Split {
  int b, unit, pieces, pad;
};

struct Workspace {
  Split* splits;            // [kMaxCtas]
  float2* stats;            // [kMaxCtas][2][R]: reference maximum (log2), sum
  float* part;              // [kMaxCtas][2][R][DP]
};
template <int DP, int R>
__host__ __device__ inline Workspace workspace_view(void* ws) {
  Workspace w;
  w.splits = static_cast<Split*>(ws);
  w.stats = reinterpret_cast<float2*>(w.splits + kMaxCtas);
  w.part = reinterpret_cast<float*>(w.stats + kMaxCtas * 2 * R);
  return w;
}
size_t workspace_of(int DP, int R) {
  return kMaxCtas * (sizeof(Split) + 2 * R * (sizeof(float2) + DP * sizeof(float)));
}

template <int D, int R, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PagedLaunch a,
                           const __grid_constant__ Geometry geo) {
  using L = Smem<D, R>;
  constexpr int DP = L::kDP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  auto bar = [&](int i) { return sb + L::kOffBar + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffMisc + 4);
  long long* scan = reinterpret_cast<long long*>(smem + L::kOffMisc + 8);      // [7]
  int* found = reinterpret_cast<int*>(smem + L::kOffMisc + 72);                // the piece's first sequence
  long long* found_at = reinterpret_cast<long long*>(smem + L::kOffMisc + 80);
  int4* rows = reinterpret_cast<int4*>(smem + L::kOffRows);
  float* ref = reinterpret_cast<float*>(smem + L::kOffRef);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Workspace ws = workspace_view<DP, R>(a.workspace);

  if (tid == 0) {
    for (int i = 0; i < 2 * L::kSlots; ++i) mbar_init(bar(i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kBarQFull + i), 1);
      mbar_init(bar(L::kBarQEmpty + i), 1);
      mbar_init(bar(L::kBarSFull + i), 1);
      mbar_init(bar(L::kBarSEmpty + i), 128);
      mbar_init(bar(L::kBarPFull + i), 128);
      mbar_init(bar(L::kBarPEmpty + i), 1);
    }
    mbar_init(bar(L::kBarDone), 1);
    mbar_init(bar(L::kBarSync), 128);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }

  // All that the kernel before this one on the stream wrote: lengths, pages, q, and the workspace
  // that an earlier call's joining kernel still reads.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) ws.splits[blockIdx.x].pieces = 0;

  // This CTA's piece: the tiles of all sequences before each thread's share of them, then the
  // sequence in which the piece begins.
  const int share = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(a.B, tid * share), b_hi = min(a.B, b_lo + share);
  long long sum = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    sum += span_of(a, b).ntiles;
    if (blockIdx.x == 0 && (a.seq_lens[b] < 0 || a.seq_lens[b] > (a.table_width << a.page_shift)))
      atomicCAS(a.status, 0, kStatusIndex);
  }
  sum *= geo.units;
  long long before = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += y;
  }
  if (lane == 31) scan[warp] = before;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before -= sum;
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long start = per * blockIdx.x;
  const long long piece = min(per, total - start);
  if (piece > 0 && start >= before && start < before + sum) {
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = static_cast<long long>(span_of(a, b).ntiles) * geo.units;
      if (start < before + n) {
        *found = b;
        *found_at = start - before;
        break;
      }
      before += n;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // Sequences without a position have no tile: their rows are written here.
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (span_of(a, b).ntiles != 0) continue;
    const long long n = static_cast<long long>(a.H) * a.T;
    for (long long i = tid; i < n * (D / 8); i += kThreads)
      reinterpret_cast<uint4*>(a.o + b * n * D)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (long long i = tid; i < n; i += kThreads) a.lse[b * n + i] = -CUDART_INF_F;
  }

  Walk w;
  w.left = piece;
  w.b = 0;
  w.unit = w.tile = 0;
  if (piece > 0) {
    w.b = *found;
    w.s = span_of(a, w.b);
    w.unit = static_cast<int>(*found_at / w.s.ntiles);
    w.tile = static_cast<int>(*found_at % w.s.ntiles);
  }

  if (warp == 4 || warp == 6) {
    // ------------------------------------------------------------------ loads
    // A box of a small page takes its lane some hundred clocks to issue, so K and V have a warp each.
    const int kv = warp == 4 ? 0 : 1;
    const CUtensorMap* map = kv == 0 ? &tmK : &tmV;
    const int slots = kv == 0 ? L::kKSlots : L::kVSlots, full = kv == 0 ? L::kBarKFull : L::kBarVFull,
              empty = kv == 0 ? L::kBarKEmpty : L::kBarVEmpty;
    const uint32_t ring = sb + (kv == 0 ? 0 : L::kOffV);
    const int box_rows = min(kTile, 1 << a.page_shift), pages = kTile / box_rows;
    int fills = 0, u = 0;
    bool ok = true;
    // This lane's page of a tile: the table's entry is read a tile ahead and looked at only when it is
    // needed, so that nothing waits for the read; kNone where the lane has none to load.
    constexpr int kNone = INT_MIN;
    auto entry = [&](const Walk& w, int tile) {
      const long long j = static_cast<long long>(w.s.tile0 + tile) * kTile + lane * box_rows;
      if (lane >= pages || j >= w.s.len || j + box_rows <= w.s.first) return kNone;
      return max(a.block_table[static_cast<long long>(w.b) * a.table_width + (j >> a.page_shift)], -1);
    };
    int next = w.more() ? entry(w, w.tile) : kNone;
    while (ok && w.more()) {
      if (kv == 0) {
        const int qbuf = u % L::kBufs;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarQEmpty + qbuf), ((u / L::kBufs) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) {
          const int hk = w.unit / geo.groups, group = w.unit % geo.groups;
          const int q_row = (w.b * a.H + hk * (a.H / a.Hkv)) * a.T + group * R;
          mbar_arrive_expect_tx(bar(L::kBarQFull + qbuf), L::kQ);
          for (int c = 0; c < L::kNBox; ++c)
            tma_load_3d(sb + L::kOffQ + qbuf * L::kQ + c * R * 128, &tmQ, bar(L::kBarQFull + qbuf), c * 64, q_row, 0);
        }
        ++u;
      }
      const int end = w.tile + w.count();
      for (int t = w.tile; ok && t < end; ++t) {
        const int page = next;
        const long long j = static_cast<long long>(w.s.tile0 + t) * kTile + lane * box_rows;
        if (t + 1 < end) {
          next = entry(w, t + 1);
        } else {
          Walk n = w;
          n.next(a, geo.units);
          next = n.more() ? entry(n, n.tile) : kNone;
        }
        // pool row of the page's first position in the tile, or -1
        int cur = -1;
        if (page >= 0 && page < a.num_pages) cur = static_cast<int>(page_row_of(page, a.Hkv, w.unit / geo.groups, j, a.page_shift));
        else if (page != kNone) atomicCAS(a.status, 0, kStatusIndex);
        const unsigned valid = __ballot_sync(0xffffffffu, cur >= 0);
        const uint32_t bytes = static_cast<uint32_t>(__popc(valid)) * box_rows * 128 * L::kPartBoxes;
#pragma unroll
        for (int part = 0; part < L::kParts; ++part) {
          const int slot = fills % slots;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(empty + slot), ((fills / slots) & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            if (bytes > 0) mbar_arrive_expect_tx(bar(full + slot), bytes);
            else mbar_arrive(bar(full + slot));
          }
          __syncwarp();
          if (cur >= 0) {
#pragma unroll
            for (int c = 0; c < L::kPartBoxes; ++c)
              tma_load_3d(ring + slot * L::kSlot + c * kBox + lane * box_rows * 128, map, bar(full + slot),
                          (part * L::kPartBoxes + c) * 64, cur, 0);
          }
          ++fills;
        }
      }
      w.next(a, geo.units);
    }
    __syncwarp();
    if (!ok) {
      if (lane == 0) raise_error(a.status, abort_flag, kStatusTimeout);
      for (int f = max(0, fills - slots); f < fills; ++f) mbar_wait_drain(bar(full + f % slots), (f / slots) & 1);
      for (int q = max(0, u - L::kBufs); q < u; ++q)
        mbar_wait_drain(bar(L::kBarQFull + q % L::kBufs), (q / L::kBufs) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0 && w.more()) {
      constexpr uint32_t kIdS = idesc_16(128, R, false, false, F16);
      constexpr uint32_t kIdO = idesc_16(128, R, true, false, F16);        // A = V^T: MN-major
      const int n = static_cast<int>(w.left);
      int is = 0, ip = 0, u = 0;             // next S^T, next P V, unit of the next S^T
      int ks = 0, vs = 0;                    // parts of K and V taken so far (kParts a tile)
      int unit_end = w.count();              // first tile of the next unit
      uint32_t firsts = 1u;                  // bit i % 32: tile i is its unit's first
      bool ok = true;
      long long t0 = clock64();
      // Whichever product has its operands goes next; P V first, as it frees a slot.
      while (ip < n) {
        const int pbuf = ip % L::kBufs, vslot = vs % L::kVSlots, vpart = vs % L::kParts;
        if (ip < is && (vpart > 0 || mbar_test_wait(bar(L::kBarPFull + pbuf), (ip / L::kBufs) & 1)) &&
            mbar_test_wait(bar(L::kBarVFull + vslot), (vs / L::kVSlots) & 1)) {
          tc_fence_after();
          const uint32_t keep = (firsts >> (ip & 31)) & 1u ? 0u : 1u;
#pragma unroll
          for (int g = 0; g < 2; ++g)
            mma_ss_x4<128, 256, 384, 2, 4, 6>(
                tmem + 2 * R + vpart * R, sdesc_sw128(sb + L::kOffV + vslot * L::kSlot + g * 4 * 2048, kBox, 1024),
                sdesc_sw128(sb + L::kOffP + pbuf * L::kP + g * R * 128, 16, 1024), kIdO, g == 0 ? keep : 1u);
          tc_commit(bar(L::kBarVEmpty + vslot));
          ++vs;
          if (vpart == L::kParts - 1) {
            tc_commit(bar(L::kBarPEmpty + pbuf));
            ++ip;
          }
          t0 = clock64();
          continue;
        }
        const int kslot = ks % L::kKSlots, kpart = ks % L::kParts, sbuf = is & 1, qbuf = u % L::kBufs;
        if (is < n && mbar_test_wait(bar(L::kBarKFull + kslot), (ks / L::kKSlots) & 1) &&
            (kpart > 0 || (mbar_test_wait(bar(L::kBarSEmpty + sbuf), ((is >> 1) & 1) ^ 1) &&
                           mbar_test_wait(bar(L::kBarQFull + qbuf), (u / L::kBufs) & 1)))) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < L::kPartBoxes; ++c)
            mma_ss_x4<2, 4, 6, 2, 4, 6>(
                tmem + sbuf * R, sdesc_sw128(sb + kslot * L::kSlot + c * kBox, 16, 1024),
                sdesc_sw128(sb + L::kOffQ + qbuf * L::kQ + (kpart * L::kPartBoxes + c) * R * 128, 16, 1024), kIdS,
                (c > 0 || kpart > 0) ? 1u : 0u);
          tc_commit(bar(L::kBarKEmpty + kslot));
          ++ks;
          if (kpart == L::kParts - 1) {
            tc_commit(bar(L::kBarSFull + sbuf));
            ++is;
            firsts &= ~(1u << (is & 31));
            if (is == unit_end) {
              tc_commit(bar(L::kBarQEmpty + qbuf));
              firsts |= 1u << (is & 31);
              ++u;
              w.next(a, geo.units);
              unit_end = w.more() ? is + w.count() : n + 1;
            }
          }
          t0 = clock64();
          continue;
        }
        if (*abort_flag || clock64() - t0 > kWaitLimitCycles) {
          ok = false;
          break;
        }
      }
      if (!ok) raise_error(a.status, abort_flag, kStatusTimeout);
      tc_commit(bar(L::kBarDone));
      mbar_wait_drain(bar(L::kBarDone), 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax: one key a thread
    const uint32_t quad = static_cast<uint32_t>(warp * 32) << 16;
    const float scale2 = a.scale * kLog2e;
    const bool cap = a.softcap != 0.f;
    const float cap_in = cap ? a.scale / a.softcap : 0.f, cap_out = a.softcap * kLog2e;
    int i = 0;
    uint32_t sync_phase = 0;
    bool ok = true;
    // Barrier of the four warps; bounded like every wait, so that a failing CTA ends.
    auto sync = [&]() {
      mbar_arrive(bar(L::kBarSync));
      const bool done = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSync), sync_phase, abort_flag));
      sync_phase ^= 1;
      return done;
    };
    while (ok && w.more()) {
      const int n_tiles = w.count();
      const int hk = w.unit / geo.groups, r0 = w.unit % geo.groups * R;
      const int rows_here = min(R, geo.M - r0);
      const long long q_row = (static_cast<long long>(w.b) * a.H + hk * (a.H / a.Hkv)) * a.T + r0;
      const int* table = a.block_table + static_cast<long long>(w.b) * a.table_width;
      const int len = w.s.len;
      if (!(ok = sync())) break;  // the last unit's rows are read
      if (tid < R) {
        const int r = r0 + tid;
        int4 v = make_int4(-1, 0, 0, 0);
        if (tid < rows_here) {
          v.x = len - a.T + r % a.T;
          v.y = first_seen(v.x, a.window);
          v.z = a.slopes != nullptr ? __float_as_int(a.slopes[hk * (a.H / a.Hkv) + r / a.T] * kLog2e) : 0;
        }
        rows[tid] = v;
        ref[tid] = -CUDART_INF_F;
      }
      if (!(ok = sync())) break;
      // all rows see the positions from the last row's first to the first row's own
      const int all_from = first_seen(len - 1, a.window), all_to = len - a.T;
      float l[R];
#pragma unroll
      for (int n = 0; n < R; ++n) l[n] = 0.f;
      // row n's value of each warp, from lane n % 32 (two buffers: a thread may be a tile ahead of
      // one that still reads)
      auto share_row = [&](float* to, float lo, float hi) {
        if (lane < R) to[lane * 4 + warp] = lo;
        if (R > 32) to[(lane + 32) % R * 4 + warp] = hi;
      };
      auto live_at = [&](int tile) {
        const long long j = static_cast<long long>(w.s.tile0 + tile) * kTile + tid;
        return j >= w.s.first && j < len && page_of(table, a.table_width, a.page_shift, a.num_pages, j) >= 0;
      };
      bool live_next = live_at(w.tile);
      for (int t = 0; t < n_tiles; ++t, ++i) {
        const int tile = w.tile + t;
        const int j = (w.s.tile0 + tile) * kTile + tid;
        const bool live = live_next;
        if (t + 1 < n_tiles) live_next = live_at(tile + 1);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSFull + (i & 1)), (i >> 1) & 1, abort_flag));
        if (!ok) break;
        FA_CONVERGED(a.status);
        tc_fence_after();
        uint32_t x[R];
#pragma unroll
        for (int c = 0; c < R; c += 16) tmem_ld16(tmem + quad + (i & 1) * R + c, reinterpret_cast<uint32_t(&)[16]>(x[c]));
        tmem_ld_wait();
        reg_fence(x);
        tc_fence_before();
        mbar_arrive(bar(L::kBarSEmpty + (i & 1)));
        auto X = [&](int n) { return __uint_as_float(x[n]); };
        if (cap) {
          // The warp's way to tanh goes by its largest score (the two differ in the last bits), so what
          // lies in K's rows that no row sees, or is left there from an earlier tile, must not count.
          if (!live) {
#pragma unroll
            for (int n = 0; n < R; ++n) x[n] = 0u;
          }
          float most = 0.f;
#pragma unroll
          for (int n = 0; n < R; n += 2) most = fmax3_abs(most, X(n), X(n + 1));
          if (__all_sync(0xffffffffu, most * cap_in <= kTanhPolyLimit)) {
            const float tanh_c[5] = {kTanhC0, kTanhC1, kTanhC2, kTanhC3, kTanhC4};
#pragma unroll
            for (int n = 0; n < R; n += 2) {
              const float2 z = __fmul2_rn(make_float2(X(n), X(n + 1)), make_float2(cap_in, cap_in));
              const float2 th = __fmul2_rn(__fmul2_rn(z, quartic2(z, tanh_c)), make_float2(cap_out, cap_out));
              x[n] = __float_as_uint(th.x);
              x[n + 1] = __float_as_uint(th.y);
            }
          } else {
#pragma unroll
            for (int n = 0; n < R; ++n) x[n] = __float_as_uint(cap_out * tanhf(X(n) * cap_in));
          }
        } else {
#pragma unroll
          for (int n = 0; n < R; ++n) x[n] = __float_as_uint(X(n) * scale2);
        }
        if (a.slopes != nullptr) {
#pragma unroll
          for (int n = 0; n < R; ++n) {
            const int4 v = rows[n];
            x[n] = __float_as_uint(fmaf(-__int_as_float(v.z), static_cast<float>(v.x - j), X(n)));
          }
        }
        // some key of the warp is not seen by every row
        if (__any_sync(0xffffffffu, !live || j < all_from || j > all_to)) {
#pragma unroll
          for (int n = 0; n < R; ++n) {
            const int4 v = rows[n];
            if (!live || j > v.x || j < v.y) x[n] = 0xff800000u;
          }
        }
        float mine = 0.f, mine2 = 0.f;                   // the warp's maximum of row `lane` (and lane + 32)
#pragma unroll
        for (int n = 0; n < R; ++n) {
          const float v = redux_max(X(n));
          if (n < 32) mine = lane == n ? v : mine;
          else mine2 = lane == n - 32 ? v : mine2;
        }
        float* wmax = reinterpret_cast<float*>(smem + L::kOffMax) + (i & 1) * 4 * R;
        share_row(wmax, mine, mine2);
        // does a row of this warp's outgrow its reference?  (lane: its own rows)
        const bool mine_grew = (lane < R && mine > ref[lane % R] + kRescale) || (R > 32 && mine2 > ref[(lane + 32) % R] + kRescale);
        const bool grew = __any_sync(0xffffffffu, mine_grew);
        int* flags = reinterpret_cast<int*>(smem + L::kOffFlags) + (i & 1) * 4;
        if (lane == 0) flags[warp] = grew;
        if (!(ok = sync())) break;
        const int4 any = *reinterpret_cast<const int4*>(flags);
        // every thread reads the same flags, so the branch is uniform
        if (any.x | any.y | any.z | any.w) {
          if (tid < R) {
            const float4 v = *reinterpret_cast<const float4*>(wmax + 4 * tid);
            const float was = ref[tid], now = fmaxf(was, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
            ref[R + tid] = now == -CUDART_INF_F ? 1.f : ex2_approx(was - now);
            ref[tid] = now;
          }
          if (!(ok = sync())) break;
#pragma unroll
          for (int n = 0; n < R; ++n) l[n] *= ref[R + n];
          if (t > 0) {
            // O^T of the tiles so far: the last product must have been added
            ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarPEmpty + (i - 1) % L::kBufs), ((i - 1) / L::kBufs) & 1, abort_flag));
            if (!ok) break;
            FA_CONVERGED(a.status);
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < (DP + 127) / 128; ++h)
#pragma unroll
              for (int c = 0; c < R; c += 16) {
                uint32_t o[16];
                const uint32_t at = tmem + quad + 2 * R + h * R + c;
                tmem_ld16(at, o);
                tmem_ld_wait();
                reg_fence(o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ref[R + c + e]);
                tmem_st16(at, o);
              }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // the buffer's last product must have read it
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarPEmpty + i % L::kBufs), ((i / L::kBufs) & 1) ^ 1, abort_flag));
        if (!ok) break;
        // P^T as the K-major operand: row n holds 64 keys in 128 bytes, two boxes
        uint8_t* p_at = smem + L::kOffP + (i % L::kBufs) * L::kP + (tid >> 6) * (R * 128) + (tid & 7) * 2;
        const int chunk = (tid & 63) >> 3;
#pragma unroll
        for (int c = 0; c < R; c += 16) {
          float m[16];
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(ref + c + e);
            m[e] = v.x, m[e + 1] = v.y, m[e + 2] = v.z, m[e + 3] = v.w;
          }
          uint16_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p = ex2_approx(X(c + e) - (m[e] == -CUDART_INF_F ? 0.f : m[e]));
            l[c + e] += p;
            pk[e] = static_cast<uint16_t>(pack16<F16>(p, 0.f));
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<uint16_t*>(p_at + (c + e) * 128 + ((chunk ^ (e & 7)) << 4)) = pk[e];
        }
        if (__any_sync(0xffffffffu, !live)) {
          // V rows that nothing may see.  The tile's V has landed in its slots only if an earlier
          // tile's is out of them, so the product before comes first.
          if (i > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarPEmpty + (i - 1) % L::kBufs), ((i - 1) / L::kBufs) & 1, abort_flag));
#pragma unroll
          for (int part = 0; part < L::kParts; ++part) {
            const int f = i * L::kParts + part, slot = f % L::kVSlots;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(L::kBarVFull + slot), (f / L::kVSlots) & 1, abort_flag));
            if (!ok) break;
            if (live) continue;
#pragma unroll
            for (int c = 0; c < L::kPartBoxes; ++c)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(smem + L::kOffV + slot * L::kSlot + c * kBox + tid * 128 + q * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          if (!ok) break;
        }
        __syncwarp();
        fence_async_smem();
        mbar_arrive(bar(L::kBarPFull + i % L::kBufs));
      }
      if (!ok) break;
      // The unit's end in this piece.  Sums over the keys' threads: each step of the butterfly
      // halves the rows that a lane holds, so lane i is left with row i / (32 / R) (R = 64: two).
#pragma unroll
      for (int d = 16, h = R / 2; d > 0; d >>= 1, h >>= 1) {
        if (h >= 1) {
#pragma unroll
          for (int n = 0; n < R / 2; ++n) {
            if (n >= h) break;
            const bool up = (lane & d) != 0;
            const float give = up ? l[n] : l[n + h], keep = up ? l[n + h] : l[n];
            l[n] = keep + __shfl_xor_sync(0xffffffffu, give, d);
          }
        } else {
          l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
        }
      }
      float* wsum = reinterpret_cast<float*>(smem + L::kOffSum);
#pragma unroll
      for (int n = 0; n < (R > 32 ? 2 : 1); ++n)
        if (R >= 32 || lane % (R >= 32 ? 1 : 32 / R) == 0) wsum[((R >= 32 ? lane * (R / 32) : lane / (R >= 32 ? 1 : 32 / R)) + n) * 4 + warp] = l[n];
      if (!(ok = sync())) break;
      const bool whole = n_tiles == w.s.ntiles;
      const int part = static_cast<int>(blockIdx.x) * 2 + (w.tile == 0 ? 1 : 0);
      auto row_sum = [&](int n) {
        const float4 v = *reinterpret_cast<const float4*>(wsum + 4 * n);
        return (v.x + v.y) + (v.z + v.w);
      };
      if (tid < rows_here) {
        const float total_l = row_sum(tid), m = ref[tid];
        if (whole) a.lse[q_row + tid] = total_l == 0.f ? -CUDART_INF_F : (m + log2f(total_l)) * kLn2;
        else ws.stats[part * R + tid] = make_float2(m, total_l);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarPEmpty + (i - 1) % L::kBufs), ((i - 1) / L::kBufs) & 1, abort_flag));
      if (!ok) break;
      FA_CONVERGED(a.status);
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < (DP + 127) / 128; ++h) {
        const int d = h * 128 + tid;
#pragma unroll
        for (int c = 0; c < R; c += 16) {
          if (c >= rows_here) break;
          uint32_t o[16];
          tmem_ld16(tmem + quad + 2 * R + h * R + c, o);
          tmem_ld_wait();
          reg_fence(o);
          float f[16];
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float total_l = row_sum(c + e);
              f[e] = total_l == 0.f ? 0.f : rcp_approx(total_l);     // 2^-23, against a rounding to 16 bits
            }
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int n = c + e;
            if (n >= rows_here || d >= D) continue;
            if (whole) a.o[(q_row + n) * D + d] = static_cast<uint16_t>(pack16<F16>(__uint_as_float(o[e]) * f[e], 0.f));
            else ws.part[(static_cast<size_t>(part) * R + n) * DP + d] = __uint_as_float(o[e]);
          }
        }
      }
      tc_fence_before();
      if (!whole && w.tile == 0 && tid == 0) {
        // the pieces behind this one that hold the rest
        const long long rest = w.s.ntiles - n_tiles;
        ws.splits[blockIdx.x] = Split{w.b, w.unit, static_cast<int>((rest + per - 1) / per) + 1, 0};
      }
      w.next(a, geo.units);
    }
    if (!ok) raise_error(a.status, abort_flag, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// Joins the pieces of the unit that begins in CTA blockIdx.x's piece, row blockIdx.y.  Every warp
// finds the common maximum and the sum over all pieces, a lane for each; the warps take turns at the
// pieces' O, a lane D / 32 neighbouring columns.  All latency (an L2 read of what another SM has just
// written takes most of a microsecond), so O's loads, kFlight pieces a warp, go out before the
// factors are known.  At D = 256, with twice the registers in flight, half the warps.
template <int D>
constexpr int kJoinWarps = D == 256 ? 4 : 8;
template <int D, int R, bool F16>
__global__ void __launch_bounds__(32 * kJoinWarps<D>) paged_join_kernel(const __grid_constant__ PagedLaunch a,
                                                                        const __grid_constant__ Geometry geo) {
  constexpr int DP = tile_dim(D), E = D / 32, kFlight = D == 256 ? 5 : 10, kWarps = kJoinWarps<D>;
  __shared__ float sh_o[kWarps][D], sh_f[kMaxCtas];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Workspace ws = workspace_view<DP, R>(a.workspace);
  const Split s = ws.splits[blockIdx.x];
  const int n = blockIdx.y, r0 = s.unit % geo.groups * R;
  if (s.pieces == 0 || r0 + n >= geo.M) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // piece 0 is this CTA's second part, the others are the next CTAs' first
  auto part = [&](int i) { return (static_cast<int>(blockIdx.x) + i) * 2 + (i == 0 ? 1 : 0); };
  float p[kFlight][E];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int at = i0 + k * kWarps;
      const float* src = ws.part + (static_cast<size_t>(part(at)) * R + n) * DP + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) p[k][e] = 0.f;
      if (at < s.pieces) {
#pragma unroll
        for (int e = 0; e < E; ++e) p[k][e] = src[e];
      }
    }
  };
  load(warp);
  constexpr int kMost = (kMaxCtas + 31) / 32;
  float2 st[kMost];
  float m = -CUDART_INF_F, l = 0.f, o[E] = {};
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    st[c] = c * 32 + lane < s.pieces ? ws.stats[part(c * 32 + lane) * R + n] : make_float2(-CUDART_INF_F, 0.f);
    m = fmaxf(m, st[c].x);
  }
  m = redux_max(m);
  const float ref = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    const float f = ex2_approx(st[c].x - ref);                 // the piece's factor
    l = fmaf(f, st[c].y, l);
    if (warp == 0 && c * 32 + lane < s.pieces) sh_f[c * 32 + lane] = f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  __syncthreads();
  for (int i0 = warp; i0 < s.pieces; i0 += kWarps * kFlight) {
    if (i0 != warp) load(i0);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = i0 + k * kWarps;
      const float f = i < s.pieces ? sh_f[i] : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(f, p[k][e], o[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sh_o[warp][lane * E + e] = o[e];
  __syncthreads();
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long long row = (static_cast<long long>(s.b) * a.H + s.unit / geo.groups * (a.H / a.Hkv)) * a.T + r0 + n;
  for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sh_o[w][d];
    a.o[row * D + d] = static_cast<uint16_t>(pack16<F16>(sum * inv, 0.f));
  }
  if (threadIdx.x == 0) a.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// Rows of a group: the fewest that hold M, so that the products and exponentials of absent rows
// stay few; at D = 256 two key-value tiles leave room for 32.
int group_rows(int M, int D) { return M <= 16 ? 16 : (M <= 32 || D == 256 ? 32 : 64); }

template <int D, int R, bool F16>
cudaError_t launch_impl(const PagedLaunch& a, cudaStream_t stream) {
  using L = Smem<D, R>;
  Geometry geo;
  geo.M = a.H / a.Hkv * a.T;
  geo.groups = (geo.M + R - 1) / R;
  geo.units = a.Hkv * geo.groups;
  CUtensorMap tmQ, tmK, tmV;
  const long long pool_rows = (static_cast<long long>(a.num_pages) * a.Hkv) << a.page_shift;
  const int box_rows = a.page_shift < 7 ? 1 << a.page_shift : kTile;
  if (encode_tmap_3d(&tmQ, a.q, D, static_cast<long long>(a.B) * a.H * a.T, 1, R, F16) != 0 ||
      encode_tmap_3d(&tmK, a.k_pages, D, pool_rows, 1, box_rows, F16) != 0 ||
      encode_tmap_3d(&tmV, a.v_pages, D, pool_rows, 1, box_rows, F16) != 0)
    return cudaErrorInvalidValue;
  auto kern = paged_attention_kernel<D, R, F16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int ctas = a.num_sms < kMaxCtas ? a.num_sms : kMaxCtas;
  // Both launched as programmatic dependents: their set-up overlaps the end of the kernel before,
  // and griddepcontrol.wait holds what depends on it.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, kern, tmQ, tmK, tmV, a, geo)) != cudaSuccess) return e;
  cfg.gridDim = dim3(ctas, geo.M < R ? geo.M : R);
  cfg.blockDim = dim3(32 * kJoinWarps<D>);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, R, F16>, a, geo);
}

template <int D, bool F16>
cudaError_t launch_rows(const PagedLaunch& a, cudaStream_t stream) {
  switch (group_rows(a.H / a.Hkv * a.T, D)) {
    case 16: return launch_impl<D, 16, F16>(a, stream);
    case 32: return launch_impl<D, 32, F16>(a, stream);
    default:
      if constexpr (D == 256) return cudaErrorInvalidValue;
      else return launch_impl<D, 64, F16>(a, stream);
  }
}

template <bool F16>
cudaError_t launch_type(const PagedLaunch& a, cudaStream_t stream) {
  switch (a.D) {
    case 32: return launch_rows<32, F16>(a, stream);
    case 64: return launch_rows<64, F16>(a, stream);
    case 96: return launch_rows<96, F16>(a, stream);
    case 128: return launch_rows<128, F16>(a, stream);
    case 256: return launch_rows<256, F16>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

size_t paged_workspace_bytes(int H, int Hkv, int T, int D) {
  return workspace_of(tile_dim(D), group_rows(H / Hkv * T, D));
}

cudaError_t launch_paged_attention(const PagedLaunch& a, cudaStream_t stream) {
  return a.f16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace fa
