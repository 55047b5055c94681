// fa_mask.cu -- builds the mask plan of the score-modified attention: per query row the interval
// of keys that it sees, and per 128-row tile what the kernels may skip (layout: MaskPlan).
//
// Every mask offered is an interval [lo_i, hi_i) per row i:
//   documents   runs of equal ids: lo, hi = first row of i's run, one past its last; id < 0: nothing
//   causal      hi = min(hi, i + 1)
//   prefix      hi = max(i + 1, prefix) (causal, without documents)
//   window w    lo = max(lo, i - w + 1), and without causal hi = min(hi, i + w)
//
// One CTA per batch element.  The rows' run starts become one bit each (a ballot per warp, ids read
// once, coalesced); a scan over the N / 32 words gives each word the last start before it and the
// first one after it, so a row finds its run with a bit scan in its own word.  Bound by latency,
// not by its 4 bytes read and 8.2 written a row: 1024 threads of one SM walk all N rows (15 us for the
// documents of 16384 rows, 5 us for a prefix mask of 2777).
#include <climits>
#include <cstdint>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kThreads = 1024;

// Inclusive scan over the CTA's threads with `op`; `buf` holds 32 ints.
template <typename Op>
__device__ __forceinline__ int block_scan(int x, int* buf, int identity, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x = op(y, x);
  }
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = buf[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, d);
      if (lane >= d) y = op(z, y);
    }
    buf[lane] = y;
  }
  __syncthreads();
  const int before = warp > 0 ? buf[warp - 1] : identity;
  __syncthreads();
  return op(before, x);
}

__global__ void __launch_bounds__(kThreads) mask_plan_kernel(int* __restrict__ plan, const int* __restrict__ documents,
                                                             const int* __restrict__ prefix, int N, int causal,
                                                             int window) {
  extern __shared__ int sh[];
  const int b = blockIdx.x, B = gridDim.x;
  const int nt = (N + 127) / 128, npad = nt * 128, nw = npad / 32;
  int* tile_lo = sh;                 // [nt] smallest key seen by a row of the tile
  int* tile_hi = tile_lo + nt;       // [nt] one past the largest
  int* scan_buf = tile_hi + nt;      // [32]
  unsigned* starts = reinterpret_cast<unsigned*>(scan_buf + 32);   // [nw] (documents only, as the next two)
  int* last_before = reinterpret_cast<int*>(starts + nw);          // [nw] last run start in the words before
  int* first_after = last_before + nw;                              // [nw] first run start in the words after
  unsigned* padding = reinterpret_cast<unsigned*>(first_after + nw);   // [nw] rows with a negative id
  const MaskPlan v = mask_plan_view(plan, B, N);
  int2* rows = const_cast<int2*>(v.rows) + static_cast<size_t>(b) * npad;
  int2* order = const_cast<int2*>(v.order) + static_cast<size_t>(b) * nt;
  int4* tiles = const_cast<int4*>(v.tiles) + static_cast<size_t>(b) * nt;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int* doc = documents != nullptr ? documents + static_cast<size_t>(b) * N : nullptr;

  for (int t = threadIdx.x; t < nt; t += kThreads) {
    tile_lo[t] = INT_MAX;
    tile_hi[t] = 0;
  }
  if (doc != nullptr) {
    for (int w0 = warp; w0 < nw; w0 += 8 * (kThreads / 32)) {
      int id[8], before[8];                              // eight words' loads in flight
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = (w0 + u * (kThreads / 32)) * 32 + lane;
        id[u] = i < N ? doc[i] : 0;
        before[u] = lane == 0 && i > 0 && i <= N ? doc[i - 1] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int w = w0 + u * (kThreads / 32), i = w * 32 + lane;
        const int left = __shfl_up_sync(0xffffffffu, id[u], 1);
        const unsigned first = __ballot_sync(0xffffffffu, i < N && (i == 0 || id[u] != (lane == 0 ? before[u] : left)));
        const unsigned pad = __ballot_sync(0xffffffffu, i < N && id[u] < 0);
        if (lane == 0 && w < nw) starts[w] = first, padding[w] = pad;
      }
    }
    __syncthreads();
    // each thread owns `per` consecutive words
    const int per = (nw + kThreads - 1) / kThreads;
    const int w0 = threadIdx.x * per, w1 = min(nw, w0 + per);
    int last = -1, first = INT_MAX;
    for (int w = w0; w < w1; ++w)
      if (starts[w] != 0u) last = w * 32 + 31 - __clz(starts[w]);
    for (int w = w1 - 1; w >= w0; --w)
      if (starts[w] != 0u) first = w * 32 + __ffs(starts[w]) - 1;
    // starts grow with the position: a running maximum from the left, a running minimum from the right
    const int upto = block_scan(last, scan_buf, -1, [](int a, int c) { return max(a, c); });
    int before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 31) scan_buf[warp] = upto;
    __syncthreads();
    if (lane == 0) before = warp > 0 ? scan_buf[warp - 1] : -1;
    __syncthreads();
    int carry = before;
    for (int w = w0; w < w1; ++w) {
      last_before[w] = carry;
      if (starts[w] != 0u) carry = w * 32 + 31 - __clz(starts[w]);
    }
    // suffix minimum: warp-level shuffles down, then over the warps
    int x = first;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, x, d);
      if (lane + d < 32) x = min(x, y);
    }
    if (lane == 0) scan_buf[warp] = x;
    __syncthreads();
    int after = __shfl_down_sync(0xffffffffu, x, 1);
    if (lane == 31) after = INT_MAX;
    for (int w = warp + 1; w < kThreads / 32; ++w) after = min(after, scan_buf[w]);
    carry = after;
    for (int w = w1 - 1; w >= w0; --w) {
      first_after[w] = carry;
      if (starts[w] != 0u) carry = w * 32 + __ffs(starts[w]) - 1;
    }
  }
  __syncthreads();

  const int pre = prefix != nullptr ? min(prefix[b], N) : 0;
#pragma unroll 2
  for (int w = warp; w < nw; w += kThreads / 32) {
    const int i = w * 32 + lane;
    int lo = 0, hi = N;
    if (i >= N) {
      hi = 0;
    } else {
      if (doc != nullptr) {
        const unsigned bits = starts[w];
        const unsigned upto = bits & (0xffffffffu >> (31 - lane));
        const unsigned past = lane == 31 ? 0u : bits & (0xffffffffu << (lane + 1));
        lo = upto != 0u ? w * 32 + 31 - __clz(upto) : last_before[w];
        hi = past != 0u ? w * 32 + __ffs(past) - 1 : min(first_after[w], N);
        if ((padding[w] >> lane) & 1u) hi = lo;
      }
      if (causal) hi = min(hi, max(i + 1, pre));
      if (window > 0) {
        lo = max(lo, i - window + 1);
        if (!causal && i < N - window) hi = min(hi, i + window);
      }
      if (hi <= lo) lo = hi = 0;
    }
    rows[i] = make_int2(lo, hi);
    const int min_lo = __reduce_min_sync(0xffffffffu, hi > lo ? lo : INT_MAX);
    const int max_hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&tile_lo[w >> 2], min_lo);
      atomicMax(&tile_hi[w >> 2], max_hi);
    }
  }
  __syncthreads();
  // Key tile kt is met by the query tiles whose range holds it; every mask here makes them
  // neighbours, up to tiles of rows that see nothing.  Work of a query block: its two tiles' ranges.
  int* q_work = scan_buf + 32;       // [nt] over the run starts, which are read
  int* k_work = q_work + nt;         // [nt]
  const int nqb = (nt + 1) / 2;
  __syncthreads();
  // eight threads an item; whole warps go round, so that the shuffles are full
  const int part = threadIdx.x & 7;
  for (int t0 = 0; t0 < nt; t0 += kThreads / 8) {
    const int t = t0 + static_cast<int>(threadIdx.x >> 3);
    int q_first = INT_MAX, q_end = 0;
    if (t < nt) {
      for (int q = part; q < nt; q += 8) {
        if (tile_hi[q] > t * 128 && tile_lo[q] < t * 128 + 128) {
          q_first = min(q_first, q);
          q_end = q + 1;
        }
      }
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
      q_first = min(q_first, __shfl_xor_sync(0xffffffffu, q_first, d));
      q_end = max(q_end, __shfl_xor_sync(0xffffffffu, q_end, d));
    }
    if (t < nt && part == 0) {
      int4 r = make_int4(0, 0, 0, 0);
      if (tile_hi[t] > 0) {
        r.x = tile_lo[t] / 128;
        r.y = (tile_hi[t] + 127) / 128;
      }
      if (q_end > 0) {
        r.z = q_first;
        r.w = q_end;
      }
      tiles[t] = r;
      k_work[t] = r.w - r.z;
      q_work[t] = r.y - r.x;
    }
  }
  __syncthreads();
  int* block_work = k_work + nt;     // [nqb]
  for (int t = threadIdx.x; t < nqb; t += kThreads) block_work[t] = q_work[2 * t] + (2 * t + 1 < nt ? q_work[2 * t + 1] : 0);
  __syncthreads();
  // place of each item: the items with more work, and those with as much before it
  for (int t0 = 0; t0 < nt; t0 += kThreads / 8) {
    const int t = t0 + static_cast<int>(threadIdx.x >> 3);
    int k_at = 0, q_at = 0;
    if (t < nt) {
      const int kw = k_work[t], qw = t < nqb ? block_work[t] : 0;
      for (int o = part; o < nt; o += 8) k_at += k_work[o] > kw || (k_work[o] == kw && o < t);
      if (t < nqb)
        for (int o = part; o < nqb; o += 8) q_at += block_work[o] > qw || (block_work[o] == qw && o < t);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) {
      k_at += __shfl_xor_sync(0xffffffffu, k_at, d);
      q_at += __shfl_xor_sync(0xffffffffu, q_at, d);
    }
    if (t < nt && part == 0) {
      order[k_at].x = t;
      order[t < nqb ? q_at : t].y = t;                   // past the blocks: never read
    }
  }
}

}  // namespace

cudaError_t launch_mask_plan(int* plan, const int* documents, const int* prefix, int B, int N, int causal, int window,
                             cudaStream_t stream) {
  const size_t nt = (static_cast<size_t>(N) + 127) / 128;
  const size_t bytes = (2 * nt + 32 + (documents != nullptr ? 4 * 4 * nt : 3 * nt)) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(mask_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(bytes));
  if (e != cudaSuccess) return e;
  mask_plan_kernel<<<B, kThreads, bytes, stream>>>(plan, documents, prefix, N, causal, window);
  return cudaGetLastError();
}

}  // namespace fa
