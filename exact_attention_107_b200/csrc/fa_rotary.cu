// fa_rotary.cu -- rotary positions, alone (queries and keys of a sequence) and on the way into a
// paged key-value cache.
//
// Row x at position p turns its first R columns, pair by pair, by the angles whose cosines and
// sines row p of the table holds (fp32, cos[R/2] then sin[R/2]; the caller makes it in 64 bits):
//     a' = a cos - b sin,   b' = b cos + a sin
// with (a, b) = columns (i, i + R/2) in the half layout and (2i, 2i + 1) in the interleaved one;
// columns R.. are copied.  The gradient is the transpose: sin changes sign (`inverse`).  Products
// and sums are fp32, rounded once.
//
// Bound by memory: every element is read once and written once (16-byte accesses), the table row
// from L1 / L2.  A unit of a row is 8 columns, or 8 and their 8 partners (half layout with R a
// multiple of 16).  A thread keeps one unit of one token: it unpacks the angles once and turns up
// to kHeads heads of the token at a time, so that many loads are in flight.  Threads are laid out
// (unit, head, token): in a token-major input neighbouring threads read neighbouring bytes.
// Measured: 8 x 4096 tokens of 16 + 4 heads, D = 128, half layout 57 us (5.9 TB/s); 32767 tokens of
// 8 + 8 heads, interleaved, R = 64: 51 us (5.4 TB/s); append of 5 x 2000 ragged rows 22.8 us.  Half
// layouts with R not a multiple of 16 are bound by their shared-memory reads of single values: R = 66
// takes twice R = 128's time.  The launch bound of four blocks an SM holds threads to 64 registers:
// the append's ordinary half layout spills 32 bytes there and is faster than with three blocks all
// the same (launch_layout), the odd half layouts spill 36 to 48.
#include <cstdint>

#include "fa_internal.h"
#include "paged_index.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;

// How the pairs of a unit lie.
//   kHalfWide     half layout, R a multiple of 16: the thread holds both columns of its pairs
//   kInterleaved  pairs are neighbours; R a multiple of 8, so a unit turns whole or not at all
//   kHalfOdd, kInterleavedOdd   other R: the angles are read one by one, and the half layout's
//                 partners come out of shared memory, where the block leaves its rows
enum Layout { kHalfWide = 0, kInterleaved = 1, kHalfOdd = 2, kInterleavedOdd = 3 };

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = unpack16_lo<F16>(w[i]);
    f[2 * i + 1] = unpack16_hi<F16>(w[i]);
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack16<F16>(f[0], f[1]), pack16<F16>(f[2], f[3]), pack16<F16>(f[4], f[5]), pack16<F16>(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
  f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
  f[4] = y.x, f[5] = y.y, f[6] = y.z, f[7] = y.w;
}

// The heads of a token: `H` query heads, then `Hkv` key heads, then (paged) `Hkv` value heads.
template <int LAYOUT, bool F16, bool PAGED>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryLaunch a) {
  extern __shared__ uint4 staged[];                            // kHalfOdd: [token][head lane][kHeads][unit]
  constexpr bool kWide = LAYOUT == kHalfWide;
  const int u = threadIdx.x, lanes = blockDim.y;
  const int heads = a.H + a.Hkv * (PAGED ? 2 : 1);
  const unsigned tok = blockIdx.x * blockDim.z + threadIdx.z;
  const bool here = tok < static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N);
  if (LAYOUT != kHalfOdd && !here) return;
  const int b = here ? static_cast<int>(tok / static_cast<unsigned>(a.N)) : 0;
  const int n = here ? static_cast<int>(tok - static_cast<unsigned>(b) * static_cast<unsigned>(a.N)) : 0;
  const int half = a.R / 2, rot_units = kWide ? a.R / 16 : (a.R + 7) / 8;
  const int col0 = kWide && u >= rot_units ? 8 * u + half : 8 * u;
  const bool pair = kWide && u < rot_units;                    // this thread holds columns col0 and col0 + half

  const int fresh = PAGED && a.new_lens != nullptr ? a.new_lens[b] : a.N;
  uint4 x[kHeads], y[kHeads];
  bool on[kHeads];
  const long long q_at = b * a.q_stride[0] + n * a.q_stride[2] + col0;
  const long long k_at = b * a.k_stride[0] + n * a.k_stride[2] + col0;
  const long long v_at = PAGED ? b * a.v_stride[0] + n * a.v_stride[2] + col0 : 0;
  auto load = [&](int head0) {
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = head0 + i * lanes;
      on[i] = here && h < heads;
      x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
      if (!on[i] || (PAGED && n >= fresh)) continue;           // behind the sequence's last row: zeros
      const uint16_t* src = h < a.H ? a.q + (q_at + h * a.q_stride[1])
                            : !PAGED || h < a.H + a.Hkv ? a.k + (k_at + (h - a.H) * a.k_stride[1])
                                                        : a.v + (v_at + (h - a.H - a.Hkv) * a.v_stride[1]);
      x[i] = __ldcs(reinterpret_cast<const uint4*>(src));
      if (pair) y[i] = __ldcs(reinterpret_cast<const uint4*>(src + half));
    }
  };
  load(threadIdx.y);

  // position, and where the token's key and value go
  bool real = true, write = true;                              // real: not a row behind its sequence's last
  long long p = n, page_row = 0;                               // page_row: of key head 0 in the pool
  if (PAGED) {
    const AppendSlot at = append_slot(a.seq_lens[b], fresh, a.N, n,
                                      a.block_table + static_cast<long long>(b) * a.table_width, a.table_width,
                                      a.page_shift, a.num_pages);
    real = at.real;
    p = at.position;
    write = at.page >= 0;
    page_row = page_row_of(at.page, a.Hkv, 0, p, a.page_shift);
    // A key whose angles the table does not hold stays out of the cache: every thread of the token
    // decides alike, those of its values and of columns that do not turn too.
    if (a.R > 0 && p >= a.table_rows) write = false;
    if (here && ((real && !write) || fresh < 0)) atomicCAS(a.status, 0, kStatusIndex);
  } else if (a.positions != nullptr) {
    p = a.positions[static_cast<long long>(b) * a.position_stride + n];
  }
  // A position outside the table is reported and left unturned.
  bool turn = here && u < rot_units && real;
  if (turn && (p < 0 || p >= a.table_rows)) {
    atomicCAS(a.status, 0, kStatusIndex);
    turn = false;
  }
  // c: cosine of column j's pair; s: factor of column j's partner (first of a pair: minus the sine)
  float c[8], s[8];
  if (turn) {
    const float* row = a.table + p * a.R;
    if (kWide) {
      load8(row + 8 * u, c);
      load8(row + half + 8 * u, s);
    } else if (LAYOUT == kInterleaved) {
      const float4 cc = *reinterpret_cast<const float4*>(row + 4 * u);
      const float4 ss = *reinterpret_cast<const float4*>(row + half + 4 * u);
      c[0] = c[1] = cc.x, c[2] = c[3] = cc.y, c[4] = c[5] = cc.z, c[6] = c[7] = cc.w;
      s[0] = -ss.x, s[1] = ss.x, s[2] = -ss.y, s[3] = ss.y, s[4] = -ss.z, s[5] = ss.z, s[6] = -ss.w, s[7] = ss.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = 8 * u + j;
        const int at = LAYOUT == kInterleavedOdd ? col >> 1 : (col < half ? col : col - half);
        const bool in = col < a.R;
        c[j] = in ? row[at] : 1.f;
        s[j] = in ? row[half + at] : 0.f;
        if (LAYOUT == kInterleavedOdd ? (j & 1) == 0 : col < half) s[j] = -s[j];
      }
    }
    if (a.inverse) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = -s[j];
    }
  }

  for (int head0 = threadIdx.y;;) {
    const uint16_t* mine = nullptr;                            // kHalfOdd: this thread's rows in shared memory
    if (LAYOUT == kHalfOdd) {
      uint4* rows = staged + (threadIdx.z * lanes + threadIdx.y) * kHeads * blockDim.x;
#pragma unroll
      for (int i = 0; i < kHeads; ++i)
        if (on[i]) rows[i * blockDim.x + u] = x[i];
      mine = reinterpret_cast<const uint16_t*>(rows);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = head0 + i * lanes;
      if (!on[i]) continue;
      const bool is_q = h < a.H, is_v = PAGED && h >= a.H + a.Hkv;
      uint16_t* dst;
      if (is_q) {
        dst = a.q_out + ((static_cast<long long>(b) * a.H + h) * a.N + n) * a.D + col0;
      } else if (PAGED) {
        if (!real || !write) continue;
        const int hk = is_v ? h - a.H - a.Hkv : h - a.H;
        dst = (is_v ? a.v_out : a.k_out) + (page_row + (static_cast<long long>(hk) << a.page_shift)) * a.D + col0;
      } else {
        dst = a.k_out + ((static_cast<long long>(b) * a.Hkv + (h - a.H)) * a.N + n) * a.D + col0;
      }
      uint4 lo = x[i], hi = y[i];
      if (turn && !is_v) {
        float f[8], o[8];
        unpack8<F16>(x[i], f);
        if (kWide) {
          float g[8], o2[8];
          unpack8<F16>(y[i], g);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j] = f[j] * c[j] - g[j] * s[j];
            o2[j] = g[j] * c[j] + f[j] * s[j];
          }
          hi = pack8<F16>(o2);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float partner = f[j ^ 1];
            if (LAYOUT == kHalfOdd) {
              const int col = col0 + j;
              // columns past R have s = 0, and their own value is one that is there
              const int other = col >= a.R ? col : (col < half ? col + half : col - half);
              partner = unpack16_lo<F16>(mine[i * blockDim.x * 8 + other]);
              if (col >= a.R) partner = 0.f;
            }
            if (LAYOUT == kInterleavedOdd && col0 + j >= a.R) partner = 0.f;
            o[j] = f[j] * c[j] + partner * s[j];
          }
        }
        lo = pack8<F16>(o);
      }
      *reinterpret_cast<uint4*>(dst) = lo;
      if (pair) *reinterpret_cast<uint4*>(dst + half) = hi;
    }
    head0 += kHeads * lanes;
    // the same for every thread of the block: the first head lane decides
    if (head0 - static_cast<int>(threadIdx.y) >= heads) break;
    if (LAYOUT == kHalfOdd) __syncthreads();                   // the rows are read
    load(head0);
  }
}

template <int LAYOUT, bool F16, bool PAGED>
cudaError_t launch_layout(const RotaryLaunch& a, cudaStream_t stream) {
  const int heads = a.H + a.Hkv * (PAGED ? 2 : 1);
  const int units = LAYOUT == kHalfWide ? a.R / 16 + (a.D - a.R) / 8 : a.D / 8;
  // Heads a thread takes: kHeads at a time, and twice as many where there is work for every SM
  // anyway, as a thread's set-up (position, page, angles) costs as much as its four heads.  Ragged
  // append of 5 x 2000 tokens, 24 heads: 22.7 us with four, 20.7 with eight (19.5 with four blocks
  // an SM, the launch bound above); interleaved backward of 32767 tokens, 16 heads: 57.6 and 51.4 us.
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const int once = (heads + kHeads - 1) / kHeads;
  int lanes = tokens * units * once >= 1024LL * 148 ? (heads + 2 * kHeads - 1) / (2 * kHeads) : once;
  if (lanes > kThreads / units) lanes = kThreads / units;
  int per_block = kThreads / (units * lanes);
  if (per_block > 64) per_block = 64;                          // the grid's z limit of a block
  if (per_block > tokens) per_block = static_cast<int>(tokens);
  const dim3 block(units, lanes, per_block);
  const size_t smem = LAYOUT == kHalfOdd ? sizeof(uint4) * units * lanes * per_block * kHeads : 0;
  rotary_kernel<LAYOUT, F16, PAGED><<<static_cast<unsigned>((tokens + per_block - 1) / per_block), block, smem, stream>>>(a);
  return cudaGetLastError();
}

template <bool F16, bool PAGED>
cudaError_t launch_type(const RotaryLaunch& a, cudaStream_t stream) {
  if (a.R == 0) return launch_layout<kInterleaved, F16, PAGED>(a, stream);
  if (a.interleaved)
    return a.R % 8 == 0 ? launch_layout<kInterleaved, F16, PAGED>(a, stream)
                        : launch_layout<kInterleavedOdd, F16, PAGED>(a, stream);
  return a.R % 16 == 0 ? launch_layout<kHalfWide, F16, PAGED>(a, stream) : launch_layout<kHalfOdd, F16, PAGED>(a, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream) {
  if (a.paged) return a.f16 ? launch_type<true, true>(a, stream) : launch_type<false, true>(a, stream);
  return a.f16 ? launch_type<true, false>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace fa
