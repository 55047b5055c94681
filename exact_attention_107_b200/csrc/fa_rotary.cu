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
// Bound by memory: every element is read once and written once (16-byte loads and stores), the
// table row from L1 / L2.  Work is laid out over (token, head, unit): a unit is 8 columns
// (interleaved, or a half layout whose halves do not split into 8s, where the partner columns are
// read one by one from L1), or 8 + 8 partner columns (half layout with R a multiple of 16).
// Consecutive threads take consecutive units, then heads of one token, which is the order of
// token-major inputs; each thread handles up to kHeads heads of its token, so the angles are read
// and unpacked once and several loads are in flight.
#include <cstdint>

#include "fa_internal.h"
#include "paged_index.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

enum Layout { kHalfWide = 0, kInterleaved = 1, kHalfOdd = 2 };

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
template <bool F16>
__device__ __forceinline__ float load16(const uint16_t* p) {
  return unpack16_lo<F16>(static_cast<uint32_t>(*p));
}

// The heads of a token: `H` query heads, then `Hkv` key heads, then (paged) `Hkv` value heads.
template <int LAYOUT, bool F16, bool PAGED, int HEADS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryLaunch a, int tokens_per_block,
                                                          int units, int head_lanes) {
  const int heads = a.H + a.Hkv * (PAGED ? 2 : 1);
  const int width = head_lanes * units;                        // work items of a token
  const int tokens = a.B * a.N;
  const int rot_units = LAYOUT == kHalfWide ? a.R / 16 : units;
  for (int l = threadIdx.x; l < tokens_per_block * width; l += kThreads) {
    const int tok = static_cast<int>(blockIdx.x) * tokens_per_block + l / width;
    if (tok >= tokens) return;
    const int item = l % width;
    const int head0 = item / units, u = item % units;
    const int b = tok / a.N, n = tok % a.N;

    // position, and where the token's key and value go
    bool real = true;                                          // false: a row behind its sequence's last
    long long p = n;
    long long page_row = 0;                                    // (page * Hkv) * page_size + slot
    bool write = true;
    if (PAGED) {
      const AppendSlot at = append_slot(a.seq_lens[b], a.new_lens != nullptr ? a.new_lens[b] : a.N, a.N, n,
                                        a.block_table + static_cast<long long>(b) * a.table_width, a.table_width,
                                        a.page_shift, a.num_pages);
      real = at.real;
      p = at.position;
      write = at.page >= 0;
      page_row = page_row_of(at.page, a.Hkv, 0, p, a.page_shift);
      if (real && !write) atomicCAS(a.status, 0, kStatusIndex);
    } else if (a.positions != nullptr) {
      p = a.positions[static_cast<long long>(b) * a.position_stride + n];
    }
    // A position outside the table is reported and left unturned.
    bool turn = u < rot_units && a.R > 0 && real;
    if (turn && (p < 0 || p >= a.table_rows)) {
      atomicCAS(a.status, 0, kStatusIndex);
      turn = false;
    }
    float c[8], s[8];
    const float* row = a.table + (turn ? p * a.R : 0);
    if (LAYOUT == kHalfWide) {
      if (turn) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(row + 8 * u + i);
          const float4 y = *reinterpret_cast<const float4*>(row + a.R / 2 + 8 * u + i);
          c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
          s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int col = 8 * u + i;
        const int pair = LAYOUT == kInterleaved ? col >> 1 : (col < a.R / 2 ? col : col - a.R / 2);
        const bool in = turn && col < a.R;
        c[i] = in ? row[pair] : 1.f;
        s[i] = in ? row[a.R / 2 + pair] : 0.f;
        // the sign of the partner's term: minus for the first of a pair
        if (LAYOUT == kInterleaved ? (i & 1) == 0 : col < a.R / 2) s[i] = -s[i];
      }
    }
    if (a.inverse) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
    const int col0 = LAYOUT == kHalfWide ? (u < rot_units ? 8 * u : 8 * u + a.R / 2) : 8 * u;

    uint4 x[HEADS], y[HEADS];
    const uint16_t* src[HEADS];
    uint16_t* dst[HEADS];
    bool on[HEADS], value[HEADS];
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const int h = head0 + i * head_lanes;
      on[i] = h < heads;
      value[i] = PAGED && h >= a.H + a.Hkv;
      src[i] = nullptr;
      dst[i] = nullptr;
      if (!on[i]) continue;
      if (h < a.H) {
        src[i] = a.q + b * a.q_stride[0] + h * a.q_stride[1] + n * a.q_stride[2];
        dst[i] = a.q_out + ((static_cast<long long>(b) * a.H + h) * a.N + n) * a.D;
      } else {
        const int hk = value[i] ? h - a.H - a.Hkv : h - a.H;
        const long long* st = value[i] ? a.v_stride : a.k_stride;
        src[i] = (value[i] ? a.v : a.k) + b * st[0] + hk * st[1] + n * st[2];
        if (PAGED) {
          on[i] = real && write;
          dst[i] = (value[i] ? a.v_out : a.k_out) + (page_row + (static_cast<long long>(hk) << a.page_shift)) * a.D;
        } else {
          dst[i] = a.k_out + ((static_cast<long long>(b) * a.Hkv + hk) * a.N + n) * a.D;
        }
      }
      if (!on[i]) continue;
      src[i] += col0;
      dst[i] += col0;
      x[i] = *reinterpret_cast<const uint4*>(src[i]);
      if (LAYOUT == kHalfWide && u < rot_units) y[i] = *reinterpret_cast<const uint4*>(src[i] + a.R / 2);
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      if (!on[i]) continue;
      if (PAGED && !real) {                                    // only query heads get here
        *reinterpret_cast<uint4*>(dst[i]) = make_uint4(0u, 0u, 0u, 0u);
        if (LAYOUT == kHalfWide && u < rot_units) *reinterpret_cast<uint4*>(dst[i] + a.R / 2) = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      if (!turn || value[i]) {
        *reinterpret_cast<uint4*>(dst[i]) = x[i];
        if (LAYOUT == kHalfWide && u < rot_units) *reinterpret_cast<uint4*>(dst[i] + a.R / 2) = y[i];
        continue;
      }
      float f[8], g[8], o[8];
      unpack8<F16>(x[i], f);
      if (LAYOUT == kHalfWide) {
        unpack8<F16>(y[i], g);
        float o2[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = f[j] * c[j] - g[j] * s[j];
          o2[j] = g[j] * c[j] + f[j] * s[j];
        }
        *reinterpret_cast<uint4*>(dst[i] + a.R / 2) = pack8<F16>(o2);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float partner = 0.f;
          if (LAYOUT == kInterleaved) {
            partner = f[j ^ 1];
          } else {
            const int col = col0 + j;
            if (col < a.R) partner = load16<F16>(src[i] + j + (col < a.R / 2 ? a.R / 2 : -(a.R / 2)));
          }
          o[j] = f[j] * c[j] + partner * s[j];
        }
      }
      *reinterpret_cast<uint4*>(dst[i]) = pack8<F16>(o);
    }
  }
}

template <int LAYOUT, bool F16, bool PAGED, int HEADS>
cudaError_t launch_heads(const RotaryLaunch& a, cudaStream_t stream) {
  const int heads = a.H + a.Hkv * (PAGED ? 2 : 1);
  const int units = LAYOUT == kHalfWide ? a.R / 16 + (a.D - a.R) / 8 : a.D / 8;
  const int head_lanes = (heads + HEADS - 1) / HEADS;
  const long long width = static_cast<long long>(head_lanes) * units;
  int per_block = static_cast<int>(kThreads / width);
  if (per_block < 1) per_block = 1;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  rotary_kernel<LAYOUT, F16, PAGED, HEADS>
      <<<static_cast<unsigned>((tokens + per_block - 1) / per_block), kThreads, 0, stream>>>(a, per_block, units, head_lanes);
  return cudaGetLastError();
}

template <int LAYOUT, bool F16, bool PAGED>
cudaError_t launch_layout(const RotaryLaunch& a, cudaStream_t stream) {
  return launch_heads<LAYOUT, F16, PAGED, 1>(a, stream);
}

template <bool F16, bool PAGED>
cudaError_t launch_type(const RotaryLaunch& a, cudaStream_t stream) {
  if (a.R == 0 || a.interleaved) return launch_layout<kInterleaved, F16, PAGED>(a, stream);
  return a.R % 16 == 0 ? launch_layout<kHalfWide, F16, PAGED>(a, stream) : launch_layout<kHalfOdd, F16, PAGED>(a, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream) {
  if (a.paged) return a.f16 ? launch_type<true, true>(a, stream) : launch_type<false, true>(a, stream);
  return a.f16 ? launch_type<true, false>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace fa
