// fa_paged.cu -- attention of a few new tokens over a paged key-value cache.
#include <cstdint>
#include <math_constants.h>

#include "fa_internal.h"
#include "paged_index.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// One CTA per query row; its four warps take every fourth key each, a lane D / 32 columns.
template <int D, bool F16>
__global__ void __launch_bounds__(128) paged_attention_kernel(const __grid_constant__ PagedLaunch a) {
  constexpr int E = D / 32;
  const int t = blockIdx.x % a.T, h = blockIdx.x / a.T % a.H, b = blockIdx.x / a.T / a.H;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = (static_cast<long long>(b) * a.H + h) * a.T + t;
  const int hk = h / (a.H / a.Hkv);
  const int len = min(a.seq_lens[b], a.table_width << a.page_shift);
  if (len != a.seq_lens[b] && threadIdx.x == 0) atomicCAS(a.status, 0, kStatusIndex);
  const int p = len - a.T + t;                     // this row's position
  const int first = first_seen(p, a.window);
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = unpack16_lo<F16>(a.q[row * D + e * 32 + lane]);
    acc[e] = 0.f;
  }
  float m = -CUDART_INF_F, l = 0.f;
  const float slope = a.slopes != nullptr ? a.slopes[h] : 0.f;
  for (int j = first + warp; j <= p; j += 4) {
    const int page = page_of(a.block_table + static_cast<long long>(b) * a.table_width, a.table_width, a.page_shift, a.num_pages, j);
    if (page < 0) {
      if (lane == 0) atomicCAS(a.status, 0, kStatusIndex);
      continue;
    }
    const long long base = page_row_of(page, a.Hkv, hk, j, a.page_shift) * D;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], unpack16_lo<F16>(a.k_pages[base + e * 32 + lane]), s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale;
    if (a.softcap != 0.f) s = a.softcap * tanhf(s / a.softcap);
    s = (s - slope * static_cast<float>(p - j)) * kLog2e;
    const float m_new = fmaxf(m, s);
    const float alpha = exp2f(m - m_new), w = exp2f(s - m_new);
    l = l * alpha + w;
    m = m_new;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * alpha + w * unpack16_lo<F16>(a.v_pages[base + e * 32 + lane]);
  }
  __shared__ float sm[4], sl[4], sa[4][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int e = 0; e < E; ++e) sa[warp][e * 32 + lane] = acc[e];
  __syncthreads();
  if (warp != 0) return;
  m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  l = 0.f;
  float o[E] = {};
  for (int w = 0; w < 4; ++w) {
    const float f = sm[w] == -CUDART_INF_F ? 0.f : exp2f(sm[w] - m);
    l += f * sl[w];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += f * sa[w][e * 32 + lane];
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.o[row * D + e * 32 + lane] = static_cast<uint16_t>(pack16<F16>(o[e] * inv, 0.f));
  if (lane == 0) a.lse[row] = l == 0.f ? -CUDART_INF_F : (m / kLog2e + logf(l));
}

template <bool F16>
cudaError_t launch_type(const PagedLaunch& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(a.B) * a.H * a.T;
  switch (a.D) {
    case 32: paged_attention_kernel<32, F16><<<grid, 128, 0, stream>>>(a); break;
    case 64: paged_attention_kernel<64, F16><<<grid, 128, 0, stream>>>(a); break;
    case 96: paged_attention_kernel<96, F16><<<grid, 128, 0, stream>>>(a); break;
    case 128: paged_attention_kernel<128, F16><<<grid, 128, 0, stream>>>(a); break;
    default: paged_attention_kernel<256, F16><<<grid, 128, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace

size_t paged_workspace_bytes(int, int, int, int, int, int) { return 16; }

cudaError_t launch_paged_attention(const PagedLaunch& a, cudaStream_t stream) {
  return a.f16 ? launch_type<true>(a, stream) : launch_type<false>(a, stream);
}

}  // namespace fa
