// fa_internal.h -- launch interfaces between the C ABI (fa_api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

constexpr int kStatusLaunch = 6;   // FA_ERR_LAUNCH (a kernel found its launch unusable)
constexpr int kStatusTimeout = 7;  // FA_ERR_TIMEOUT
constexpr int kStatusIndex = 13;   // FA_ERR_INDEX (a page, position or length outside its table)

// Order of the CTAs of a (head, tile) grid.  Heads are taken in groups of `hg` whose
// data fits in L2 together; inside a group the order is tile-major (tile 0 of every
// head of the group first, then tile 1, ...), so that with causal masking the heaviest
// tiles of a group start first, and CTAs that run at the same time share their heads'
// K/V (forward) or Q/dO/dQ (backward) through L2 instead of re-reading device memory.
struct WorkItem {
  int bh, tile;
};
__host__ __device__ inline WorkItem grouped_order(int cta, int BH, int ntiles, int hg) {
  const long long per_group = static_cast<long long>(hg) * ntiles;
  const int g = static_cast<int>(cta / per_group);
  const int local = static_cast<int>(cta - g * per_group);
  const int gh = (BH - g * hg) < hg ? (BH - g * hg) : hg;     // the last group may be smaller
  return {g * hg + local % gh, local / gh};
}

// What the score-modified paths add to a call (the MOD instances of the forward and
// fused backward kernels).  All pointers are device pointers.
struct ScoreMods {
  const int* plan;      // key intervals and tile ranges (see MaskPlan), or null: full / causal by `causal`
  const float* slopes;  // per query head, or null: no distance bias
  float softcap;        // 0: none
  int H, Hkv;           // query and key-value heads per batch element
  int causal;           // without a plan: 1 = key j visible to query i iff j <= i
  // softcap: out tanh(in s) = s (poly[0] + poly[1] s^2 + ...) for |s| <= poly_limit, set by
  // set_cap_poly.  poly_limit < 0 (coefficients beyond the floats' normal range): s stands for
  // tanh(in s) itself.
  float poly[5], poly_limit;
};
// The polynomial of out tanh(in s) (coefficients of tanh: kTanhC0 .. kTanhC4).
inline void set_cap_poly(ScoreMods* m, double in, double out, const float (&tanh_c)[5], float limit) {
  m->poly_limit = static_cast<float>(limit / in);
  double power = in * out;
  for (int j = 0; j < 5; ++j, power *= in * in) {
    const double c = tanh_c[j] * power;
    m->poly[j] = static_cast<float>(c);
    if (!(c * c > 1e-72 && c * c < 1e72)) m->poly_limit = -1.f;
  }
  if (m->poly_limit < 0.f) {
    m->poly[0] = static_cast<float>(out);
    m->poly[1] = m->poly[2] = m->poly[3] = 0.f;
    m->poly[4] = 1e-37f;          // nothing next to poly[0]; -inf still gives -inf, not inf * 0
  }
}

// Layout of a mask plan for B batch elements of N rows (int32, 16-byte aligned), Npad = N
// rounded up to a multiple of 128, nt = Npad / 128:
//   rows    [B][Npad]  int2  (lo, hi): row i sees the keys lo <= j < hi (padding rows: 0, 0)
//   tiles   [B][nt]    int4  (first, end) key tile that query tile t meets, (first, end) query tile
//                            that key tile t meets; first = end where there is none
//   order   [B][nt]    int2  x: the key tiles, those that meet most query tiles first; y: the same
//                            for blocks of two query tiles ((nt + 1) / 2 of them): long work items
//                            started last leave the other SMs idle at the end
struct MaskPlan {
  const int2* rows;
  const int4* tiles;
  const int2* order;
};
__host__ __device__ inline size_t mask_plan_ints(size_t B, size_t N) {
  const size_t npad = (N + 127) / 128 * 128;
  return B * (2 * npad + (4 + 2) * (npad / 128));
}
__host__ __device__ inline MaskPlan mask_plan_view(const int* plan, int B, int N) {
  const size_t npad = (static_cast<size_t>(N) + 127) / 128 * 128;
  MaskPlan v;
  v.rows = reinterpret_cast<const int2*>(plan);
  v.tiles = reinterpret_cast<const int4*>(v.rows + B * npad);
  v.order = reinterpret_cast<const int2*>(v.tiles + B * (npad / 128));
  return v;
}
// Builds a plan from optional document ids (B, N) and prefix lengths (B) (fa_mask.cu).
cudaError_t launch_mask_plan(int* plan, const int* documents, const int* prefix, int B, int N, int causal, int window,
                             cudaStream_t stream);

// Shared by the C-ABI files: per-device status word and SM count of the current device, and
// tensor-map encoding (fa_api.cu).  Both return an fa_status.
int device_info(int** status, int* num_sms);
int encode_tmap_3d(CUtensorMap* map, const void* ptr, long long d0, long long d1, long long d2, int box_rows, bool f16);

// Rotary positions and cache append (fa_rotary.cu).  Strides are in elements: batch, head, token.
struct RotaryLaunch {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_out, *v_out;   // paged: k_out / v_out are the page pools
  long long q_stride[3], k_stride[3], v_stride[3];
  const float* table;                // (table_rows, R): cos[R/2], sin[R/2]
  const int* positions;              // rotary: (B or 1, N), or null: 0 .. N-1
  long long position_stride;         // elements between batch elements (0: shared)
  const int *block_table, *seq_lens, *new_lens;   // paged (new_lens may be null: N for all)
  int B, H, Hkv, N, D, R, table_rows, table_width, num_pages, page_shift;
  int interleaved, inverse, f16, paged;
  int* status;
};
cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t stream);

// Attention of T new tokens a sequence over a paged cache (fa_paged.cu).
struct PagedLaunch {
  const uint16_t *q, *k_pages, *v_pages;   // q (B,H,T,D); pages (num_pages, Hkv, page, D)
  const int *block_table, *seq_lens;       // (B, table_width), (B)
  const float* slopes;                     // (H) or null
  uint16_t* o;
  float* lse;
  void* workspace;
  int B, H, Hkv, T, D, num_pages, page_shift, table_width, window, f16;
  float scale, softcap;
  int* status;
  int num_sms;
};
size_t paged_workspace_bytes(int H, int Hkv, int T, int D);
cudaError_t launch_paged_attention(const PagedLaunch& a, cudaStream_t stream);

// bf16 / fp16 forward (fa_fwd_sm100.cu).  Tensor maps are 3-D (D, N, B*H) of the
// element type with 64 x 128 x 1 boxes (O: 64 x 32 x 1) and 128-byte swizzle.
struct FwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmO;
  float* lse;
  int BH, N, D;
  float scale;
  int causal;
  int f16;           // element type: 0 = bf16, 1 = fp16
  int hg;            // heads per L2 group (grouped_order)
  int* status;
  int num_sms;
};
cudaError_t launch_fwd_16(const FwdLaunch& a, cudaStream_t stream);
// Score-modified forward (head dims up to 128); a.BH counts query heads, tmK / tmV key-value heads.
cudaError_t launch_fwd_mod(const FwdLaunch& a, const ScoreMods& m, cudaStream_t stream);
// Head dimension 256 (fa_fwd_d256_sm100.cu): one query tile per CTA, same tensor maps.
cudaError_t launch_fwd_d256(const FwdLaunch& a, cudaStream_t stream);

// fp32 forward (fa_fwd_f32.cu), plain pointers.
cudaError_t launch_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse,
                           int BH, int N, int D, float scale, int causal, int* status, cudaStream_t stream);

// Backward stages (fa_bwd_sm100.cu).  The workspace holds, per (b, h) and per row of
// N padded up to a multiple of 128 (Npad): ws_nl = -lse * log2(e) (padding: -inf)
// and ws_delta = rowsum(dO * O) (padding: 0).
struct BwdLaunch {
  CUtensorMap tmQ, tmK, tmV, tmdO;   // loads (query box rows: 64 for dK/dV, 128 for dQ)
  CUtensorMap tmdQ, tmdK, tmdV;      // stores (32-row boxes)
  const void* o;
  const void* dO;
  const float* lse;
  float* ws_nl;
  float* ws_delta;
  float* ws_dq;      // fp32 dQ accumulator of the fused path (B*H*Npad*DK floats), or null
  int BH, N, Npad, D;
  int DK;            // columns of the kernels' tiles: 64 (D <= 64) or 128 (D in {96, 128})
  int hg;            // heads per L2 group (grouped_order)
  float scale;
  int causal;
  int f16;           // element type of q, k, v, o, dO and the gradients: 0 = bf16, 1 = fp16
  int* status;
  int num_sms;
};
cudaError_t launch_bwd_preprocess(const BwdLaunch& a, cudaStream_t stream);
cudaError_t launch_bwd_dkdv(const BwdLaunch& a, cudaStream_t stream);
cudaError_t launch_bwd_dq(const BwdLaunch& a, cudaStream_t stream);
// Fused backward (fa_bwd_fused_sm100.cu), DK in {64, 128}: dK, dV written, dQ added into
// ws_dq (which the preprocess kernel zeroed); then dq_finish writes scale * ws_dq to dq.
cudaError_t launch_bwd_fused(const BwdLaunch& a, cudaStream_t stream);
// Score-modified fused backward; a.BH counts query heads, tmK / tmV / tmdK / tmdV key-value heads.
cudaError_t launch_bwd_fused_mod(const BwdLaunch& a, const ScoreMods& m, cudaStream_t stream);
cudaError_t launch_bwd_dq_finish(const BwdLaunch& a, void* dq, cudaStream_t stream);
// Head dimension 256 (fa_bwd_d256_sm100.cu): two CTAs per tile, one per half of D.
cudaError_t launch_bwd_dkdv_d256(const BwdLaunch& a, cudaStream_t stream);
cudaError_t launch_bwd_dq_d256(const BwdLaunch& a, cudaStream_t stream);

}  // namespace fa
