/*
 * fa.h -- C ABI of libfa.so: exact, IO-aware tiled attention for NVIDIA B200 (sm_100a).
 *
 * The operation (all entry points):
 *     S   = scale * Q K^T                (N x N per batch b and head h)
 *     S_ij = -inf for j > i               (only when causal != 0; top-left aligned)
 *     P   = softmax(S) row-wise,  O = P V
 *     lse_i = ln( sum_j exp(S_ij) )       (natural-log logsumexp of the scaled scores)
 * This is the attention of the three-line PyTorch form in "CUDA-kernel-level
 * optimisation: why Flash Attention is 5-10x faster than native PyTorch"
 * (guanweilu.cn, section "three lines of PyTorch"), computed the way its
 * section "three tricks" and "LLM paper notes #8: FlashAttention" (adg.csdn.net,
 * sections "tiling", "online softmax", "recomputation") describe: Q/K/V tiles
 * staged on chip, an online softmax with a running max and sum, no N x N matrix
 * in device memory, and a backward pass that recomputes P from lse.
 *
 * Conventions shared by every entry point
 *   - Layout: every tensor is contiguous (B, H, N, D), head dimension innermost
 *     (the layout of naive_attention in "Flash Attention principles: making
 *     Transformers faster", ijyty.com, section "memory bottleneck").  lse and
 *     delta are contiguous (B, H, N) float32.
 *   - Pointers are DEVICE pointers (cudaMalloc'd or equivalent) on the current
 *     device, 16-byte aligned.  The caller owns and allocates every buffer; the
 *     library never allocates or frees device memory.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Every call is asynchronous on that stream; the library does no
 *     host synchronisation.
 *   - Supported: B, H, N >= 1; D in {32, 64, 96, 128} for bf16 and fp16 (32
 *     and 96 run the 64- and 128-column kernels on zero-filled columns, so
 *     they cost what 64 and 128 cost), and D = 256 (forward: one query tile
 *     per CTA; backward: two CTAs per tile, one per half of D); D in
 *     {32, 64, 128} for fp32; Nq == Nk == N; causal in {0, 1}; ceil(N/256)*B*H < 2^31 (and
 *     B*H <= 65535 for fa_fwd_f32).
 *   - Return value: FA_OK (0) or an fa_status code.  Arguments are validated
 *     before anything is launched; on an error nothing is launched and no
 *     output is touched.  Errors are never thrown across the ABI.
 *   - Device-side failures (a pipeline wait that exceeded its time limit) do
 *     not trap: the kernel records FA_ERR_TIMEOUT in a device status word and
 *     returns; fa_device_status() reads (and optionally clears) that word.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_NULL = 1,             /* a required pointer is NULL                      */
  FA_ERR_SHAPE = 2,            /* B, H or N out of range, or index overflow       */
  FA_ERR_HEADDIM = 3,          /* unsupported head dimension D                    */
  FA_ERR_ALIGN = 4,            /* a pointer is not 16-byte aligned                */
  FA_ERR_UNSUPPORTED_ARCH = 5, /* current device is not sm_100 (B200)             */
  FA_ERR_LAUNCH = 6,           /* cudaLaunch / tensor-map encoding failed         */
  FA_ERR_TIMEOUT = 7,          /* a device-side wait exceeded its limit           */
  FA_ERR_WORKSPACE = 8,        /* workspace NULL or smaller than required         */
  FA_ERR_CUDA = 9,             /* another CUDA runtime error                      */
  FA_ERR_ARG = 10,             /* another invalid argument (scale not finite ...) */
  FA_ERR_NOALLOC_CAPACITY = 11, /* problem too large for fa_bwd_noalloc's scratch  */
  FA_ERR_DEBUG_CHECK = 12,     /* a device-side check of the debug build failed   */
  FA_ERR_INDEX = 13            /* device data: a page, position or length outside its table */
} fa_status;

/* Element type of the entry points that take a `dtype`. */
typedef enum { FA_BF16 = 0, FA_F16 = 1 } fa_dtype;

/* Forward, bf16 in / bf16 out, fp32 accumulation (tcgen05 tensor cores).
 * Q/K/V tiles staged on chip and an online softmax with a running max and sum
 * that rescales the partial output ("LLM paper notes #8: FlashAttention",
 * adg.csdn.net, sections "tiling" and "online softmax"); lse is saved for the
 * backward ("recomputation").
 *   q, k, v : (B,H,N,D) bf16, read only.
 *   o       : (B,H,N,D) bf16, written (O = P V, rounded to nearest even).
 *   lse     : (B,H,N) float32, written (natural-log logsumexp of scale*q.k).
 *   scale   : the softmax scale (e.g. 1/sqrt(D)); must be finite and > 0.
 *   causal  : 0 = full attention, 1 = key j allowed for query i iff j <= i. */
int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
           int B, int H, int N, int D, float scale, int causal, void* stream);

/* Forward with fp16 (IEEE binary16) q, k, v and o instead of bf16; otherwise
 * identical to fa_fwd (fp32 accumulation and softmax, fp32 lse).  FP16 is the
 * element type in which "CUDA-kernel-level optimisation: why Flash Attention is
 * 5-10x faster than native PyTorch" (guanweilu.cn, section "three lines of
 * PyTorch") and "Flash Attention principles: making Transformers faster"
 * (ijyty.com, section "memory bottleneck") size the N x N matrices.  P is
 * rounded to fp16 for the P V product, so it carries 3 more mantissa bits than
 * on the bf16 path.  Values of O beyond the fp16 range (|x| > 65504) become
 * +-inf. */
int fa_fwd_f16(const void* q, const void* k, const void* v, void* o, float* lse,
               int B, int H, int N, int D, float scale, int causal, void* stream);

/* Forward in fp32 throughout (fp32 in, fp32 FFMA arithmetic, fp32 out), for
 * callers that need ~1e-6 relative accuracy.  Same arguments as fa_fwd with
 * float32 tensors.  Computes the same tiled online softmax as fa_fwd ("LLM paper
 * notes #8: FlashAttention", adg.csdn.net, sections "tiling" and "online
 * softmax"), with every product and exponential in fp32. */
int fa_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse,
               int B, int H, int N, int D, float scale, int causal, void* stream);

/* ---------------------------------------------------------------------------
 * Backward.  The gradients of O = softmax(S) V for a scalar loss, with P
 * recomputed from lse instead of stored ("LLM paper notes #8: FlashAttention",
 * adg.csdn.net, section "recomputation"; guanweilu.cn, section "three tricks"):
 *     dV = P^T dO,  dP = dO V^T,  delta_i = sum_d dO_id O_id,
 *     dS = P * (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q.
 * Workspace layout (device memory owned by the caller, 16-byte aligned), with
 * Npad = N rounded up to a multiple of 128 and R = B*H*Npad rows:
 *   [0, R) floats            nl_i    = -lse_i * log2(e)   (padding rows: -inf)
 *   [R, 2R) floats           delta_i = sum_d dO_id * O_id (padding rows: 0)
 *   [2R, 2R + R*DK) floats   fp32 dQ accumulator of fa_bwd (head dims up to 128;
 *                            DK = 64 for D <= 64, 128 for D in {96, 128}); per
 *                            128-row query tile a block of 128 x DK floats laid
 *                            out [DK/4][128 rows][4].
 * ------------------------------------------------------------------------- */

/* Bytes of device workspace fa_bwd and fa_bwd_f16 need: 4 * R * (2 + DK) for
 * D <= 128 (statistics and dQ accumulator), 8 * R for D = 256 (statistics only).
 * A multiple of 1024.  Returns 0 for an unsupported shape. */
size_t fa_bwd_workspace_size(int B, int H, int N, int D);

/* Bytes of device workspace fa_bwd_deterministic and its stages (fa_bwd_dkdv,
 * fa_bwd_dq) need: the statistics only, 8 * R.  Returns 0 for an unsupported shape. */
size_t fa_bwd_deterministic_workspace_size(int B, int H, int N, int D);

/* Backward, bf16 (recomputes P from lse; never stores an N x N matrix).
 *   q, k, v, o, dO : (B,H,N,D) bf16 inputs; o and lse must be the outputs of
 *                    fa_fwd for the same q, k, v, scale and causal.
 *   lse            : (B,H,N) float32 from fa_fwd.
 *   dq, dk, dv     : (B,H,N,D) bf16, overwritten (not accumulated into).
 *   workspace      : device buffer of at least fa_bwd_workspace_size() bytes;
 *                    contents on entry ignored, clobbered on exit.
 * For D <= 128 one kernel per 128-key tile computes dK, dV and each tile's
 * contribution dS K to dQ, which it adds into the workspace's fp32 accumulator
 * with reductions in L2; equivalent to fa_bwd_preprocess, fa_bwd_dkdvdq and
 * fa_bwd_dq_finish on the same stream.  The order of those fp32 additions varies
 * from run to run, so dQ is reproducible to rounding (not bit for bit); dK and
 * dV are.  For D = 256 it runs the three-stage path of fa_bwd_deterministic. */
int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
           const float* lse, void* dq, void* dk, void* dv,
           void* workspace, size_t workspace_bytes,
           int B, int H, int N, int D, float scale, int causal, void* stream);

/* Backward with fp16 q, k, v, o, dO, dq, dk, dv (o and lse from fa_fwd_f16);
 * otherwise identical to fa_bwd, with the same workspace.  P and dS are rounded
 * to fp16 for the tensor-core products; gradients beyond the fp16 range become
 * +-inf. */
int fa_bwd_f16(const void* q, const void* k, const void* v, const void* o, const void* dO,
               const float* lse, void* dq, void* dk, void* dv,
               void* workspace, size_t workspace_bytes,
               int B, int H, int N, int D, float scale, int causal, void* stream);

/* Backward, bf16 only, bit-for-bit reproducible: the same formulas as fa_bwd in
 * three stages with no atomics (fa_bwd_preprocess, fa_bwd_dkdv, fa_bwd_dq):
 * every output tile is owned by one CTA, at the price of a second pass that
 * recomputes S and dP for dQ.  Workspace: at least
 * fa_bwd_deterministic_workspace_size() bytes (fa_bwd's workspace also fits). */
int fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const void* dO,
                         const float* lse, void* dq, void* dk, void* dv,
                         void* workspace, size_t workspace_bytes,
                         int B, int H, int N, int D, float scale, int causal, void* stream);

/* Backward stage 1 (bf16): fills nl and delta from O, dO and lse (delta is the
 * row sum the softmax gradient subtracts, "recomputation", adg.csdn.net).  When
 * the workspace holds the dQ accumulator (workspace_bytes >=
 * fa_bwd_workspace_size and D <= 128) it is zeroed too. */
int fa_bwd_preprocess(const void* o, const void* dO, const float* lse,
                      void* workspace, size_t workspace_bytes,
                      int B, int H, int N, int D, void* stream);

/* Fused backward stage 2 (bf16, D <= 128): dK, dV (overwritten) and the dQ
 * contributions added into the accumulator that fa_bwd_preprocess zeroed.  Each
 * 128-key tile is owned by one CTA that walks the query tiles, recomputing P
 * from lse ("recomputation", adg.csdn.net).  Workspace: fa_bwd_workspace_size(). */
int fa_bwd_dkdvdq(const void* q, const void* k, const void* v, const void* dO,
                  void* workspace, size_t workspace_bytes, void* dk, void* dv,
                  int B, int H, int N, int D, float scale, int causal, void* stream);

/* Fused backward stage 3 (bf16, D <= 128): dq = scale * accumulator, rounded to
 * bf16 (the "dQ finish" of the backward).  Workspace: fa_bwd_workspace_size(). */
int fa_bwd_dq_finish(const void* workspace, size_t workspace_bytes, void* dq,
                     int B, int H, int N, int D, float scale, void* stream);

/* Deterministic stage 2 (bf16): dK, dV (overwritten), reading the statistics that
 * stage 1 filled.  Each 128-key tile is owned by one CTA that walks the query
 * rows, recomputing P from lse ("recomputation", adg.csdn.net), so dK and dV
 * need no atomics.  Workspace: fa_bwd_deterministic_workspace_size(). */
int fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dO,
                const void* workspace, size_t workspace_bytes, void* dk, void* dv,
                int B, int H, int N, int D, float scale, int causal, void* stream);

/* Deterministic stage 3 (bf16): dQ (overwritten), reading the statistics that
 * stage 1 filled.  Each 256-query block is owned by one CTA that walks the key
 * tiles and recomputes S, P and dP for them, so dQ needs no atomics.
 * Workspace: fa_bwd_deterministic_workspace_size(). */
int fa_bwd_dq(const void* q, const void* k, const void* v, const void* dO,
              const void* workspace, size_t workspace_bytes, void* dq,
              int B, int H, int N, int D, float scale, int causal, void* stream);

/* Size of the fixed device scratch array that fa_bwd_noalloc uses (8 MiB). */
#define FA_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)

/* Backward that allocates nothing and takes no workspace (bf16 only).  The paper
 * has no counterpart to this entry point; it exists for callers that cannot
 * allocate device memory -- code that a host framework hands only its input and
 * output buffers, with all device memory planned up front and no workspace or
 * allocator available to the operator.
 *   Same arguments, layout and errors as fa_bwd_deterministic minus the workspace,
 *     and the same results bit for bit (it runs the same three kernels).
 *   Scratch: a fixed FA_NOALLOC_SCRATCH_BYTES array in the library's own device
 *     memory (held by every GPU that loads the library until the process exits).
 *     Limit: fa_bwd_deterministic_workspace_size(B, H, N, D) <= FA_NOALLOC_SCRATCH_BYTES,
 *     i.e. B*H*ceil(N/128)*128 <= 1,048,576 rows; larger problems return
 *     FA_ERR_NOALLOC_CAPACITY before anything is launched.
 *   Set-up: the first call on a device looks up the array's device address
 *     (with that device current); make that first call before any stream capture.
 *     A failed lookup is not remembered: the next call on that device tries again.
 *   Sharing: every call uses the same array; nothing in it needs to start at zero
 *     (each call rewrites what it reads), but calls whose work overlaps on the GPU
 *     (unordered streams) race on it. */
int fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dO,
                   const float* lse, void* dq, void* dk, void* dv,
                   int B, int H, int N, int D, float scale, int causal, void* stream);

/* ---------------------------------------------------------------------------
 * Score-modified attention: shared key-value heads, interval masks, capped scores
 * and a distance bias, forward and backward, bf16 and fp16 (dtype), D in
 * {32, 64, 96, 128}.  For query row i and key j of query head h:
 *     s   = scale * q_i . k_j
 *     x   = softcap * tanh(s / softcap)      (softcap > 0; 0: x = s)
 *           (softcap log2(e) and scale / softcap have to be finite floats)
 *     x  -= slopes[h] * |i - j|              (slopes given: float32 (H))
 *     P   = softmax of x over the keys that row i sees,  O = P V,
 *     lse = ln(sum over them of exp(x)).
 * A row that sees no key has O = 0 and lse = -inf, and gives no gradient.
 * q, o, dO, dq are (B,H,N,D), lse (B,H,N); k, v, dk, dv are (B,Hkv,N,D) with H a
 * multiple of Hkv: query head h reads key-value head h / (H / Hkv), and dk, dv sum
 * over the query heads that share one.  Which keys a row sees is given by a plan
 * (fa_mask_plan, with causal = 0 here), or without one (plan NULL) by `causal`.
 * Values must be finite in every row, masked ones included: a masked key takes
 * weight 0, and 0 times an infinity is not 0 (as in fa_fwd).  Finite ones may be as
 * large as the type allows: a masked pair's products do not count, even where they
 * leave the fp32 range.
 * ------------------------------------------------------------------------- */

/* Bytes of a mask plan for B batch elements of N rows; 0 if out of range (N up to
 * 262144). */
size_t fa_mask_plan_size(int B, int N);

/* Builds the plan of an interval mask, to be used by any number of calls with the
 * same B and N.  documents (int32 (B,N)) or NULL: rows i and j see each other only if
 * every row from i to j carries the same id; a row with a negative id sees nothing
 * and is not seen.  causal: key j allowed for query i iff j <= i; prefix (int32 (B))
 * or NULL: or j < prefix[b] (causal only; not with documents or a window).
 * window > 0: only i - j < window, and without causal also j - i < window. */
int fa_mask_plan(void* plan, size_t plan_bytes, const int* documents, const int* prefix,
                 int B, int N, int causal, int window, void* stream);

/* Forward. */
int fa_fwd_mod(const void* q, const void* k, const void* v, void* o, float* lse,
               const void* plan, const float* slopes, float softcap,
               int B, int H, int Hkv, int N, int D, float scale, int causal, int dtype, void* stream);

/* Backward: o and lse from fa_fwd_mod with the same arguments; workspace of at least
 * fa_bwd_workspace_size(B, H, N, D) bytes, contents ignored.  As in fa_bwd the fp32
 * additions into dQ run in varying order (reproducible to rounding); dK and dV are
 * deterministic. */
int fa_bwd_mod(const void* q, const void* k, const void* v, const void* o, const void* dO,
               const float* lse, void* dq, void* dk, void* dv,
               void* workspace, size_t workspace_bytes,
               const void* plan, const float* slopes, float softcap,
               int B, int H, int Hkv, int N, int D, float scale, int causal, int dtype, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions, and the paged key-value cache.  bf16 and fp16 (dtype), D in
 * {32, 64, 96, 128, 256}.
 * The table is float32 (table_rows, R): row p holds the R/2 cosines, then the R/2
 * sines, of position p's angles.  The first R columns (even, 2 <= R <= D) turn in
 * pairs (a, b) -> (a cos - b sin, b cos + a sin), pair i being columns (i, i + R/2),
 * or (2i, 2i + 1) when interleaved; the rest is copied.
 * Strides are in elements, for (batch, head, token), multiples of 8; the D columns of
 * a row are contiguous.
 * Index data (positions, pages, lengths) is read on the device: a value outside its
 * table is never followed; the kernel records FA_ERR_INDEX in the device status word
 * and leaves a row at such a position unturned (in q_out, k_out), does not write a key
 * and value that have no page or, where keys turn, no row of the rotary table, and reads
 * keys of such a page as absent.
 * ------------------------------------------------------------------------- */

/* q_out, k_out <- q, k with their rows turned; outputs contiguous (B,H,N,D) and
 * (B,Hkv,N,D).  H = 0 or Hkv = 0 leaves that tensor out (its pointers may be NULL).
 * positions: int32, row b at positions + b * position_stride, or NULL: 0 .. N-1.
 * inverse = 1 turns by the negative angles: the gradient of inverse = 0. */
int fa_rotary(const void* q, const void* k, void* q_out, void* k_out, const float* table,
              const int* positions, const long long* q_strides, const long long* k_strides,
              long long position_stride, int table_rows, int B, int H, int Hkv, int N, int D, int R,
              int interleaved, int inverse, int dtype, void* stream);

/* Writes the keys and values of new tokens into the pages of their sequences, turning
 * the keys (and q into q_out) by their positions on the way.
 *   k, v        (B,Hkv,T,D); q, q_out (B,H,T,D) or H = 0 without; q_out contiguous.
 *   k_pages, v_pages (num_pages, Hkv, page_size, D) contiguous, page_size a power of
 *               two from 8 to 256.
 *   block_table int32 (B, table_width): page of positions [i page_size, (i+1) page_size).
 *   seq_lens    int32 (B): length of each sequence WITH its new tokens.
 *   new_lens    int32 (B), new tokens of each sequence (0 to T), or NULL: T.  Token t
 *               of sequence b has position seq_lens[b] - new_lens[b] + t; rows
 *               t >= new_lens[b] are not written, their q_out rows are zero.  A count
 *               outside 0 to T writes nothing (FA_ERR_INDEX).
 *   table       or NULL with R = 0: nothing turns. */
int fa_paged_append(const void* k, const void* v, void* k_pages, void* v_pages, const void* q, void* q_out,
                    const int* block_table, const int* seq_lens, const int* new_lens, const float* table,
                    const long long* k_strides, const long long* v_strides, const long long* q_strides,
                    int table_rows, int table_width, int num_pages, int page_size,
                    int B, int H, int Hkv, int T, int D, int R, int interleaved, int dtype, void* stream);

/* Largest number of new tokens and of sequences of one fa_paged_attention call. */
#define FA_PAGED_MAX_TOKENS 64
#define FA_PAGED_MAX_BATCH 4096

/* Bytes of device workspace fa_paged_attention needs; 0 for an unsupported shape. */
size_t fa_paged_workspace_size(int B, int H, int Hkv, int T, int D);

/* Attention of the last T tokens of each sequence (T = 1: one new token) over its
 * paged cache, which already holds them (fa_paged_append).  q, o (B,H,T,D) contiguous,
 * lse (B,H,T) float32.  Row t of sequence b has position p = seq_lens[b] - T + t and
 * sees the keys j <= p, with window > 0 only those with p - j < window; x as in
 * fa_fwd_mod with |i - j| = p - j.  A row with p < 0 (a sequence shorter than T, or
 * empty) has O = 0 and lse = -inf.  Table entries past a sequence's last page, or wholly
 * before every row's window, and the slots behind its last position are never used,
 * whatever they hold.
 * Lengths beyond the table (table_width * page_size) are cut to it, with FA_ERR_INDEX.
 * workspace: contents ignored and clobbered; calls that may overlap on the GPU need one
 * each.  Results do not vary from run to run. */
int fa_paged_attention(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                       const int* seq_lens, void* o, float* lse, void* workspace, size_t workspace_bytes,
                       const float* slopes, float softcap, int window, int table_width, int num_pages,
                       int page_size, int B, int H, int Hkv, int T, int D, float scale, int dtype, void* stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* fa_status_string(int status);

/* Reads the device status word of the current device (synchronises the
 * device first).  Returns FA_OK or the first FA_ERR_* a kernel recorded;
 * if reset != 0 the word is cleared afterwards.  Kernels record
 * FA_ERR_TIMEOUT (a pipeline wait ran out) and FA_ERR_LAUNCH (a launch they
 * cannot use); the debug build of the library (libfa_debug.so, compiled with
 * FA_DEBUG_CHECKS) also records FA_ERR_DEBUG_CHECK when a computed index falls
 * outside its buffer or a warp reaches a warp-collective tensor-memory
 * operation diverged, and skips that access instead of performing it. */
int fa_device_status(int reset);

/* Library version, major*10000 + minor*100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_H_ */
