/*
 * prefill_ops.h -- per-kernel entry points of the KV-shared prefill library.
 *
 * Each call runs ONE of the library's CUDA kernels (the same launchers the
 * prefill pass uses) on caller-provided device buffers, waits for it, and
 * returns a status (PF_OK or a negative PF_E_* from prefill.h).  They exist
 * so that every step of the pass can be checked on its own against a
 * reference.  Weights are passed as host pointers and uploaded for the call.
 * Calls are synchronous on `stream` (a cudaStream_t or NULL).
 *
 * Matrices are row-major.  bf16/fp16 buffers hold raw 16-bit values.  The A
 * operand of every GEMM (a_dev, bf16 [a_rows][K]) must have a_rows >= 128
 * rows allocated (rows beyond M are read but their results are dropped) and
 * K a multiple of 64.
 */
#ifndef PREFILL_OPS_H
#define PREFILL_OPS_H

#include <stdint.h>

#include "prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* out[m][n] = sum_k A[m][k] W[n][k] (fp32 [M][N]); W [N][K] in wtype
   (PF_W_Q4_0 blocks or fp32, computed as bf16).  bn: N-tile, 64, 128 or 256
   (192 with Q4_0). */
int pfop_linear_f32(int32_t wtype, const void* w_host, int32_t N, int32_t K, int32_t bn, const void* a_dev,
                    int32_t a_rows, int32_t M, float* out_dev, void* stream);

/* x[m][n] += (A W^T)[m][n] (fp32 [M][N], in place); if xb_dev != NULL also
   xb[m][n] = bf16(new x[m][n]).  N must be a multiple of 32. */
int pfop_linear_resid(int32_t wtype, const void* w_host, int32_t N, int32_t K, const void* a_dev, int32_t a_rows,
                      int32_t M, float* x_dev, void* xb_dev, void* stream);

/* h[m][f] = act(A Wg^T)[m][f] * (A Wu^T)[m][f] (bf16 [M][F]); act 0 =
   gelu_tanh (GeGLU), 1 = silu (SwiGLU).  F a multiple of 64.  Gate and up
   rows are interleaved in tiles of 256 rows when F is a multiple of 128, of
   192 (Q4_0) when F is a multiple of 96, else of 128. */
int pfop_linear_glu(int32_t wtype, const void* wg_host, const void* wu_host, int32_t F, int32_t K, int32_t act,
                    const void* a_dev, int32_t a_rows, int32_t M, void* h_dev, void* stream);

/* out[m][p] = bf16(gelu_tanh((A W^T)[m][p]) * ple[m*ple_stride + p]) (bf16
   [M][P]); ple bf16.  P a multiple of 32 (the per-layer-embedding gate). */
int pfop_linear_ple(int32_t wtype, const void* w_host, int32_t P, int32_t K, const void* a_dev, int32_t a_rows,
                    int32_t M, const void* ple_dev, int32_t ple_stride, void* out_dev, void* stream);

/* Q/K/V projection with half-split RoPE at positions pos0+m (angle
   pos * base^(-2i/hd), i < hd/2, pairing i with i+hd/2):
   q_out fp16 [M][Hq*hd]; if wk_host/wv_host are not NULL, K (rotated) and V
   go to the fp16 caches kc/vc [max_ctx][Hkv*hd] at rows pos0+m. */
int pfop_linear_qkv(int32_t wtype, const void* wq_host, const void* wk_host, const void* wv_host, int32_t Hq,
                    int32_t Hkv, int32_t hd, int32_t K, float rope_base, const void* a_dev, int32_t a_rows,
                    int32_t M, int32_t pos0, int32_t max_ctx, void* q_dev, void* kc_dev, void* vc_dev, void* stream);

/* Causal GQA attention: q fp16 [M][Hq*hd] at positions pos_base+m, K/V fp16
   [positions][Hkv*hd] with keys [0, kv_len) valid; out bf16 [M][Hq*hd].
   mode 0: any M.  The (query row, query head of a KV head's group) pairs
   form 128-row blocks; keys are folded in 64-key chunks, the chunks in at
   most four groups (as many as keep the launch to one wave of CTAs, at
   least four chunks a group); one CTA per (row block, KV head, group),
   then an ordered merge of the group states of rows whose keys span
   several groups.
   mode 1: one row (M == 1) at position pos_base, the form the KV-shared
   layers use for the output row (G4 section 1: after the pruning those
   layers carry that row only): the keys [0, pos_base] are cut into 64-key
   tiles and the tiles into ranges over up to 144 CTAs in clusters of four;
   each CTA streams its range once (online softmax, fp32 accumulation), a
   cluster folds its four range states in rank order, and the last cluster
   of each KV head merges the cluster states in cluster order, all in one
   launch.  Its bits depend on pos_base only, not on the launch; they differ
   from mode 0's in rounding. */
int pfop_attention(int32_t mode, const void* q_dev, const void* k_dev, const void* v_dev, int32_t M, int32_t Hq,
                   int32_t Hkv, int32_t hd, int32_t pos_base, int32_t kv_len, void* out_dev, void* stream);

/* y[i] = bf16(rmsnorm(x[row0+i]) * (1 + g)) for i < M (x fp32 [.][D]); if
   xcopy_dev != NULL, xcopy[i] = x[row0+i]. */
int pfop_rmsnorm(const float* x_dev, int32_t row0, int32_t M, int32_t D, const float* g_host, float eps, void* y_dev,
                 float* xcopy_dev, void* stream);

/* x[t] = E[tok_t] (fp32 [T][D]); if ple_host != NULL, ple[t] = bf16(E_ple[tok_t] *
   ple_scale) (bf16 [T][LP]).  Tables in wtype.  tok_dev: int32 device. */
int pfop_embed(int32_t wtype, const void* tok_host, const void* ple_host, int32_t vocab, int32_t D, int32_t LP,
               float ple_scale, const int32_t* tok_dev, int32_t T, float* x_dev, void* ple_dev, void* stream);

/* The KV image copy kernel.  dir 0: cache -> image (writes the 16-byte header
   `header`, then n_seg segments of copy_bytes); dir 1: image -> cache.
   Segment s is at s*cache_seg_halves halves in the cache and at
   16 + s*img_seg_bytes bytes in the image.  The kernel moves 16-byte
   vectors: cache_dev and image_dev 16-byte aligned, cache_seg_halves a
   multiple of 8, img_seg_bytes and copy_bytes multiples of 16, else
   PF_E_ARG (checked before any CUDA call). */
int pfop_kv_copy(int32_t dir, void* cache_dev, int64_t cache_seg_halves, void* image_dev, int64_t img_seg_bytes,
                 int32_t n_seg, int64_t copy_bytes, const int32_t* header4, void* stream);

/* out[n] = sum_k a[k] W[n][k] (fp32 [N]) for ONE row a (bf16 [K]) with the
   one-token projection kernel that a one-token ubatch uses (generation
   after the prompt): CUDA cores stream W once (wtype as in pfop_linear_f32,
   bn its tile width: 64, 128, 256, or 192 for Q4_0), fp32 dot products,
   k-part sums added in a fixed order.  If iters > 0 the call is then repeated `iters` times and *us
   receives the mean device time per launch (CUDA events on `stream`). */
int pfop_linear_row(int32_t wtype, const void* w_host, int32_t N, int32_t K, int32_t bn, const void* a_dev,
                    float* out_dev, int32_t iters, float* us, void* stream);

/* Check of the failure path of the bounded waits (the library's own error
   convention; the pages have no counterpart).  Runs the GEMM of
   pfop_linear_f32 (no k-split) with the copy producer of CTA 0 issuing
   nothing from pipeline stage `withhold_stage` on, so no copy is left in
   flight for the tensor-core and dequantisation warps that wait for that
   stage: their waits give up after their bound (about 2 s of SM clock),
   every warp unwinds (copies already issued are drained, TMEM is freed), and
   the call returns PF_E_DEVICE_TIMEOUT with the GPU context still usable.
   withhold_stage < 0 (or past the CTA's last stage) runs the plain GEMM and
   returns PF_OK.  Synchronous on `stream`. */
int pfop_linear_wait_test(int32_t wtype, const void* w_host, int32_t N, int32_t K, int32_t bn, const void* a_dev,
                          int32_t a_rows, int32_t M, float* out_dev, int32_t withhold_stage, void* stream);

/* Time the GEMM kernel: upload W once, run `warmup` then `iters` launches of
   out = A W^T (fp32 [M][N]) and return the mean device time per launch in
   *us (CUDA events on `stream`).  split: k-splits on single CTAs (0 = the
   library's choice for this shape; -1 = no split, 2-CTA pairs sharing
   256-row tcgen05 MMAs, Q4_0 with bn 128, 192 or 256 only).  bn 192 takes
   Q4_0 weights only. */
int pfop_linear_bench(int32_t wtype, const void* w_host, int32_t N, int32_t K, int32_t bn, int32_t split,
                      const void* a_dev, int32_t a_rows, int32_t M, float* out_dev, int32_t warmup, int32_t iters,
                      float* us, void* stream);

/* Time the attention kernels of pfop_attention (same arguments and modes):
   `warmup` untimed calls, then `iters` timed ones, each bracketed by its own
   CUDA events on `stream`; *us = mean device time per call (the single-row
   kernel, or the prefill kernel plus the group-state merge when it runs).  If scrub_dev is
   not NULL, scrub_bytes of it (a caller-owned device buffer larger than L2)
   are overwritten before every timed call, outside the events, so that each
   call reads K/V from HBM (cold L2).  Reading K/V once is the op's
   algorithmic traffic: kv_len * Hkv * hd * 2 bytes for each of K and V.
   Returns PF_E_DEVICE_TIMEOUT if a bounded wait gave up. */
int pfop_attention_bench(int32_t mode, const void* q_dev, const void* k_dev, const void* v_dev, int32_t M, int32_t Hq,
                         int32_t Hkv, int32_t hd, int32_t pos_base, int32_t kv_len, void* out_dev, void* scrub_dev,
                         int64_t scrub_bytes, int32_t warmup, int32_t iters, float* us, void* stream);

/* Time the KV image copy kernel of pfop_kv_copy (same layout arguments and
   alignment rules; the image header written by dir 0 is all zeros here)
   like pfop_attention_bench: mean device time per launch in *us, optional
   L2 scrub of scrub_dev before every timed launch.  The copy reads and
   writes n_seg * copy_bytes bytes each. */
int pfop_kv_copy_bench(int32_t dir, void* cache_dev, int64_t cache_seg_halves, void* image_dev, int64_t img_seg_bytes,
                       int32_t n_seg, int64_t copy_bytes, void* scrub_dev, int64_t scrub_bytes, int32_t warmup,
                       int32_t iters, float* us, void* stream);

/* The single-row split-K attention of pfop_attention (mode 1) without any
   memory allocation, for callers that may not allocate device memory at this
   point (a fixed memory budget already handed out, a server that forbids
   allocation after start-up, an embedder whose allocator owns the device).
   The page set this library follows has no counterpart for this call.
   q fp16 [Hq*hd] at position pos; K/V fp16 [positions][Hkv*hd] with keys
   [0, kv_len) valid, pos < kv_len; out bf16 [Hq*hd].
   Scratch: one fixed device array of 2^19 floats (2 MiB) per GPU that loads
   the library, kept until exit.  A call needs the merge tickets (Hkv ints,
   rounded up to 4) and Hkv*C*(Hq/Hkv*hd + 32) floats of folded states, C
   being the clusters of four key ranges per KV head (at most 36/Hkv, at
   least 1), plus 4 for an error word: any shape of up to 1024 query heads
   of 256 fits; larger requests return PF_E_ARG without touching the GPU,
   and so do
   shapes the kernels do not take (head_dim other than 64 or 256, n_head not
   a multiple of n_head_kv, a group size not dividing 16, q/k/v not 16-byte
   aligned).  All calls share the array, so calls that overlap on the GPU
   race: order them on one stream or with events.  Each call clears the
   tickets it uses.  The first call on a device looks up the array's device
   address with that device current (cudaGetSymbolAddress); make that first
   call before capturing any stream.  Synchronous on `stream`. */
int pfop_attention_split_noalloc(const void* q_dev, const void* k_dev, const void* v_dev, int32_t Hq, int32_t Hkv,
                                 int32_t hd, int32_t pos, int32_t kv_len, void* out_dev, void* stream);

/* How the GEMMs of the pfop_* calls run (process-wide, for every later
   call): 0 = as the library picks per matrix shape (the default), 1 = every
   Q4_0 matrix with 128-, 192- or 256-row tiles in 2-CTA pairs (tcgen05
   .cta_group::2, no k-split), -1 = never in pairs.  Lets the same checks run
   on both forms; no effect on prefill contexts.  PF_E_ARG for other modes. */
int pfop_set_gemm_pairs(int32_t mode);

/* ---- host-only: the stored form of the weights (no GPU needed) ----
   The library repacks every matrix at create into the order and layout its
   kernels read; these two calls return that form so that it can be checked
   on its own.

   pfop_qkv_row_order: the stored row order of a layer's Q|K|V projection
   (128-row tiles).  order[i] = the source row of stored row i, counting
   rows of [Wq; Wk; Wv] (Wq: Hq*hd rows, then Wk and Wv: Hkv*hd rows each;
   with_kv = 0: a Q-only projection), or -1 for a zero row padding the last
   tile.  A Q or K head wider than a tile is cut into hd/128 tiles: tile j
   of the head holds dims j*64 .. j*64+63 of each half of the head, so that
   every RoPE pair (i, i + hd/2) lies in one tile; narrower heads and V rows
   stay in order.  Returns the number of stored
   rows (a multiple of 128), or PF_E_ARG (hd odd, hd above 128 and not a
   multiple of it, cap too small).

   pfop_repack_q4: a Q4_0 matrix [N][K] (K a multiple of 64) in tiles of bn
   rows (64, 128, 192 or 256; N padded with zero rows to a multiple of bn).
   Tile (t, kb), for t < ceil(N/bn) and 64-wide k-block kb < K/64, is bn*36
   contiguous bytes at ((t * K/64) + kb) * bn*36: first the 16 nibble bytes
   of 32-element block h (h = 0, 1: elements kb*64 + h*32 ..) of row r at
   (h*bn + r)*16, then that block's fp16 scale at bn*32 + (h*bn + r)*2.
   Padding rows hold nibble bytes 0x88 and scale 0 (value 0).  With dst NULL
   returns the byte count; otherwise writes it to dst (host memory,
   dst_bytes at least that) and returns it; PF_E_ARG for bad shapes. */
int32_t pfop_qkv_row_order(int32_t Hq, int32_t Hkv, int32_t hd, int32_t with_kv, int32_t* order, int32_t cap);
int64_t pfop_repack_q4(const void* w_host, int32_t N, int32_t K, int32_t bn, void* dst, int64_t dst_bytes);

/* ---- several sequences in one call ----
   Unlike the calls above, the calls below only enqueue work on `stream` (of
   the current device), allocate nothing and may be recorded into a CUDA
   graph; arguments are checked on the host before any CUDA call.

   The attention calls work on one layer's K and V in the layout in which
   prefill_ubatch_seqs keeps them: [cells][Hkv*hd], a sequence's cells one
   after another.  The buffers are the caller's own: a prefill context gives
   out no address of its cache (kv_save copies sequence 0 out of it).

   A run is n_rows consecutive rows of one sequence that continue it at
   position pos0; the sequence's position p lives in cache cell cell0 + p.
   The rows of run r follow those of run r-1 in q and out (runs with
   n_rows 0 are allowed and skipped).  K and V of the run's own rows are in
   the cache already, at cells cell0 + pos0 .. cell0 + pos0 + n_rows - 1. */
typedef struct pfop_attn_run {
  int32_t n_rows;
  int32_t pos0;
  int32_t cell0;
} pfop_attn_run;

/* Causal GQA attention of up to 128 runs in one call: q fp16 [T][Hq*hd], T
   the runs' rows in all, K/V fp16 [n_cells][Hkv*hd], out bf16 [T][Hq*hd]
   (rows from T on are not touched).  Row i of a run sees its sequence's
   positions 0 .. pos0 + i, scores scaled by 1 / sqrt(hd).  Cells of no run's
   positions 0 .. pos0 + n_rows - 1 are never used, whatever they hold; the
   runs' own cells must hold finite values (an infinity or NaN in V reaches
   the rows of its run that do not see it too, but no other run's).  Scores
   may be as large as finite q and k make them.  Probabilities are rounded to
   fp16 before P V, sums and states are fp32.  A row's bits depend on its
   position, its keys and the shapes of the call's runs, not on the other
   runs' values; a repeated call gives the same bits.
   work_dev: device scratch of the call, 256-byte aligned, work_bytes of it
   at least pfop_attention_work_bytes of the runs; its first 4096 bytes must
   be zero before its first call.  Calls that share a scratch must not
   overlap on the GPU (one stream, or events; two recorded graphs that share
   one may not run at once).
   PF_E_ARG: hd other than 64 or 256; n_head above 1024 or not a multiple of
   n_head_kv with a group size dividing 16; more than 128 runs or 2^20 rows; a
   run past n_cells or position 2^30; n_cells above 2^31 - 1024; q, k, v not
   16-byte or out not 32-byte aligned; a scratch too small; 2^30 units of work
   or more.  Units of work: for every KV head and every block of 256 / (n_head /
   n_head_kv) rows of a run (half as many in small calls at hd 64) the 128-key
   chunks up to its last row's position, and 3 (hd 256) or 4 (hd 64).  One
   prompt of 2^20 rows with 32 heads over 8 of 64 is about 2^29. */
int pfop_attention_packed(const void* q_dev, const void* k_dev, const void* v_dev, int64_t n_cells, int32_t Hq,
                          int32_t Hkv, int32_t hd, const pfop_attn_run* runs, int32_t n_runs, void* out_dev,
                          void* work_dev, int64_t work_bytes, void* stream);

/* Attention of drafted token trees over the runs' caches (one row per
   drafted token): like pfop_attention_packed, but row i of a run sees its
   sequence's positions 0 .. pos0 - 1 (the context) and those drafted tokens
   j of its run (position pos0 + j) whose bit j % 64 of
   mask_dev[row * mask_words + j / 64] is set.  mask_dev: uint64, device, a
   row for every row of q; mask_words 1 .. 4 (at most 256 drafted tokens a
   run, n_rows <= 64 * mask_words); bits from n_rows on are ignored.  A row
   that sees nothing (pos0 0 and no bit set) gives zeros.  One row with its
   own bit set is a plain decoding step.  Units of work count the whole run's
   chunks for every block. */
int pfop_attention_tree(const void* q_dev, const void* k_dev, const void* v_dev, int64_t n_cells, int32_t Hq,
                        int32_t Hkv, int32_t hd, const pfop_attn_run* runs, int32_t n_runs, const uint64_t* mask_dev,
                        int32_t mask_words, void* out_dev, void* work_dev, int64_t work_bytes, void* stream);

/* Scratch bytes that either call needs for these runs on the current device
   (host only; without a device, as on a GB300; at least 4096), or PF_E_ARG.
   Runs that the tree call does not take (more than 256 rows, or too much work
   as a tree) get what pfop_attention_packed needs. */
int64_t pfop_attention_work_bytes(int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs, int32_t n_runs);

/* Wait for `stream` and report whether a call using this scratch gave up a
   bounded wait (PF_E_DEVICE_TIMEOUT: the results of that call and of those
   after it are invalid; all of them have ended).  Then it makes the scratch
   as good as new, for any stream, before it returns; until it is called the
   scratch must not be used for further results.  Not to be recorded. */
int pfop_attention_status(void* work_dev, void* stream);

/* Log probabilities over a vocabulary, for every row of logits [rows][ld]
   (the first `vocab` values of each row; ltype PF_L_F32 or PF_L_BF16):
     logp[r]    = x[tok[r]] - logsumexp(x)     (tok, logp NULL: skipped)
     entropy[r] = -sum_v p[v] log p[v]         (NULL: skipped)
     top_id[r][i], top_logp[r][i], i < n_top: the n_top most probable tokens
       and their log probabilities, most probable first, the lower id first
       where two are equal (n_top 0: skipped; at most 32, at most vocab).
   All outputs are fp32 (top_id int32), rows dense.  -inf logits are allowed
   (probability 0).  A token outside [0, vocab) gives logp NaN.  A row
   without a distribution (a NaN, +inf, or only -inf) gives NaN throughout
   and top_id -1, and so does a row of which a copy did not arrive within the
   bound of the library's waits (about 2 s of SM clock): with no scratch there
   is no error word to tell the two apart.  Enqueue only, no scratch,
   recordable.
   PF_E_ARG: rows < 0, vocab < 1 or >= 2^30, ld < vocab, n_top outside
   [0, min(32, vocab)], missing or misaligned buffers (logits to their
   element, outputs to 4 bytes). */
#define PF_L_F32 0
#define PF_L_BF16 1
int pfop_logprobs(int32_t ltype, const void* logits_dev, int64_t ld, int32_t rows, int32_t vocab,
                  const int32_t* tok_dev, int32_t n_top, float* logp_dev, float* entropy_dev, int32_t* top_id_dev,
                  float* top_logp_dev, void* stream);

/* Last error message of a pfop_* call on this thread. */
const char* pfop_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PREFILL_OPS_H */
