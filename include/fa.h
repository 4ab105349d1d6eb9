/* Exact tiled attention for GB300 (sm_103a): the C ABI.
 *
 * What the library computes, for every batch b and head h (all tensors
 * contiguous, layout (B, H, N, d), d innermost):
 *
 *     O = softmax(scale * Q K^T  [+ causal mask]) V,   LSE_i = ln sum_j exp(scale * q_i . k_j)
 *
 * the definition of wiki.ai-engineering.at "Flash Attention" (section "Das
 * Grundproblem") and johe.ru "Flash Attention: ускорить attention в 6 раз без
 * потери точности" (section "Введение").  It is evaluated tile by tile with the
 * online-softmax recurrence of the first page (section "Lösung: Online
 * Softmax"), so the N x N score matrix never exists in device memory.  The
 * result equals standard attention up to floating-point rounding; only the
 * order of operations differs (second page, "Почему это точно?").
 *
 * Conventions shared by every entry point:
 *  - q, k, v, o, dO, dq, dk, dv, caches: bf16 (__nv_bfloat16) device pointers,
 *    16-byte aligned, contiguous (B, H, N, d); d is 64 or 128.
 *  - lse, D and every workspace: fp32 device pointers, 16-byte aligned.
 *  - scale is passed explicitly (1/sqrt(d) is the usual choice); it must be
 *    finite and > 0.
 *  - causal: 0 or 1.  The mask is aligned bottom-right: query i sees key j iff
 *    j <= i + (Nk - Nq).  A query that sees no key gets O = 0, LSE = -inf and
 *    zero gradients.
 *  - stream: a cudaStream_t passed as void* (NULL = the legacy default stream).
 *    Every call is asynchronous on it; nothing is synchronised.  Kernels are
 *    launched as programmatic dependents of the work before them on the stream
 *    (their setup may overlap its end), but each waits for that work to
 *    complete before it reads or writes any buffer, so stream order holds as
 *    for ordinary launches.
 *  - Ownership: the caller allocates and owns every buffer, workspaces
 *    included.  The library allocates no device memory and keeps no state
 *    besides a device-side error word and host-side caches (the tensor-map
 *    encoder's entry point, each device's SM count, and which kernels'
 *    shared-memory limits have been raised on which device).
 *  - Errors: return codes only (fa_status); arguments are validated before
 *    anything is launched, and an invalid call launches nothing.  No fallback
 *    implementation exists: an unsupported shape is an error, never a slower
 *    path.  Device-side waits are bounded; a wait that runs out records
 *    FA_ERR_TIMEOUT in the error word, the kernel releases what it holds and
 *    returns, and fa_get_last_device_error() reports it.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = -1, /* null pointer, non-positive size, bad scale or flag */
    FA_ERR_UNSUPPORTED = -2, /* d not in {64, 128}, sizes beyond 32-bit tile indexing */
    FA_ERR_ALIGNMENT = -3,   /* a pointer not 16-byte aligned */
    FA_ERR_WORKSPACE = -4,   /* workspace null or smaller than the *_workspace_bytes query */
    FA_ERR_CUDA = -5,        /* a CUDA runtime/driver call failed (launch, tensor map) */
    FA_ERR_TIMEOUT = -6      /* a device-side bounded wait ran out (see fa_get_last_device_error) */
} fa_status;

/* Forward pass (tiled attention with online softmax, one fused kernel).
 * q [B,H,Nq,d], k/v [B,H,Nk,d] bf16 in; o [B,H,Nq,d] bf16 and lse [B,H,Nq]
 * fp32 out (natural log of the row's sum of exp(scale * q.k)).  Source: the
 * "Tiling Algorithm" and "Lösung: Online Softmax" sections of
 * wiki.ai-engineering.at "Flash Attention"; each output row leaves the chip
 * exactly once (johe.ru, section "Проблема 2: DRAM bottleneck", the count of
 * memory round trips).  Requires B, H, Nq, Nk >= 1. */
int fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
           int B, int H, int Nq, int Nk, int d, float scale, int causal, void *stream);

/* Query rows per work tile fa_fwd takes for these sizes on the current device:
 * 256 (two 128-row query tiles share every key/value block) or 128 (split-KV
 * tiles: the key blocks of one 128-row tile alternate between two softmax
 * groups, merged at the end with the log-sum-exp weights, the combine of
 * wiki.ai-engineering.at "Flash Attention", section "Lösung: Online
 * Softmax").  The choice minimises the busiest SM's share of a static
 * persistent schedule; it only changes the rounding order.  Returns a negative
 * fa_status for invalid sizes or no usable device.  Host-only; launches
 * nothing. */
int fa_fwd_tile_rows(int B, int H, int Nq, int Nk, int d, int causal);

/* The static schedule of the persistent grids (the forward's work tiles, the
 * backward's key and query tiles): n_items work items listed in chunks of
 * chunk_items (heads whose streamed operands fit in L2 together), taken by
 * `grid` CTAs.  per_chunk != 0 (causal lists, heaviest item first in each
 * chunk): each chunk in its own rounds of alternating direction, odd chunks
 * starting reversed; otherwise, or when a chunk is smaller than the grid,
 * rounds of alternating direction over the whole list.  Writes owner[i] = the
 * CTA that takes item i (owner: n_items ints, host memory).  Returns FA_OK,
 * FA_ERR_INVALID_ARG for bad sizes or a null owner, or FA_ERR_INVALID_ARG if
 * an item would be taken twice (never: the schedule is a partition).
 * Host-only; launches nothing. */
int fa_work_schedule(int n_items, int chunk_items, int grid, int per_chunk, int *owner);

/* Causal sliding-window forward: like fa_fwd with causal = 1, except that
 * query i sees only the `window` (>= 1) keys ending at its diagonal, keys j
 * with i + Nk - Nq - window < j <= i + Nk - Nq (the fixed-window local
 * attention of johe.ru "Flash Attention: ...", section "Альтернативы").  Only
 * the key blocks inside a tile's window are loaded and multiplied. */
int fa_fwd_window(const void *q, const void *k, const void *v, void *o, float *lse,
                  int B, int H, int Nq, int Nk, int d, float scale, int window, void *stream);

/* Forward over a padded batch of sequences of different lengths (a mask
 * variant of fa_fwd: zimaspace.com "Wie reduziert Flash Attention ...",
 * masking is applied to the tile scores before the softmax).  seqlens_q and
 * seqlens_k are device int32 [B]: sequence b has seqlens_q[b] <= Nq query
 * rows and seqlens_k[b] <= Nk keys, stored in the first rows of its
 * [H, Nq, d] / [H, Nk, d] slices.  Row i < seqlens_q[b] attends to keys
 * j < seqlens_k[b] (causal: also j <= i + seqlens_k[b] - seqlens_q[b]).  Rows
 * past seqlens_q[b] get O = 0 and LSE = -inf.  Query and key tiles wholly past a
 * sequence are skipped.  Padding positions of q, k and v must hold finite
 * values (their contents do not change the result).  A length outside
 * [0, Nq] / [0, Nk] is clamped and recorded as FA_ERR_INVALID_ARG in the
 * device error word.  Other conventions as fa_fwd; both length pointers are
 * required (FA_ERR_INVALID_ARG if null) and 4-byte aligned. */
int fa_fwd_varlen(const void *q, const void *k, const void *v, void *o, float *lse,
                  const int *seqlens_q, const int *seqlens_k,
                  int B, int H, int Nq, int Nk, int d, float scale, int causal, void *stream);

/* Bytes of workspace fa_fwd_fp8 needs: a transposed copy of V,
 * [B*H, 128, Nk rounded up to 16] bytes.  Returns 0 for invalid sizes. */
size_t fa_fwd_fp8_workspace_bytes(int B, int H, int Nk, int d);

/* FP8 forward with block scales (johe.ru "Flash Attention: ...", sections
 * "Flash Attention 3": block-scaled attention, and "Flash Attention 4": FP8).
 * q [B,H,Nq,128], k and v [B,H,Nk,128] as e4m3 bytes (OCP FP8, no infinities).
 * The value an element stands for is its e4m3 value times its scale:
 *  q_scale fp32 [B*H, ceil(Nq/128)]: one per 128-row block of q;
 *  k_scale fp32 [B*H, ceil(Nk/128)]: one per 128-row block of k;
 *  v_scale fp32 [B*H]: one per head of v.
 * Computes the forward of fa_fwd on those values: o [B,H,Nq,128] bf16 and lse
 * [B,H,Nq] fp32.  Scores accumulate in fp32.  P = exp(S - m) is rounded to
 * e4m3 (relative error <= 2^-4, or 2^-10 absolute below 2^-6) for the value
 * product, and the result is multiplied by v_scale / l.  d must be 128
 * (FA_ERR_UNSUPPORTED otherwise).  workspace: at least
 * fa_fwd_fp8_workspace_bytes(B,H,Nk,d) bytes, 16-byte aligned; it receives V^T
 * (one extra pass over V) so that both products take K-major operands. */
int fa_fwd_fp8(const void *q, const void *k, const void *v, const float *q_scale, const float *k_scale,
               const float *v_scale, void *o, float *lse, int B, int H, int Nq, int Nk, int d, float scale,
               int causal, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of fp32 workspace fa_bwd needs: the row terms D [B,H,Nq] (dQ is
 * accumulated on chip, in a pass of its own).  Returns 0 for invalid sizes. */
size_t fa_bwd_workspace_bytes(int B, int H, int Nq, int Nk, int d);

/* Backward pass (johe.ru, section "Стадии вычисления", pass 2: gradients are
 * recomputed from the same tiles, P is rebuilt from the saved LSE instead of
 * being stored).  Inputs: q, k, v, o (the forward output), lse (the forward's
 * LSE), dO [B,H,Nq,d] the upstream gradient.  Outputs dq [B,H,Nq,d],
 * dk/dv [B,H,Nk,d] bf16.  Steps: D_i = sum_c dO_ic O_ic (fp32); per key tile,
 * S = scale QK^T recomputed, P = exp(S - LSE), dV += P^T dO, dP = dO V^T,
 * dS = P (dP - D), dK += scale dS^T Q; per query tile, dQ += scale dS K.  All
 * accumulation is fp32 on chip; each gradient is rounded to bf16 once.  The
 * result is deterministic (no atomics).  workspace must hold at least
 * fa_bwd_workspace_bytes(B,H,Nq,Nk,d) bytes; its contents on entry do not
 * matter. */
int fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
           const void *dO, void *dq, void *dk, void *dv,
           int B, int H, int Nq, int Nk, int d, float scale, int causal,
           void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_bwd_fused needs: D [B,H,Nq] as for fa_bwd, then an
 * fp32 dQ accumulator [B,H,Nq,d].  Returns 0 for invalid sizes and for
 * d != 128. */
size_t fa_bwd_fused_workspace_bytes(int B, int H, int Nq, int Nk, int d);

/* The same backward as fa_bwd (same arguments, outputs and tolerance) in one
 * pass over the key tiles instead of two: besides dK and dV, each 128-key
 * CTA computes its share of dQ = scale dS K as dQ^T = K^T dS^T on the tensor
 * cores and adds it to the fp32 accumulator in the workspace with reduce-adds,
 * so S and dP are rebuilt once per tile pair instead of twice (johe.ru, section
 * "Стадии вычисления", pass 2; the dQ product is one of the five).  The order
 * of those fp32 additions varies from run to run, so dq is not bit-for-bit
 * reproducible (dk and dv are).  Launches: the preprocess (which also zeroes
 * the accumulator), the pass, and a conversion of the accumulator to bf16 dq.
 * d = 128 only (FA_ERR_UNSUPPORTED otherwise).  workspace must hold at least
 * fa_bwd_fused_workspace_bytes(B,H,Nq,Nk,d) bytes, 16-byte aligned; its
 * contents on entry do not matter. */
int fa_bwd_fused(const void *q, const void *k, const void *v, const void *o, const float *lse,
                 const void *dO, void *dq, void *dk, void *dv,
                 int B, int H, int Nq, int Nk, int d, float scale, int causal,
                 void *workspace, size_t workspace_bytes, void *stream);

/* Backward of fa_fwd_window (same window, same conventions as fa_bwd). */
int fa_bwd_window(const void *q, const void *k, const void *v, const void *o, const float *lse,
                  const void *dO, void *dq, void *dk, void *dv,
                  int B, int H, int Nq, int Nk, int d, float scale, int window,
                  void *workspace, size_t workspace_bytes, void *stream);

/* Backward of fa_fwd_varlen (same lengths, same conventions as fa_bwd).
 * Gradient rows past a sequence's length (dq past seqlens_q[b], dk and dv
 * past seqlens_k[b]) are written as zeros.  dO must be finite in padding rows
 * too; lse is fa_fwd_varlen's (-inf in padding rows). */
int fa_bwd_varlen(const void *q, const void *k, const void *v, const void *o, const float *lse,
                  const void *dO, void *dq, void *dk, void *dv,
                  const int *seqlens_q, const int *seqlens_k,
                  int B, int H, int Nq, int Nk, int d, float scale, int causal,
                  void *workspace, size_t workspace_bytes, void *stream);

/* The three steps of fa_bwd, for callers that schedule them (or time them)
 * separately; fa_bwd is exactly these three launches in this order, except
 * that it launches each as a programmatic dependent of the one before: the
 * dK/dV pass sets up and loads K/V while the preprocess ends, and the dQ pass
 * may start on SMs that the last dK/dV CTAs leave free.  Every read of D still
 * follows the preprocess, and the dQ grid completes only after the dK/dV grid.
 *  fa_bwd_preprocess: delta [B,H,Nq] fp32 = rowsum(dO o O).
 *  fa_bwd_dkdv: dk, dv [B,H,Nk,d] from q, k, v, lse, delta, dO; each
 *    128-key tile is one work item of a persistent grid (at most one CTA per
 *    SM), P and dS rebuilt on chip for every query tile it sees.
 *  fa_bwd_dq: dq [B,H,Nq,d] from q, k, v, lse, delta, dO; each 128-query
 *    tile is one work item.  dkdv and dq only read delta, so they may run in any
 *    order (or concurrently) after the preprocess.
 * Same conventions and errors as fa_bwd. */
int fa_bwd_preprocess(const void *o, const void *dO, float *delta, int B, int H, int Nq, int d,
                      void *stream);
int fa_bwd_dkdv(const void *q, const void *k, const void *v, const float *lse, const float *delta,
                const void *dO, void *dk, void *dv, int B, int H, int Nq, int Nk, int d, float scale,
                int causal, void *stream);
int fa_bwd_dq(const void *q, const void *k, const void *v, const float *lse, const float *delta,
              const void *dO, void *dq, int B, int H, int Nq, int Nk, int d, float scale, int causal,
              void *stream);

/* fa_bwd_dkdv on CTA pairs (d = 128 only; FA_ERR_UNSUPPORTED for d = 64):
 * the two CTAs of a cluster take key tiles 2t and 2t + 1 of a head and issue
 * every product once for both as a tcgen05.mma with cta_group::2 (M = 256
 * keys), each CTA loading only the half of the B operand that it contributes.
 * Same arguments, outputs and tolerance as fa_bwd_dkdv (the same sums, split
 * differently across the tensor cores).  It needs more synchronisation
 * between the two CTAs than it saves in shared-memory reads, so it is slower
 * than fa_bwd_dkdv, which fa_bwd uses (johe.ru "Flash Attention: ...",
 * section "Flash Attention 4": kernels for the newest tensor cores).  The
 * caller's stream must allow cluster launches (every CUDA stream does). */
int fa_bwd_dkdv_pair(const void *q, const void *k, const void *v, const float *lse, const float *delta,
                     const void *dO, void *dk, void *dv, int B, int H, int Nq, int Nk, int d, float scale,
                     int causal, void *stream);

/* Bytes of fp32 workspace fa_decode needs for num_splits partials (<= 0:
 * for min(16, ceil(Nk / 256)) splits, the most the automatic count takes).
 * Host only, no device call.  Returns 0 for invalid sizes. */
size_t fa_decode_workspace_bytes(int B, int H, int Nk, int d, int num_splits);

/* Split-KV decode: one query token per (b, h) against a KV cache.  The key
 * cache is streamed, not shrunk (zimaspace.com "Wie reduziert Flash Attention
 * den Speicherverkehr ...", section "Weniger IO bedeutet nicht, dass der
 * KV-Cache entfällt").  The Nk keys are cut into num_splits contiguous chunks of
 * ceil(Nk / num_splits) keys; each chunk yields a partial output and partial
 * LSE, and the partials are merged with the max-shifted rescaling of the
 * online-softmax recurrence (wiki.ai-engineering.at "Flash Attention",
 * "Lösung: Online Softmax").  With d = 128 and Nk a multiple of 128 the
 * chunks are read by the tensor-core kernel of
 * fa_decode_paged (the cache as one page per sequence), whose chunks are
 * rounded up to whole 128-key stages, so trailing chunks may be empty; every
 * other shape takes a kernel of 16-byte loads.  The result is the same up to
 * rounding either way.  q [B,H,d], kcache/vcache [B,H,Nk,d] bf16 in;
 * o [B,H,d] bf16 out; lse [B,H] fp32 out, may be NULL.  num_splits <= 0 lets
 * the library choose: min(16, ceil(Nk / 256)) on the tensor-core kernel; on
 * the other kernel the count in 1 .. min(16, ceil(Nk / 256)) whose
 * (b, h, split) grid costs the fewest waves of resident CTAs times keys per
 * split (ties: fewer splits).  Otherwise 1 <= num_splits <= 256.  workspace:
 * at least fa_decode_workspace_bytes(B,H,Nk,d,num_splits) bytes. */
int fa_decode(const void *q, const void *kcache, const void *vcache, void *o, float *lse,
              int B, int H, int Nk, int d, float scale, int num_splits,
              void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of fp32 workspace fa_decode_paged needs (partials of B*Hq heads);
 * num_splits <= 0 (automatic) returns the size for 16 splits, the most the
 * automatic choice takes. */
size_t fa_decode_paged_workspace_bytes(int B, int Hq, int d, int num_splits);

/* Decode against a paged KV cache with grouped-query heads (the serving
 * layout: johe.ru "Flash Attention: ...", section "Альтернативы",
 * PagedAttention keeps the cache in fixed-size pages; grouped-query heads
 * share one kv head).  For every sequence b and query head h it computes the
 * same result as fa_decode against the sequence's first seq_lens[b] tokens
 * in logical order, with query head h reading kv head h / (Hq / Hkv).
 *  q [B, Hq, d] bf16; k_pages, v_pages [num_pages, Hkv, page_size, d] bf16
 *  (a page holds page_size consecutive tokens of one kv head);
 *  block_table [B, max_pages] int32: physical page of each logical page;
 *  seq_lens [B] int32, 1 <= seq_lens[b] <= max_pages * page_size;
 *  o [B, Hq, d] bf16; lse [B, Hq] fp32 or NULL.
 * num_splits <= 0 lets the library choose (from B, the heads, the longest
 * possible sequence max_pages * page_size and the SM count; at most 16).
 * Each sequence is cut into num_splits (1..256) contiguous chunks of
 * ceil(seq_lens[b] / num_splits) tokens (rounded up to whole 128-token stages
 * on the tensor-core path: page_size a multiple of 8), merged as in
 * fa_decode.  Every K/V
 * row is read once per group of up to 16 query heads on that path (4 on the
 * general one).  Tokens past seq_lens[b] in a page are never used, whatever
 * they hold.  Host checks: Hq % Hkv
 * == 0, d in {64, 128}, alignment, workspace.  The table and lengths live in
 * device memory and are checked by the kernel: a page index outside
 * [0, num_pages) or a length out of range is never dereferenced; it is read
 * as zeros and recorded as FA_ERR_INVALID_ARG in the device error word
 * (fa_get_last_device_error). */
int fa_decode_paged(const void *q, const void *k_pages, const void *v_pages, const int *block_table,
                    const int *seq_lens, void *o, float *lse, int B, int Hq, int Hkv, int page_size,
                    int max_pages, int num_pages, int d, float scale, int num_splits, void *workspace,
                    size_t workspace_bytes, void *stream);

/* ---- Rotary positions and a paged KV cache held in 8 bits -------------------
 * A serving step with them: fa_rope on the queries, fa_cache_append_fp8 on the
 * new keys (rotated on the way) and values, fa_decode_paged_fp8, and, when a
 * sequence has outgrown its budget, fa_cache_evict_fp8.  (The cache stays in
 * memory and is streamed: zimaspace.com "Wie reduziert Flash Attention ...",
 * section "Weniger IO bedeutet nicht, dass der KV-Cache entfaellt"; 8 bits
 * halve what is streamed.)
 *
 * The cache: k_pages, v_pages e4m3 bytes [num_pages, Hkv, page_size, d] (OCP
 * FP8, no infinities); k_scale, v_scale fp32 [num_pages, Hkv, page_size /
 * scale_block], one per block of scale_block consecutive tokens of a page and
 * kv head, positive and finite.  An element stands for its e4m3 value times its
 * block's scale.  scale_block divides page_size and is at most 128; any page
 * size >= 1.  block_table int32 [B, max_pages]: physical page of each logical
 * page; seq_lens int32 [B], 0 <= seq_lens[b] <= max_pages * page_size <= 2^30.
 * Scales, tables, lengths, positions, lse and weights need 4-byte alignment
 * only.  A length out of range is clamped, a page index outside [0, num_pages)
 * is never dereferenced (reads give zeros, writes are left out); either is
 * recorded as FA_ERR_INVALID_ARG in the device error word.  num_pages * Hkv *
 * page_size must stay below 2^32 - 1 (FA_ERR_UNSUPPORTED). */

/* Turns per position for fa_rope and fa_cache_append_fp8: turns[i] =
 * inv_freq[i] / (2 pi) modulo whole turns, in units of 2^-64 turn: the quotient
 * as a double has it (within 2^-52 of itself), rounded to 2^-65 turn; -x gives
 * the negative of x's.  inv_freq[i] (finite, host memory) is pair i's angle per
 * position in radians; scalings for long contexts change these frequencies (and
 * the magnitude below).  n >= 1.  Host only; copy the n values to the device. */
int fa_rope_table(const double *inv_freq, int n, uint64_t *turns);

/* Rotary positions.  x and y: bf16 [B, H, N, d] with element strides (sb, sh,
 * sn, 1), multiples of 8 (FA_ERR_ALIGNMENT) and >= 0; those of a dimension of
 * size 1 are ignored.  y's elements must be distinct (FA_ERR_INVALID_ARG); y may
 * be x with the same strides, but may not overlap it otherwise.  For token
 * (b, n) at position p = positions[b * N + n] (int32 [B, N], any value; NULL: n)
 * the pair i < rot / 2 turns by the angle a = p * inv_freq[i]:
 *     y1 = magnitude (x1 cos a - x2 sin a),  y2 = magnitude (x2 cos a + x1 sin a)
 * where the pair is columns (2i, 2i + 1) if interleaved, else (i, i + rot / 2);
 * columns from rot on are copied.  inverse = 1 turns by -a with the same
 * magnitude: the transpose, i.e. the gradient of x from the gradient of y.  The
 * angle of the table's turns is reduced exactly at any position, and its cos and
 * sin are within 2^-23; the table itself is off by at most 2^-52 |p inv_freq[i]| +
 * 2^-62 |p| radians (below 2^-24 up to 2^27 radians).  Computed in fp32, rounded
 * to bf16 once.  rot: a multiple of 16
 * (FA_ERR_UNSUPPORTED), 16 <= rot <= d; turns: device [rot / 2], 16-byte
 * aligned; magnitude finite.  B * N <= 2^31 - 1, B * H <= 2^24. */
int fa_rope(const void *x, void *y, long long x_sb, long long x_sh, long long x_sn, long long y_sb,
            long long y_sh, long long y_sn, const int *positions, const uint64_t *turns, int B, int H, int N,
            int d, int rot, int interleaved, float magnitude, int inverse, void *stream);

/* Writes new tokens into the cache.  k, v: bf16 [B, Hkv, N, d] with strides as
 * fa_rope's x.  Sequence b has seq_lens[b] tokens in the cache and gets its
 * first n_b = new_lens[b] (0..N; NULL: N) tokens at seq_lens[b], seq_lens[b] + 1,
 * ...; tokens that would not fit max_pages * page_size are left out and
 * recorded.  seq_lens is not changed, and a sequence with n_b = 0 is not
 * touched, nor its table's pages looked at.  B * Hkv * N <= 2^31 - 1 and
 * N <= 2^29 (FA_ERR_UNSUPPORTED).  If turns is not NULL, K is rotated first
 * as by fa_rope (same arguments; positions NULL: seq_lens[b] + i) and rounded
 * to bf16: the result is, bit for bit, that of fa_rope followed by this call
 * without turns.  With turns NULL, rot, interleaved, magnitude and positions
 * are ignored.
 * Scales: s = the smallest power of two >= 2^-126 with amax <= 448 s over the
 * finite new elements of the block; if the block holds earlier tokens of the
 * sequence, the larger of s and its present scale.  If that grows the scale, the
 * block's earlier tokens are rescaled to it (exact unless they become
 * subnormal).  Elements are rounded to nearest, infinities saturate at 448
 * times the scale, NaN stays NaN.  Slots behind the new tokens keep their
 * bytes.  No page may be written for two sequences at once. */
int fa_cache_append_fp8(const void *k, const void *v, long long k_sb, long long k_sh, long long k_sn,
                        long long v_sb, long long v_sh, long long v_sn, void *k_pages, void *v_pages,
                        float *k_scale, float *v_scale, const int *block_table, const int *seq_lens,
                        const int *new_lens, const int *positions, const uint64_t *turns, int B, int Hkv, int N,
                        int d, int rot, int interleaved, float magnitude, int page_size, int scale_block,
                        int max_pages, int num_pages, void *stream);

/* Bytes of workspace fa_decode_paged_fp8 needs; max_tokens = max_pages *
 * page_size, weights = 1 if it is given accumulated weights.  Those take fp32
 * scores of every query row (rounded up to 4 per kv head) and slot of the table
 * besides the partials, 4 * B * Hq * Nq * max_tokens bytes, whatever the lengths
 * are: give such calls a table no wider than the longest sequence needs.  Returns
 * 0 for invalid sizes.  Host only, no device call. */
size_t fa_decode_paged_fp8_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int max_tokens, int weights);

/* Attention of the last Nq (1..16) tokens of each sequence over the 8-bit
 * cache, which holds them already: one token, or a few drafted ones.  q, o: bf16
 * [B, Hq, Nq, d]; lse fp32 [B, Hq, Nq] or NULL.  Query head h reads kv head h /
 * (Hq / Hkv); query t sees the tokens j <= seq_lens[b] - Nq + t (the bottom-right
 * mask of fa_fwd).  A query that sees none (an empty sequence) gets O = 0,
 * LSE = -inf.  Scores and sums are fp32; for the value product only, a softmax
 * weight times its block's V scale is rounded to fp16: by 2^-11 of itself, or,
 * where it is below 2^-25 of the largest one of its row, by 2^-36 of that.
 * weights fp32 [B, Hkv, max_pages * page_size] or NULL: weights[b, kvh, j] +=
 * the sum of token j's attention weights over the group's heads and the Nq
 * queries (what fa_cache_evict_fp8 selects by); tokens >= seq_lens[b] are left
 * as they are.
 * The tokens of all sequences are dealt out evenly, by their lengths, to the
 * CTAs that run at once, so there is no number of splits to choose.  Results do
 * not depend on the run (fixed order of additions), but for rounding on the
 * batch that a sequence is in.  Steps of 128 tokens over all sequences at full
 * capacity, kv heads and tiles of 32 query rows must stay below 2^31
 * (FA_ERR_UNSUPPORTED).  Tokens past seq_lens[b] are never used, and one that a
 * query does not see does not reach it, whatever it holds (a padded draft's NaN
 * too).  No output may overlap an input or the cache (o = q:
 * FA_ERR_INVALID_ARG).  workspace: 16-byte aligned, at least
 * fa_decode_paged_fp8_workspace_bytes(...); contents do not matter; calls that
 * may overlap need one each. */
int fa_decode_paged_fp8(const void *q, const void *k_pages, const void *v_pages, const float *k_scale,
                        const float *v_scale, const int *block_table, const int *seq_lens, void *o, float *lse,
                        float *weights, int B, int Hq, int Hkv, int Nq, int page_size, int scale_block,
                        int max_pages, int num_pages, int d, float scale, void *workspace, size_t workspace_bytes,
                        void *stream);

/* Eviction by accumulated attention weight: per sequence b and kv head, the
 * min(seq_lens[b], keep) tokens that stay are the last `recent` (0..keep) and,
 * of the others, the keep - recent with the largest weights[b, kvh, j]; of equal
 * ones (+0 = -0) the lowest index, and NaN counts as largest.  A sequence of at
 * most keep tokens keeps all.  The kept tokens are copied in order into the
 * pages of new_table int32 [B, new_max_pages] (keep <= new_max_pages *
 * page_size), from slot 0 on.  Those pages must be disjoint from every page that
 * the call reads and from each other's; the source pages stay as they are (they
 * may be shared), so a page can be freed by its owner afterwards.  A block's
 * scale is the largest of its tokens' source scales; tokens of smaller scale
 * are rescaled to it.  Outputs: new_lens int32 [B]; kept int32 and new_weights
 * fp32 [B, Hkv, new_max_pages * page_size]: the source index of each kept token
 * and its weight, then -1 and 0 (so new_weights goes on accumulating).  No
 * output may overlap an input (new_lens = seq_lens or new_weights = weights:
 * FA_ERR_INVALID_ARG).  Rotation stays as it was applied: later tokens go on with
 * their own positions. */
int fa_cache_evict_fp8(void *k_pages, void *v_pages, float *k_scale, float *v_scale, const int *block_table,
                       const int *seq_lens, const float *weights, const int *new_table, int *new_lens,
                       float *new_weights, int *kept, int B, int Hkv, int page_size, int scale_block,
                       int max_pages, int new_max_pages, int num_pages, int d, int keep, int recent, void *stream);

/* ---- Long contexts out of the paged bf16 cache -------------------------------
 * The cache of fa_decode_paged (k_pages, v_pages bf16 [num_pages, Hkv, page_size,
 * d], block_table int32 [B, max_pages], seq_lens int32 [B]), its writer and two
 * ways to read less of it: fa_cache_append writes new tokens, the keys rotated on
 * the way; fa_select_blocks and fa_decode_blocks attend to the blocks that a
 * score from bounds of their keys selects; fa_decode_shared reads a prefix that
 * all sequences have in common once for the whole batch.  (The cache is
 * streamed, not shrunk: zimaspace.com "Wie reduziert Flash Attention ...",
 * section "Weniger IO bedeutet nicht, dass der KV-Cache entfaellt"; pages: johe.ru
 * "Flash Attention: ...", section "Альтернативы", PagedAttention.)
 *
 * Any page size >= 1 (fa_decode_shared: a multiple of 8).  A block is `block`
 * consecutive tokens of a page and kv head; block divides page_size and is at
 * most 128.  Tables, lengths, positions, lists of blocks and lse need 4-byte
 * alignment only.  0 <= seq_lens[b] <= max_pages * page_size <= 2^30.  A length
 * out of range is clamped, a page index outside [0, num_pages) is never
 * dereferenced (reads give zeros, writes are left out); either is recorded as
 * FA_ERR_INVALID_ARG in the device error word.  num_pages * Hkv * page_size must
 * stay below 2^32 - 1 (FA_ERR_UNSUPPORTED). */

/* Writes new tokens into the cache.  k, v, strides, seq_lens, new_lens, turns,
 * rot, interleaved, magnitude and positions as for fa_cache_append_fp8: sequence b
 * gets its first n_b tokens at seq_lens[b], seq_lens[b] + 1, ..., the keys rotated
 * as by fa_rope if turns is not NULL, and rounded to bf16 once.  bounds: bf16
 * [num_pages, Hkv, page_size / block, 2, d] or NULL: the smallest and the largest
 * element of each key column over the block's tokens, as they are stored (NaN
 * where one of them is NaN).  Those of a block that tokens of the sequence before
 * seq_lens[b] are in are widened, those of a block that starts with new tokens
 * are replaced.  With bounds NULL, block is ignored.  Slots behind the new
 * tokens keep their contents.  No page may be written for two sequences at once. */
int fa_cache_append(const void *k, const void *v, long long k_sb, long long k_sh, long long k_sn, long long v_sb,
                    long long v_sh, long long v_sn, void *k_pages, void *v_pages, void *bounds, const int *block_table,
                    const int *seq_lens, const int *new_lens, const int *positions, const uint64_t *turns, int B,
                    int Hkv, int N, int d, int rot, int interleaved, float magnitude, int page_size, int block,
                    int max_pages, int num_pages, void *stream);

/* Bytes of workspace fa_select_blocks needs; max_blocks = max_pages * page_blocks.
 * 12 bytes per kv head and block of the table, whatever the lengths are.  Returns
 * 0 for invalid sizes.  Host only, no device call. */
size_t fa_select_blocks_workspace_bytes(int B, int Hkv, int max_blocks);

/* The blocks that the last Nq (1..16) tokens of each sequence are to attend to.
 * q bf16 [B, Hq, Nq, d]; bounds bf16 [num_pages, Hkv, page_blocks, 2, d] as
 * fa_cache_append keeps them, page_blocks = page_size / block.  No key of a block
 * gives a row r of q more than u_r = sum_c max(q_rc, 0) max_c + min(q_rc, 0) min_c
 * (before the scale); the block's score is the largest u_r of the kv head's Hq /
 * Hkv x Nq rows.  blocks int32 [B, Hkv, keep] out: of the n_b = ceil(seq_lens[b] /
 * block) blocks of sequence b the first `first` ones, the last `recent` ones
 * (first + recent <= keep) and, of the others, the keep - first - recent of
 * largest score, in ascending order; all of them and -1 behind them if n_b <= keep.
 * The choice is that of exact scores, but for what is below 2^-58 of the largest
 * sum_c |q_rc| |bound_c|: of equal ones (+0 = -0) the lowest index stays; NaN (also
 * an infinite bound times zero) counts as largest.  Where a query element or a bound
 * is not finite, or all of a kv head's bounds are zero, its scores are summed in fp64,
 * which takes a hundred times as long (milliseconds for thousands of blocks); several
 * hundred equal scores around the last that stays take several times as long.  recent should
 * cover the Nq tokens.  workspace: 16-byte aligned, at least
 * fa_select_blocks_workspace_bytes(...); contents do not matter; calls that may
 * overlap need one each. */
int fa_select_blocks(const void *q, const void *bounds, const int *block_table, const int *seq_lens, int *blocks, int B,
                     int Hq, int Hkv, int Nq, int block, int page_blocks, int max_pages, int num_pages, int d, int keep,
                     int first, int recent, void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_decode_blocks needs.  Returns 0 for invalid sizes.  Host
 * only, no device call. */
size_t fa_decode_blocks_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d);

/* Attention of the last Nq (1..16) tokens of each sequence over listed blocks of
 * the cache, which holds them already.  q, o bf16 [B, Hq, Nq, d]; lse fp32 [B, Hq,
 * Nq] or NULL; blocks int32 [B, Hkv, keep]: distinct blocks of the sequence, in any
 * order (a block listed twice counts twice).  Of a list the first min(keep, n_b)
 * entries are looked at, n_b = ceil(seq_lens[b] / block); negative ones are
 * skipped, ones >= n_b too, and recorded as FA_ERR_INVALID_ARG.  Query head h reads
 * kv head h / (Hq / Hkv); query t sees the tokens j <= seq_lens[b] - Nq + t of the
 * listed blocks.  A query that sees none gets O = 0, LSE = -inf.  Scores and sums
 * are fp32; for the value product a softmax weight is rounded to 16 bits (2^-17).
 * Results do not depend on the run (fixed order of additions), but for rounding on
 * the batch that a sequence is in.  Tokens past seq_lens[b] are never used, and one
 * that a query does not see does not reach it, whatever it holds.  (B + 4) x Hkv x
 * tiles x (steps + 2) must stay below 2^31 (FA_ERR_UNSUPPORTED), with steps = (max_pages *
 * page_size + block) / 64, rounded up, and the tiles that a kv head's Hq / Hkv x Nq
 * query rows make: of 8 rows, of 16 if there are more, of 32 if there are more than
 * 16.  No output may overlap an input (o = q: FA_ERR_INVALID_ARG).  workspace as for
 * fa_select_blocks. */
int fa_decode_blocks(const void *q, const void *k_pages, const void *v_pages, const int *block_table,
                     const int *seq_lens, const int *blocks, void *o, float *lse, int B, int Hq, int Hkv, int Nq,
                     int page_size, int block, int keep, int max_pages, int num_pages, int d, float scale,
                     void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace fa_decode_shared needs.  Returns 0 for invalid sizes.  Host
 * only, no device call. */
size_t fa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d);

/* Attention of the last Nq (1..16) tokens of each sequence over the whole cache,
 * where the first shared_len[0] tokens are the same for all sequences (a system
 * prompt, a document with many questions, samples of one prompt).  q, o, lse and the
 * mask as for fa_decode_blocks with every block listed.  shared_len: device int32
 * [1], 0 <= shared_len[0] <= max_pages * page_size, any number of tokens.
 * seq_lens[b] counts the shared tokens too.  A sequence with seq_lens[b] - Nq >=
 * shared_len[0] takes part: its first shared_len[0] tokens are read through the
 * table's row of the first sequence that takes part (its own entries for whole
 * shared pages are not looked at), the others through its own row.  Others (a slot
 * without a sequence, or a shorter one) read all their tokens through their own
 * row.  For the product of a shared token's weight and value the weight is rounded
 * to bf16 (2^-8), or to 16 bits (2^-17) in small batches with narrow tables; for own
 * tokens it is to 16 bits.  Errors, workspace (its size:
 * fa_decode_shared_workspace_bytes) and the rest as for fa_decode_blocks (in its limit
 * block is 1, and the tiles are of 8 rows up to 16 rows, and up to 32 where B * Hkv
 * <= 128); page_size must be a multiple of 8 (FA_ERR_UNSUPPORTED). */
int fa_decode_shared(const void *q, const void *k_pages, const void *v_pages, const int *block_table,
                     const int *seq_lens, const int *shared_len, void *o, float *lse, int B, int Hq, int Hkv, int Nq,
                     int page_size, int max_pages, int num_pages, int d, float scale, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Size of the scratch array that fa_decode_noalloc uses instead of a workspace. */
#define FA_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

/* Split-KV decode exactly like fa_decode, for callers that cannot allocate
 * device memory when they need a decode step.  Examples: a serving loop or
 * plugin host that hands this library only its input and output buffers and
 * owns every other byte of device memory; a real-time path that must never
 * call the allocator, because cudaMalloc/cudaFree may synchronise the whole
 * device and may fail once memory is fragmented; C callers with no access to
 * the framework allocator that owns the tensors.
 * Not a step of the method: the pages have no counterpart; it only changes
 * where the split partials live.  Instead of a caller workspace, the partials
 * go to one fixed array of FA_DECODE_NOALLOC_SCRATCH_BYTES compiled into the
 * library (every GPU that loads the library holds it until the process exits).
 * Arguments mean what they mean for fa_decode; the caller still passes q, the
 * caches, o and (optionally) lse.  A problem whose partials would need more
 * than the array (fa_decode_workspace_bytes(B,H,Nk,d,num_splits) >
 * FA_DECODE_NOALLOC_SCRATCH_BYTES) is rejected with FA_ERR_WORKSPACE before
 * anything is launched.  The call allocates nothing.  The first call on each
 * device looks up the array's device address (with that device current) and
 * caches it; make that first call before any stream capture.  All calls share
 * the one array: calls that may overlap on the GPU (different streams, no
 * ordering between them) race on it, so order them.  Nothing in the array has
 * to start at zero (every partial is written before it is read), and it keeps
 * the last call's partials. */
int fa_decode_noalloc(const void *q, const void *kcache, const void *vcache, void *o, float *lse,
                      int B, int H, int Nk, int d, float scale, int num_splits, void *stream);

/* Synchronises `stream`, then reads and clears the device error word of the
 * current device.  Returns FA_OK, the first code a kernel recorded
 * (FA_ERR_TIMEOUT: a bounded wait ran out; FA_ERR_INVALID_ARG: a device-side
 * argument check failed, e.g. a page index), or FA_ERR_CUDA if synchronising
 * or reading failed.  If `detail` is not NULL it
 * receives 4 ints: code, site (which wait), block index, and an auxiliary
 * value (the wait's phase), all 0 when no error was recorded. */
int fa_get_last_device_error(void *stream, int *detail);

/* Watchdog self-test (failure detection without a GPU fault): launches one
 * thread that waits on a barrier nothing ever arrives on, with a limit of
 * timeout_ns (1e3 .. 1e9).  The wait runs out, the kernel records
 * FA_ERR_TIMEOUT (site 19, the self-test site) in the error word and returns;
 * fa_get_last_device_error(stream, ...) then reports it and clears the word.
 * The device stays usable.  Returns the launch status. */
int fa_selftest_wait_timeout(uint64_t timeout_ns, void *stream);

/* Sets the limit of every device-side wait, in nanoseconds, for kernels
 * launched after the call (default 2e9; values below 1e6 are raised to 1e6).
 * Returns the previous value. */
uint64_t fa_set_wait_timeout_ns(uint64_t ns);

/* Static description of a status code. */
const char *fa_status_string(int status);

/* Library version, as major * 10000 + minor * 100 + patch. */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
