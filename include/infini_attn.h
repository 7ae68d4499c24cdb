/*
 * infini_attn.h -- C ABI of the B200 (sm_100a) Infini-attention forward library.
 *
 * What is computed (AI Wiki "Infini-Attention", "What happens inside the Infini-attention
 * block?" and "How does the compressive memory work?"; the Hugging Face reproduction
 * analysis, "Infini-Attention Mechanism", steps 1-6):
 *
 *   The length-L sequence of every (batch b, query head h) is cut into segments of N
 *   tokens, processed in order; when N does not divide L the last segment is shorter
 *   (L mod N tokens) and is processed the same way, its update included.  For segment s
 *   and query row q_t:
 *     A_dot = causal softmax(q_t K_s^T / sqrt(d)) V_s     keys of segment s only, j <= t
 *     A_mem = sigma(q_t) M_{s-1} / (sigma(q_t) . z_{s-1}) sigma(x) = ELU(x) + 1; 0 while the
 *                                                          denominator is exactly 0
 *     out_t = g_h A_mem + (1 - g_h) A_dot                  g_h = 1 / (1 + exp(-beta[h]))
 *   After the segment the memory of its key/value head advances:
 *     linear: M_s = M_{s-1} + sigma(K_s)^T V_s
 *     delta : M_s = M_{s-1} + sigma(K_s)^T (V_s - sigma(K_s) M_{s-1} / (sigma(K_s) z_{s-1}))
 *             (one batch update per segment; a row whose denominator is 0 predicts 0)
 *     both  : z_s = z_{s-1} + sum_t sigma(K_{s,t})
 *   Query head h reads key/value head h / (H / Hkv) (grouped-query attention).
 *
 * Layouts: row-major, contiguous, on the device:
 *   q, out  [B, H,   L, d]        k, v  [B, Hkv, L, d]        beta [H] float
 *   M0, M_out [B, Hkv, d, d] float (row = key feature, column = value feature)
 *   z0, z_out [B, Hkv, d]    float
 *
 * Conventions shared by every entry point:
 *   - All pointers are DEVICE pointers owned by the caller; the library keeps none of them
 *     after the call returns.  Every pointer must be 16-byte aligned.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream) and
 *     runs asynchronously: results are valid once that stream has synchronised.
 *   - M0 / z0 may be NULL (an empty memory: zeros).  M_out / z_out may alias M0 / z0
 *     exactly (in-place state update); a partial overlap is INFINI_ERR_INVALID_ARG.  out
 *     must not overlap any input.
 *   - Preconditions not checked: z0 >= 0 elementwise (sigma > 0 then makes a zero
 *     denominator mean an empty memory); inputs finite.
 *   - On an argument error nothing is launched and nothing is written.  Nothing aborts,
 *     throws or traps; every failure is an int status below.
 *   - Scratch: the call allocates its workspace (per-segment memory snapshots; the size
 *     is infini_attn_workspace_bytes) stream-ordered on `stream` from a memory pool the
 *     library owns on each device, and frees it on the same stream.  The pool keeps freed
 *     memory for the next call (up to the largest workspace used so far).
 */
#ifndef INFINI_ATTN_H
#define INFINI_ATTN_H

#include <stdint.h>

#if defined(__GNUC__)
#define INFINI_API __attribute__((visibility("default")))
#else
#define INFINI_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *infini_stream_t;

enum {
    INFINI_UPDATE_LINEAR = 0, /* M += sigma(K)^T V                      */
    INFINI_UPDATE_DELTA = 1   /* M += sigma(K)^T (V - sigma(K) M / den) */
};

enum {
    INFINI_OK = 0,
    INFINI_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size or position, bad rule,
                                   partial overlap of a state output with its input        */
    INFINI_ERR_UNSUPPORTED = 2, /* valid but not built: d not in {32, 64, 128}, N % 64 != 0 */
    INFINI_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed                      */
    INFINI_ERR_OOM = 4,         /* the workspace allocation failed                           */
    INFINI_ERR_TIMEOUT = 5,     /* a bounded device wait gave up (infini_attn_device_status) */
    INFINI_ERR_PAGE = 6         /* a kernel met a page number or row outside the paged cache
                                   (infini_attn_device_status)                             */
};

/*
 * Infini-attention forward, bf16 activations (q, k, v, out are __nv_bfloat16; arithmetic
 * in fp32, memory M / z in fp32, out rounded to nearest-even).
 *
 *   B, H, Hkv : batch, query heads, key/value heads (H % Hkv == 0)
 *   L, N, d   : sequence length, segment length, head dimension (L need not be a
 *               multiple of N: the final L mod N tokens form a shorter last segment)
 *   update_rule : INFINI_UPDATE_LINEAR or INFINI_UPDATE_DELTA
 * Returns INFINI_OK or an error status.
 */
INFINI_API int infini_attn_fwd(const void *q, const void *k, const void *v, const float *beta,
                    const float *M0, const float *z0, void *out, float *M_out, float *z_out,
                    int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t N, int64_t d,
                    int update_rule, infini_stream_t stream);

/* The same operation with fp32 activations (q, k, v, out are float); identical parameters. */
INFINI_API int infini_attn_fwd_f32(const void *q, const void *k, const void *v, const float *beta,
                        const float *M0, const float *z0, void *out, float *M_out,
                        float *z_out, int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t N,
                        int64_t d, int update_rule, infini_stream_t stream);

/*
 * Backward pass: the gradients of  <dout, out> + <dM, M_out> + <dz, z_out>  of the forward
 * above (same q, k, v, beta, M0, z0, N, update rule) with respect to every input, through
 * the local attention, the retrieval, the gate and the memory recurrence of every segment
 * (AI Wiki "Infini-Attention", "How is an Infini-attention model trained?": gradients flow
 * through the memory from segment to segment).  A quotient whose denominator is 0 (an
 * empty memory) is 0 and passes no gradient.
 *
 *   dout [B, H, L, d] (activation dtype): gradient of out;  dM [B, Hkv, d, d], dz [B, Hkv, d]
 *     fp32: gradients of M_out, z_out (NULL = zero)
 *   dq [B, H, L, d], dk / dv [B, Hkv, L, d] (activation dtype), dbeta [H], dM0 [B, Hkv, d, d],
 *     dz0 [B, Hkv, d] fp32: written; dbeta, dM0 and dz0 may be NULL (not written)
 *
 * infini_attn_bwd takes bf16 activations, infini_attn_bwd_f32 fp32 ones; all arithmetic is
 * fp32.  Outputs must not overlap any input or each other.  The call recomputes the
 * forward's memory and softmax statistics itself and allocates its workspace (fp32, about
 * 4 x (q + 3 k) bytes plus 3 memory snapshots per segment) like the forward.  Shapes,
 * alignment, streams and errors as for infini_attn_fwd.
 */
INFINI_API int infini_attn_bwd(const void *q, const void *k, const void *v, const float *beta,
                               const float *M0, const float *z0, const void *dout,
                               const float *dM, const float *dz, void *dq, void *dk, void *dv,
                               float *dbeta, float *dM0, float *dz0, int64_t B, int64_t H,
                               int64_t Hkv, int64_t L, int64_t N, int64_t d, int update_rule,
                               infini_stream_t stream);
INFINI_API int infini_attn_bwd_f32(const void *q, const void *k, const void *v,
                                   const float *beta, const float *M0, const float *z0,
                                   const void *dout, const float *dM, const float *dz, void *dq,
                                   void *dk, void *dv, float *dbeta, float *dM0, float *dz0,
                                   int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t N,
                                   int64_t d, int update_rule, infini_stream_t stream);

/*
 * The memory after the whole sequence, without the outputs (bf16 keys / values; the _f32
 * variant takes fp32 ones): M_out / z_out exactly as infini_attn_fwd would leave them, from
 * the forward's memory kernels alone.  With M0 = z0 = NULL this is the increment of a
 * sequence chunk under the additive rule, the quantity ranks exchange when one sequence is
 * cut across devices (the memory before a chunk is M0 plus the increments of the chunks
 * before it).  Arguments, layouts, aliasing and errors as for infini_attn_fwd, without q,
 * beta and out.
 */
INFINI_API int infini_attn_state(const void *k, const void *v, const float *M0, const float *z0,
                                 float *M_out, float *z_out, int64_t B, int64_t Hkv, int64_t L,
                                 int64_t N, int64_t d, int update_rule, infini_stream_t stream);
INFINI_API int infini_attn_state_f32(const void *k, const void *v, const float *M0,
                                     const float *z0, float *M_out, float *z_out, int64_t B,
                                     int64_t Hkv, int64_t L, int64_t N, int64_t d,
                                     int update_rule, infini_stream_t stream);

/*
 * Token-by-token decode (bf16 activations; the _f32 variant takes fp32 ones).  One call
 * processes one new token of every (batch, head) at offset `pos` of its current segment
 * and gives the output the forward would give that token:
 *   - local attention over the current segment's keys at offsets 0..pos: rows 0..pos-1 of
 *     the cache, then this token's own key and value, which the call writes into row pos;
 *   - retrieval from (M, z), the memory from before the current segment;
 *   - the gate, as in the forward.
 * When pos == N - 1 the segment is complete: after the output, the call folds all N cached
 * rows into (M, z) in place (the linear or delta update of the forward), and the next
 * token starts a new segment at pos = 0.  At the end of a stream whose last segment is
 * shorter, infini_attn_fold folds the rows cached so far; feeding a whole sequence this way
 * then leaves the forward's M_out / z_out in (M, z).
 *
 *   q [B, H, d], k / v [B, Hkv, d]: this token;  out [B, H, d]
 *   k_cache / v_cache [B, Hkv, N, d]: the current segment's keys and values (caller-owned;
 *     rows >= pos are not read)
 *   M [B, Hkv, d, d], z [B, Hkv, d] fp32: read, and updated in place when pos == N - 1
 *     (start a stream with zeros, or with a forward's M_out / z_out)
 *   0 <= pos < N; N any positive length; d in {32, 64, 128}
 * Everything runs on `stream`, and neither call allocates memory (both may be captured in
 * a CUDA graph).  out must not overlap any other buffer; caches, M and z must not overlap
 * one another.
 */
INFINI_API int infini_attn_decode_step(const void *q, const void *k, const void *v,
                                       const float *beta, void *k_cache, void *v_cache,
                                       int64_t pos, float *M, float *z, void *out, int64_t B,
                                       int64_t H, int64_t Hkv, int64_t N, int64_t d,
                                       int update_rule, infini_stream_t stream);
INFINI_API int infini_attn_decode_step_f32(const void *q, const void *k, const void *v,
                                           const float *beta, void *k_cache, void *v_cache,
                                           int64_t pos, float *M, float *z, void *out,
                                           int64_t B, int64_t H, int64_t Hkv, int64_t N,
                                           int64_t d, int update_rule, infini_stream_t stream);

/*
 * Fold the first n rows (0 <= n <= N; 0 does nothing) of every chain's cache into (M, z),
 * in place, with the update rule of the forward: the end of a stream whose last segment is
 * shorter than N.  Layouts as for infini_attn_decode_step; no allocation.
 */
INFINI_API int infini_attn_fold(const void *k_cache, const void *v_cache, int64_t n, float *M,
                                float *z, int64_t B, int64_t Hkv, int64_t N, int64_t d,
                                int update_rule, infini_stream_t stream);
INFINI_API int infini_attn_fold_f32(const void *k_cache, const void *v_cache, int64_t n,
                                    float *M, float *z, int64_t B, int64_t Hkv, int64_t N,
                                    int64_t d, int update_rule, infini_stream_t stream);

/*
 * Rotary positions.  The first `rot` channels of every head of q and k are turned in pairs by
 * the angle position * freq[i], i < rot / 2, and scaled:
 *     y1 = scale (x1 cos a - x2 sin a),   y2 = scale (x2 cos a + x1 sin a)
 * Pair i is channels (i, i + rot / 2), or (2 i, 2 i + 1) when `interleaved`; channels >= rot are
 * copied.  Apply it before infini_attn_fwd: the forward takes rotated q and k.  Angles are
 * formed and reduced in 64 bits, so positions far into a stream keep their fraction.
 *
 *   q [B, H, L, d], k [B, Hkv, L, d]: read through q_strides / k_strides, three element
 *     strides (batch, head, token) in HOST memory; NULL = contiguous.  The last dimension is
 *     contiguous; element alignment suffices (16-byte aligned rows are faster).  k may be NULL
 *     (with k_out): q alone.
 *   q_out, k_out: contiguous; each may be its own (contiguous) input
 *   freq [rot / 2] double (rot even, 0 <= rot <= d);  positions [B, L] int64 (8-byte alignment), or
 *     NULL: token t is at start + t.  Negative positions are valid.
 * The _bwd entries map the gradients of q_out, k_out to those of q, k with the same arguments
 * (the angle negated); they take the gradients in the place of q, k.
 */
INFINI_API int infini_attn_rotary(const void *q, const void *k, void *q_out, void *k_out,
                                  const double *freq, const int64_t *positions, int64_t start,
                                  const int64_t *q_strides, const int64_t *k_strides, int64_t B,
                                  int64_t H, int64_t Hkv, int64_t L, int64_t d, int64_t rot,
                                  int interleaved, float scale, infini_stream_t stream);
INFINI_API int infini_attn_rotary_f32(const void *q, const void *k, void *q_out, void *k_out,
                                      const double *freq, const int64_t *positions, int64_t start,
                                      const int64_t *q_strides, const int64_t *k_strides, int64_t B,
                                      int64_t H, int64_t Hkv, int64_t L, int64_t d, int64_t rot,
                                      int interleaved, float scale, infini_stream_t stream);
INFINI_API int infini_attn_rotary_bwd(const void *dq_out, const void *dk_out, void *dq, void *dk,
                                      const double *freq, const int64_t *positions, int64_t start,
                                      const int64_t *q_strides, const int64_t *k_strides, int64_t B,
                                      int64_t H, int64_t Hkv, int64_t L, int64_t d, int64_t rot,
                                      int interleaved, float scale, infini_stream_t stream);
INFINI_API int infini_attn_rotary_bwd_f32(const void *dq_out, const void *dk_out, void *dq, void *dk,
                                          const double *freq, const int64_t *positions, int64_t start,
                                          const int64_t *q_strides, const int64_t *k_strides,
                                          int64_t B, int64_t H, int64_t Hkv, int64_t L, int64_t d,
                                          int64_t rot, int interleaved, float scale,
                                          infini_stream_t stream);

/*
 * Decode over a paged cache: a batch whose sequences are at different places.
 *
 *   k_pages, v_pages [P, Hkv, page, d] (activation dtype): a pool of P pages, `page` rows each
 *     (a power of two; other sizes are INFINI_ERR_UNSUPPORTED)
 *   page_table [B, max_pages] int32: row r of sequence b lies in page page_table[b][r / page],
 *     slot r % page, the same for every key/value head.  Entries past a sequence's rows are not
 *     read.  Sequences may share pages that no call writes.
 *   lens [B] int32: rows each sequence has in the cache; negative: a padding entry of the
 *     batch, which reads and writes no page.  Calls do not change lens (all layers of a model
 *     share it): the caller adds the rows it appended.
 *   weights [P, Hkv, page] float: per row, the softmax weight it has received so far, summed
 *     over the group's query heads and the steps (NULL: not kept)
 * No entry allocates memory; all may be captured in a graph.  A workspace, where one is asked
 * for, holds nothing between calls, and calls that may overlap on the GPU need one each.
 * page_table and lens are read on the device: a page number outside [0, P), or a row past the
 * table's end, is never followed.  Such a row is left out (not read, not written; the new row of a
 * decode step is attended to all the same), and infini_attn_device_status reports INFINI_ERR_PAGE.
 * page_table, lens, counts, dst_table, lens_out and the decode step's beta need 4-byte alignment,
 * positions 8-byte, the strided k and v of infini_attn_paged_append that of an element.
 *
 * infini_attn_paged_append: rows lens[b] .. lens[b] + counts[b] - 1 become the first counts[b]
 * tokens of k, v [B, Hkv, T, d] (strides as for infini_attn_rotary; counts [B] int32, NULL: T
 * for every sequence; a count beyond T counts as T), and their weights 0.  T * Hkv may not
 * exceed 2^30.  Only decode steps add to weights: an eviction right behind a prompt finds ties, and
 * keeps the lowest rows and the recent ones, unless the caller writes weights of its own.
 */
INFINI_API int infini_attn_paged_append(const void *k, const void *v, const int64_t *k_strides,
                                        const int64_t *v_strides, void *k_pages, void *v_pages,
                                        float *weights, const int32_t *page_table,
                                        const int32_t *lens, const int32_t *counts, int64_t B,
                                        int64_t Hkv, int64_t T, int64_t d, int64_t P, int64_t page,
                                        int64_t max_pages, infini_stream_t stream);
INFINI_API int infini_attn_paged_append_f32(const void *k, const void *v, const int64_t *k_strides,
                                            const int64_t *v_strides, void *k_pages, void *v_pages,
                                            float *weights, const int32_t *page_table,
                                            const int32_t *lens, const int32_t *counts, int64_t B,
                                            int64_t Hkv, int64_t T, int64_t d, int64_t P,
                                            int64_t page, int64_t max_pages,
                                            infini_stream_t stream);

/*
 * infini_attn_paged_decode_step: one new token of every sequence, the counterpart of
 * infini_attn_decode_step with a row count per sequence:
 *   - rot > 0: q and k are rotated first, as by infini_attn_rotary, at positions [B] int64
 *     (NULL: lens);
 *   - k, v become row lens[b] (its weight starts at 0); with k = v = NULL nothing is appended
 *     and the attention spans the cached rows alone;
 *   - softmax attention of q over rows 0 .. lens[b]; a sequence without rows gives 0;
 *   - with beta, M and z (all or none): the retrieval from (M, z) with the rotated q and the
 *     gate, as in the forward given rotated q and k (with rot > 0 the retrieval so depends on the
 *     positions); M and z are read only;
 *   - with weights: every row's softmax weight, summed over the group's query heads, is added.
 *     The pages of a sequence must then be its own.
 * Padding entries (lens < 0) give rows of 0.
 *   q [B, H, d], k / v [B, Hkv, d], out [B, H, d];  out and the workspace overlap nothing.
 *   workspace: infini_attn_paged_decode_workspace_bytes(B, H, Hkv, d, P, page, weights != NULL):
 *     about (296 + B * Hkv) * (d + 2) * 4 bytes per query head of a group, and with weights
 *     P * page * H * 4 more (every cached row's scores)
 * The rows of all sequences are shared out over the SMs by the device, whatever the lengths; up
 * to eight query heads of a group share one reading of its rows, larger groups read them again.
 * Results do not depend on the run: nothing is summed in an order that may change.
 */
INFINI_API int infini_attn_paged_decode_step(
    const void *q, const void *k, const void *v, void *k_pages, void *v_pages,
    const int32_t *page_table, const int32_t *lens, const float *beta, const float *M,
    const float *z, float *weights, const double *freq, const int64_t *positions, void *out,
    void *workspace, int64_t workspace_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t d,
    int64_t P, int64_t page, int64_t max_pages, int64_t rot, int interleaved, float scale,
    infini_stream_t stream);
INFINI_API int infini_attn_paged_decode_step_f32(
    const void *q, const void *k, const void *v, void *k_pages, void *v_pages,
    const int32_t *page_table, const int32_t *lens, const float *beta, const float *M,
    const float *z, float *weights, const double *freq, const int64_t *positions, void *out,
    void *workspace, int64_t workspace_bytes, int64_t B, int64_t H, int64_t Hkv, int64_t d,
    int64_t P, int64_t page, int64_t max_pages, int64_t rot, int interleaved, float scale,
    infini_stream_t stream);
INFINI_API int64_t infini_attn_paged_decode_workspace_bytes(int64_t B, int64_t H, int64_t Hkv,
                                                            int64_t d, int64_t P, int64_t page,
                                                            int with_weights);

/*
 * infini_attn_paged_evict: cut every sequence to `budget` rows.  Of its n = lens[b] rows every
 * key/value head keeps the last `recent` (<= budget) and, of the others, those of the highest
 * weights (ties: the lowest row; a NaN counts as the highest), min(n, budget) in all.  They are
 * copied with their weights, in their old order, to rows 0, 1, ... of the pages dst_table
 * [B, dst_pages] (dst_pages * page >= budget); every other row of the pool stays as it was.  The
 * destination pages are written, so they must be in no other sequence and not among the pages of
 * page_table; only a sequence of at most `budget` rows may name its own pages (in the same
 * order), and nothing of it moves then.
 *   lens_out [B]: min(lens[b], budget) (may not be lens itself)
 *   kept [B, Hkv, budget] int32: the old rows of the kept ones, ascending, -1 past the last
 *   M, z (both or none): the rows not kept are folded in, in place, as one update of the
 *     forward's rule, with the keys as the cache holds them (rotated ones rotated).
 *     INFINI_UPDATE_DELTA is not built: INFINI_ERR_UNSUPPORTED.
 *   workspace: infini_attn_paged_evict_workspace_bytes(B, Hkv, d, page, max_pages, budget,
 *     M != NULL): nothing without a memory; else 4 bytes for every row of the table beyond the
 *     budget and key/value head, and about (148 + B * Hkv) * d * d * 4
 * budget may not exceed 2^30.
 * A wait of the fold's that gives up is reported as INFINI_ERR_TIMEOUT by
 * infini_attn_device_status.  The rows are selected and copied all the same, and the pages of
 * page_table still hold the others.  M then has the complete sums of some heads (folded by one block
 * alone) and is as it was for all others; z is as it was.  Fold again from copies of M and z.  Until
 * the record is read, later calls fold nothing: they select and copy, and leave M and z.
 */
INFINI_API int infini_attn_paged_evict(void *k_pages, void *v_pages, float *weights,
                                       const int32_t *page_table, const int32_t *lens,
                                       const int32_t *dst_table, int32_t *lens_out, int32_t *kept,
                                       float *M, float *z, void *workspace, int64_t workspace_bytes,
                                       int64_t B, int64_t Hkv, int64_t d, int64_t P, int64_t page,
                                       int64_t max_pages, int64_t dst_pages, int64_t budget,
                                       int64_t recent, int update_rule, infini_stream_t stream);
INFINI_API int infini_attn_paged_evict_f32(void *k_pages, void *v_pages, float *weights,
                                           const int32_t *page_table, const int32_t *lens,
                                           const int32_t *dst_table, int32_t *lens_out,
                                           int32_t *kept, float *M, float *z, void *workspace,
                                           int64_t workspace_bytes, int64_t B, int64_t Hkv,
                                           int64_t d, int64_t P, int64_t page, int64_t max_pages,
                                           int64_t dst_pages, int64_t budget, int64_t recent,
                                           int update_rule, infini_stream_t stream);
INFINI_API int64_t infini_attn_paged_evict_workspace_bytes(int64_t B, int64_t Hkv, int64_t d,
                                                           int64_t page, int64_t max_pages,
                                                           int64_t budget, int with_memory);

/*
 * Allocation-free variant of infini_attn_fwd (bf16 activations); same parameters, same
 * results.  The pages have no counterpart to this entry point: it exists for callers that
 * may not allocate device memory while they run, for example a serving loop whose device
 * memory is planned and handed out by its own allocator up front (a stream-ordered
 * allocation there could fail when that allocator holds nearly all of HBM, or stall the
 * loop while the driver's pool grows), or a host program that gives plugins buffers but
 * no allocation rights.  This call makes no cudaMalloc / cudaFree / cudaMallocAsync /
 * cudaFreeAsync call and calls no allocating library routine.
 *
 *   - Its workspace is a fixed device array of INFINI_NOALLOC_SCRATCH_BYTES inside the
 *     library; every GPU that loads the library holds that array until the process exits.
 *     A problem whose workspace exceeds it is rejected with INFINI_ERR_UNSUPPORTED, before
 *     anything is launched.  The size that counts is what the kernels chosen for the
 *     problem need: infini_attn_workspace_bytes is an upper bound over all of them, and the
 *     fused 64-token paths need much less.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call before any
 *     stream capture begins.
 *   - All calls on a device share that device's one array, which keeps the last call's
 *     contents.  Calls on the same device that overlap on the GPU (issued on different
 *     streams or from different host threads without ordering between them) race and
 *     corrupt each other's results: order them on one stream or with events.  Calls on
 *     different devices do not interfere.  Nothing in the array has to start at zero: each
 *     call writes every workspace byte it reads before reading it.
 */
#define INFINI_NOALLOC_SCRATCH_BYTES (16ull << 20)
INFINI_API int infini_attn_fwd_noalloc(const void *q, const void *k, const void *v,
                                       const float *beta, const float *M0, const float *z0,
                                       void *out, float *M_out, float *z_out, int64_t B,
                                       int64_t H, int64_t Hkv, int64_t L, int64_t N, int64_t d,
                                       int update_rule, infini_stream_t stream);

/* Bytes of workspace one call allocates for these sizes (an upper bound over the kernels
 * the call may choose; 0 on invalid sizes). */
INFINI_API int64_t infini_attn_workspace_bytes(int64_t B, int64_t Hkv, int64_t L, int64_t N, int64_t d);

/*
 * Synchronises `stream`, then reports whether a bounded wait inside a kernel of this
 * library gave up since the last check: INFINI_ERR_TIMEOUT (and the record is cleared),
 * INFINI_OK, or INFINI_ERR_CUDA if the synchronisation itself failed.  A kernel whose wait
 * gave up stops early and leaves part of its outputs unwritten.  The record is sticky:
 * until it is read here, later launches of the waiting kernels return without work.
 * INFINI_ERR_PAGE if instead a paged entry met a page number or row outside its cache since the
 * last check (cleared too; later launches are not affected).  Where both happened, the timeout is
 * reported first and the other record by the next call.
 */
INFINI_API int infini_attn_device_status(infini_stream_t stream);

/* Static, NUL-terminated description of a status code. */
INFINI_API const char *infini_attn_status_string(int status);

/* Library version: major * 10000 + minor * 100 + patch. */
INFINI_API int infini_attn_version(void);

/*
 * Launch tracing (off by default).  While enabled, every kernel this library enqueues is
 * bracketed by two CUDA events recorded on the call's stream.  infini_attn_trace_enable(1)
 * starts a new trace (clearing the previous one); it returns the previous setting.
 * infini_attn_trace_report synchronises on the recorded events, adds them to a per-kernel
 * table and writes it as JSON, {"<kernel>": {"launches": n, "ms": total}, ...}
 * (NUL-terminated, truncated to len - 1 bytes; buf may be NULL), and returns the size
 * the full report needs.  Reporting does not clear the table.
 */
INFINI_API int infini_attn_trace_enable(int on);
INFINI_API int64_t infini_attn_trace_report(char *buf, int64_t len);

/*
 * Test hooks: they let the library's failure paths be exercised without a real failure.
 * None of them is needed for normal use, and all are off by default.
 *
 * infini_attn_test_fail_allocations(n): the next n workspace allocations of this process
 *   fail as an exhausted device would make them fail: the calls return INFINI_ERR_OOM before
 *   anything is launched or written.  n = 0 turns the hook off.  INFINI_ERR_INVALID_ARG if
 *   n < 0.
 * infini_attn_test_wait_limit(cycles): the bound every device wait of the current device
 *   applies, in SM clock cycles (default about 0.5 s at the top clock; cycles <= 0 restores
 *   it).  A wait that reaches it gives up as described for infini_attn_device_status.
 * infini_attn_test_withhold_publish(on): on the current device, the first unit of every head
 *   in the fused 64-token kernel (additive rule, d = 64, N = 64, at most 64 units of 128
 *   tokens per head) skips publishing its memory aggregate, so the later units'
 *   waits for it run out: the call's outputs are then incomplete and
 *   infini_attn_device_status reports INFINI_ERR_TIMEOUT.  Nothing traps or hangs.  In
 *   infini_attn_paged_evict's fold the first warp of every block that loads rows loads none, with
 *   the same end.
 * The last two copy to device variables synchronously (INFINI_ERR_CUDA if that fails); use
 * them while no call of this library is running on the device.
 */
INFINI_API int infini_attn_test_fail_allocations(int n);
INFINI_API int infini_attn_test_wait_limit(int64_t cycles);
INFINI_API int infini_attn_test_withhold_publish(int on);

#ifdef __cplusplus
}
#endif

#endif /* INFINI_ATTN_H */
