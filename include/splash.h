/*
 * splash.h -- C ABI of the GB300 (sm_103a) block-sparse masked attention
 * library (libsplash.so).
 *
 * The operation is the forward pass of "Splash" attention: a mask made of a
 * causal part, a local window and document segment IDs, joined by AND, is
 * preprocessed into a sparse execution table (MaskInfo), and an attention
 * kernel walks only the non-empty key/value blocks of each query block with an
 * online softmax, writing O and the per-row log-sum-exp.
 *
 * Sources:
 *   "Pallas Kernels and Splash Attention" (CMU 11-868 Lecture 13 notes):
 *     §5.1 online softmax; §5.2 the Flash kernel body (m, l, o accumulators,
 *     alpha rescale, deferred normalisation), MHA/GQA; §5.4 soft cap;
 *     §6.1 empty / partial / full blocks; §6.2 MaskInfo (block_mask,
 *     partial_mask_blocks, mask_next, bounds_start / bounds_end); §6.3 the
 *     Splash grid over active blocks and the residual LSE; §6.4 segment IDs
 *     and masks joined by AND.
 *   "The maths and infra behind core LLM operations" (joto.ai): sections
 *     "Causal Mask" (skip blocks above the diagonal, mask only the diagonal
 *     ones) and "LSE and Online Softmax" (LSE = m + log l).
 *
 * Conventions that hold for every call:
 *   - All tensors are caller-owned.  Pointers documented as "device" must be
 *     device memory of the current CUDA device; "host" pointers are ordinary
 *     host memory.  Nothing is retained after a call returns except inside a
 *     splash_mask_info handle.
 *   - `cuda_stream` is a cudaStream_t (NULL = the legacy default stream).
 *     Kernels are launched asynchronously on it.
 *   - No call throws, exits or traps.  Invalid arguments are detected on the
 *     host before any launch and reported as a status; the output buffers are
 *     then untouched.
 *   - Tensor layouts are dense row-major (contiguous), innermost dimension
 *     last.
 */
#ifndef SPLASH_H
#define SPLASH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SPLASH_OK = 0,
    SPLASH_ERR_INVALID_ARG = 1,    /* NULL pointer, negative size, bad flag */
    SPLASH_ERR_SHAPE = 2,          /* sizes inconsistent with each other or with the MaskInfo */
    SPLASH_ERR_UNSUPPORTED = 3,    /* valid, but outside what this build implements */
    SPLASH_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
    SPLASH_ERR_DEVICE_TIMEOUT = 5, /* a kernel's bounded wait ran out (see splash_last_device_error) */
    SPLASH_ERR_OOM = 6,            /* device allocation failed */
    SPLASH_ERR_DEVICE_CHECK = 7    /* a kernel's bounds check rejected table contents */
} splash_status;

/*
 * The joint mask (AND of the enabled parts), "Pallas Kernels and Splash
 * Attention" §6.1 and §6.4.  Query position i and key position j are 0-based
 * within their sequence; for batch row b the pair is allowed when
 *     (!causal || j <= i)
 *  && (window_left  < 0 || i - j <= window_left)
 *  && (window_right < 0 || j - i <= window_right)
 *  && (q_segment_ids == NULL || q_segment_ids[b][i] == kv_segment_ids[b][j]).
 * A window of W keys including the query itself is window_left = W - 1.
 */
typedef struct {
    int32_t causal;                 /* 0 or 1 */
    int64_t window_left;            /* inclusive distance to the left; -1 = unbounded */
    int64_t window_right;           /* inclusive distance to the right; -1 = unbounded */
    const int32_t *q_segment_ids;   /* device int32 [batch][Lq], or NULL for no document mask */
    const int32_t *kv_segment_ids;  /* device int32 [batch][Lk]; NULL means "same as q_segment_ids"
                                       (then Lq must equal Lk) */
    int32_t batch;                  /* rows of the segment arrays; ignored when q_segment_ids is NULL */
} splash_mask_spec;

/* Opaque, library-owned MaskInfo; freed by splash_mask_info_destroy. */
typedef struct splash_mask_info splash_mask_info;

/*
 * splash_build_mask_info -- preprocess a mask into the sparse execution table
 * ("Pallas Kernels and Splash Attention" §6.2, §6.3, §6.6).
 *
 * Every (bq x bk) block of the [Lq, Lk] mask is classified as empty (0),
 * partial (1) or full (2) (block_mask).  Active (non-empty) blocks are listed
 * in row-major order (q-block ascending, then kv-block ascending) as
 * active_rows / active_cols, with row_ptr giving each q-block row's range
 * (CSR) and bounds_start / bounds_end flagging the first / last active block
 * of a row.  Each partial block's bq x bk element pattern (1 = allowed) is
 * deduplicated by exact content in first-occurrence order into
 * partial_mask_blocks; mask_next[g] is the pattern index of active block g, or
 * -1 when the block is full.
 *
 * With segment IDs the table has B_mask = spec->batch batch rows (one per
 * segment-array row); without them B_mask = 1 and it serves every batch row
 * and head.  Rows are then ordered (b_mask, q-block).
 *
 *   spec        host pointer to the mask; its segment arrays are device memory
 *               and are read on `cuda_stream` before this call returns.
 *   Lq, Lk      sequence lengths (> 0).  When one is not a multiple of its
 *               block, the grid is padded to nq = ceil(Lq/bq) by
 *               nk = ceil(Lk/bk) whole blocks and the padding positions are
 *               masked (§2.3: ragged edges are padded so that every block has
 *               the same size); a block holding padding is never full.
 *   bq, bk      block sizes; this build supports bk in {64, 128} and
 *               bq in {64, 128, 256} (the worked example of "Pallas Kernels
 *               and Splash Attention" §6.2 already uses bq != bk).
 *   cuda_stream stream for the build kernels.
 *   out         receives a new handle (set to NULL on error).
 *
 * Synchronisation: the build kernels are queued on `cuda_stream` and the
 * call returns without waiting, in the usual case: the pattern buffer is
 * sized from a bound known before the build (band-only masks: at most
 * 2 * (ceil((bq-1)/bk) + 1) partial blocks per q-block row, plus one block per
 * row and the last row on a ragged grid; with segment IDs: the number of
 * blocks the causal / window part alone leaves non-empty, since segments only
 * remove pairs).  Only when that bound's bit-packed patterns would exceed
 * 256 MB does the call wait once on `cuda_stream` for the exact pattern
 * count; that path is not capturable in a CUDA graph.  The table may be used
 * by later work on `cuda_stream` at once (work on another stream must wait
 * for it); the totals reach the host only when splash_mask_info_counts or
 * splash_mask_info_to_host asks for them.  A first build allocates the
 * table's device memory (cudaMalloc, which synchronises the device); a
 * rebuild into a handle whose buffers are large enough can then be captured
 * into a CUDA graph on `cuda_stream` (with the attention calls that use it);
 * after a replay, synchronise the stream before asking for the totals.
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA, OOM; *out is NULL then.
 */
splash_status splash_build_mask_info(const splash_mask_spec *spec, int64_t Lq, int64_t Lk,
                                     int32_t bq, int32_t bk, void *cuda_stream,
                                     splash_mask_info **out);

/*
 * splash_mask_info_rebuild -- the same computation as splash_build_mask_info,
 * written into an existing handle whose buffers are reused when they are large
 * enough (no device allocation then).  The handle's previous contents are
 * replaced; on error the handle is left empty but valid (destroy it or rebuild
 * it).  Same synchronisation as splash_build_mask_info.
 */
splash_status splash_mask_info_rebuild(splash_mask_info *mi, const splash_mask_spec *spec,
                                       int64_t Lq, int64_t Lk, int32_t bq, int32_t bk,
                                       void *cuda_stream);

/*
 * splash_mask_info_shape -- host-side read of the table's geometry.
 *   batch_rows = B_mask, nq = Lq/bq, nk = Lk/bk.  Any output may be NULL.
 */
splash_status splash_mask_info_shape(const splash_mask_info *mi, int32_t *batch_rows, int64_t *nq,
                                     int64_t *nk, int32_t *bq, int32_t *bk);

/*
 * splash_mask_info_counts -- totals of the table:
 *   num_active    active blocks A (over all batch rows),
 *   num_partial   partial blocks,
 *   num_patterns  distinct partial patterns P,
 *   allowed_pairs allowed (query, key) pairs summed over the batch rows (the
 *                 "useful" entries of the score matrix).  This output is an
 *                 extension of the table the pages describe: the FLOP counts
 *                 of the benchmark are taken from it.
 * After an asynchronous build the first call waits for the build's kernels
 * and copies the totals from the device (later calls read the host copy).
 * Any output may be NULL.
 */
splash_status splash_mask_info_counts(const splash_mask_info *mi, int64_t *num_active,
                                      int64_t *num_partial, int64_t *num_patterns,
                                      int64_t *allowed_pairs);

/*
 * splash_mask_info_to_host -- copy the table into caller-allocated HOST arrays
 * (synchronous).  Sizes: block_mask [B_mask*nq*nk], row_ptr [B_mask*nq + 1],
 * active_rows / active_cols / mask_next / bounds_start / bounds_end [A],
 * partial_mask_blocks [P*bq*bk] (one byte per element, 1 = allowed; the
 * device keeps the patterns bit-packed and they are expanded here).  Any
 * pointer may be NULL to skip that array.
 */
splash_status splash_mask_info_to_host(const splash_mask_info *mi, int8_t *block_mask,
                                       int32_t *row_ptr, int32_t *active_rows,
                                       int32_t *active_cols, int32_t *mask_next,
                                       uint8_t *bounds_start, uint8_t *bounds_end,
                                       uint8_t *partial_mask_blocks);

/*
 * splash_mask_info_set_pattern_source -- where the attention forward takes the
 * element masks of partial blocks from:
 *   SPLASH_PATTERNS_STORED (default): the deduplicated partial_mask_blocks;
 *   SPLASH_PATTERNS_FROM_POSITIONS: computed in the kernel from the query and
 *     key positions (causal / window bounds and ragged-length padding) and,
 *     for a table built with segment IDs, from the segment arrays, the
 *     alternative of "Pallas Kernels and Splash Attention" §6.6 (no pattern
 *     reads; the results are identical).  With segment IDs every forward
 *     call (splash_attention_fwd, _fwd_mle, _fwd_split, _fwd_host) must pass
 *     the arrays the table was built from (same values; device memory, read
 *     by the kernel); a NULL q_segment_ids there returns INVALID_ARG.
 * The setting stays with the handle across rebuilds.  The backward always
 * reads the stored patterns.  Errors: INVALID_ARG (NULL handle, unknown
 * source).
 */
#define SPLASH_PATTERNS_STORED 0
#define SPLASH_PATTERNS_FROM_POSITIONS 1
splash_status splash_mask_info_set_pattern_source(splash_mask_info *mi, int32_t source);

/* Frees the handle and its device memory (NULL is a no-op).  Work queued on
 * other streams that still reads the table must be complete first. */
void splash_mask_info_destroy(splash_mask_info *mi);

/*
 * splash_attention_fwd -- block-sparse masked attention forward
 * ("Pallas Kernels and Splash Attention" §5.1-§5.4, §6.3).
 *
 * For every batch b, query head h and query i, with kv head g = h / (Hq/Hkv):
 *   s_j  = scale * q[b,h,i,:] . k[b,g,j,:]              (fp32 accumulation)
 *   s_j  = softcap * tanh(s_j / softcap)                 (only if softcap > 0)
 *   over the keys j allowed by the MaskInfo's mask:
 *   out[b,h,i,:] = sum_j exp(s_j - m) v[b,g,j,:] / sum_j exp(s_j - m)
 *   lse[b,h,i]   = m + ln(sum_j exp(s_j - m))            (natural log)
 * Rows with no allowed key get out = 0 and lse = -inf.  Only the MaskInfo's
 * active blocks are loaded or computed; partial blocks are masked element by
 * element from partial_mask_blocks (or from positions and segment IDs, see
 * splash_mask_info_set_pattern_source).
 *
 *   q    device bf16 [B][Hq][Lq][dqk]      k  device bf16 [B][Hkv][Lk][dqk]
 *   v    device bf16 [B][Hkv][Lk][dv]      (all 16-byte aligned)
 *   q_segment_ids, kv_segment_ids  the device arrays the MaskInfo was built
 *        from, or NULL.  Read only when the table has segment IDs and its
 *        pattern source is SPLASH_PATTERNS_FROM_POSITIONS (then q_segment_ids
 *        is required; kv_segment_ids NULL means q_segment_ids); the stored
 *        patterns already encode them otherwise.
 *   mi   a MaskInfo built for (Lq, Lk) with B_mask == 1 or B_mask == B.
 *   scale  multiplies q.k (e.g. 1/sqrt(dqk)); must be positive and finite.
 *   softcap <= 0 disables the cap (NaN or +inf is rejected).
 *   out  device bf16 [B][Hq][Lq][dv]       lse device fp32 [B][Hq][Lq]
 *
 * Supported in this build: (dqk, dv) in {(64, 64), (128, 128), (192, 128)},
 * Hq % Hkv == 0, and the MaskInfo's blocks bq == bk in {64, 128} (bk = 128
 * for dqk = 192), or bq = 256 with bk = 128.  The kernel computes in query
 * tiles of 128 rows, two per work item: with bq <= 128 the two tiles are
 * two query heads of one q-block (sharing K / V within a GQA group), with
 * bq = 256 they are the two halves of one q-block of one head and share
 * every K / V tile (this halves the K / V traffic of MHA; blocks of the
 * union that are masked for one half are computed and contribute nothing).
 * Other valid shapes return SPLASH_ERR_UNSUPPORTED.
 * Errors are returned before any launch; kernel-side bounded waits and table
 * checks are reported by splash_last_device_error.
 */
splash_status splash_attention_fwd(const void *q, const void *k, const void *v, int32_t B,
                                   int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk,
                                   int32_t dv, const int32_t *q_segment_ids,
                                   const int32_t *kv_segment_ids, const splash_mask_info *mi,
                                   float scale, float softcap, void *out, float *lse,
                                   void *cuda_stream);

/*
 * splash_attention_fwd_mle -- the same forward with the Max Logit Estimate
 * ("Pallas Kernels and Splash Attention" §5.4): every row's softmax reference
 * is the constant max_logit (natural-log units, the same units as s_j after
 * scale and soft cap) instead of a running maximum, so no block maximum is
 * taken and the accumulator is never rescaled (alpha = 1):
 *   out = sum_j exp(s_j - c) v_j / sum_j exp(s_j - c),  lse = c + ln sum_j exp(s_j - c)
 * which equals splash_attention_fwd's result (c cancels) while c is in the
 * safe range of §5.4 / exercise 10: with a soft cap, c = softcap always is.
 * Outside it:
 *   - a block whose sum of exponentials (base 2, fp32) would reach 2^64
 *     (scores some 40 or more above c) moves that row's reference to the
 *     block's maximum (the overflow guard of the plain kernel), so too small a
 *     c costs time, not accuracy;
 *   - a row whose scores all lie more than about 87 below c underflows: its
 *     sum flushes to 0 and it gets out = 0, lse = -inf, like a fully masked
 *     row (the underflow the lecture warns about; not detected).
 *   max_logit  finite (else SPLASH_ERR_INVALID_ARG)
 * Other arguments, supported shapes and errors as for splash_attention_fwd.
 */
splash_status splash_attention_fwd_mle(const void *q, const void *k, const void *v, int32_t B,
                                       int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk,
                                       int32_t dv, const int32_t *q_segment_ids,
                                       const int32_t *kv_segment_ids, const splash_mask_info *mi,
                                       float scale, float softcap, float max_logit, void *out,
                                       float *lse, void *cuda_stream);

/*
 * splash_attention_fwd_host -- splash_attention_fwd for tensors in host
 * memory: copies q, k, v to the caller's device buffers, runs the forward and
 * copies out and lse back, overlapping the three.  The work is cut into
 * contiguous chunks (whole GQA groups of one batch row when the MaskInfo is
 * shared by the batch; the whole batch at once for a per-batch table) and
 * pipelined on library-owned streams: host -> device copies of one chunk,
 * the attention of the previous one and device -> host copies of the one
 * before run at the same time.  Ordered after prior work on cuda_stream;
 * work queued on cuda_stream afterwards waits for the last copy back.
 *
 *   q_host, k_host, v_host   host bf16, layouts as splash_attention_fwd
 *   out_host, lse_host       host bf16 [B][Hq][Lq][dv] and fp32 [B][Hq][Lq]
 *   q_dev .. lse_dev         device buffers of the full sizes (caller-owned,
 *                            overwritten; alignment as splash_attention_fwd)
 * Host buffers should be page-locked (cudaHostAlloc / cudaHostRegister):
 * copies from pageable memory are correct but do not overlap.  Other
 * arguments, supported shapes and errors as for splash_attention_fwd.
 */
splash_status splash_attention_fwd_host(const void *q_host, const void *k_host, const void *v_host,
                                        int32_t B, int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk,
                                        int32_t dqk, int32_t dv, const int32_t *q_segment_ids,
                                        const int32_t *kv_segment_ids, const splash_mask_info *mi,
                                        float scale, float softcap, void *out_host, float *lse_host,
                                        void *q_dev, void *k_dev, void *v_dev, void *out_dev,
                                        float *lse_dev, void *cuda_stream);

/* Largest num_splits accepted by the split-KV entry points. */
#define SPLASH_MAX_SPLITS 256

/*
 * splash_attention_fwd_split -- the same forward with each q-block row's
 * active list cut into num_splits consecutive ranges ("split-KV"), each a
 * separate work item, so that rows with many active blocks and few rows in
 * total (long keys, few queries) still fill the GPU.  For split s (blocks
 * [nb*s/num_splits, nb*(s+1)/num_splits) of a row with nb active blocks), with
 * J_s its allowed keys and R = B*Hq*Lq:
 *   o_part[s][b][h][i][:]  = sum_{j in J_s} exp(s_j - lse_s) v[b,g,j,:]   (fp32)
 *   lse_part[s][b][h][i]   = ln sum_{j in J_s} exp(s_j)
 * with o_part = 0 and lse_part = -inf where J_s is empty.  splash_attention_merge
 * turns them into out / lse equal to splash_attention_fwd's: this is the merge
 * of softmax segments through their log-sum-exp ("The maths and infra behind
 * core LLM operations" (joto.ai), "LSE and Online Softmax"; "Pallas Kernels
 * and Splash Attention" §5.1).
 *
 *   num_splits  1 .. SPLASH_MAX_SPLITS (splits beyond a row's block count are
 *               empty)
 *   o_part      device fp32 [num_splits][B][Hq][Lq][dv], 32-byte aligned
 *   lse_part    device fp32 [num_splits][B][Hq][Lq]
 * Both are caller-owned workspace, fully overwritten.  Other arguments,
 * supported shapes and errors as for splash_attention_fwd.
 */
splash_status splash_attention_fwd_split(const void *q, const void *k, const void *v, int32_t B,
                                         int32_t Hq, int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk,
                                         int32_t dv, const int32_t *q_segment_ids,
                                         const int32_t *kv_segment_ids, const splash_mask_info *mi,
                                         float scale, float softcap, int32_t num_splits, float *o_part,
                                         float *lse_part, void *cuda_stream);

/*
 * splash_attention_merge -- combines split-KV partials (layout above, rows =
 * B*Hq*Lq):  m = max_s lse_part[s][r];  lse[r] = m + ln sum_s exp(lse_part[s][r] - m);
 * out[r][:] = sum_s exp(lse_part[s][r] - lse[r]) o_part[s][r][:]  (bf16);
 * rows whose splits are all empty get out = 0, lse = -inf.
 *   o_part  device fp32, 16-byte aligned     lse_part  device fp32
 *   dv      64 or 128 (else SPLASH_ERR_UNSUPPORTED)
 *   out     device bf16 [rows][dv], 16-byte aligned    lse  device fp32 [rows]
 */
splash_status splash_attention_merge(const float *o_part, const float *lse_part, int32_t num_splits,
                                     int64_t rows, int32_t dv, void *out, float *lse, void *cuda_stream);

/*
 * splash_attention_bwd -- gradients of splash_attention_fwd with respect to
 * q, k and v for an upstream gradient dout, from the forward's out and lse
 * ("Pallas Kernels and Splash Attention" §6.3: the forward's residual outputs
 * serve the backward; "The maths and infra behind core LLM operations"
 * (joto.ai), "LSE and Online Softmax": the probabilities are recomputed from
 * the scores and LSE, P_ij = exp(s_ij - lse_i), instead of being stored).
 * With dP_ij = dout_i . v_j, D_i = dout_i . out_i and
 *   dS_ij = P_ij (dP_ij - D_i)  (times 1 - tanh^2(scale q.k / softcap) with a cap):
 *   dv[b,g,j,:] = sum over heads h of group g, allowed i: P_ij dout[b,h,i,:]
 *   dk[b,g,j,:] = scale * sum over h, i: dS_ij q[b,h,i,:]
 *   dq[b,h,i,:] = scale * sum over allowed j: dS_ij k[b,g,j,:]
 * (masked pairs contribute nothing; a key no query sees gets dk = dv = 0).
 * Only the MaskInfo's active blocks are computed, visited column by column:
 * the first call after each build (or rebuild) of the MaskInfo makes a
 * column-major copy of the table inside it (device memory allocated on
 * first use, hence the non-const handle), and later calls reuse it; a call
 * on another stream waits for the copy's completion.
 *
 *   q, k, v, mi, scale, softcap   exactly as given to the forward
 *   out  device bf16 [B][Hq][Lq][dv], lse device fp32 [B][Hq][Lq]: the forward's outputs
 *   dout device bf16 [B][Hq][Lq][dv]
 *   dq   device bf16 [B][Hq][Lq][dqk]   dk device bf16 [B][Hkv][Lk][dqk]
 *   dv_out device bf16 [B][Hkv][Lk][dv]   (all fully overwritten)
 *   workspace  device, 16-byte aligned, at least
 *              splash_attention_bwd_workspace_size(B, Hq, Lq, dqk) bytes
 *              (an fp32 dq accumulator, D and a copy of lse, over whole
 *              256-row blocks per head); caller-owned, overwritten.
 * All device pointers 16-byte aligned.  Supported: dqk == dv in {64, 128}
 * and MaskInfo blocks bk = 128 with bq = 128 or 256 (a 256-row q-block is
 * taken as two 128-row halves), any Lq / Lk (ragged lengths as in the
 * forward); other valid shapes return SPLASH_ERR_UNSUPPORTED.  dq is accumulated with fp32 atomic additions, so
 * its last bits may differ between runs; dk and dv are deterministic.
 * Errors as for splash_attention_fwd.
 */
splash_status splash_attention_bwd_workspace_size(int32_t B, int32_t Hq, int64_t Lq, int32_t dqk,
                                                  size_t *bytes);
splash_status splash_attention_bwd(const void *q, const void *k, const void *v, const void *out,
                                   const float *lse, const void *dout, int32_t B, int32_t Hq,
                                   int32_t Hkv, int64_t Lq, int64_t Lk, int32_t dqk, int32_t dv,
                                   const int32_t *q_segment_ids, const int32_t *kv_segment_ids,
                                   splash_mask_info *mi, float scale, float softcap, void *dq,
                                   void *dk, void *dv_out, void *workspace, size_t workspace_bytes,
                                   void *cuda_stream);

/*
 * ---------------------------------------------------------------------------
 * Serving: rotary positions, a paged key/value cache, attention of new tokens
 * ---------------------------------------------------------------------------
 * The calls above work on contiguous keys.  The three below surround them: q
 * and k are rotated by position before the forward (splash_rope; its inverse
 * turns the gradients back after the backward), keys and values of served
 * sequences are kept in pages (splash_paged_append), and new tokens attend to
 * the pages (splash_paged_decode).  Their arguments come in one struct each;
 * struct_bytes is sizeof the struct, so that a caller compiled against
 * another layout is refused (INVALID_ARG).
 *
 * All three only queue kernels on cuda_stream and can be captured into a CUDA
 * graph; what lives in device memory (positions, lengths, the block table)
 * may change between replays.  Indices read on the device are checked there:
 * one out of range touches no memory outside the tensors and is reported by
 * splash_last_device_error as SPLASH_ERR_DEVICE_CHECK.
 */

/* A bf16 tensor [B][H][L][d]: d contiguous, the other strides in elements
 * (multiples of 8, so that every row starts on 16 bytes; ptr 16-byte aligned).
 * The stride of a dimension of size 1 is not read.  Inputs may repeat rows
 * (stride 0); outputs may not overlap themselves. */
typedef struct {
    void *ptr;
    int64_t stride_b, stride_h, stride_l;
} splash_view;

/* A cache tensor [num_pages][Hkv][page_size][d]: d contiguous, strides in
 * elements, rows and ptr 16-byte aligned.  Pages stored token by token
 * ([num_pages][page_size][Hkv][d]) are this tensor with the strides of the
 * head and the token exchanged. */
typedef struct {
    void *ptr;
    int64_t stride_page, stride_head, stride_token;
} splash_cache_view;

#define SPLASH_CACHE_BF16 0
#define SPLASH_CACHE_E4M3 1 /* stores x / scale[kv head], rounded to nearest even, saturated at +-448 */

/*
 * splash_rope -- rotary positions.  For a token at position p and every pair
 * (a, b) of its row's rotated dimensions, with c = table[p][i] and
 * s = table[p][rot_dim/2 + i] for pair i:
 *   forward (inverse = 0):  a' = a c - b s,   b' = b c + a s
 *   gradient (inverse = 1): a' = a c + b s,   b' = b c - a s
 * (the rotation is linear, so its gradient is the transposed rotation).  The
 * rotated dimensions are [rot_offset, rot_offset + rot_dim); pair i is
 * (i, i + rot_dim/2) of them, or (2i, 2i + 1) when interleaved.  The others
 * are copied.  Computed in fp32, rounded once.
 *
 *   q, q_out, k, k_out  views with Hq / Hkv heads; k.ptr NULL = no k.  An
 *               output is the input's own view (in place) or does not
 *               overlap any input.
 *   positions   device int32, [b][l] at positions[b * positions_stride_b + l]
 *               (stride 0: the same for every b).  A negative position is the
 *               identity (padding); one >= table_rows also, and is reported.
 *   table       device fp32 [table_rows][rot_dim], cosines then sines,
 *               16-byte aligned
 *   d           multiple of 16, <= 512;  rot_dim a positive multiple of 16;
 *               rot_offset a multiple of 8; rot_offset + rot_dim <= d
 * Errors: INVALID_ARG (NULL, alignment, strides, flags), SHAPE (rotated
 * dimensions outside d), UNSUPPORTED (sizes), CUDA.
 */
typedef struct {
    uint64_t struct_bytes;
    splash_view q, q_out, k, k_out;
    const int32_t *positions;
    int64_t positions_stride_b;
    const float *table;
    int64_t table_rows;
    int64_t L;
    int32_t B, Hq, Hkv, d;
    int32_t rot_dim, rot_offset, interleaved, inverse;
} splash_rope_args;
splash_status splash_rope(const splash_rope_args *args, void *cuda_stream);

/*
 * splash_paged_append -- writes the keys and values of new tokens into a paged
 * cache, rotating them on the way.  Token (b, l) of sequence
 * s = seq_ids ? seq_ids[b][l] : b at position p = positions[b][l] goes to page
 * block_table[s][p / page_size], row p % page_size:
 *   k_cache[page][h][row] = rotated k[b][h][l]    v_cache[...] = v[b][h][l]
 * (divided by k_scale[h] / v_scale[h] and rounded to e4m3 in an 8-bit cache;
 * the rotated key is rounded once, from fp32).  Optionally also
 *   q_out = rotated q        (q.ptr not NULL)
 *   k_out = rotated k, bf16  (k_out.ptr not NULL: for splash_attention_fwd)
 * With table NULL nothing is rotated.  Nothing else in the cache is written.
 *
 * A token with a negative position is padding: no cache row is written, its
 * q_out / k_out rows are copies of q / k.  A position outside the table of
 * rotations or the block table's row, a page outside [0, num_pages) or a
 * sequence outside [0, num_seqs) is reported and treated the same way (q_out
 * and k_out are rotated where the position has a rotation).  Two tokens of
 * one call must not share a cache row; if they do, each of its elements is
 * one of the two.
 *
 *   seq_ids     device int32 [b][l] (stride as positions) or NULL: b.  This
 *               is how a row of packed documents is appended.
 *   block_table device int32 [num_seqs][max_pages], row stride
 *               block_table_stride; entries of pages not written are not read
 *   page_size   a power of two, 16 .. 1024; max_pages * page_size < 2^31 - 65535
 *   dqk, dv     multiples of 16, <= 512
 *   k_scale, v_scale  device fp32 [Hkv], both required for e4m3, else ignored
 * The rotation's arguments and the errors are as for splash_rope.
 */
typedef struct {
    uint64_t struct_bytes;
    splash_view q, q_out, k, k_out, v;
    splash_cache_view k_cache, v_cache;
    const float *k_scale, *v_scale;
    const int32_t *block_table;
    int64_t block_table_stride;
    const int32_t *positions;
    int64_t positions_stride_b;
    const int32_t *seq_ids;
    int64_t seq_ids_stride_b;
    const float *table;
    int64_t table_rows;
    int64_t L, num_pages;
    int32_t B, Hq, Hkv, dqk, dv;
    int32_t num_seqs, max_pages, page_size, cache_type;
    int32_t rot_dim, rot_offset, interleaved;
} splash_paged_append_args;
splash_status splash_paged_append(const splash_paged_append_args *args, void *cuda_stream);

/* Most new tokens per sequence in one splash_paged_decode call. */
#define SPLASH_MAX_NEW_TOKENS 16

/*
 * splash_paged_decode -- attention of each sequence's newest Lq tokens over
 * its paged cache (which already holds their keys).  Sequence b has
 * n = seq_lens[b] cached tokens; its query l sits at position p = n - Lq + l
 * and sees the keys j <= p, and with window_left >= 0 only those with
 * p - j <= window_left.  For query head h and g = h / (Hq/Hkv):
 *   s_j = scale * q[b,h,l,:] . k[j,:]   (times k_scale[g] for e4m3; capped as
 *         in splash_attention_fwd when softcap > 0)
 *   out[b,h,l,:] = sum_j exp(s_j - lse) v[j,:]   (times v_scale[g] for e4m3)
 *   lse[b,h,l]   = ln sum_j exp(s_j)
 * A query that sees no key (n = 0, or p < 0) gets out = 0 and lse = -inf.
 * This equals splash_attention_fwd over the gathered keys with the mask
 * causal from the sequence's end.  Cache rows that no query sees (past n, or
 * before the window) are not read, nor are the block table's entries for
 * them, so they may hold anything; rows that only some of the queries see do
 * not reach the others, whatever they hold.
 *
 * A negative n counts as 0 and one above max_pages * page_size as that; a page
 * outside [0, num_pages) reads as keys and values of zero; each is reported.
 *
 *   q           view [B][Hq][Lq][dqk]
 *   out         device bf16 [B][Hq][Lq][dv] dense, 16-byte aligned
 *   lse         device fp32 [B][Hq][Lq]
 *   workspace   device, 16-byte aligned, at least
 *               splash_paged_decode_workspace_size bytes for the same sizes;
 *               overwritten, holds nothing between calls.  Two calls that may
 *               run at the same time need two workspaces.
 * Supported: (dqk, dv) in {(64, 64), (128, 128), (192, 128)}, Hq % Hkv == 0,
 * 1 <= Lq <= SPLASH_MAX_NEW_TOKENS, page_size a power of two in 16 .. 1024,
 * max_pages * page_size < 2^31 - 65535, B <= 65535, and fewer than 2^31 steps of
 * 16 keys (at most max_pages * page_size / 16 + 1, or window_left / 16 + 4) over
 * all sequences, KV heads and groups of 16 of the Hq/Hkv * Lq rows.  The result
 * does not depend on timing: the same inputs give the same bits on the same GPU.
 * The cache is read once for every 32 of the Hq/Hkv * Lq rows.
 *
 * Precision: scores, softmax statistics and sums are fp32, out is rounded once.
 * The product with the values takes each probability to 2^-16 of it for a bf16
 * cache; for an e4m3 one to 2^-11, or 2^-22 with at most 8 of the Hq/Hkv * Lq
 * rows, and those below 2^-32 of the largest count in lse but not in out (below
 * out's own rounding up to 2^23 such keys).
 */
typedef struct {
    uint64_t struct_bytes;
    splash_view q;
    splash_cache_view k_cache, v_cache;
    const float *k_scale, *v_scale;
    const int32_t *block_table;
    int64_t block_table_stride;
    const int32_t *seq_lens;
    void *out;
    float *lse;
    void *workspace;
    uint64_t workspace_bytes;
    int64_t num_pages, window_left;
    int32_t B, Hq, Hkv, Lq, dqk, dv;
    int32_t max_pages, page_size, cache_type;
    float scale, softcap;
    int32_t reserved; /* 0 */
} splash_paged_decode_args;
splash_status splash_paged_decode(const splash_paged_decode_args *args, void *cuda_stream);
/* *bytes = the workspace of a call with these sizes (0: none, workspace may be
 * NULL): INVALID_ARG, SHAPE or UNSUPPORTED where the call itself would be. */
splash_status splash_paged_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t Lq, int32_t dqk, int32_t dv,
                                                 int32_t max_pages, int32_t page_size, int32_t cache_type,
                                                 int64_t window_left, size_t *bytes);

/*
 * ---------------------------------------------------------------------------
 * Several position axes, trees of drafted tokens, upkeep of the paged cache
 * ---------------------------------------------------------------------------
 * Images and video have positions in time, height and width; a draft model
 * proposes a tree of continuations that is checked at once; samples and beams
 * fork a sequence.  The calls below go with the three above, in their manner
 * (struct_bytes, kernels queued on cuda_stream, capturable, device indices
 * checked on the device).  One step with drafts is
 *   splash_paged_append_axes   keys and values of the drafts, slot n + l, turned by depth
 *   splash_paged_tree_decode   their attention over the cache and their own branch
 *   splash_paged_compact       the accepted branch's tokens to the slots n, n + 1, ...
 * and one with forks splash_paged_remap, then splash_paged_copy for each layer.
 */

/* Most position axes of a rotation. */
#define SPLASH_MAX_AXES 4

/*
 * splash_rope_axes -- splash_rope where pair i turns by the position of axis
 * axes[i]: c = table[positions[axes[i]][b][l]][i], s likewise.  (The table's
 * columns are the frequencies of the pairs, whatever their axis: one ladder for
 * all pairs or one for each axis is a matter of the table.)  The gradient
 * (inverse = 1) is the transposed rotation.  A negative position is the identity
 * for the pairs of its axis; one >= table_rows also, and is reported.
 *
 *   rope        the arguments of splash_rope; its positions are device int32
 *               [num_axes][B][L], axis a at positions_stride_a * a
 *   axes        host, rot_dim / 2 entries below num_axes
 *   num_axes    1 .. SPLASH_MAX_AXES
 * Errors as for splash_rope (an axis >= num_axes among axes: INVALID_ARG; more than
 * SPLASH_MAX_AXES: UNSUPPORTED).
 */
typedef struct {
    uint64_t struct_bytes;
    splash_rope_args rope;
    int64_t positions_stride_a;
    const uint8_t *axes;
    int32_t num_axes;
    int32_t reserved; /* 0 */
} splash_rope_axes_args;
splash_status splash_rope_axes(const splash_rope_axes_args *args, void *cuda_stream);

/*
 * splash_paged_append_axes -- splash_paged_append where a token's slot and its
 * rotation are apart: it is stored at append.positions[b][l] and turned by
 * rot_positions[axis][b][l], pair by pair as in splash_rope_axes.  With one axis
 * this stores a tree of drafts (slots in a row, rotations by depth); with more,
 * images and video.  A negative slot is padding, as in splash_paged_append;
 * q_out / k_out are rotated all the same.  A rotation position >= table_rows is
 * reported and the token not stored.
 *
 *   append      the arguments of splash_paged_append; table required
 *   rot_positions  device int32 [num_axes][B][L], strides in elements
 *   axes, num_axes as for splash_rope_axes
 */
typedef struct {
    uint64_t struct_bytes;
    splash_paged_append_args append;
    const int32_t *rot_positions;
    int64_t rot_positions_stride_a, rot_positions_stride_b;
    const uint8_t *axes;
    int32_t num_axes;
    int32_t reserved; /* 0 */
} splash_paged_append_axes_args;
splash_status splash_paged_append_axes(const splash_paged_append_axes_args *args, void *cuda_stream);

/* Most tokens of a tree in one splash_paged_tree_decode call. */
#define SPLASH_MAX_TREE_TOKENS 64

/*
 * splash_paged_tree_decode -- splash_paged_decode for a tree of T = decode.Lq
 * new tokens instead of a chain.  Sequence b has n = seq_lens[b] cached tokens,
 * the tree's in the slots n - T .. n - 1 (token l in slot n - T + l) behind a
 * context of n - T.  parents[b][l] is -1 for a token that continues the context,
 * else the token that it continues, an earlier one.  With depth(l) the number
 * of l's ancestors in the tree, token l sits at position n - T + depth(l) and
 * sees the context, its ancestors and itself (with window_left >= 0 only those
 * whose position is at most window_left before its own).  out and lse as in
 * splash_paged_decode; a chain (parents l - 1) gives that call's result.
 *
 * A parent below -1 marks padding: the token sees nothing (out = 0,
 * lse = -inf), and neither do its descendants; a sequence may thus have fewer
 * tokens than T.  A parent that is not an earlier token (>= l) counts as padding
 * and is reported.  Tokens whose slot is negative (n < T) are padding too.
 * Cache rows that no token sees are not read, or do not reach a result; rows
 * that some tokens see do not reach the others, whatever they hold.
 *
 *   decode      the arguments of splash_paged_decode, with 1 <= Lq <=
 *               SPLASH_MAX_TREE_TOKENS; the workspace is that of
 *               splash_paged_tree_decode_workspace_size
 *   parents     device int32 [B][T], row stride parents_stride_b (0: one tree)
 * Supported sizes as for splash_paged_decode but for Lq, and for the number of
 * steps: those of 64 keys (at most max_pages * page_size / 64 + 1, or (window_left +
 * T) / 64 + 3) and nine more, over all sequences, KV heads and groups of 256 rows (of
 * 128, up to 128 rows), are to be fewer than 2^31; with at most 16 of the Hq/Hkv * T
 * rows those of splash_paged_decode are too.  The caches' strides are below 2^40 bytes, and a page's tokens do not share a row (stride_token > 0).  The cache is read
 * once for every 256 of the Hq/Hkv * T rows.  The result does not depend on timing:
 * the same inputs give the same bits on the same GPU.
 *
 * Precision as splash_paged_decode: for a bf16 cache each probability is taken
 * to 2^-16 of it, for an e4m3 one to 2^-11.
 */
typedef struct {
    uint64_t struct_bytes;
    splash_paged_decode_args decode;
    const int32_t *parents;
    int64_t parents_stride_b;
} splash_paged_tree_decode_args;
splash_status splash_paged_tree_decode(const splash_paged_tree_decode_args *args, void *cuda_stream);
splash_status splash_paged_tree_decode_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t T, int32_t dqk,
                                                      int32_t dv, int32_t max_pages, int32_t page_size,
                                                      int32_t cache_type, int64_t window_left, size_t *bytes);

/*
 * splash_paged_compact -- moves tokens inside their sequences: the token at
 * position src[b][m] becomes the one at start[b] + m, in K and V of every head,
 * for m = 0, 1, ... up to the row's end or its first negative entry.  This keeps
 * the accepted branch of a tree (start = the context's length), or what an
 * eviction leaves of a sequence.  All other rows stay as they are; the
 * sequence's new length and the pages behind it are the caller's (see
 * splash_paged_remap).
 *
 * Positions ascend: src[b][m] >= start[b] + m and src[b][m] > src[b][m - 1], so
 * that no source is overwritten before it is read.  A row's list ends at the
 * first entry that breaks this, lies outside the block table's row or is on a
 * page outside [0, num_pages) (as source or destination), which is reported.
 * Sequences that share a page must not write to it, and K and V caches do not
 * overlap (one and the same for both: INVALID_ARG).
 *
 *   src         device int32 [B][moves], row stride src_stride
 *   start       device int32 [B], >= 0 (a negative one: reported, nothing moves)
 *   caches, block_table, page_size, dqk, dv  as for splash_paged_append
 * Errors: INVALID_ARG, UNSUPPORTED, CUDA as for splash_paged_append.
 */
typedef struct {
    uint64_t struct_bytes;
    splash_cache_view k_cache, v_cache;
    const int32_t *block_table;
    int64_t block_table_stride;
    const int32_t *src;
    int64_t src_stride;
    const int32_t *start;
    int64_t num_pages, moves;
    int32_t B, Hkv, dqk, dv, max_pages, page_size, cache_type;
    int32_t reserved; /* 0 */
} splash_paged_compact_args;
splash_status splash_paged_compact(const splash_paged_compact_args *args, void *cuda_stream);

/*
 * splash_paged_remap -- a new block table from an old one: sequences fork, grow,
 * shrink, begin and end, pages are shared by reference count, copied on write,
 * given out and released.  New row i takes over the first keep[i] tokens of row
 * parents[i] (negative: of none, keep counts as 0) and gets pages for
 * max(room[i], keep[i]) tokens.  With P = page_size, row i has the columns
 * j < ceil(max(room, keep) / P), the others are -1:
 *   (j + 1) P <= keep[i]       the parent's page, shared;
 *   j P < keep[i] < (j + 1) P  the parent's page if no other row uses it.  Of
 *                              several rows that keep part of a page which
 *                              nobody else uses, the first keeps it; the others
 *                              get a fresh page and an entry in copies;
 *   j P >= keep[i]             a fresh page.
 * refs[p] counts the uses of page p: those by rows of the old table (every entry
 * in [0, num_pages) is one) and any others, which stay.  refs_out = refs - uses
 * by the old table + uses by the new one.  Fresh pages are those with refs = 0,
 * in ascending order, given out in the order of (i, j).  So this call forks
 * (equal parents), reserves (room above the old one), truncates or rolls back
 * (keep below it), frees (rows of the old table without heirs) and admits
 * (parents = -1); pages released by it are free from the next call on.
 *
 * Where the free pages do not suffice, *short_pages is the number that is
 * missing, their columns are -1 and their copies are left out: the caller drops
 * the results and tries fewer rows.  (The old table and refs are still there
 * unless refs_out was refs.)  The page contents are copied by splash_paged_copy,
 * once for each layer that goes by this table.
 *
 * A parent >= num_rows counts as negative, a keep beyond the parent's row as its
 * end, a room beyond the new row as that, and a negative keep as 0; a page outside
 * [0, num_pages) among the kept ones counts as absent (its column is -1).  Each is
 * reported, and so are counts that become negative.
 *
 *   block_table device int32 [num_rows][max_pages], row stride block_table_stride
 *   new_table   device int32 [new_rows][max_pages], row stride new_table_stride;
 *               must not overlap block_table
 *   parents, keep, room  device int32 [new_rows]
 *   refs, refs_out  device int32 [num_pages] (may be the same array)
 *   copies      device int32 [new_rows][3]: source page, destination page, rows
 *               to copy, or -1, -1, 0
 *   short_pages device int32 [1]
 *   workspace   device, 16-byte aligned, of splash_paged_remap_workspace_size
 *               bytes; overwritten, holds nothing between calls
 * num_rows may be 0 (block_table is not read).  Errors: INVALID_ARG (also where
 * new_table overlaps block_table, or refs_out a part of refs); UNSUPPORTED
 * (page_size, tables of 2^31 entries or more, rows more than 2^29 apart); CUDA.
 */
typedef struct {
    uint64_t struct_bytes;
    const int32_t *block_table;
    int64_t block_table_stride;
    int32_t *new_table;
    int64_t new_table_stride;
    const int32_t *parents, *keep, *room, *refs;
    int32_t *refs_out, *copies, *short_pages;
    void *workspace;
    uint64_t workspace_bytes;
    int64_t num_pages;
    int32_t num_rows, new_rows, max_pages, page_size;
} splash_paged_remap_args;
splash_status splash_paged_remap(const splash_paged_remap_args *args, void *cuda_stream);
splash_status splash_paged_remap_workspace_size(int64_t num_pages, int32_t new_rows, size_t *bytes);

/*
 * splash_paged_copy -- for every entry (source page, destination page, n) of
 * copies: rows 0 .. n - 1 of the source page to the destination page, in K and V
 * of every head.  Entries with a negative page or n <= 0 are skipped; pages or n
 * past their ends are reported and skipped.  A page that is a destination may not
 * be in another entry.
 *
 *   copies      device int32 [count][3], dense
 *   caches      as for splash_paged_append
 */
typedef struct {
    uint64_t struct_bytes;
    splash_cache_view k_cache, v_cache;
    const int32_t *copies;
    int64_t num_pages;
    int32_t count, Hkv, dqk, dv, page_size, cache_type;
} splash_paged_copy_args;
splash_status splash_paged_copy(const splash_paged_copy_args *args, void *cuda_stream);

/*
 * splash_classify_blocks_noalloc -- the block classification of a mask
 * (block_mask and its totals), computed without allocating any device memory.
 * The pages have no counterpart: this exists for callers that must not call
 * cudaMalloc, such as a process whose device memory is owned by its own pool
 * allocator under a fixed budget, where an allocation outside the pool can fail
 * or break the pool's accounting.
 *
 * It runs the same classification as splash_build_mask_info, but its working
 * memory (per-row counters, segment summaries, the list of blocks the
 * summaries cannot decide, totals; about 640 KiB) is a fixed array inside the
 * library's module, present on every GPU that loads the library until the
 * process exits.  The first call on a device looks that array up (once per
 * device, under a lock).  Every call ends by copying the totals to the host
 * and synchronising `cuda_stream`, so it cannot be called while that stream
 * is being captured into a CUDA graph.
 *
 *   spec, Lq, Lk, bq, bk  as for splash_build_mask_info.
 *   block_mask  device int8 [B_mask][nq][nk], caller-allocated: 0 empty,
 *               1 partial, 2 full (identical to the MaskInfo's block_mask).
 *   totals      host int64 [4]: active blocks, partial blocks, allowed
 *               (query, key) pairs, and the largest active-block count of a
 *               q-block row.
 * Limits: B_mask * nq <= 16384 and B_mask * nk <= 16384; larger masks return
 * SPLASH_ERR_UNSUPPORTED before any launch.  All calls share the one array
 * (its counters are cleared at the start of each call), so calls that
 * overlap on the GPU -- other streams or other host threads -- race and must
 * be serialised by the caller.
 */
splash_status splash_classify_blocks_noalloc(const splash_mask_spec *spec, int64_t Lq, int64_t Lk,
                                             int32_t bq, int32_t bk, int8_t *block_mask,
                                             int64_t *totals, void *cuda_stream);

/*
 * splash_last_device_error -- synchronises `cuda_stream`, then reads and
 * clears the device error word that the library's kernels set when a bounded
 * wait runs out (SPLASH_ERR_DEVICE_TIMEOUT) or a table entry fails a bounds
 * check (SPLASH_ERR_DEVICE_CHECK).  Returns SPLASH_OK when no kernel
 * reported anything, SPLASH_ERR_CUDA when the synchronisation itself fails.
 */
splash_status splash_last_device_error(void *cuda_stream);

/*
 * splash_debug_wait_selftest -- launches one tiny kernel whose mbarrier wait
 * can never be satisfied (nothing arrives on it), bounded by timeout_ns
 * nanoseconds, and returns what splash_last_device_error then reports
 * (SPLASH_ERR_DEVICE_TIMEOUT when the bound works).  It exercises the same
 * bounded-wait helper the attention kernel uses, without faulting or hanging
 * the device.  timeout_ns must be in (0, 2e9].
 */
splash_status splash_debug_wait_selftest(uint64_t timeout_ns, void *cuda_stream);

/*
 * splash_kernel_launches -- number of kernels this library has launched in
 * this process so far (all devices, all entry points).  Host-side counter,
 * thread-safe; for accounting in benchmarks.
 */
uint64_t splash_kernel_launches(void);

/*
 * splash_shard_items -- the share of one rank when a workload is split
 * across `world` GPUs by (batch, KV head) groups (host logic, no device
 * work).  "Pallas Kernels and Splash Attention" §5.2: heads are independent,
 * and the query heads of a GQA group read the same K / V, so a group is
 * never split: the n = B * Hkv groups, in (batch, KV head) row-major order,
 * are dealt in balanced contiguous ranges, rank r taking groups
 * [floor(n r / world), floor(n (r + 1) / world)).  Group g covers batch
 * g / Hkv and query heads (g % Hkv) * (Hq / Hkv) ... + Hq / Hkv - 1, which
 * in the [B][H][L][d] layouts of q, k, v, out and lse is one contiguous
 * range of memory per tensor, so a rank passes sub-tensors of the caller's
 * tensors as a problem of (end - begin) batch rows with Hq / Hkv query heads
 * and one KV head (with segment IDs, row g / Hkv of the segment array for
 * each group).  The ranges of ranks 0 .. world-1 tile [0, n) with no gap or
 * overlap; a rank may get an empty range when world > n.
 *   B, Hkv        batch size and KV heads of the whole workload (> 0)
 *   world, rank   number of ranks (> 0) and this rank (0 <= rank < world)
 *   begin, end    out: this rank's half-open range of groups
 * Errors: SPLASH_ERR_INVALID_ARG for null outputs or values out of range.
 * Thread-safe, no side effects.
 */
splash_status splash_shard_items(int32_t B, int32_t Hkv, int32_t world, int32_t rank, int64_t *begin,
                                 int64_t *end);

/*
 * splash_schedule_head_group -- the forward's item order across heads, as
 * the attention call chooses it (host logic, no device work): the number of
 * heads (256-row q-blocks) or head pairs whose items are dealt together.
 * The kernel deals its items in rounds of `grid` (one per CTA), rows longest
 * first, all heads of a row together; when the rows reach across the keys
 * (dense_rows: no window, no segment IDs) and the K / V of all heads
 * (kv_bytes) exceeds 64 MB, the items are ordered by groups of heads whose
 * K / V fits that budget, and among the group sizes from half the largest
 * such size up to it, the one whose items (items_per_head per head) leave
 * the fewest in a partial round.  Returns npairs when no grouping applies.
 *   dense_rows      1 if the mask has neither a window nor segment IDs
 *   items_per_head  work items per head (pair): q-block rows x batch x splits
 *   npairs          heads (256-row q-blocks) or head pairs
 *   kv_bytes        bytes of all heads' K and V
 *   grid            CTAs of the launch (min(items, SMs))
 * Invalid arguments (npairs < 1, items_per_head < 1, grid < 1, kv_bytes < 0)
 * return 0.  The pages have no counterpart (their grid is scheduled by the
 * TPU compiler); this is the GB300 kernel's own work order, exposed so that
 * it can be checked without a GPU.  Thread-safe, no side effects.
 */
int32_t splash_schedule_head_group(int32_t dense_rows, int64_t items_per_head, int32_t npairs, int64_t kv_bytes,
                                   int64_t grid);

/* Static description of a status code (never NULL). */
const char *splash_status_string(splash_status status);

/* Library version string, e.g. "splash-gb300 0.1 sm_103a". */
const char *splash_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPLASH_H */
