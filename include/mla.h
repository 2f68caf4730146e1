/*
 * mla.h -- C ABI of libmla.so: absorbed Multi-head Latent Attention decode on
 * NVIDIA B200 (sm_100a).
 *
 * What is computed (one new query token per sequence, s_q = 1):
 *
 *   Each cached token t of sequence b is one 576-wide bf16 row
 *       row_t = [ c_t (512 latent dims) | k_rope_t (64 rope dims) ],
 *   shared by every query head ("Multi-head Latent Attention" glossary entry,
 *   teaching abstraction: the cache holds the latent c^KV plus one decoupled
 *   rope key shared across heads).
 *
 *   The absorbed query of head h is q'_h = [ q_nope_h W_UK[h] (512) | q_rope_h (64) ]
 *   (glossary, "why absorb in decode": q^C (W^UK)^T; FlashMLA issue #16
 *   "up matrix is not involved?": q goes from [bs, H, 128] to [bs, H, 512]
 *   concatenated with q_rope [bs, H, 64], and the attention output is
 *   [bs, H, 512]).
 *
 *   mla_decode computes, for every (b, h), with T = cache_seqlens[b]:
 *       s_t  = softmax_scale * <q'_h, row_t>          (all 576 dims: content + rope score)
 *       lse  = ln sum_t exp(s_t)                      (natural log, scale included)
 *       out  = sum_t exp(s_t - lse) * row_t[0:512]    (values = the latent itself)
 *   and mla_absorb_o lifts out to per-head values: out_h W_UV[h]
 *   (glossary: sum_t p_t (c_t W^UV) = (sum_t p_t c_t) W^UV).
 *
 * Conventions shared by every entry point
 *   - Pointers marked "device" must be device memory of the current CUDA device;
 *     "host" pointers are host memory.  Every tensor is dense, row-major, with the
 *     layout given; base addresses must be 16-byte aligned.
 *   - The caller owns every tensor; the library never frees or retains them past
 *     the call.  The library owns only its workspace and a per-device error word.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *     stream).  No entry point below synchronises the host except
 *     mla_get_device_error and mla_set_workspace.
 *   - Errors found on the host (null pointer, unsupported size, misalignment)
 *     return a status before anything is launched.  Errors found on the device
 *     (a page id outside [0, num_pages), a bounded wait that ran out) set the
 *     per-device error word, read by mla_get_device_error; the affected
 *     sequences' outputs are NaN.  (Of a call whose wait ran out, mla_decode,
 *     mla_decode_multi, mla_decode_noalloc, mla_absorb_q and the fp32 mla_absorb_o
 *     do not mark what they left undone: discard all its outputs.)  No kernel traps.
 *   - Fixed widths: latent 512, rope 64 (row 576), page 64 tokens, and for the
 *     absorption GEMMs 128 no-rope query dims and 128 value dims.  Heads 1..128.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* mla_stream_t; /* same handle as cudaStream_t */

typedef enum {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1,     /* null pointer, negative size, misaligned address      */
  MLA_ERR_UNSUPPORTED = 2,     /* a size outside what the kernels handle (e.g. H > 128) */
  MLA_ERR_WORKSPACE = 3,       /* workspace too small and cannot grow (external, or capture) */
  MLA_ERR_CUDA = 4,            /* a CUDA runtime call failed; see mla_last_error_message */
  MLA_ERR_DEVICE_BAD_PAGE = 5, /* device: a block-table entry outside [0, num_pages)   */
  MLA_ERR_DEVICE_TIMEOUT = 6,  /* device: a bounded wait gave up                        */
  MLA_ERR_DEVICE_BAD_POSITION = 7 /* device: a rotation position outside the table      */
} mla_status_t;

enum {
  MLA_D_LATENT = 512,
  MLA_D_ROPE = 64,
  MLA_D_QK = 576,
  MLA_PAGE_TOKENS = 64,
  MLA_D_NOPE = 128,
  MLA_D_V = 128,
  MLA_MAX_HEADS = 128
};

/*
 * mla_decode -- split-KV absorbed decode against the (paged) latent cache.
 *
 * q             device bf16 [batch, heads, 576]: q'_h = [q_nope W_UK | q_rope].
 * kv_cache      device bf16.  Paged (block_table != NULL): [num_pages, 64, 576],
 *               token t of sequence b is row t % 64 of page block_table[b][t / 64]
 *               (glossary, capacity section: the latent cache can still be paged
 *               into blocks).  Contiguous (block_table == NULL):
 *               [batch, max_blocks * 64, 576]; num_pages is ignored.
 * block_table   device int32 [batch, max_blocks], or NULL.  Entries at or beyond
 *               ceil(T_b / 64) are never read.
 * cache_seqlens device int32 [batch], 0 <= T_b <= max_blocks * 64 (read on the
 *               device only; never copied to the host).
 * out           device fp32 [batch, heads, 512], fully overwritten.
 * lse           device fp32 [batch, heads], natural-log sum of exp(scaled score),
 *               fully overwritten.  T_b = 0 gives out = 0, lse = -inf.
 * softmax_scale multiplies the whole 576-dim dot product (1/sqrt(192) for
 *               128 no-rope + 64 rope query dims, as the glossary's runnable check
 *               scales by 1/sqrt(d_k + d_r)).
 * Rows of a last page beyond T_b, and unused block-table entries, may hold
 * anything (NaN included); they do not affect the result.
 * Uses the library workspace (split partials and per-sequence records): see
 * mla_workspace_size / mla_set_workspace.  The split of each sequence depends
 * only on (batch, heads, cache_seqlens, the device's SM count), never on page
 * ids, so a paged and a contiguous cache holding the same rows give
 * bit-identical results.
 */
mla_status_t mla_decode(const void* q, const void* kv_cache, const int32_t* block_table,
                        const int32_t* cache_seqlens, float* out, float* lse,
                        int batch, int heads, int num_pages, int max_blocks,
                        float softmax_scale, mla_stream_t stream);

/*
 * mla_decode_multi -- mla_decode with s_q query tokens per sequence (multi-token
 * prediction, speculative verification): the s_q new tokens are the last s_q
 * cached rows of each sequence, and each attends causally.
 *
 * q       device bf16 [batch, s_q, heads, 576]
 * out     device fp32 [batch, s_q, heads, 512], fully overwritten
 * lse     device fp32 [batch, s_q, heads], fully overwritten
 * Query i (0 <= i < s_q) of sequence b sits at position T_b - s_q + i and attends
 * to the cached tokens t <= T_b - s_q + i, i.e. the first T_b - s_q + 1 + i rows;
 * a query whose window is empty (T_b < s_q - i) gets out = 0, lse = -inf.  The
 * pages describe single-token decode only; this is the causal reading of several
 * new tokens appended to the cache before the call.  Each query row is computed as
 * in mla_decode (s_q = 1 gives exactly mla_decode), with the s_q x heads rows of a
 * sequence sharing every load of its cached rows.
 * s_q >= 1, heads <= 128 and s_q * heads <= 2048, else MLA_ERR_UNSUPPORTED.
 * Up to 128 rows share one pass over the cache; more rows run as groups of 128,
 * each group reading the cache again.  Every other
 * argument, the workspace, determinism and error behaviour are those of
 * mla_decode (mla_workspace_size takes s_q * heads as its heads).
 */
mla_status_t mla_decode_multi(const void* q, const void* kv_cache, const int32_t* block_table,
                              const int32_t* cache_seqlens, float* out, float* lse,
                              int batch, int s_q, int heads, int num_pages, int max_blocks,
                              float softmax_scale, mla_stream_t stream);

/*
 * mla_absorb_q -- key absorption, H independent GEMMs [batch x 128] x [128 x 512].
 *
 * q_nope  device bf16 [batch, heads, 128]
 * q_rope  device bf16 [batch, heads, 64]
 * w_uk    device bf16 [heads, 128, 512]; row i of head h holds the latent weights of
 *         key dim i (the glossary's W^UK_h transposed), so
 * q_out   device bf16 [batch, heads, 576] receives
 *         q_out[b,h,0:512]   = q_nope[b,h,:] W_UK[h]   (fp32 accumulate, bf16 round-to-nearest-even)
 *         q_out[b,h,512:576] = q_rope[b,h,:]           (copied)
 * (glossary, "why absorb in decode", first identity; FlashMLA issue #16.)
 */
mla_status_t mla_absorb_q(const void* q_nope, const void* q_rope, const void* w_uk, void* q_out,
                          int batch, int heads, mla_stream_t stream);

/*
 * mla_absorb_o -- value absorption, H independent GEMMs [batch x 512] x [512 x 128].
 *
 * out_latent device fp32 [batch, heads, 512] (mla_decode's out); rounded to bf16
 *            (nearest-even) on load, fp32 accumulate.
 * w_uv       device bf16 [heads, 512, 128]
 * out        device fp32 [batch, heads, 128] = out_latent[b,h,:] W_UV[h]
 * (glossary, "why absorb in decode", second identity; FlashMLA issue #16: the
 * [bs, H, 512] output is projected independently of the attention kernel.)
 */
mla_status_t mla_absorb_o(const float* out_latent, const void* w_uv, float* out,
                          int batch, int heads, mla_stream_t stream);

/*
 * mla_decode_noalloc -- mla_decode for callers that cannot allocate device memory.
 *
 * The pages have no counterpart of this call; it exists for callers such as a
 * serving runtime that has already reserved all device memory for its own pool,
 * or latency-critical paths that cannot absorb cudaMalloc's implicit device
 * synchronisation.  Arguments, layouts, results and errors are those of
 * mla_decode.  Instead of the workspace, it uses one 32 MiB static device array
 * that each GPU loading the library holds until exit; it never calls cudaMalloc or
 * cudaFree.  Sizes whose split partials and per-sequence records do not fit are
 * rejected with MLA_ERR_UNSUPPORTED before any launch; to fit, it may split over fewer workers
 * than mla_decode, so results match mla_decode within rounding, not bit for bit.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress).  All calls on a device share the array (it keeps the last
 * call's contents; nothing in it must start at zero): calls that overlap on the GPU
 * race and must be serialised by the caller.
 */
mla_status_t mla_decode_noalloc(const void* q, const void* kv_cache, const int32_t* block_table,
                                const int32_t* cache_seqlens, float* out, float* lse,
                                int batch, int heads, int num_pages, int max_blocks,
                                float softmax_scale, mla_stream_t stream);

/*
 * mla_append -- write new tokens' rows into the latent cache, the position rotation
 * applied on the way, and rotate the same tokens' query parts.  One launch.
 *
 * Sequence b appends n_b tokens; cache_seqlens[b] = T_b is its length with them, so its
 * new tokens are its last n_b cached rows, as in mla_decode_multi.  Token n (the i-th of
 * sequence b) goes to row r = T_b - n_b + i and is rotated to position
 * p = r + pos_offset[b]:
 *     row r of sequence b  = [ c_kv[n] (512) | R(p) k_rope[n] (64) ]
 *     q_out[n, h]          = R(p) q_rope[n, h]
 * R(p) turns pair i of the 32 pairs by the angle of cos_sin[p]: (x, y) ->
 * (x c - y s, x s + y c), computed in fp32 and rounded once to bf16.  Pair i is dims
 * (2i, 2i + 1) if interleaved = 1, (i, i + 32) if 0.
 *
 * c_kv       device bf16 [tokens, 512], consecutive tokens c_kv_stride elements apart
 * k_rope     device bf16 [tokens, 64], k_rope_stride elements apart
 * q_rope     device bf16 [tokens, heads, 64] with strides q_stride_token, q_stride_head, or
 *            NULL (then q_out is NULL and heads is ignored)
 * q_out      device bf16, likewise with its own strides, its vectors apart from one another;
 *            may be q_rope itself with the same strides (rotation in place), and must not
 *            overlap it otherwise
 * cos_sin    device fp32 [max_pos, 64]: 32 cosines, then 32 sines, of each position
 * cu_tokens  device int32 [batch + 1], ascending: sequence b's new tokens are
 *            cu_tokens[b] .. cu_tokens[b+1] (none is allowed); tokens at or beyond
 *            cu_tokens[batch] are padding: nothing is read into the cache or written for
 *            them.  NULL: every sequence appends tokens / batch.
 * pos_offset device int32 [batch], or NULL for 0 (e.g. the length of a shared prefix whose
 *            pages are not in block_table)
 * block_table, kv_cache, cache_seqlens: as in mla_decode (block_table NULL = contiguous)
 * Strides are elements, multiples of 8 (that of a single token or head may be anything);
 * vectors are dense.  A token whose length, row or
 * page id is invalid sets MLA_ERR_DEVICE_BAD_PAGE, one whose position is outside
 * [0, max_pos) MLA_ERR_DEVICE_BAD_POSITION: no cache row is written for it and its q_out
 * is NaN.  Two tokens given the same cache row race.
 */
mla_status_t mla_append(const void* c_kv, const void* k_rope, const void* q_rope, void* q_out, const float* cos_sin,
                        const int32_t* cu_tokens, const int32_t* cache_seqlens, const int32_t* pos_offset,
                        const int32_t* block_table, void* kv_cache, int64_t c_kv_stride, int64_t k_rope_stride,
                        int64_t q_stride_token, int64_t q_stride_head, int64_t q_out_stride_token,
                        int64_t q_out_stride_head, int tokens, int batch, int heads, int num_pages, int max_blocks,
                        int max_pos, int interleaved, mla_stream_t stream);

/*
 * mla_decode_window -- absorbed decode over a sliding window and the first tokens.
 *
 * Query i (0 <= i < s_q) of sequence b sits at position p = T_b - s_q + i, as in
 * mla_decode_multi, and attends to the cached tokens t <= p with
 *     t < sinks   or   t > p - window,
 * i.e. the last `window` tokens up to its own, and the first `sinks` tokens of the
 * sequence.  window >= 1, sinks >= 0; a window of at least T_b is plain causal decode.
 *
 * q       device bf16 [batch, s_q, heads, 576]
 * out     device bf16 [batch, s_q, heads, 512], fully overwritten: the softmax weights are
 *         rounded to bf16 for the tensor cores, so out is given with that precision
 *         (mla_absorb_o_bf16 takes it); sums and split partials are fp32
 * lse     device fp32 [batch, s_q, heads], fully overwritten
 * A query that sees no token gets out = 0, lse = -inf.  Block-table entries of pages
 * wholly outside the sinks and every query's window are never read (such pages may have
 * been given back), and what a query does not see never reaches it: cached rows outside
 * its sight, other sequences and other queries may hold anything, NaN included.
 * s_q, heads, kv_cache, block_table, cache_seqlens, softmax_scale, errors: as in
 * mla_decode_multi.
 * workspace: device memory of at least mla_decode_window_workspace_size bytes, 256-byte
 * aligned, the caller's: calls that may overlap on the GPU (streams, captured graphs)
 * need one each.  It holds nothing between calls.  Results depend on (batch, s_q, heads,
 * window, sinks, cache_seqlens, max_blocks, the device's SMs), not on page ids or on what
 * ran before: the same call gives the same bits.  (max_blocks bounds the pages, from which
 * the width of the query tiles and the split of short calls are chosen: it may move a
 * result by its rounding.)
 */
size_t mla_decode_window_workspace_size(int batch, int s_q, int heads);
mla_status_t mla_decode_window(const void* q, const void* kv_cache, const int32_t* block_table,
                               const int32_t* cache_seqlens, void* out, float* lse, int batch, int s_q, int heads,
                               int num_pages, int max_blocks, int window, int sinks, float softmax_scale, void* workspace,
                               size_t workspace_bytes, mla_stream_t stream);

/*
 * mla_decode_shared -- absorbed decode of a batch whose sequences begin with the same
 * cached tokens (a system prompt, a document): the prefix is attended to once for all
 * rows of the batch, packed into tiles, instead of once per sequence.
 *
 * The cache of sequence b is the prefix's P = prefix_len[0] tokens followed by its own
 * T_b = cache_seqlens[b] tokens.  Query i sits at position P + T_b - s_q + i and attends
 * to every token up to its own.
 *
 * kv_cache     device bf16 [num_pages, 64, 576]
 * prefix_table device int32 [prefix_blocks]: the prefix's pages in order
 * prefix_len   device int32 [1], 0 <= P <= prefix_blocks * 64 (read on the device only)
 * block_table  device int32 [batch, max_blocks]: pages of each sequence's own tokens; the
 *              first of them starts a page, whatever P is
 * cache_seqlens device int32 [batch], the own tokens, 0 <= T_b <= max_blocks * 64
 * q, out, lse, s_q, heads, softmax_scale, workspace, empty queries, errors, sight: as in
 * mla_decode_window (prefix_blocks counts like max_blocks; an invalid prefix_len makes every
 * row NaN, an invalid length or own page the rows of its sequence).
 * The host sees the tables' widths, not the lengths.  Spare columns of block_table may cost a
 * short call 3 to 6 % (7 sequences of 16 heads behind 1,000 tokens 12.9 us with exact tables,
 * 13.3 to 13.8 with 512 columns: the split of short calls is only for tables that cannot hold many
 * pages); longer calls take the same time.
 */
size_t mla_decode_shared_workspace_size(int batch, int s_q, int heads);
mla_status_t mla_decode_shared(const void* q, const void* kv_cache, const int32_t* prefix_table, const int32_t* prefix_len,
                               const int32_t* block_table, const int32_t* cache_seqlens, void* out, float* lse, int batch,
                               int s_q, int heads, int num_pages, int prefix_blocks, int max_blocks, float softmax_scale,
                               void* workspace, size_t workspace_bytes, mla_stream_t stream);

/*
 * mla_absorb_o_bf16 -- mla_absorb_o for the bf16 out_latent of mla_decode_window and
 * mla_decode_shared (device bf16 [batch, heads, 512]; fp32 accumulate, fp32 out).
 */
mla_status_t mla_absorb_o_bf16(const void* out_latent, const void* w_uv, float* out, int batch, int heads,
                               mla_stream_t stream);

/* Bytes of workspace mla_decode needs on the current device for these sizes. */
size_t mla_workspace_size(int batch, int heads, int max_blocks);

/*
 * Give the library a caller-owned device buffer (>= 256-byte aligned) as the
 * current device's workspace; NULL returns to library-owned, grow-only storage
 * (allocated with cudaMalloc on first need, refused while `stream` is capturing a
 * graph).  The buffer must stay valid while calls that use it may run.  Blocks
 * until the device is idle before switching.
 */
mla_status_t mla_set_workspace(void* dev_ptr, size_t bytes);

/*
 * Synchronise `stream`, then read and clear the current device's error word.
 * Returns MLA_OK, MLA_ERR_DEVICE_BAD_PAGE, MLA_ERR_DEVICE_TIMEOUT or
 * MLA_ERR_DEVICE_BAD_POSITION, the first that was set (or MLA_ERR_CUDA if the
 * synchronisation itself failed).  Other threads' calls go on during the wait.
 */
mla_status_t mla_get_device_error(mla_stream_t stream);

/* Static text for a status code. */
const char* mla_status_string(mla_status_t status);

/* Detail of the last host-side error on this thread (static storage, never NULL). */
const char* mla_last_error_message(void);

/* ---------------------------------------------------------------------------
 * Testing and measurement hooks.  They change how work is split or which decode
 * kernel runs, never what is computed.
 * ------------------------------------------------------------------------- */
typedef enum {
  MLA_KNOB_NUM_WORKERS = 0,     /* > 0: force the number of split workers; 0 = auto         */
  MLA_KNOB_MIN_PAGES = 1,       /* > 0: minimum pages per worker; 0 = auto                  */
  MLA_KNOB_DECODE_KERNEL = 2,   /* 0 = auto (3); 2 = CTA pair split by latent dims, partial
                                   scores exchanged through distributed shared memory;
                                   3 = CTA pair split by heads, pair-wide tcgen05 MMAs       */
  MLA_KNOB_WAIT_LIMIT = 3,      /* > 0: time limit of bounded device waits in ms; 0 = 2000  */
  MLA_KNOB_WITHHOLD_ARRIVE = 4, /* 1: the decode kernel's producer skips one load, so the
                                   consumer's bounded wait must run out (timeout test)      */
  MLA_KNOB_SPLIT_POLICY = 5,    /* 0 = auto: one whole sequence per worker when batch <= the
                                   worker count and the longest sequence is at most 16 pages
                                   above the split quota, else split; 1 = always split;
                                   2 = whole sequences whenever batch <= the worker count.
                                   A forced MLA_KNOB_NUM_WORKERS always splits.             */
  MLA_KNOB_PIECE_COST = 6,      /* pages a split charges each sequence for its fixed cost
                                   (q' staging, pipeline fill, epilogue) when it lays the
                                   sequences end to end and cuts equal shares: 0 = auto (8,
                                   a multiple of the 4-page step, so pieces of step-aligned
                                   sequences stay aligned); k > 0: min(k - 1, 256) pages 
                                   (1 = split by pages alone)                               */
  MLA_KNOB_ROW_TILE = 7         /* query rows per tile of mla_decode_window and _shared: 16,
                                   32 or 128; any other value = auto                        */
} mla_knob_t;
mla_status_t mla_set_knob(mla_knob_t knob, int value);
int mla_get_knob(mla_knob_t knob);
/* Which decode kernel mla_decode runs for `heads` under the current knobs:
   2 or 3 (MLA_KNOB_DECODE_KERNEL's numbering), -1 = none handles it. */
int mla_selected_decode_kernel(int heads);

/*
 * Per-launch device timing.  While enabled, every mla_decode records CUDA events
 * around each of its launches on its stream.  mla_timing_read synchronises on the
 * last event and writes the summed milliseconds since enabling into ms[0..2] --
 * ms[0] the split schedule (no launch of its own: every decode CTA derives its page
 * range from the lengths, so this is the empty interval between two events), ms[1]
 * the decode, ms[2] the combine -- and the number of recorded calls into *calls; it
 * then clears the record.
 */
mla_status_t mla_timing_enable(int enable);
mla_status_t mla_timing_read(float ms[3], int* calls);

#ifdef __cplusplus
}
#endif
#endif /* MLA_H_ */
