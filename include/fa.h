/*
 * fa.h -- C ABI of the GB300 (sm_103a) fused exact-attention library.
 *
 * The library computes exact scaled-dot-product attention
 *     O = softmax(scale * Q K^T) V
 * as one fused kernel per call: Q, K, V are tiled, the scores S and the
 * probabilities P never reach global memory, and an online softmax (running
 * row max m and denominator l, the partial O rescaled when the max moves) is
 * kept per query row. This is the algorithm of "Lesson 1: FlashAttention core
 * idea" §3-§4 and of "FlashAttention and Triton" §19.4-§19.6. The backward
 * pass keeps only one number per query row from the forward pass (the
 * log-sum-exp, "Lesson 1" §5) and recomputes S and P tile by tile.
 *
 * Conventions shared by every entry point
 *  - Tensors are dense, contiguous, row-major [B, H, N, d] (d fastest);
 *    per-row statistics are [B, H, N] float32.
 *  - Every pointer argument is a DEVICE pointer (cudaMalloc / PyTorch CUDA
 *    memory on the current device) unless stated otherwise. The caller owns
 *    all buffers and the stream; the library allocates no device memory and
 *    keeps no pointer after the call returns.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Work is enqueued asynchronously; FA_OK means "validated and
 *    launched", not "finished".
 *  - No call throws; errors are returned as fa_status. Arguments are validated
 *    before anything is launched: on any error nothing is enqueued.
 *  - Attention is non-causal, without mask or dropout, unless an _ex or
 *    _varlen entry point is given FA_CAUSAL.
 *
 * dtypes and head sizes
 *  - FA_BF16: bf16 Q/K/V/O/dO/dQ/dK/dV, float32 accumulation, d in {64, 128}.
 *    Runs on the tcgen05 tensor cores. Pointers 16-byte aligned.
 *  - FA_F32 : float32 everything, 1 <= d <= 128, CUDA-core FFMA arithmetic.
 *    Pointers 4-byte aligned.
 *  - Any N >= 1 (ragged last tiles are masked), B >= 1, H >= 1,
 *    B*H*N*d < 2^31 elements per tensor.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null/misaligned pointer, non-positive size, bad scale, small workspace */
  FA_ERR_UNSUPPORTED = 2, /* valid but not implemented (e.g. bf16 with d not in {64,128}) */
  FA_ERR_CUDA = 3,        /* a CUDA runtime/driver call or a launch failed */
  FA_ERR_TIMEOUT = 4      /* a kernel gave up on a bounded wait (reported by fa_check_device_status) */
} fa_status;

typedef enum { FA_F32 = 0, FA_BF16 = 1 } fa_dtype;

/*
 * Forward pass.  "Lesson 1" §4 (tiled forward, query tiles outer, key/value
 * tiles inner, online softmax, O_i / l_i at the end).
 *   Q, K, V : [B,H,N,d] inputs, dtype `dt`.
 *   O       : [B,H,N,d] output, dtype `dt`.
 *   LSE     : [B,H,N] float32 output, LSE = m + ln(l) of the scaled scores
 *             scale * q.k (natural log). The backward pass consumes it.
 *   scale   : finite, > 0 (the pages use 1/sqrt(d)).
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (before launch), FA_ERR_CUDA.
 */
fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                 int B, int H, int N, int d, float scale, fa_dtype dt, void* stream);

/* Flags of the _ex and _varlen entry points. */
#define FA_CAUSAL 1 /* query row r attends to keys c <= r of its own sequence */
/* Backward stages (fa_bwd_ex / fa_bwd_varlen); no stage bit = all three, in order. */
#define FA_STAGE_PREPROCESS (1 << 8)
#define FA_STAGE_MAIN (2 << 8)
#define FA_STAGE_DQ_CONVERT (4 << 8)
#define FA_STAGE_MASK (7 << 8)

/*
 * fa_fwd with flags: 0 or FA_CAUSAL. Causal attention is not on the source
 * pages; it is the plainest adjacent variant of the definition for
 * self-attention: row r of softmax(scale * Q K^T) is taken over keys
 * c <= r only (the others get weight 0), O and LSE defined over those keys.
 * Query tiles skip key tiles past their diagonal. Errors: as fa_fwd, plus
 * FA_ERR_INVALID_ARG for unknown flags.
 */
fa_status fa_fwd_ex(const void* Q, const void* K, const void* V, void* O, float* LSE,
                    int B, int H, int N, int d, float scale, int flags, fa_dtype dt, void* stream);

/*
 * Bytes of device scratch with which fa_fwd_ws shortens this problem's
 * forward on the CURRENT device; 0 when it gains nothing (or on invalid
 * arguments). Only bf16, non-causal problems are split.
 */
size_t fa_fwd_workspace_bytes(int B, int H, int N, int d, int flags, fa_dtype dt);

/*
 * The schedule fa_fwd_ws uses: *n_full units (batch*head, 256-query block)
 * run whole, then *n_tail units run as *splits key ranges each (*splits = 1,
 * *n_tail = 0: nothing split). resident_ctas > 0 plans for a GPU running
 * that many forward CTAs at once (host only, no GPU needed); 0 plans for the
 * current device. The rule: with W CTAs at once and U units, the U mod W
 * units of the last wave are split into min(W / (U mod W), 4, key tiles / 4)
 * ranges when that is at least 2 and U >= W (bf16, non-causal only).
 * bf16 d = 64 problems that run on the four-query-tile kernel (causal or
 * not, B*H*ceil(N/512) >= 3/4 of W) are never split.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (as fa_fwd_ex).
 */
fa_status fa_fwd_plan(int B, int H, int N, int d, int flags, fa_dtype dt, int resident_ctas,
                      int* n_full, int* n_tail, int* splits);

/*
 * fa_fwd_ex with scratch for the tail of the schedule. The forward runs one
 * CTA per (batch*head, 256-query block) unit, one CTA per SM; when the last
 * wave of CTAs is only partly filled, its units are split into 2-4 key
 * ranges, each range runs as a CTA of its own and leaves a partial result in
 * the scratch, and a second kernel on the same stream combines the parts by
 * their maxima and sums ("Lesson 1: FlashAttention core idea" §3). O and LSE
 * are the same attention (other rounding order within fp32).
 *   workspace       : device scratch of >= fa_fwd_workspace_bytes() bytes,
 *                     256-byte aligned, contents on entry irrelevant, used by
 *                     one call at a time (stream-ordered); NULL (or a
 *                     problem that needs none) runs the plain schedule.
 * Errors: as fa_fwd_ex, plus FA_ERR_INVALID_ARG for a non-NULL workspace
 * that is too small or misaligned.
 */
fa_status fa_fwd_ws(const void* Q, const void* K, const void* V, void* O, float* LSE,
                    void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                    float scale, int flags, fa_dtype dt, void* stream);

/*
 * Variable-length batch (packed layout, no padding): B sequences of
 * different lengths, sequence b holding rows cu_seqlens[b] ..
 * cu_seqlens[b+1]-1 of the packed tensors. Each sequence is attended to
 * separately (keys of other sequences get weight 0); with FA_CAUSAL row r
 * of a sequence sees its keys 0..r.
 *   Q, K, V, O : [total, H, d] (rows of all sequences back to back, then
 *                heads, d fastest), dtype `dt`.
 *   LSE        : [H, total] float32 output.
 *   cu_seqlens : DEVICE int32 [B+1], cu_seqlens[0] = 0, non-decreasing,
 *                cu_seqlens[B] = total; every length <= max_seqlen <= total
 *                (max_seqlen sizes the grid). The kernels check each pair:
 *                a sequence whose offsets break these rules is skipped
 *                (nothing of it is read or written) and fa_check_device_status
 *                then returns FA_ERR_INVALID_ARG.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (as fa_fwd; H*total*d <
 * 2^31, B*H <= 65535), FA_ERR_CUDA.
 */
fa_status fa_fwd_varlen(const void* Q, const void* K, const void* V, void* O, float* LSE,
                        const int* cu_seqlens, int B, int H, int total, int max_seqlen, int d,
                        float scale, int flags, fa_dtype dt, void* stream);

/*
 * Bytes of device scratch that fa_bwd needs for this problem on the CURRENT
 * device (0 on invalid arguments). The caller allocates it; its contents on
 * entry do not matter. Holds the fp32 dQ accumulator, per-row statistics
 * derived from D = rowsum(dO o O) and the LSE, the main kernel's unit
 * counter and, when the schedule splits its tail (fa_bwd_plan), the split
 * units' fp32 partial dK and dV.
 */
size_t fa_bwd_workspace_bytes(int B, int H, int N, int d, fa_dtype dt);

/*
 * The schedule of the bf16 backward's main kernel for this problem (no GPU
 * work). Its work items are (batch*head, 128-key tile) units, taken by a
 * persistent grid of one CTA per SM (non-causal: item w by CTA w mod W, in
 * order);
 * when the last round of items fills at most half of the SMs, its *n_tail
 * units run as *splits ranges of query tiles each, one item per range, and the dQ-convert
 * stage adds their partial dK and dV up ("Lesson 1: FlashAttention core
 * idea" §5: dK_j and dV_j are sums over the query tiles). *n_full units run
 * whole (*splits = 1, *n_tail = 0: nothing split). The rule, with W CTAs at
 * once and U units: splits = min(W / (U mod W), 4, query tiles / 4) when that
 * is at least 2 and U >= W; bf16, fixed length, non-causal only. The partial
 * sums are part of fa_bwd_workspace_bytes().
 *   resident_ctas : W; 0 plans for the current device.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (as fa_bwd_ex).
 */
fa_status fa_bwd_plan(int B, int H, int N, int d, int flags, fa_dtype dt, int resident_ctas,
                      int* n_full, int* n_tail, int* splits);

/*
 * Backward pass with recomputation.  "Lesson 1" §5: with P rebuilt from the
 * saved statistics, dV = P^T dO, dP = dO V^T,
 * dS = P o (dP - rowsum(dO o O)) * scale, dQ = dS K, dK = dS^T Q.
 * (rowsum(dP o P) over a full row equals rowsum(dO o O) because O = P V.)
 *   Q, K, V, O, dO : [B,H,N,d] inputs, dtype `dt` (O from fa_fwd).
 *   LSE            : [B,H,N] float32 from fa_fwd.
 *   dQ, dK, dV     : [B,H,N,d] outputs, dtype `dt`.
 *   workspace      : device scratch of >= fa_bwd_workspace_bytes() bytes,
 *                    256-byte aligned, not used by another call in flight.
 * Errors: as fa_fwd, plus FA_ERR_INVALID_ARG when the workspace is too small.
 */
fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                 size_t workspace_bytes, int B, int H, int N, int d, float scale, fa_dtype dt,
                 void* stream);

/*
 * One stage of fa_bwd, for callers that schedule or time the stages
 * separately. Same arguments and validation as fa_bwd, plus `stage`:
 *   FA_BWD_PREPROCESS (0): per-row statistics from D = rowsum(dO o O) and
 *                          the LSE into the workspace; zero the workspace's
 *                          dQ accumulator and (bf16) the main stage's unit
 *                          counter.
 *   FA_BWD_MAIN       (1): recompute P tile by tile; write dK, dV (the
 *                          split units of fa_bwd_plan: partial sums into the
 *                          workspace); add dQ into the workspace accumulator
 *                          (for bf16 without the softmax scale). Needs stage
 *                          0 done since the last main stage on this
 *                          workspace (a causal bf16 problem takes its units
 *                          from that counter).
 *   FA_BWD_DQ_CONVERT (2): workspace dQ accumulator -> dQ in dtype `dt`
 *                          (bf16: the scale is applied here), and the split
 *                          units' partial dK, dV added up into dK, dV.
 *                          Needs stage 1.
 * Stages run in that order on one workspace; fa_bwd == stages 0, 1, 2.
 * Errors: as fa_bwd, plus FA_ERR_INVALID_ARG for an unknown stage.
 */
typedef enum { FA_BWD_PREPROCESS = 0, FA_BWD_MAIN = 1, FA_BWD_DQ_CONVERT = 2 } fa_bwd_stage_id;

/*
 * fa_bwd with flags: FA_CAUSAL and/or stage bits (FA_STAGE_PREPROCESS,
 * FA_STAGE_MAIN, FA_STAGE_DQ_CONVERT; none = all three). The workspace is the
 * same as fa_bwd's. Pass the flags given to fa_fwd_ex. With FA_CAUSAL the
 * gradients are those of the causal definition: P is zero above the
 * diagonal, so key tiles skip the query tiles before their diagonal.
 * Errors: as fa_bwd, plus FA_ERR_INVALID_ARG for unknown flags.
 */
fa_status fa_bwd_ex(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                    const float* LSE, void* dQ, void* dK, void* dV, void* workspace,
                    size_t workspace_bytes, int B, int H, int N, int d, float scale, int flags,
                    fa_dtype dt, void* stream);

/* Scratch bytes for fa_bwd_varlen (0 on invalid sizes). */
size_t fa_bwd_varlen_workspace_bytes(int B, int H, int total, int max_seqlen, int d, fa_dtype dt);

/*
 * Backward pass of fa_fwd_varlen: same packed layout ([total, H, d] tensors,
 * LSE [H, total], device cu_seqlens), flags and stage bits as fa_bwd_ex,
 * workspace of >= fa_bwd_varlen_workspace_bytes() bytes, 256-byte aligned.
 * Errors: as fa_fwd_varlen, plus FA_ERR_INVALID_ARG for a small workspace.
 */
fa_status fa_bwd_varlen(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                        const float* LSE, void* dQ, void* dK, void* dV, const int* cu_seqlens,
                        void* workspace, size_t workspace_bytes, int B, int H, int total,
                        int max_seqlen, int d, float scale, int flags, fa_dtype dt, void* stream);

fa_status fa_bwd_stage(int stage, const void* Q, const void* K, const void* V, const void* O,
                       const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                       void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                       float scale, fa_dtype dt, void* stream);

/*
 * Fused row softmax: Y[r, :] = softmax(scale * X[r, :]) for each of `rows`
 * rows of `cols` elements. The fusion example of "FlashAttention and Triton"
 * §19.11: one pass per row (a ragged tail reads as -inf), max, exp, sum and
 * divide without intermediate arrays, so each element is read and written
 * once. X, Y: dense row-major [rows, cols], dtype `dt` (fp32 or bf16, the
 * arithmetic in fp32); they may alias (in place). 1 <= cols <= 32768,
 * rows >= 1, rows * cols < 2^31, scale finite and > 0.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (cols > 32768), FA_ERR_CUDA.
 */
fa_status fa_softmax_rows(const void* X, void* Y, int rows, int cols, float scale, fa_dtype dt,
                          void* stream);

/*
 * KV-cache decode: attention of Nq new queries per head against Nk cached
 * keys and values, O = softmax(scale * Q K^T) V and LSE = ln sum exp(scale *
 * Q K^T) per query row, every query seeing every key (no mask). The use case
 * is the inference remark of "Interview Q15: FlashAttention" (decoding with a
 * KV cache). The keys are cut into contiguous splits processed in parallel,
 * each with the online softmax of "Lesson 1: FlashAttention core idea" §3;
 * the split results (normalised output and log-sum-exp) are merged with the
 * same (m, l) rule by a second kernel. Nothing of size Nq x Nk reaches
 * global memory.
 *   Q, O : [B,H,Nq,d] bf16 (for grouped-query attention pass the G query
 *          heads that share one K/V head as Nq = G rows).
 *   K, V : [B,H,Nk,d] bf16, the cache; only the first Nk rows are read.
 *   LSE  : [B,H,Nq] float32 output (natural log, as fa_fwd).
 *   workspace : device scratch of >= fa_decode_workspace_bytes() bytes,
 *          256-byte aligned, not used by another call in flight; contents on
 *          entry do not matter (split outputs and log-sum-exps, fp32).
 *   dt   : FA_BF16 only; d in {64, 128}; 1 <= Nq <= 16; 1 <= Nk <= 2^30;
 *          B*H <= 65535. Q, K, V, O 16-byte aligned, LSE 4-byte aligned.
 * One query per head runs on CUDA cores (bandwidth-bound); 2..16 queries
 * run both products on the tensor cores with the queries padded to 16.
 * Errors: FA_ERR_INVALID_ARG (pointers, sizes, scale, small workspace),
 * FA_ERR_UNSUPPORTED (FA_F32, d, Nq > 16), FA_ERR_CUDA.
 */
fa_status fa_decode(const void* Q, const void* K, const void* V, void* O, float* LSE,
                    void* workspace, size_t workspace_bytes, int B, int H, int Nq, int Nk, int d,
                    float scale, fa_dtype dt, void* stream);

/*
 * Bytes of scratch fa_decode needs for this problem on the CURRENT device
 * (the split count depends on its SM count); 0 on invalid arguments or a
 * failed device query.
 */
size_t fa_decode_workspace_bytes(int B, int H, int Nq, int Nk, int d, fa_dtype dt);

/*
 * The split plan fa_decode uses: *splits key ranges of *keys_per_split keys
 * (a multiple of 64; the last range may be shorter), chosen to fill whole
 * waves of resident CTAs. resident_ctas > 0 plans for a GPU that holds that
 * many decode CTAs at once (no device access, for tests and capacity
 * planning); resident_ctas == 0 queries the current device. Returns
 * FA_ERR_INVALID_ARG on bad sizes or null outputs, FA_ERR_CUDA if the device
 * query fails.
 */
fa_status fa_decode_plan(int B, int H, int Nq, int Nk, int d, int resident_ctas, int* splits,
                         int* keys_per_split);

/*
 * Paged key/value cache: a pool of pages, each holding `page_size` keys (and
 * values) of every K/V head. Element e of row r of head h of page p of the
 * keys is k[p * k_page_stride + h * k_head_stride + r * k_row_stride + e],
 * the values likewise, so both orders of a page (heads of rows, rows of
 * heads) and views of a larger tensor are covered. The struct lives on the
 * host and is read during the call only.
 *   k, v      : DEVICE bf16, 16-byte aligned, not aliased with each other.
 *   page_size : a multiple of 8 in [8, 65536].
 *   d         : 64 or 128, contiguous.
 *   strides   : in elements, multiples of 8, >= d (of an axis of extent 1:
 *               ignored); distinct (page, head, row) must not overlap.
 * A sequence b owns the pages block_tables[b * max_pages ..]: its key j is row
 * j mod page_size of page block_tables[b * max_pages + j / page_size]. Entries
 * past a sequence's last page are never read. block_tables and seq_lens are
 * DEVICE int32 arrays, so that a captured graph follows their contents. The
 * kernels check what they read there: a sequence with a negative length, a
 * length beyond max_pages pages, or a page outside [0, num_pages) makes
 * fa_check_device_status return FA_ERR_INVALID_ARG; nothing outside the pool
 * is read or written, and that sequence's results are undefined.
 */
typedef struct {
  void* k;
  void* v;
  int num_pages, kv_heads, page_size, d;
  long long k_page_stride, k_head_stride, k_row_stride;
  long long v_page_stride, v_head_stride, v_row_stride;
} fa_paged_kv;

/* Flag of fa_kv_append: rotate the pairs (2i, 2i+1) instead of (i, i + rot_dim/2). */
#define FA_ROPE_INTERLEAVED 2

/*
 * Append the new tokens of a batch to a paged cache, the keys (and, if given,
 * the queries) rotated by their position on the way. A rotated pair (a, b) at
 * position p becomes
 *     (a cos[p][i] - b sin[p][i],  a sin[p][i] + b cos[p][i])
 * for the pairs i < rot_dim / 2 of each head; elements from rot_dim on, and
 * all values, are copied. The arithmetic is fp32, rounded once to bf16.
 *   K, V      : new keys and values, packed tokens [total, Hkv, d] bf16, the
 *               heads of a token contiguous, tokens k_stride / v_stride
 *               elements apart (a slice of a fused projection will do).
 *   Q, Qout   : queries [total, Hq, d] (tokens q_stride apart) and their
 *               rotated copy (tokens qout_stride apart; may be Q itself with
 *               the same stride); both NULL and Hq = 0: keys and values only.
 *   cu_seqlens: DEVICE int32 [B+1]: sequence b's new tokens are the packed
 *               tokens cu_seqlens[b] .. cu_seqlens[b+1]-1. Packed tokens
 *               before cu_seqlens[0] and from cu_seqlens[B] on are padding:
 *               what they hold does not matter, and nothing is written for
 *               them (nor their rows of Qout). NULL: every sequence has total / B (exactly) tokens.
 *   seq_lens  : the sequences' lengths AFTER this append (what the attention
 *               calls then take): new token i of n goes to key
 *               seq_lens[b] - n + i. seq_lens[b] = 0 marks a padding
 *               sequence: its tokens are skipped.
 *   cos, sin  : DEVICE fp32 [max_positions, rot_dim / 2]; rot_dim = 0 (and
 *               NULL): no rotation, Qout is a copy of Q.
 *   positions : DEVICE int32 [total] rotary positions of the packed tokens;
 *               NULL: the token's key index in the cache.
 *   rot_dim   : a multiple of 16, 0 <= rot_dim <= d.
 * No two new tokens may name the same (page, row); which of them such a row
 * would hold, element by element, is undefined. K, V, Q, Qout 16-byte
 * aligned; strides multiples of 8 and >= heads * d; cos, sin 16-byte aligned.
 * On the device: a token whose key index is negative or past max_pages pages,
 * whose page is outside the pool or whose position is outside
 * [0, max_positions) is skipped (its Qout row too) and reported like a bad
 * length above; so are all tokens of a sequence whose offsets are not within
 * 0 <= cu_seqlens[b] <= cu_seqlens[b+1] <= total. (Where offsets decrease,
 * tokens of other sequences may be left out as well; none is stored but at the
 * key that its own sequence's offsets give it.)
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (FA_F32, d, rot_dim,
 * page_size), FA_ERR_CUDA.
 */
fa_status fa_kv_append(const void* K, const void* V, long long k_stride, long long v_stride,
                       const void* Q, void* Qout, long long q_stride, long long qout_stride, int Hq,
                       const fa_paged_kv* cache, const int* block_tables, int max_pages,
                       const int* seq_lens, const int* cu_seqlens, int B, int total,
                       const float* cos, const float* sin, int rot_dim, int max_positions,
                       const int* positions, int flags, fa_dtype dt, void* stream);

/*
 * Decode against a paged cache: attention of the Nq newest tokens of each
 * sequence, whose keys are already in the cache (fa_kv_append), over that
 * sequence's seq_lens[b] keys. Query i of the Nq sees the keys
 * j < seq_lens[b] - Nq + 1 + i: its own and all before it (Nq = 1: all).
 * A query that sees no key (seq_lens[b] = 0, or fewer keys than new tokens)
 * gets O = 0 and LSE = -inf. What stands in the pages behind a sequence's
 * last key, NaN included, and in keys and values a query does not see has no
 * influence on its row.
 * The query heads h * Hq/Hkv .. (h + 1) * Hq/Hkv - 1 share K/V head h, whose
 * keys and values are loaded once for up to 32 rows (query heads times new
 * tokens), twice for more, the second time mostly from L2: G * Nq <= 64 rows,
 * G = Hq / Hkv.
 * A key whose score is -inf has weight zero, also where a row sees no other.
 *   Q   : [B,Hq,Nq,d] bf16; q_strides: NULL (dense) or 3 HOST values, the
 *         element strides of batch, head and row, multiples of 8 and >= d (of
 *         an axis of extent 1: ignored); 16-byte aligned.
 *   O   : as Q, o_strides likewise; must not overlap Q or the cache.
 *   LSE : [B,Hq,Nq] float32, dense (natural log, as fa_fwd).
 *   workspace : device scratch of >= fa_decode_paged_workspace_bytes() bytes,
 *         256-byte aligned, contents on entry irrelevant, not used by another
 *         call in flight.
 * The keys of all sequences and heads are laid end to end and cut into equal
 * shares, one per resident CTA, on the device: lengths may change between
 * replays of a captured graph. Scores, maxima and sums in fp32; each weight is
 * rounded to bf16 once for its product with the values (the sum of weights takes
 * it unrounded), O once at the end. Results are the same on every run. 1 <= B * Hkv <= 2^24, seq_lens[b] <= 2^30.
 * Errors: FA_ERR_INVALID_ARG (pointers, sizes, Hq not a multiple of Hkv,
 * strides, scale, small workspace), FA_ERR_UNSUPPORTED (FA_F32, d,
 * page_size, G * Nq > 64), FA_ERR_CUDA.
 */
fa_status fa_decode_paged(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                          const int* block_tables, int max_pages, const int* seq_lens, void* O,
                          const long long* o_strides, float* LSE, void* workspace,
                          size_t workspace_bytes, int B, int Hq, int Nq, float scale, fa_dtype dt,
                          void* stream);

/* Scratch bytes fa_decode_paged needs on the CURRENT device; 0 on invalid arguments. */
size_t fa_decode_paged_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, fa_dtype dt);

/*
 * fa_decode_paged for a batch whose sequences all continue one prefix (a
 * system prompt, a document, the prompt of many samples): every query sees
 * the prefix_len keys of the pages prefix_pages[0 .. ceil(prefix_len /
 * page_size) - 1] (DEVICE int32), then its own sequence's keys as in
 * fa_decode_paged. block_tables and seq_lens describe the sequences' OWN keys
 * only (their key 0 follows the prefix; a prefix may end inside a page, the
 * rest of which is not read). The prefix is loaded once per K/V head and 256
 * query rows of the batch (B * G * Nq; further blocks of 256 mostly find it in
 * L2), and its partial result is merged with the own keys' by maximum and sum.
 *   prefix_len : HOST value, 0 <= prefix_len <= 2^30 (0: fa_decode_paged).
 *   workspace  : >= fa_decode_shared_workspace_bytes() bytes, as above.
 * Limits and errors: as fa_decode_paged, plus FA_ERR_INVALID_ARG for a
 * negative prefix_len or missing prefix_pages. A prefix page outside the pool
 * is reported by fa_check_device_status; every row is then undefined.
 */
fa_status fa_decode_shared(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                           const int* prefix_pages, int prefix_len, const int* block_tables,
                           int max_pages, const int* seq_lens, void* O, const long long* o_strides,
                           float* LSE, void* workspace, size_t workspace_bytes, int B, int Hq, int Nq,
                           float scale, fa_dtype dt, void* stream);

/* Scratch bytes fa_decode_shared needs on the CURRENT device; 0 on invalid arguments. */
size_t fa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int Nq, int prefix_len, int d,
                                        fa_dtype dt);

/*
 * How fa_decode_shared shares a GPU between the prefix and the own keys: a
 * prefix of more than 32 rows (B * G * Nq) runs as a kernel of its own, of
 * *prefix_ctas CTAs (one per SM), its keys cut into *key_ranges ranges; the own
 * keys take the other SMs meanwhile, and all SMs afterwards. 0 and 0 without
 * such a kernel. The own keys' lengths are on the device, so this choice, which
 * a captured graph keeps, is made for any of them: of the table's size it only
 * uses that sequences cannot be longer (from 2048 keys on, nothing). sms > 0
 * plans for a GPU of that many SMs, 65536 at most (no device access); sms == 0:
 * the current device. FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED as fa_decode_shared;
 * FA_ERR_CUDA if the device query fails.
 */
fa_status fa_decode_shared_plan(int B, int Hq, int Hkv, int Nq, int prefix_len, int d, int page_size,
                                int max_pages, int sms, int* key_ranges, int* prefix_ctas);

/*
 * Causal attention of packed prompts with grouped heads. Sequence b has the
 * query tokens cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 and the keys
 * cu_seqlens_k[b] .. cu_seqlens_k[b+1]-1 of packed tensors; of its n tokens and
 * m keys, token i sees the keys j <= m - n + i (the tokens are the newest of
 * the sequence; n = m: a whole prompt, row r sees keys 0..r). A token that sees
 * no key (m < n) gets O = 0 and LSE = -inf. Query heads h * Hq/Hkv ..
 * (h + 1) * Hq/Hkv - 1 share K/V head h.
 *   Q, O : [total_q, Hq, d] bf16, K, V: [total_k, Hkv, d] bf16: the heads of a
 *          token contiguous, tokens *_stride elements apart (a slice of a fused
 *          projection will do; of one token: ignored), multiples of 8 and >=
 *          heads * d; 16-byte aligned. O must not overlap the inputs.
 *   LSE  : [Hq, total_q] float32, dense (natural log, as fa_fwd_varlen).
 *   cu_seqlens_q, cu_seqlens_k : DEVICE int32 [B+1], non-decreasing; they may
 *          be one array. Tokens before the first offset and from the last one
 *          on are padding: not read, and their rows of O and LSE are not
 *          written. What stands outside a sequence's keys, NaN included, has no
 *          influence on it; values that are not finite reach every row of
 *          their own sequence whose tile reads them, as in a product with
 *          weight zero.
 *   max_seqlen_q, max_seqlen_k : HOST upper bounds of the sequences' tokens and
 *          keys, at least 1 and at most total_q and total_k; with total_q they
 *          size the launch.
 *   workspace : device scratch of >= fa_prompt_fwd_workspace_bytes() bytes,
 *          256-byte aligned, contents on entry irrelevant, not used by another
 *          call in flight; it lets few queries with many keys be split into key
 *          ranges. NULL: they are not split.
 * Scores, maxima and sums in fp32; each weight is rounded to bf16 once for its
 * product with the values (the sum of weights takes it unrounded), O once at
 * the end. Results are the same on every run.
 * On the device: a sequence whose offsets do not lie within the tensors in
 * order, or whose lengths exceed the given bounds, is left out (nothing of it
 * is read or written) and fa_check_device_status returns FA_ERR_INVALID_ARG.
 * Where offsets run back, so that sequences lie upon one another, what the
 * call's sequences get is undefined (and reported); nothing is written past
 * their rows or the workspace.
 * Limits: bf16, d 64 or 128, Hq / Hkv <= 128, totals <= 2^30, B * Hkv <= 2^24,
 * and the rows of all blocks below 2^31: 256 Hkv times total_q / t + B or B
 * ceil(max_seqlen_q / t), whichever is less, t = 2 floor(128 / (Hq / Hkv))
 * tokens to a block (sequences of one token: B * Hkv < 2^23).
 * Errors: FA_ERR_INVALID_ARG (pointers, sizes, strides, scale, small
 * workspace), FA_ERR_UNSUPPORTED (FA_F32, d, the limits), FA_ERR_CUDA.
 */
fa_status fa_prompt_fwd(const void* Q, const void* K, const void* V, long long q_stride, long long k_stride,
                        long long v_stride, void* O, long long o_stride, float* LSE, const int* cu_seqlens_q,
                        const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                        int max_seqlen_k, void* workspace, size_t workspace_bytes, int d, float scale, fa_dtype dt,
                        void* stream);

/*
 * Scratch bytes with which fa_prompt_fwd (or fa_prompt_paged, max_seqlen_k =
 * max_pages * page_size, or 2^30 where that is more) splits this problem on the
 * CURRENT device; 0 when it does not (or on invalid arguments).
 */
size_t fa_prompt_fwd_workspace_bytes(int B, int Hq, int Hkv, int total_q, int max_seqlen_q, int max_seqlen_k, int d,
                                     fa_dtype dt);

/*
 * fa_prompt_fwd over a paged cache, which already holds the tokens' own keys
 * and values (fa_kv_append) and those of earlier turns: sequence b has the
 * first seq_lens[b] keys of its pages (DEVICE int32 arrays, as in
 * fa_decode_paged; a length or a page out of range is reported likewise, and
 * that sequence's results are undefined). For more new tokens than
 * fa_decode_paged takes. Arguments, limits and errors otherwise as there.
 */
fa_status fa_prompt_paged(const void* Q, long long q_stride, const fa_paged_kv* cache, const int* block_tables,
                          int max_pages, const int* seq_lens, void* O, long long o_stride, float* LSE,
                          const int* cu_seqlens_q, int B, int Hq, int total_q, int max_seqlen_q, void* workspace,
                          size_t workspace_bytes, float scale, fa_dtype dt, void* stream);

/* Scratch bytes for fa_prompt_bwd on the CURRENT device (0 on invalid sizes, or sizes past its limits). */
size_t fa_prompt_bwd_workspace_bytes(int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                                     int max_seqlen_k, int d, fa_dtype dt);

/*
 * Backward pass of fa_prompt_fwd: dQ like Q, dK and dV like K and V, the
 * gradients of a K/V head summed over the query heads that share it (in fp32,
 * in a fixed order; dQ is added up over the keys by the memory system, in an
 * order that differs from run to run: up to a rounding of fp32 per addition
 * before its one rounding to bf16). A token that sees no key has dQ = 0; keys
 * that no token sees (their sequence has none) dK = dV = 0. Rows outside all
 * sequences are not read, and not written in the outputs.
 *   O, dO [total_q, Hq, d]; LSE [Hq, total_q] from fa_prompt_fwd; dQ, dK, dV:
 *   strides between tokens as in fa_prompt_fwd, no overlap with each other (a
 *   fused projection's gradient will do: three slices of one tensor) or the
 *   inputs. workspace: >= fa_prompt_bwd_workspace_bytes() bytes, 256-byte
 *   aligned, contents on entry irrelevant, not used by another call in flight.
 * A sequence that is left out gets no gradients; where sequences lie upon one
 * another, gradients are undefined, as the results of fa_prompt_fwd.
 * Limits and errors as fa_prompt_fwd, plus Hkv <= 65535, and the workspace's
 * rows, 128 Hkv (total_q / floor(128 / G) + B + 1), below 2^31.
 */
fa_status fa_prompt_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO, long long q_stride,
                        long long k_stride, long long v_stride, long long o_stride, long long do_stride,
                        const float* LSE, void* dQ, void* dK, void* dV, long long dq_stride, long long dk_stride,
                        long long dv_stride, const int* cu_seqlens_q, const int* cu_seqlens_k, void* workspace,
                        size_t workspace_bytes, int B, int Hq, int Hkv, int total_q, int total_k, int max_seqlen_q,
                        int max_seqlen_k, int d, float scale, fa_dtype dt, void* stream);

/* Flag of the calls below: older keys' weights are added to, not set. */
#define FA_ACCUMULATE 4

/*
 * The attention weight that each key of a prompt got:
 *     w[b][h][j] = sum over the Hq/Hkv query heads of K/V head h and the counted
 *                  tokens i that see key j of exp(scale * q_i . k_j - LSE_i),
 * after fa_prompt_fwd, whose arguments and LSE it takes. One number per key by
 * which fa_kv_evict decides what stays in a cache.
 *   W      : float32, W[b * w_batch_stride + h * w_head_stride + j], j < w_keys
 *            (j: the key's index in its sequence, as in the cache); rows must not
 *            overlap. Elements from a sequence's length on, and all of a sequence
 *            without tokens, are left as they are.
 *   window : only the last `window` tokens of a sequence count; 0: all.
 *   flags  : FA_ACCUMULATE: the weights of keys that are older than the tokens
 *            (j < m - n) are added to what W holds; the tokens' own keys have
 *            none yet, and theirs are set. 0: all are set.
 * Scores, exponentials and sums in fp32 (sums of sums with a compensation term),
 * in a fixed order. Limits and errors as fa_prompt_fwd, plus FA_ERR_INVALID_ARG
 * for window < 0, unknown flags and overlapping rows of W; a sequence longer than
 * w_keys is left out and reported like one longer than max_seqlen_k.
 */
fa_status fa_prompt_key_weights(const void* Q, const void* K, long long q_stride, long long k_stride, const float* LSE,
                                float* W, long long w_batch_stride, long long w_head_stride, int w_keys,
                                const int* cu_seqlens_q, const int* cu_seqlens_k, int B, int Hq, int Hkv, int total_q,
                                int total_k, int max_seqlen_q, int max_seqlen_k, int window, int d, float scale,
                                int flags, fa_dtype dt, void* stream);

/* The same after fa_prompt_paged: keys in a paged cache (its values are not read). */
fa_status fa_prompt_key_weights_paged(const void* Q, long long q_stride, const fa_paged_kv* cache,
                                      const int* block_tables, int max_pages, const int* seq_lens, const float* LSE,
                                      float* W, long long w_batch_stride, long long w_head_stride, int w_keys,
                                      const int* cu_seqlens_q, int B, int Hq, int total_q, int max_seqlen_q, int window,
                                      float scale, int flags, fa_dtype dt, void* stream);

/*
 * The same for a decoding step, after fa_decode_paged: Q, strides, tables, lengths
 * and limits as there, LSE [B, Hq, Nq] its result. Every key of seq_lens[b] gets
 * the weight of the Nq newest tokens' query heads; W and FA_ACCUMULATE as above
 * (the new keys are the last Nq). The keys are read once, the values not.
 */
fa_status fa_decode_key_weights(const void* Q, const long long* q_strides, const fa_paged_kv* cache,
                                const int* block_tables, int max_pages, const int* seq_lens, const float* LSE, float* W,
                                long long w_batch_stride, long long w_head_stride, int w_keys, int B, int Hq, int Nq,
                                float scale, int flags, fa_dtype dt, void* stream);

/*
 * Eviction from a paged cache by weight. Of the first seq_lens[b] keys of each
 * sequence and K/V head stay the `recent` newest ones and, of the others, those
 * with the largest weights (of equal ones the older; NaN counts as the largest),
 * min(seq_lens[b], budget) in all. They keep their order: the i-th that stays
 * moves, with its value, to row i mod page_size of page new_tables[b * new_pages
 * + i / page_size]. Keys keep the rotation they were stored with; give
 * fa_kv_append `positions` afterwards.
 *   new_tables : block_tables itself, of max_pages pages (B = 1: or fewer): in
 *          place (no page may then be in two sequences' tables; the pages behind
 *          the last key that stays are free afterwards). Otherwise pages that no
 *          old table holds in use, each once; the old ones are left as they are,
 *          and may be shared.
 *   new_lens   : DEVICE int32 [B], min(seq_lens[b], budget); may be seq_lens.
 *   W          : float32 weights as above, read. new_W: the weights of what stays,
 *          in its order, from element 0 of each row on (strides likewise, rows
 *          must not overlap; the rest of a row is left as it is); may be W, with
 *          W's strides, and overlaps it in no other way.
 *   kept       : DEVICE int32 [B, Hkv, budget]: the index that each key that stays
 *          had, -1 behind the last one.
 *   budget     : HOST value >= 1; 0 <= recent <= budget.
 * new_pages pages must hold min(budget, w_keys, max_pages pages) keys. On
 * the device: a sequence whose length is negative, past max_pages pages or past
 * w_keys is left as it is (kept -1, new_lens as seq_lens), and, like a page outside
 * the pool (whose rows are not moved), reported by fa_check_device_status.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED (FA_F32, d, page_size; B or
 * kv_heads > 65535, budget > 2^30), FA_ERR_CUDA.
 */
fa_status fa_kv_evict(const fa_paged_kv* cache, const int* block_tables, int max_pages, const int* seq_lens,
                      const int* new_tables, int new_pages, int* new_lens, const float* W, long long w_batch_stride,
                      long long w_head_stride, int w_keys, float* new_W, long long new_w_batch_stride,
                      long long new_w_head_stride, int* kept, int B, int budget, int recent, fa_dtype dt, void* stream);

/*
 * fa_bwd without a caller-provided workspace, for callers that cannot
 * allocate device memory (for example code running inside a host application
 * that owns all device memory through its own pool, or a serving path where
 * cudaMalloc is not allowed). The paper has no counterpart to this entry point:
 * it is a deployment convenience around fa_bwd.
 * Same arguments, results and errors as fa_bwd, minus the workspace. The
 * scratch is one library-owned device array of
 * FA_BWD_NOALLOC_MAX_WORKSPACE_BYTES per device, held until process exit;
 * problems needing more (fa_bwd_workspace_bytes) return FA_ERR_UNSUPPORTED
 * without launching. All calls on a device share that array: calls whose
 * kernels may overlap on the GPU race and must be ordered by the caller. The
 * first call on each device looks up the array's address; make it before any
 * stream capture. Allocates nothing.
 */
#define FA_BWD_NOALLOC_MAX_WORKSPACE_BYTES ((size_t)32 << 20)

fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                         int B, int H, int N, int d, float scale, fa_dtype dt, void* stream);

/*
 * Synchronises `stream`, then reads and clears the library's device status
 * word on the current device. Returns FA_ERR_TIMEOUT if any kernel launched
 * since the last check abandoned a bounded wait (its outputs are then
 * undefined), FA_ERR_INVALID_ARG if a variable-length call met inconsistent
 * cu_seqlens (the sequences concerned were skipped) or a call on a paged cache
 * a length, a page or a position out of range (see there), FA_ERR_CUDA if the
 * stream reports an error, FA_OK otherwise.
 */
fa_status fa_check_device_status(void* stream);

/*
 * Test hook for the bounded-wait machinery: launches one block that waits on
 * a shared-memory barrier nothing will ever arrive at, giving up after
 * `limit_ns` nanoseconds (clamped to [1e3, 2e9]) and recording FA_ERR_TIMEOUT
 * in the device status word, exactly as the attention kernels do. Lets a test
 * observe the timeout path without hanging or faulting the GPU.
 */
fa_status fa_debug_timeout_probe(long long limit_ns, void* stream);

/*
 * Test hooks for the attention kernels' own abort path (bf16 only). Same
 * arguments, layout and ownership as fa_fwd / fa_bwd (dtype bf16, no causal
 * mask), plus:
 *   skip_tile  the forward's producer skips the load of key tile `skip_tile`
 *              of every CTA; the backward's producer skips the Q tile of
 *              query iteration `skip_tile` of every CTA (a CTA of the
 *              persistent grid counts its iterations over all the units it
 *              walks, in order). Neither the copy nor
 *              its expected-bytes arrival is issued, so no copy is left in
 *              flight; the consumers' bounded waits on that tile run out.
 *              Must be in [1, ceil(N / 128) - 1], else FA_ERR_INVALID_ARG.
 *   limit_ns   every bounded wait of these launches gives up after this many
 *              nanoseconds (clamped to [1e3, 2e9]).
 * Each CTA then records FA_ERR_TIMEOUT in the device status word, waits for
 * the copies and products it issued, frees its tensor memory and exits; the
 * outputs are undefined. fa_check_device_status reports (and clears) the
 * timeout, and the context stays usable for ordinary calls. Not for
 * production use: the pages have no counterpart; this exercises the bounded
 * waits every kernel here carries.
 */
fa_status fa_debug_fwd_skip_load(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                 int B, int H, int N, int d, float scale, int skip_tile,
                                 long long limit_ns, void* stream);
fa_status fa_debug_bwd_skip_load(const void* Q, const void* K, const void* V, const void* O,
                                 const void* dO, const float* LSE, void* dQ, void* dK, void* dV,
                                 void* workspace, size_t workspace_bytes, int B, int H, int N,
                                 int d, float scale, int skip_tile, long long limit_ns,
                                 void* stream);
/*
 * The same for the decode over a paged cache: arguments of fa_decode_shared
 * (dtype bf16). No CTA loads the tile `skip_tile` >= 1 of its walk (one with
 * fewer tiles works as usual), and a kernel of the prefix's own loads nothing.
 */
fa_status fa_debug_decode_skip_load(const void* Q, const long long* q_strides,
                                    const fa_paged_kv* cache, const int* prefix_pages,
                                    int prefix_len, const int* block_tables, int max_pages,
                                    const int* seq_lens, void* O, const long long* o_strides,
                                    float* LSE, void* workspace, size_t workspace_bytes, int B,
                                    int Hq, int Nq, float scale, int skip_tile, long long limit_ns,
                                    void* stream);
/*
 * fa_debug_bwd_skip_load with flags: FA_CAUSAL runs the causal backward,
 * whose persistent CTAs take their units from the device counter and pass
 * them on through the shared-memory item ring (the ring's bounded waits then
 * run out too). The workspace must hold fa_bwd_workspace_bytes for the
 * problem. Errors: as fa_debug_bwd_skip_load, plus FA_ERR_INVALID_ARG for
 * flags other than 0 and FA_CAUSAL.
 */
fa_status fa_debug_bwd_skip_load_ex(const void* Q, const void* K, const void* V, const void* O,
                                    const void* dO, const float* LSE, void* dQ, void* dK,
                                    void* dV, void* workspace, size_t workspace_bytes, int B,
                                    int H, int N, int d, float scale, int flags, int skip_tile,
                                    long long limit_ns, void* stream);

/* Static, NUL-terminated description of a status code. */
const char* fa_status_string(fa_status s);

/* Library ABI version (major * 100 + minor). */
int fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
