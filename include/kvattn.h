/*
 * kvattn.h -- C ABI of libkvattn: the generation-phase (decode) attention
 * step over a grouped-query / multi-query KV cache, for NVIDIA GB300
 * (sm_103a).
 *
 * The operation.  During generation each sequence adds one token per step.
 * Its key and value projections are written into a per-layer KV cache, and
 * its query then forms q_i . k_j products against every cached key without
 * recomputing earlier tokens ("The Basics of Transformer Inference" -- How To
 * Scale Your Model, part 7 -- the paragraph that introduces the KV cache).
 * Each query head runs its own softmax and its own weighted sum of values
 * ("Tensor Parallelism: Splitting Operations Across GPUs", section
 * "Splitting attention by head, and why decode is where it hurts").  Query
 * heads are grouped onto shared K/V heads in contiguous groups of
 * G = Hq / Hkv ("Tensor Parallelism ...", section "The GQA ceiling: a worked
 * memory audit"; multi-query attention, Hkv = 1, in "Efficiently Scaling
 * Transformer Inference", section 3 "Attention Layer Partitioning"):
 *
 *     kvh        = h / G
 *     s_j        = scale * sum_d q[b,h,d] * K[b,kvh,j,d],  0 <= j < seq_lens[b]
 *     out[b,h,:] = sum_j softmax_j(s) * V[b,kvh,j,:]
 *
 * Only the non-padding part of each sequence's cache is read ("The Basics of
 * Transformer Inference", item "Using ragged HBM reads and Paged Attention").
 *
 * Conventions for every call below.
 *  - All tensor arguments are DEVICE pointers to contiguous row-major memory
 *    owned by the caller.  The library never frees or retains them beyond the
 *    call's stream work.
 *  - bf16 is IEEE binary32's upper 16 bits (passed as void*); fp32 is float.
 *  - Every pointer must be 16-byte aligned.
 *  - Calls are asynchronous on `stream` (0 = legacy default stream) and do
 *    not synchronise the host, except that the first attention call on a
 *    (device, stream) pair, or a call needing a larger workspace than any
 *    before on that pair, allocates device memory (cudaMalloc; it may
 *    serialise with other device work).  Make such a first call before
 *    capturing a stream into a CUDA graph.  An outgrown workspace is not
 *    freed until kvattn_release(), so graphs captured with it stay valid.
 *  - Host-detected errors return a non-zero kvattn_status and launch nothing;
 *    kvattn_last_error() then gives a one-line reason (thread-local).
 *  - Device-detected errors (a length outside the cache) never fault or trap:
 *    the offending sequence is skipped and a sticky per-device error word is
 *    set, read and cleared by kvattn_check_device_error().
 *  - Thread-safe: internal caches are guarded by a mutex.  Calls on the same
 *    stream run in order, whichever host threads make them (a call's kernels are
 *    launched together: another thread's call on the stream waits for them to be);
 *    calls on different streams use separate workspaces.  cudaStreamPerThread is a
 *    stream, with a workspace, of each host thread that calls with it; the
 *    workspace of a thread that has ended is kept, too, until kvattn_release().
 *  - A stream is destroyed, and a thread that called with cudaStreamPerThread ends,
 *    only once the work of those calls has finished (synchronise the stream
 *    first): a destroyed stream's handle may come again, for a stream that would
 *    take the workspace over while the old one's kernels still use it.
 */
#ifndef KVATTN_H
#define KVATTN_H

#include <stdint.h>

#if defined(__GNUC__)
#define KVATTN_API __attribute__((visibility("default")))
#else
#define KVATTN_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream, spelled without CUDA headers. */
typedef struct CUstream_st *kvattn_stream_t;

typedef enum {
    KVATTN_OK = 0,
    KVATTN_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size, Hq % Hkv != 0, non-finite scale */
    KVATTN_ERR_UNSUPPORTED = 2,   /* D not in {64, 128, 256}, or sizes beyond the library's limits */
    KVATTN_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed (see kvattn_last_error) */
    KVATTN_ERR_OOM = 4,           /* workspace allocation failed */
    KVATTN_ERR_DEVICE_BOUNDS = 5, /* device saw seq_lens[b] outside the cache (sticky word) */
    KVATTN_ERR_TIMEOUT = 6        /* a bounded device wait gave up (sticky word) */
} kvattn_status;

/*
 * kv_append -- write this step's new key/value rows into the cache.
 *
 * Follows "The Basics of Transformer Inference", the KV-cache paragraph:
 * each token's key and value projections are written into the cache once.
 *
 *   k_cache, v_cache : bf16 [B, Hkv, Lmax, D], modified in place
 *   k_new, v_new     : bf16 [B, Hkv, D], the new token's rows
 *   seq_lens         : int32 [B] (device), the number of tokens cached
 *                      BEFORE this one; row seq_lens[b] is written.  The
 *                      array is not modified -- the caller advances it.
 *   B, Hkv, D, Lmax  : sizes; D in {64, 128, 256}
 *
 * Bit-exact copy; nothing outside row seq_lens[b] of each (b, kvh) changes.
 * A sequence with seq_lens[b] < 0 or >= Lmax is skipped on the device and
 * sets KVATTN_ERR_DEVICE_BOUNDS in the sticky error word.
 */
KVATTN_API int kv_append(void *k_cache, void *v_cache, const void *k_new,
              const void *v_new, const int32_t *seq_lens, int B, int Hkv,
              int D, int Lmax, kvattn_stream_t stream);

/*
 * gqa_decode_attn -- one decode step of grouped-query attention.
 *
 * Computes, for every sequence b and query head h (kvh = h / (Hq / Hkv)),
 *   out[b,h,:] = softmax_j(scale * q[b,h,:] . K[b,kvh,j,:]) . V[b,kvh,j,:]
 * over positions 0 <= j < seq_lens[b] (see the header comment for the
 * passages this follows).
 *
 *   q                : bf16 [B, Hq, D]
 *   k_cache, v_cache : bf16 [B, Hkv, Lmax, D]
 *   seq_lens         : int32 [B] (device), positions attended per sequence,
 *                      0 <= seq_lens[b] <= Lmax (after this step's append)
 *   out              : fp32 [B, Hq, D], written in full
 *   B, Hq, Hkv, D    : sizes; Hq % Hkv == 0; D in {64, 128, 256}
 *   Lmax             : positions allocated per (b, kvh) in the caches
 *   scale            : finite softmax scale (typically 1/sqrt(D))
 *
 * A sequence with seq_lens[b] == 0 gets an all-zero output row.  One with
 * seq_lens[b] outside [0, Lmax] gets an all-zero row and sets
 * KVATTN_ERR_DEVICE_BOUNDS in the sticky error word.
 * Limits: B <= 65535, Hkv <= 4096, Hq <= 8192, Lmax <= 2^24.
 */
KVATTN_API int gqa_decode_attn(const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *seq_lens, float *out, int B, int Hq,
                    int Hkv, int D, int Lmax, float scale,
                    kvattn_stream_t stream);

/*
 * gqa_decode_step -- one whole decode step in one call: kv_append followed
 * by gqa_decode_attn, fused into the attention kernel.
 *
 * Follows the same passages as the two calls it fuses: the new token's key
 * and value are written into the cache, then its query attends over every
 * cached position including its own ("The Basics of Transformer
 * Inference", the KV-cache paragraph).
 *
 *   q                : bf16 [B, Hq, D]
 *   k_new, v_new     : bf16 [B, Hkv, D], this step's key/value rows
 *   k_cache, v_cache : bf16 [B, Hkv, Lmax, D]; row seq_lens[b] is written
 *   seq_lens         : int32 [B] (device), tokens cached BEFORE this step
 *                      (0 <= seq_lens[b] < Lmax); not modified -- the
 *                      attention covers positions [0, seq_lens[b] + 1)
 *   out              : fp32 [B, Hq, D]
 *
 * Results are identical to kv_append then gqa_decode_attn with lengths
 * seq_lens + 1.  A sequence with seq_lens[b] outside [0, Lmax) is neither
 * appended nor attended (zero output row) and sets KVATTN_ERR_DEVICE_BOUNDS.
 */
KVATTN_API int gqa_decode_step(const void *q, const void *k_new, const void *v_new,
                               void *k_cache, void *v_cache, const int32_t *seq_lens,
                               float *out, int B, int Hq, int Hkv, int D, int Lmax,
                               float scale, kvattn_stream_t stream);

/*
 * kv_append_multi -- kv_append for T new tokens per sequence (the drafted
 * tokens of speculative sampling): token t's rows go into row
 * seq_lens[b] + t.
 *
 *   k_new, v_new : bf16 [B, T, Hkv, D]
 *   seq_lens     : int32 [B] (device), tokens cached before the T new ones;
 *                  not modified
 *   T            : 1 .. 64 (KVATTN_ERR_INVALID_ARG otherwise)
 * The rest as for kv_append; a sequence whose T rows do not all fit
 * (seq_lens[b] + T > Lmax, or seq_lens[b] < 0) is left untouched and sets
 * KVATTN_ERR_DEVICE_BOUNDS.  Bit-exact.
 */
KVATTN_API int kv_append_multi(void *k_cache, void *v_cache, const void *k_new,
                               const void *v_new, const int32_t *seq_lens, int B, int T,
                               int Hkv, int D, int Lmax, kvattn_stream_t stream);

/*
 * gqa_decode_attn_multi -- attention for T new tokens per sequence, causal
 * among themselves: the scoring pass of speculative sampling ("The Basics of
 * Transformer Inference": the big model scores a run of drafted tokens in
 * one pass, sharing the KV-cache loads among them).  The tokens' K/V rows
 * are already in the cache at positions seq_lens[b] - T .. seq_lens[b] - 1;
 * token t attends positions [0, seq_lens[b] - T + 1 + t) -- the cached prefix
 * and the new tokens up to itself -- and gets a zero row when that is empty.
 * A pass of the kernel takes hpg of a K/V head's G query heads for all T
 * tokens (hpg x T query rows, at most 64) and reads each K/V tile once for
 * all of them; when G x T rows do not fit one pass, the heads are split over
 * ceil(G / floor(64 / T)) passes of nearly equal size, each of which reads
 * the K/V head's tiles again (e.g. 48 heads sharing one K/V head: 2 passes
 * of 24 heads for T = 2, 3 of 16 for T = 4, 6 of 8 for T = 8).
 *
 *   q        : bf16 [B, T, Hq, D]
 *   k_cache, v_cache, seq_lens : as for gqa_decode_attn (seq_lens counts the
 *              new tokens too)
 *   out      : fp32 [B, T, Hq, D]
 *   T        : 1 .. 64 (one pass's rows); needs D in {128, 256}, else
 *              KVATTN_ERR_UNSUPPORTED.
 *              T = 1 is gqa_decode_attn.
 * Ownership, streams and device-side errors are those of gqa_decode_attn.
 */
KVATTN_API int gqa_decode_attn_multi(const void *q, const void *k_cache, const void *v_cache,
                                     const int32_t *seq_lens, float *out, int B, int T, int Hq,
                                     int Hkv, int D, int Lmax, float scale,
                                     kvattn_stream_t stream);

/*
 * gqa_decode_attn_window, gqa_decode_step_window -- the same two calls for a
 * local (sliding-window) attention layer: the query at position len_b - 1
 * attends only positions [max(0, len_b - window), len_b), the token itself
 * included ("The Basics of Transformer Inference", item on mixing in local
 * attention layers: a local layer caps how far back a token attends).
 *
 * Arguments, layouts, ownership and errors are those of gqa_decode_attn and
 * gqa_decode_step, plus
 *   window : positions attended at most, >= 1 (KVATTN_ERR_INVALID_ARG
 *            otherwise); window >= Lmax is the full attention.
 * Only the attended rows are read from HBM.  Cache rows in [0, len_b) must
 * hold finite values (the last tile may load rows just before the window,
 * which are then masked); rows at and past len_b may hold anything.
 */
KVATTN_API int gqa_decode_attn_window(const void *q, const void *k_cache, const void *v_cache,
                                      const int32_t *seq_lens, float *out, int B, int Hq,
                                      int Hkv, int D, int Lmax, float scale, int window,
                                      kvattn_stream_t stream);
KVATTN_API int gqa_decode_step_window(const void *q, const void *k_new, const void *v_new,
                                      void *k_cache, void *v_cache, const int32_t *seq_lens,
                                      float *out, int B, int Hq, int Hkv, int D, int Lmax,
                                      float scale, int window, kvattn_stream_t stream);

/*
 * gqa_decode_attn_multi_window -- gqa_decode_attn_multi on a local layer:
 * each of the T new tokens keeps its own window, so token t (at position
 * e_t - 1, e_t = seq_lens[b] - T + 1 + t) attends positions
 * [max(0, e_t - window), e_t), and gets a zero row when e_t <= 0.  The
 * tiles cover the union of the T windows, window + T - 1 positions, read
 * once for all tokens.  Arguments as for gqa_decode_attn_multi, plus window
 * as for gqa_decode_attn_window (>= 1; >= Lmax is gqa_decode_attn_multi).
 * Rows in [0, seq_lens[b]) must hold finite values.
 */
KVATTN_API int gqa_decode_attn_multi_window(const void *q, const void *k_cache,
                                            const void *v_cache, const int32_t *seq_lens,
                                            float *out, int B, int T, int Hq, int Hkv, int D,
                                            int Lmax, float scale, int window,
                                            kvattn_stream_t stream);

/*
 * Paged KV cache.  Instead of one contiguous [Lmax] run of rows per sequence,
 * the cache is a pool of fixed-size blocks and each sequence keeps a block
 * table mapping its logical positions to physical blocks; sequences that
 * share a prefix may point at the same blocks ("Machine Learning
 * Engineering and AI Systems at Scale", section "The key and value cache",
 * on PagedAttention; "The Basics of Transformer Inference", item "Using
 * ragged HBM reads and Paged Attention").  Position j of sequence b is row
 * j % block_size of block block_table[b, j / block_size]:
 *
 *   k_pool, v_pool : bf16 [num_blocks, Hkv, block_size, D]
 *   block_table    : int32 [B, max_blocks] (device, 4-byte aligned); a
 *                    sequence may use max_blocks * block_size positions
 *   block_size     : a power of two in [16, 2^20] (vLLM-style 16-position
 *                    blocks as well as blocks of a few hundred positions)
 *   max_blocks * block_size <= 2^24; num_blocks * Hkv < 2^31
 *
 * Table entries of blocks wholly past a sequence's length are never read;
 * pool rows at and past the length in its last block are never read either
 * (they may hold anything).  A table entry that is read and lies outside
 * [0, num_blocks) sets KVATTN_ERR_DEVICE_BOUNDS in the sticky word; that
 * block then reads as zeros (attention) or is not written (append) -- the
 * sequence's output is then meaningless but no memory outside the pool is
 * touched.  Results are those of the contiguous calls on the cache the
 * table describes.  The attention calls need D in {128, 256} (the
 * tensor-core kernel; KVATTN_ERR_UNSUPPORTED otherwise);
 * gqa_decode_attn_paged and gqa_decode_step_paged attend every position,
 * their _window forms a local window.
 */

/*
 * kv_append_paged -- kv_append / kv_append_multi into a paged pool: token t
 * of sequence b goes to position seq_lens[b] + t.
 *
 *   k_new, v_new : bf16 [B, T, Hkv, D]; T in [1, 64]
 *   seq_lens     : int32 [B] (device), tokens cached before the T new ones
 * A sequence whose T rows do not all fit in max_blocks * block_size
 * positions is left untouched and sets KVATTN_ERR_DEVICE_BOUNDS.  Bit-exact.
 */
KVATTN_API int kv_append_paged(void *k_pool, void *v_pool, const void *k_new,
                               const void *v_new, const int32_t *block_table,
                               const int32_t *seq_lens, int B, int T, int Hkv, int D,
                               int num_blocks, int block_size, int max_blocks,
                               kvattn_stream_t stream);

/*
 * gqa_decode_attn_paged -- gqa_decode_attn (T = 1) or gqa_decode_attn_multi
 * (T new tokens, causal among themselves) over a paged pool.
 *
 *   q        : bf16 [B, T, Hq, D]
 *   seq_lens : int32 [B] (device), positions attended per sequence,
 *              0 <= seq_lens[b] <= max_blocks * block_size (for T > 1 they
 *              count the new tokens too)
 *   out      : fp32 [B, T, Hq, D]
 * The rest as for gqa_decode_attn / gqa_decode_attn_multi.
 */
KVATTN_API int gqa_decode_attn_paged(const void *q, const void *k_pool, const void *v_pool,
                                     const int32_t *block_table, const int32_t *seq_lens,
                                     float *out, int B, int T, int Hq, int Hkv, int D,
                                     int num_blocks, int block_size, int max_blocks,
                                     float scale, kvattn_stream_t stream);

/*
 * gqa_decode_step_paged -- gqa_decode_step over a paged pool: the new
 * token's rows go to position seq_lens[b] (through the block table), then
 * its query attends positions [0, seq_lens[b] + 1).  Arguments as for
 * gqa_decode_step, with the pools and table above in place of the caches.
 */
KVATTN_API int gqa_decode_step_paged(const void *q, const void *k_new, const void *v_new,
                                     void *k_pool, void *v_pool, const int32_t *block_table,
                                     const int32_t *seq_lens, float *out, int B, int Hq,
                                     int Hkv, int D, int num_blocks, int block_size,
                                     int max_blocks, float scale, kvattn_stream_t stream);

/*
 * gqa_decode_attn_paged_window, gqa_decode_step_paged_window -- the two
 * paged calls on a local layer ("The Basics of Transformer Inference", the
 * items on local attention layers and on ragged reads with Paged
 * Attention): the queries attend what gqa_decode_attn_multi_window (T new
 * tokens) and gqa_decode_step_window (one new token, appended first) attend,
 * through the block table.  Arguments as for gqa_decode_attn_paged and
 * gqa_decode_step_paged, plus
 *   window : positions one query attends at most, >= 1
 *            (KVATTN_ERR_INVALID_ARG otherwise); >= max_blocks * block_size
 *            is the full attention.
 * A tile of a paged cache starts on a block boundary, so the first tile
 * read starts at the 128-position boundary at or before the window and its
 * rows before the window are masked: up to 127 positions before each
 * window are read (not attended), and their table entries must be valid
 * and their rows finite.
 */
KVATTN_API int gqa_decode_attn_paged_window(const void *q, const void *k_pool,
                                            const void *v_pool, const int32_t *block_table,
                                            const int32_t *seq_lens, float *out, int B, int T,
                                            int Hq, int Hkv, int D, int num_blocks,
                                            int block_size, int max_blocks, float scale,
                                            int window, kvattn_stream_t stream);
KVATTN_API int gqa_decode_step_paged_window(const void *q, const void *k_new, const void *v_new,
                                            void *k_pool, void *v_pool,
                                            const int32_t *block_table, const int32_t *seq_lens,
                                            float *out, int B, int Hq, int Hkv, int D,
                                            int num_blocks, int block_size, int max_blocks,
                                            float scale, int window, kvattn_stream_t stream);

/*
 * 8-bit KV cache (FP8 E4M3 codes with one fp32 scale per cached row).
 * Quantizing the KV cache to int8 / fp8 saves memory bandwidth and capacity
 * ("The Basics of Transformer Inference", item "Quantization"; "Machine
 * Learning Engineering and AI Systems at Scale", section "Quantization":
 * E4M3 is the inference format, the KV cache is the second thing to
 * quantize).  The pages give no rule; this library's: each cached row (one
 * position of one K/V head, D values) is stored as
 *     scale  = absmax(row) / 448          (1 for an all-zero row)
 *     code_d = E4M3(row_d / scale)        nearest, ties to even, saturating
 * with both divisions in IEEE binary32, and read as code value x scale.
 * E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits, subnormals, no
 * infinities, largest finite 448 (the OCP 8-bit format).  Rows must be
 * finite.
 *
 *   codes  : uint8 [B, Hkv, Lmax, D] (K and V separately)
 *   scales : fp32  [B, Hkv, Lmax]    (K and V separately)
 */

/* kv_quantize_fp8 -- quantize `rows` rows of D bf16 values (src [rows, D])
 * into codes [rows, D] and scales [rows] by the rule above: e.g. a whole
 * prefilled bf16 cache viewed as B*Hkv*Lmax rows.  D in {64, 128, 256}.
 * Bit-exact. */
KVATTN_API int kv_quantize_fp8(const void *src, void *codes, float *scales, long long rows,
                               int D, kvattn_stream_t stream);

/* kv_append_fp8 -- kv_append into an 8-bit cache: the new token's K and V
 * rows (bf16 [B, Hkv, D]) are quantized into position seq_lens[b], codes and
 * scale.  Errors as for kv_append.  Bit-exact. */
KVATTN_API int kv_append_fp8(void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                             const void *k_new, const void *v_new, const int32_t *seq_lens,
                             int B, int Hkv, int D, int Lmax, kvattn_stream_t stream);

/* gqa_decode_attn_fp8 -- gqa_decode_attn over an 8-bit cache: K[b,kvh,j,:] =
 * E4M3(k_codes[b,kvh,j,:]) * k_scale[b,kvh,j], V likewise.  The cache read
 * per position and K/V head is 2 (D + 4) bytes instead of 4 D.  q bf16
 * [B, Hq, D] (any finite value: each head enters the 8-bit products as two
 * E4M3 parts under a power-of-two scale, exact for entries down to 2^-14 of
 * the head's largest and within 2^-22 of it below), out fp32
 * [B, Hq, D]; lengths, errors and ownership as gqa_decode_attn.  A position's
 * weight, exp(score - the largest score) times its value scale over the
 * largest value scale of its head's positions (an all-zero row's scale is 1
 * and counts among them), enters with 11 significant bits down to 2^-14 and
 * to within 2^-25 below.
 * Needs D = 128 or 256: the kernel copies each position's codes in rows of
 * 128 (one 128-byte swizzled TMA box per 128 head dims); D = 64 is
 * KVATTN_ERR_UNSUPPORTED (not built: its 64-byte rows would need a layout
 * of their own).  Rows at and past seq_lens[b], codes and scales, are never
 * read. */
KVATTN_API int gqa_decode_attn_fp8(const void *q, const void *k_codes, const void *v_codes,
                                   const float *k_scale, const float *v_scale,
                                   const int32_t *seq_lens, float *out, int B, int Hq, int Hkv,
                                   int D, int Lmax, float scale, kvattn_stream_t stream);

/* gqa_decode_step_fp8 -- kv_append_fp8 followed by gqa_decode_attn_fp8 over
 * seq_lens[b] + 1 positions, in one pass over the 8-bit cache (the decode
 * step of "The Basics of Transformer Inference", KV-cache paragraph: write
 * this token's K/V, then attend, itself included): the attention kernel's
 * copy warp quantizes the new rows (the rule above, bit for bit the bytes
 * kv_append_fp8 writes) into position seq_lens[b] just before it copies the
 * tile that holds that position, so the step is one kernel launch (plus the
 * combine when a sequence is split) instead of two.  k_new, v_new: bf16
 * [B, Hkv, D], 16-byte aligned; seq_lens counts the tokens cached before
 * this step and is not modified.  A sequence with seq_lens[b] outside
 * [0, Lmax - 1] gets no append and a zero output row, and sets
 * KVATTN_ERR_DEVICE_BOUNDS.  D = 128 or 256; other arguments, errors and
 * ownership as gqa_decode_attn_fp8. */
KVATTN_API int gqa_decode_step_fp8(const void *q, const void *k_new, const void *v_new,
                                   void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                                   const int32_t *seq_lens, float *out, int B, int Hq, int Hkv,
                                   int D, int Lmax, float scale, kvattn_stream_t stream);

/*
 * Prompts into a paged cache.  A serving step takes its requests' new tokens
 * packed one request after the other -- whole prompts and single tokens
 * alike, request b's rows at [cu_seqlens[b], cu_seqlens[b+1]) -- and
 * kv_block_tables gives them blocks and slots, kv_append_slots (bf16 pool)
 * or kv_append_paged_fp8 (8-bit pool) writes their K/V rows, and
 * gqa_prefill_attn computes the prompts' own attention ("The Basics of
 * Transformer Inference", prefill and generation; "Machine Learning
 * Engineering and AI Systems at Scale", section "The key and value cache",
 * on PagedAttention); gqa_decode_attn_paged_fp8 then takes single tokens
 * over the 8-bit pool.  The first four keep no device memory: a captured
 * graph of them holds nothing of the library's and may replay beside any
 * other.  Outputs must not overlap inputs, but where that is said.  Packed
 * rows k_new, v_new (and q, k, v) may be
 * slices of wider rows, as of one fused projection: *_stride counts the
 * elements from one token's [H, D] row to the next, a multiple of 8, at
 * least H * D.  The calls run on the current device; every pointer belongs
 * to it.
 */

/*
 * kv_block_tables -- blocks and slots for each request's new tokens.
 *
 *   cached_lens : int32 [B], tokens request b has cached (c_b)
 *   new_lens    : int32 [B], tokens it adds now (n_b; 0: none)
 *   block_table : int32 [B, max_blocks], updated in place: entries
 *                 [0, ceil(c_b / block_size)) are the blocks it has,
 *                 the next ones, up to ceil((c_b + n_b) / block_size), are
 *                 taken from the free list; all others stay as they are
 *   free_blocks : int32 [num_free], a stack of free block ids of which the
 *                 first free_count[0] are left; ids are taken from its top
 *                 (entry free_count[0] - 1 first) in request order
 *   free_count, free_count_out : int32 [1], ids left before and after; the
 *                 two may be the same word
 *   cu_seqlens  : int32 [B + 1], written: cu_seqlens[b] = sum of n before b
 *   slots       : int64 [num_slots], written in full: token i of request b,
 *                 at packed row cu_seqlens[b] + i, gets slot
 *                 block_table[b, p / block_size] * block_size + p % block_size
 *                 with p = c_b + i; rows behind the last token get -1
 *   block_size  : a power of two in [16, 2^20]
 *
 * A request is served if its lengths are not negative and fit max_blocks
 * blocks, its rows end within num_slots, and the blocks wanted by it and all
 * requests before it are no more than free_count[0].  One that is not takes
 * no block, its rows get slot -1, the table entries it lacks become -1 (those
 * of packed rows below num_slots; with lengths that are negative or do not fit
 * its table row stays as it is), and KVATTN_ERR_DEVICE_BOUNDS is set; a
 * negative n counts as 0 rows.  free_count[0] outside [0, num_free] sets it
 * too and counts as 0.  cu_seqlens is capped at 2^31 - 1.
 * Limits: 1 <= B <= 65535, max_blocks * block_size <= 2^24,
 * 1 <= num_slots <= 2^28.
 */
KVATTN_API int kv_block_tables(const int32_t *cached_lens, const int32_t *new_lens,
                               int32_t *block_table, const int32_t *free_blocks,
                               const int32_t *free_count, int32_t *free_count_out,
                               int32_t *cu_seqlens, int64_t *slots, int B, int max_blocks,
                               int block_size, int num_free, int num_slots,
                               kvattn_stream_t stream);

/*
 * kv_append_slots -- write packed K/V rows to the pool rows that a slot map
 * names: row i goes to position slots[i] % block_size of block
 * slots[i] / block_size.
 *
 *   k_pool, v_pool : bf16 [num_blocks, Hkv, block_size, D], in place
 *   k_new, v_new   : bf16, N rows [Hkv, D]
 *   slots          : int64 [N] (8-byte aligned); a negative slot skips its row
 * Bit-exact; rows no slot names stay as they are.  A slot at or past
 * num_blocks * block_size skips its row and sets KVATTN_ERR_DEVICE_BOUNDS.
 * Slots must differ: of two rows with one slot either may land, in pieces of
 * 16 bytes.  D in {64, 128, 256}; 1 <= N <= 2^28.
 */
KVATTN_API int kv_append_slots(void *k_pool, void *v_pool, const void *k_new, const void *v_new,
                               const int64_t *slots, int N, int Hkv, int D, long long k_stride,
                               long long v_stride, int num_blocks, int block_size,
                               kvattn_stream_t stream);

/*
 * gqa_prefill_attn -- causal attention of whole prompts, packed.  Nothing of
 * a cache is read: it is the attention of prompts that have no token cached.
 * Rows that continue a cached prefix (cached_lens > 0 in kv_block_tables)
 * would attend each other alone here; gqa_extend_attn takes them, over a bf16
 * pool.
 *
 * For every sequence b, token i of its n_b = cu_seqlens[b+1] - cu_seqlens[b]
 * and query head h (kvh = h / (Hq / Hkv)):
 *     out[i,h,:] = softmax_j(scale * q[i,h,:] . k[j,kvh,:]) . v[j,kvh,:]
 * over max(0, i - window + 1) <= j <= i of its own sequence.
 *
 *   q          : bf16, N rows [Hq, D]; k, v: bf16, N rows [Hkv, D]
 *   cu_seqlens : int32 [B + 1] (device), non-decreasing, within [0, N]
 *   out        : bf16 [N, Hq, D], contiguous, 32-byte aligned; rows of no
 *                sequence (behind the last one, or between two) stay as they
 *                are
 *   scale      : finite; window >= 1 (>= N: the whole prompt)
 *
 * Scores, maxima and sums are held in fp32 (scale * q . k must stay finite
 * there); the weights enter the second
 * product as bf16, unnormalised, and the result is rounded once more.  A
 * sequence's own q, k and v rows must hold finite values; all other rows may
 * hold anything.  A sequence whose bounds are not
 * 0 <= cu_seqlens[b] <= cu_seqlens[b+1] <= N is skipped and sets
 * KVATTN_ERR_DEVICE_BOUNDS; of sequences that overlap either may have
 * written the shared rows.  The single-token form is gqa_decode_attn
 * (gqa_decode_attn_paged).  D in {64, 128, 256}; 1 <= N <= 2^28.
 */
KVATTN_API int gqa_prefill_attn(const void *q, const void *k, const void *v,
                                const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                                int D, long long q_stride, long long k_stride, long long v_stride,
                                float scale, int window, kvattn_stream_t stream);

/*
 * A paged 8-bit cache with one scale per block and K/V head ("The Basics of
 * Transformer Inference", item "Quantization"; "Machine Learning Engineering
 * and AI Systems at Scale", section "Quantization").  The pages give no
 * rule; this library's:
 *     row_d = E4M3(code_d) * scale[block, kvh]
 *     scale = the smallest power of two, 2^-100 at least, with
 *             absmax <= 448 * scale over the block's rows of that head
 *     code_d = E4M3(row_d / scale)      nearest, ties to even
 * The rows of a block are written over many steps, so a scale can only be
 * final once its block is full: a row that needs a larger one raises it, and
 * the codes already there are rewritten for it (E4M3(code value * old / new),
 * exact but for results below 2^-6, whose last bits are rounded away: the
 * scales are powers of two for this).  Rows must be finite.
 *
 *   codes  : uint8 [num_blocks, Hkv, block_size, D] (K and V separately)
 *   scales : fp32  [num_blocks, Hkv]                (K and V separately)
 *   block_size: a power of two in [16, 1024]; otherwise as the paged cache above
 */

/*
 * kv_append_paged_fp8 -- quantize packed K/V rows into a paged 8-bit cache:
 * token i of request b goes to position cached_lens[b] + i of its block
 * table row.
 *
 *   k_new, v_new : bf16, N rows [Hkv, D]
 *   block_table  : int32 [B, max_blocks]; cached_lens: int32 [B], tokens
 *                  cached before (not modified); cu_seqlens: int32 [B + 1]
 * A block's scale counts its first min(cached_lens[b] - start, block_size)
 * rows and the new ones: a block that starts empty forgets what it held.
 * Rows past the new ones keep their codes.  Blocks written by one call must
 * belong to one request each.  A request with negative lengths, rows outside
 * [0, N) or positions outside its table row is skipped, a table entry outside
 * [0, num_blocks) skips its block; both set KVATTN_ERR_DEVICE_BOUNDS.
 * cu_seqlens must not decrease: a request that ends before it starts is
 * skipped and reported, but then blocks of the others may stay unwritten, too.
 * Deterministic, codes and scales exact by the rule above.
 * D in {64, 128, 256} (gqa_decode_attn_paged_fp8 reads pools of 128 and 256);
 * 1 <= N <= 2^28.
 */
KVATTN_API int kv_append_paged_fp8(void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                                   const void *k_new, const void *v_new,
                                   const int32_t *block_table, const int32_t *cached_lens,
                                   const int32_t *cu_seqlens, int B, int N, int Hkv, int D,
                                   long long k_stride, long long v_stride, int num_blocks,
                                   int block_size, int max_blocks, kvattn_stream_t stream);

/*
 * gqa_decode_attn_paged_fp8 -- gqa_decode_attn over a paged 8-bit cache.
 *
 *   q   : bf16 [B, Hq, D]; seq_lens: int32 [B] (device), positions attended,
 *         0 <= seq_lens[b] <= max_blocks * block_size
 *   out : bf16 [B, Hq, D]
 * Scales may be any finite values >= 0 (scale * q . K must stay finite in
 * fp32).  A position's weight, exp(score - the largest score) times its value
 * scale over the largest value scale of its head's positions, enters the 8-bit
 * products with 11 significant bits down to 2^-14 and to within 2^-25 below:
 * n positions smaller than that are off by n 2^-25 together.  Pool rows at and
 * past a length are never read; table entries, lengths and device-side errors are those of
 * gqa_decode_attn_paged.  Its workspace is the stream's, as for the other
 * attention calls, but a call that is being captured gets one of that
 * capture's own: graphs captured on one stream may replay side by side (two
 * instances of one graph may not), and the first call on a stream may be a
 * captured one.  The graph keeps it; once the graph and all that was
 * instantiated from it are destroyed, later captures take it over.
 * kvattn_release frees it, so a graph of this call is not replayed after that.
 * D = 128 or 256.
 */
KVATTN_API int gqa_decode_attn_paged_fp8(const void *q, const void *k_codes, const void *v_codes,
                                         const float *k_scale, const float *v_scale,
                                         const int32_t *block_table, const int32_t *seq_lens,
                                         void *out, int B, int Hq, int Hkv, int D, int num_blocks,
                                         int block_size, int max_blocks, float scale,
                                         kvattn_stream_t stream);

/*
 * Serving running requests from a paged cache.  A step's tokens, packed as
 * above, are normalised and rotated on their way into attention
 * (qk_norm_rope, or kv_append_rope with the write of their K/V rows) and
 * attend what their requests have cached (gqa_extend_attn) or an encoder's
 * states (gqa_cross_attn); requests that share a prefix share its blocks
 * (kv_fork_blocks, kv_copy_blocks, kv_free_blocks), and a pool can be compacted
 * (kv_compact_blocks).  All but the two attention calls keep no device memory.
 * The calls run on the current device; every pointer belongs to it.  Outputs
 * must not overlap inputs, but where that is said.
 */

/*
 * qk_norm_rope -- norm of each query and key head and rotation by position.
 * The pages give no rule; this library's, for every row i and head of D
 * values x (fp32, rounded once at the end):
 *     y_d = x_d / sqrt(mean_d x_d^2 + eps) * weight_d
 *     (a, b) -> (a c_j - b s_j, a s_j + b c_j),  0 <= j < rope_dim / 2
 * with c_j, s_j = cos_table, sin_table[positions[i]][j] and (a, b) the values
 * j and j + rope_dim / 2 of y, or, interleaved, 2 j and 2 j + 1.  Values from
 * rope_dim on are not rotated.
 *
 *   q, k       : bf16, N rows [Hq, D] and [Hkv, D]
 *   positions  : int32 [N]
 *   cos_table, sin_table : fp32 [max_pos, rope_dim / 2], the caller's (any base
 *                or scaling)
 *   q_weight, k_weight : fp32 [D], or null: y = x for q, or for k
 *   q_out, k_out : bf16, N rows like q and k, written in full.  They may be q
 *                and k themselves, with the same strides
 *   rope_dim   : a multiple of 16 in [16, D]; eps >= 0 and finite
 * A row with a negative position (padding) becomes zeros; so does one whose
 * position is max_pos or more, which sets KVATTN_ERR_DEVICE_BOUNDS.  Squares
 * are summed in fp32, which values of 2^60 and more overflow (and below 2^-63
 * vanish: with eps = 0 a head of such values alone has no norm).
 * D in {64, 128, 256}; 1 <= N <= 2^28.
 */
KVATTN_API int qk_norm_rope(const void *q, const void *k, const int32_t *positions,
                            const float *cos_table, const float *sin_table, const float *q_weight,
                            const float *k_weight, void *q_out, void *k_out, int N, int Hq, int Hkv,
                            int D, int rope_dim, int max_pos, long long q_stride,
                            long long k_stride, long long q_out_stride, long long k_out_stride,
                            float eps, int interleaved, kvattn_stream_t stream);

/*
 * kv_append_rope -- qk_norm_rope and kv_append_slots in one pass: the rotated
 * keys and the values (copied bit for bit) go to the pool rows that slots
 * names, as kv_append_slots writes them; q_out gets the rotated queries.
 *
 *   v          : bf16, N rows [Hkv, D]; slots: int64 [N], all different
 *   k_pool, v_pool : bf16 [num_blocks, Hkv, block_size, D], in place
 * A negative slot writes no K/V row; one at or past num_blocks * block_size
 * neither, and sets KVATTN_ERR_DEVICE_BOUNDS; a row without a valid position
 * writes none whatever its slot.  The rest as qk_norm_rope.
 */
KVATTN_API int kv_append_rope(const void *q, const void *k, const void *v,
                              const int32_t *positions, const float *cos_table,
                              const float *sin_table, const float *q_weight,
                              const float *k_weight, const int64_t *slots, void *q_out,
                              void *k_pool, void *v_pool, int N, int Hq, int Hkv, int D,
                              int rope_dim, int max_pos, long long q_stride, long long k_stride,
                              long long v_stride, long long q_out_stride, float eps,
                              int interleaved, int num_blocks, int block_size,
                              kvattn_stream_t stream);

/*
 * gqa_extend_attn -- causal attention of packed tokens that continue what their
 * requests have cached, over the paged pool that holds both: a prompt taken in
 * parts, a prompt behind a shared prefix, drafted tokens, or one token of each
 * request, in any mixture.
 *
 * For every sequence b with n_b = cu_seqlens[b+1] - cu_seqlens[b] rows, token i
 * of it is at position p = seq_lens[b] - n_b + i of its block table row, and for
 * query head h (kvh = h / (Hq / Hkv))
 *     out[i,h,:] = softmax_j(scale * q[i,h,:] . K[j,kvh]) . V[j,kvh]
 * over max(0, p - window + 1) <= j <= p.
 *
 *   q          : bf16, N rows [Hq, D] (q_stride as above)
 *   k_pool, v_pool : bf16 [num_blocks, Hkv, block_size, D], the new tokens' rows
 *                written (kv_append_rope, kv_append_slots)
 *   block_table: int32 [B, max_blocks]; seq_lens: int32 [B], tokens in the cache
 *                with the new ones
 *   cu_seqlens : int32 [B + 1], non-decreasing, within [0, N]
 *   out        : bf16 [N, Hq, D], contiguous, 32-byte aligned; rows of no
 *                sequence stay as they are
 *   scale      : finite; window >= 1 (past every position: all)
 *
 * Tokens that attend nothing (n_b > seq_lens[b], the first n_b - seq_lens[b] of
 * them) get zeros.  A sequence whose bounds are not 0 <= cu_seqlens[b] <=
 * cu_seqlens[b+1] <= N is skipped, one whose length is outside [0, max_blocks *
 * block_size] gets zeros, a table entry outside [0, num_blocks) that holds
 * attended positions reads as a block of zeros; all three set
 * KVATTN_ERR_DEVICE_BOUNDS.  A sequence's q rows and the pool rows that some
 * token of it attends must hold finite values; entries and pool rows at and past
 * its length, and those before its tokens' windows, may hold anything.  Of
 * sequences whose rows overlap either may have written them.
 *
 * Scores, maxima and sums are held in fp32 (scale * q . K must stay finite
 * there), the weights enter the second product as bf16, unnormalised, and the
 * result is rounded once more.  The same call gives the same bits; how a
 * request's keys are divided, and with it the rounding, depends on the others'
 * lengths.  The workspace (41 MB on a GPU of 152 SMs at D = 128 and 256, 21 MB at
 * D = 64) is the stream's, or of a captured call's own, as for
 * gqa_decode_attn_paged_fp8: 64 and 32 MB then, or one of a graph that is gone, of
 * twice that at most.
 *
 * Single tokens, one of each request, are gqa_decode_attn_paged's as well (D = 128
 * and 256), which returns fp32 and keeps twice the bits of a weight.  This call is
 * the faster one in blocks of 16 at D = 128 and some dozen requests (32 of 64 heads
 * over 8 behind up to 8191: 103 us for 129) and for several tokens each at D = 256
 * (4 of 48 heads over 1: 56 to 60 us for 107 to 109); that one in blocks of 64 and
 * more (93 us for 101), at D = 256 (16 heads over 1: 29 us for 37, in blocks of 16 34
 * for 39) and for a single request (8 us for 11).  In blocks of 32 they are even.
 * D in {64, 128, 256}; block_size a power of two in [16, 2^20]; 1 <= N <= 2^28.
 */
KVATTN_API int gqa_extend_attn(const void *q, const void *k_pool, const void *v_pool,
                               const int32_t *block_table, const int32_t *seq_lens,
                               const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                               int D, long long q_stride, int num_blocks, int block_size,
                               int max_blocks, float scale, int window, kvattn_stream_t stream);

/*
 * gqa_cross_attn -- attention of packed tokens over all rows of another
 * sequence, such as an encoder's states: gqa_extend_attn without the causal
 * limit.  Every token of sequence b attends the positions 0 <= j < kv_lens[b] of
 * block table row b, whatever the number of its tokens; kv_lens[b] = 0 gives
 * zeros.  The states' K/V rows are written to their blocks once (kv_append_slots)
 * and may be shared (kv_fork_blocks, or the same ids in several rows, of which
 * kv_free_blocks is to be given one).  The rest as gqa_extend_attn.
 */
KVATTN_API int gqa_cross_attn(const void *q, const void *k_pool, const void *v_pool,
                              const int32_t *block_table, const int32_t *kv_lens,
                              const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                              int D, long long q_stride, int num_blocks, int block_size,
                              int max_blocks, float scale, kvattn_stream_t stream);

/*
 * Blocks with several holders.  refs, int32 [num_blocks], counts the holders
 * of each block beyond the first: 0 for a free block and for one that a single
 * request holds, so that kv_block_tables needs none of it.  The table rows'
 * entries [0, ceil(seq_lens[r] / block_size)) are the holders.  The free stack
 * is that of kv_block_tables: free_count[0] ids in free_blocks, taken from and
 * pushed onto its top.  A row is written at its request's end only, so whole
 * blocks can be shared and a partly filled one cannot: kv_fork_blocks gives a
 * fork its own.  refs must be 16-byte aligned, copies and moves 8, other int32
 * arrays 4.  Limits: R <= 65535 table rows, n <= 65535 named, num_blocks and
 * num_free <= 2^28, max_blocks * block_size <= 2^24, block_size a power of two
 * in [16, 2^20].
 */

/*
 * kv_fork_blocks -- table row children[i] becomes a fork of row parents[i].
 *
 *   block_table : int32 [R, max_blocks], in place: the child's row gets the
 *                 parent's whole blocks (refs + 1 each) and, if its last block is
 *                 partly filled, a block from the free stack for it
 *   seq_lens    : int32 [R], in place: the child's becomes the parent's
 *   copies      : int32 [n, 2], written: (parent's last block, child's), whose
 *                 rows kv_copy_blocks is to copy in each layer's pools, or
 *                 (-1, -1) where there is nothing to copy
 *   free_count, free_count_out : int32 [1]; may be the same word
 * Blocks are taken in the order of i.  Of the forks whose rows are within [0, R)
 * and whose child's length is 0, one is served if none of them before it has the
 * same child, none of them has its parent for a child, the parent's length is
 * within its row, and there is a block for it, if it wants one, beside those that
 * forks before it want.  One that is not changes nothing, has copies (-1, -1) and
 * sets KVATTN_ERR_DEVICE_BOUNDS, and so does a block id outside [0, num_blocks): a
 * table entry is copied as it is, without a count.  A free_count[0] outside [0,
 * num_free] is left as it is and counts as 0.
 */
KVATTN_API int kv_fork_blocks(int32_t *block_table, int32_t *seq_lens, int32_t *refs,
                              const int32_t *free_blocks, const int32_t *free_count,
                              const int32_t *parents, const int32_t *children, int32_t *copies,
                              int32_t *free_count_out, int n, int R, int max_blocks,
                              int block_size, int num_blocks, int num_free,
                              kvattn_stream_t stream);

/*
 * kv_free_blocks -- the named requests let go of their blocks: their table
 * entries become -1, their lengths 0, refs - 1 per block; a block that has no
 * holder left is pushed onto the free stack, in ascending order of the ids.
 *
 *   requests    : int32 [n], table rows; one named twice is freed once
 *   free_blocks : int32 [num_free], written from free_count[0] on
 * A request outside [0, R), or whose length is not within its row, is left as
 * it is; an entry outside [0, num_blocks) is only cleared; a block freed more
 * often than it is held is pushed once; blocks that the stack has no room for
 * are dropped.  All of these set KVATTN_ERR_DEVICE_BOUNDS.  With free_count[0]
 * outside [0, num_free] nothing is freed.  The stack is not searched: an entry of a
 * block that is on it already, as after a free of another row with the same ids that
 * refs does not count, is taken for its last holder's and pushes it a second time.
 */
KVATTN_API int kv_free_blocks(int32_t *block_table, int32_t *seq_lens, int32_t *refs,
                              int32_t *free_blocks, const int32_t *free_count,
                              const int32_t *requests, int32_t *free_count_out, int n, int R,
                              int max_blocks, int block_size, int num_blocks, int num_free,
                              kvattn_stream_t stream);

/*
 * kv_compact_blocks -- the held blocks of a pool moved to its front.  A block
 * is free if the stack has it and held if not; with `used` held ones, the k-th
 * held block at or past `used` moves to the k-th free one below it.
 *
 *   moves  : int32 [num_blocks / 2, 2], written in full: (from, to), for
 *            kv_copy_blocks in each layer's pools, (-1, -1) behind the last.  (Of a
 *            pool of one block nothing is written: any aligned pointer will do, and
 *            there is no call of kv_copy_blocks to make, whose n is positive.)
 *   remap  : int32 [num_blocks] (16-byte aligned), written: each held block's
 *            new id, -1 for free blocks (to rewrite other tables by)
 *   *_out  : the tables, references, stack and count after the moves; each may
 *            be its input.  Entries of a row past its length, and stack places
 *            past the count, are as before; the stack has the lowest id on top
 * A length that is not within its row leaves the row as it is; an entry that
 * names no held block becomes -1 if it was within [0, num_blocks); an id on the
 * stack that is outside or there twice counts once or not at all.  All of these
 * set KVATTN_ERR_DEVICE_BOUNDS; with free_count[0] outside [0, num_free] nothing
 * moves.
 */
KVATTN_API int kv_compact_blocks(const int32_t *block_table, const int32_t *seq_lens,
                                 const int32_t *refs, const int32_t *free_blocks,
                                 const int32_t *free_count, int32_t *block_table_out,
                                 int32_t *refs_out, int32_t *free_blocks_out,
                                 int32_t *free_count_out, int32_t *moves, int32_t *remap, int R,
                                 int max_blocks, int block_size, int num_blocks, int num_free,
                                 kvattn_stream_t stream);

/*
 * kv_copy_blocks -- block copies[i][0] to block copies[i][1], in two pools.
 *
 *   k_pool, v_pool : num_blocks blocks of block_bytes each (a multiple of 4; of
 *            16 for 16-byte vectors): a bf16 pool, 8-bit codes, or their scales
 *   copies : int32 [n, 2] (8-byte aligned); (-1, -1) copies nothing, any other
 *            id outside [0, num_blocks) neither, and sets KVATTN_ERR_DEVICE_BOUNDS
 * The blocks copied to must differ from each other and from those copied from.
 * n <= 2^28, block_bytes <= 2^32.
 */
KVATTN_API int kv_copy_blocks(void *k_pool, void *v_pool, const int32_t *copies, int n,
                              int num_blocks, long long block_bytes, kvattn_stream_t stream);

/*
 * gqa_decode_attn_noalloc -- the same computation as gqa_decode_attn, for
 * callers that must not have the library allocate device memory (for
 * example a server that gives all free GPU memory to its own pool at
 * start-up, or a loop that cannot afford the device synchronisation a
 * cudaFree brings).  The paper has no counterpart: this is a property of
 * the library, not of the method.
 *
 * Same arguments, layouts and errors as gqa_decode_attn.  It always runs the
 * CUDA-core split-KV kernel and keeps the partial results of split sequences
 * in a fixed 4 MiB device array that is part of the library (one per GPU,
 * held until the process exits); it never calls cudaMalloc or cudaFree.
 * The array's address is looked up on the first call made on each device
 * (with that device current); make that first call before capturing work on
 * the device into anything.  All calls on a device share the array: calls
 * whose GPU work overlaps (different streams with no ordering) race and may
 * return wrong results.  A call whose partials would not fit (2 x grid CTAs x
 * heads per pass x (D + 2) floats > 4 MiB, e.g. after kvattn_set_tuning
 * forced a very large grid) returns KVATTN_ERR_UNSUPPORTED and launches
 * nothing.
 */
KVATTN_API int gqa_decode_attn_noalloc(const void *q, const void *k_cache,
                                       const void *v_cache, const int32_t *seq_lens,
                                       float *out, int B, int Hq, int Hkv, int D,
                                       int Lmax, float scale, kvattn_stream_t stream);

/* Static string naming a status code. */
KVATTN_API const char *kvattn_status_string(int status);

/* Detail of the last host-side error on the calling thread ("" if none). */
KVATTN_API const char *kvattn_last_error(void);

/*
 * Synchronises `stream`, then returns and clears the current device's sticky
 * error word (KVATTN_OK if no device-side error was seen since the last
 * check), or KVATTN_ERR_CUDA if synchronisation itself failed.
 */
KVATTN_API int kvattn_check_device_error(kvattn_stream_t stream);

/*
 * Frees every workspace the library holds on every device (after a device
 * synchronisation), when the calls that other host threads are making have
 * launched their kernels.  Later calls allocate again on demand.
 */
KVATTN_API void kvattn_release(void);

/*
 * Test and ablation knobs (process-wide; 0 restores the automatic choice).
 *   force_path : 0 auto, 1 CUDA-core FMA kernel, 2 tensor-core kernel
 *   num_ctas   : 0 auto, else the persistent grid size of the attention
 *                kernel (a small value forces long multi-CTA splits); also that
 *                of gqa_prefill_attn, gqa_extend_attn, gqa_cross_attn,
 *                kv_block_tables and the split of
 *                kv_append_paged_fp8
 * Returns KVATTN_ERR_INVALID_ARG for values out of range.
 */
KVATTN_API int kvattn_set_tuning(int force_path, int num_ctas);

/*
 * Test knob for the failure handling (process-wide; 0 restores the default).
 * Every wait inside the tensor-core split-KV kernel is bounded; this sets
 * how many polls its pipeline waits make before giving up -- the softmax
 * threads' waits for scores and for finished P.V products, and the MMA
 * thread's polling while nothing is ready.  A kernel that gives up sets the
 * device error word to KVATTN_ERR_TIMEOUT (read by kvattn_check_device_error),
 * lets every copy and MMA it already issued finish, frees its tensor memory
 * and returns; the output of that call is undefined.  Waits for work already
 * issued keep their default limit.  With a very small value (1) a call is
 * sure to give up, which is how the tests exercise this path.  It shortens
 * gqa_prefill_attn's, gqa_extend_attn's and gqa_cross_attn's waits for scores,
 * probabilities and P.V products the same way, and in the 8-bit kernels the MMA warp's polling (the other waits
 * there end with it).  Always returns KVATTN_OK.
 */
KVATTN_API int kvattn_set_wait_limit(unsigned int polls);

/*
 * Measurement hook (process-wide).  With two events given (cudaEvent_t
 * handles, owned by the caller), every later attention call records
 * `before` on its stream just before its split-KV kernel and `after` just
 * after it, so that cudaEventElapsedTime(before, after) is that kernel's
 * duration alone (gqa_prefill_attn, gqa_extend_attn and gqa_cross_attn record
 * nothing).
 * The records sit between the kernel and its neighbours on
 * the stream, so they also end the programmatic overlap with them: use it to
 * time, not in production.  Pass (NULL, NULL) to stop; one NULL alone is
 * KVATTN_ERR_INVALID_ARG.
 */
KVATTN_API int kvattn_set_kernel_events(void *before, void *after);

/* How a call with these sizes would run (host-side planning only; no GPU
 * work).  num_sms <= 0 queries the current device. */
typedef struct {
    int path;            /* 1 FMA, 2 tensor core */
    int tile_positions;  /* positions per pipeline tile */
    int heads_per_cta;   /* query heads one CTA pass serves */
    int head_groups;     /* passes per (b, kvh): ceil(G / heads_per_cta) */
    int stages;          /* shared-memory pipeline depth */
    int threads;         /* threads per CTA */
    int num_ctas;        /* persistent grid size */
    int smem_bytes;      /* dynamic shared memory per CTA */
    int64_t workspace_bytes; /* partial (m, l, o) buffer this call needs */
} kvattn_plan;

KVATTN_API int kvattn_get_plan(int B, int Hq, int Hkv, int D, int Lmax, int num_sms,
                    kvattn_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* KVATTN_H */
