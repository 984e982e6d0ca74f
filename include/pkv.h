/*
 * pkv.h - C ABI of the paged KV attention library for GB300 (sm_103a).
 *
 * What it computes.  Exact softmax attention of every new token of a flat,
 * variable-length serving batch over its request's context, where the context
 * K/V live in a paged cache of 16-token blocks named by per-request block
 * tables, plus the slot-mapped write of the new tokens' K/V into that cache.
 * The batch description follows "Model execution" (vLLM internals notes),
 * section "Flattening a step": query_start_loc, seq_lens, block_table and
 * slot_mapping; the method follows "Inside the engine: kernels, CUDA graphs
 * and the life of a request", sections "Never materialise the TxT matrix"
 * (online softmax), "Prefill has a full grid; decode at batch 1 has almost
 * none" (split-KV partials merged by a second reduction kernel) and
 * "Attention over a block table, not a contiguous tensor" (16-token blocks
 * gathered through a block table).
 *
 * Conventions for every entry point.
 *   - Device pointers are CUDA device addresses on the current device; the
 *     caller allocates and owns every buffer.  The library never allocates,
 *     frees or synchronises: each call validates its host arguments, enqueues
 *     kernels on `stream` (a cudaStream_t; NULL = legacy default stream) and
 *     returns.  All pointers to tensors must be 16-byte aligned.
 *   - Host-checkable errors return a status and enqueue nothing.
 *   - Data-dependent errors (a block ID or slot outside the cache, a request
 *     with more new tokens than context, a query_start_loc that is not a
 *     valid prefix sum) cannot be seen on the host without a sync.  Kernels
 *     skip the offending access, never trap, and OR a PKV_FLAG_* bit into
 *     *error_flag (a device int32 the caller zeroes and reads later) when
 *     error_flag is non-NULL.  Outputs of the affected rows are unspecified.
 *   - Tensors are dense and row-major in the shapes given; the KV cache is
 *     two tensors (K and V), each [num_blocks, block_size, num_kv_heads,
 *     head_dim], i.e. [num_slots, num_kv_heads, head_dim] with
 *     slot = block_id * block_size + offset.
 *   - Supported: block_size 16; head_dim 64 or 128; num_q_heads a multiple of
 *     num_kv_heads; dtype PKV_F32 or PKV_BF16 (same dtype for Q, K, V and
 *     the output), or an 8-bit E4M3 cache with bf16 Q and output through the
 *     _e4m3 entry points, or a 4-bit E2M1 cache of pages (pkv_write_e2m1)
 *     through the _e2m1 ones.  Arithmetic is fp32 with fp32 accumulation; the
 *     tensor-core prefill rounds P to bf16 for its P.V product.  On tensor cores
 *     over E4M3 and E2M1 codes q rows are scaled and narrowed and P is rounded to
 *     f16, as those entry points say.  The rotated writes and latent attention have
 *     sizes and layouts of their own, given with their entry points.
 *
 * Entry points: pkv_write / pkv_write_e4m3 / pkv_write_e2m1 (slot-mapped write),
 * pkv_read_e2m1 (cached rows read back), pkv_stage_inputs
 * (a step's packed inputs copied to the device), pkv_num_splits
 * / pkv_num_splits_e2m1 and pkv_workspace_bytes (split-KV sizing),
 * pkv_attention_varlen and its variants _window (sliding window), _e4m3 (8-bit
 * cache), _e4m3_window, _e2m1 (4-bit cache) and _noalloc (no caller
 * workspace), pkv_write_attention_varlen / _e4m3 / _e2m1 (write and attend in
 * one call, the write folded into the decode kernel for decode steps), pkv_cascade_splits / pkv_cascade_workspace_bytes /
 * pkv_cascade_attention / _e4m3 (requests sharing a block-aligned prefix),
 * pkv_rotate_write / _e4m3 / _e2m1 (queries and keys turned by their positions, keys and
 * values stored), pkv_write_latent, pkv_latent_workspace_bytes,
 * pkv_latent_attention_varlen and pkv_expanded_attention_varlen (latent attention: its
 * cache, and both its forms),
 * pkv_build_metadata (the step's flat-batch metadata, host only) and
 * pkv_status_string.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,    /* null/misaligned pointer, bad size or count */
    PKV_ERR_UNSUPPORTED = 2,    /* valid request this build does not implement */
    PKV_ERR_WORKSPACE = 3,      /* workspace missing or smaller than required */
    PKV_ERR_CUDA = 4,           /* a CUDA runtime call or launch failed */
    PKV_ERR_DEVICE_CHECK = 5,   /* reserved for callers mapping *error_flag */
    PKV_ERR_DEVICE_TIMEOUT = 6  /* reserved for callers mapping *error_flag */
} pkv_status;

typedef enum { PKV_F32 = 0, PKV_BF16 = 1 } pkv_dtype;

/* Bits a kernel ORs into *error_flag. */
#define PKV_FLAG_BAD_BLOCK   1  /* block_table entry outside [0, num_blocks) */
#define PKV_FLAG_BAD_SLOT    2  /* slot_mapping entry >= num_blocks * block_size */
#define PKV_FLAG_BAD_LENGTHS 4  /* q_len > seq_len, q_len > max_query_len,
                                   seq_len > max_blocks_per_seq * block_size, or
                                   query_start_loc not a prefix sum ending at
                                   num_tokens */
#define PKV_FLAG_TIMEOUT     8  /* a pipeline wait gave up (about 2 s bound) */

/* Requests with at most this many new tokens take the split-KV decode path;
 * longer ones take the tiled prefill path. */
#define PKV_DECODE_MAX_QLEN 4

/*
 * pkv_write - store each new token's K and V at its slot.
 *
 * "Model execution", section "Flattening a step": slot_mapping gives, per new
 * token, the physical slot block_id * block_size + offset its K and V go to;
 * "Inside the engine ...", section "Attention over a block table ...": the
 * KV-write kernel scatters into non-contiguous blocks.
 *
 *   k_new, v_new   device, [num_tokens, num_kv_heads, head_dim], dtype.
 *   slot_mapping   device int64 [num_tokens]; a negative slot (a padding
 *                  token) is skipped; a slot >= num_blocks * block_size is
 *                  skipped and flagged PKV_FLAG_BAD_SLOT.
 *   k_cache, v_cache  device, [num_blocks, block_size, num_kv_heads, head_dim].
 *   error_flag     device int32 or NULL.
 * Slots not named by slot_mapping keep their contents.  Two tokens naming
 * the same slot leave its contents unspecified (parts of either's rows).
 * num_tokens == 0 is a no-op returning PKV_OK.
 */
pkv_status pkv_write(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                     int64_t num_tokens, void* k_cache, void* v_cache, int64_t num_blocks,
                     int block_size, int num_kv_heads, int head_dim, pkv_dtype dtype,
                     int32_t* error_flag, void* stream);

/*
 * pkv_write_e4m3 - pkv_write into an 8-bit E4M3 cache.
 *
 * "Model execution", section "Where it breaks" (an FP8 KV cache is a backend
 * feature) and "Anatomy of a serving engine", the FP8-cache exercise of its
 * KV-memory arithmetic: the cache holds one byte per element.  The pages fix
 * no format; this library reads it as E4M3 (sign, 4 exponent bits with bias
 * 7, 3 mantissa bits; subnormals m/8 * 2^-6; largest finite 448; no
 * infinities; S.1111.111 is NaN) with one fp32 scale per cache tensor: a
 * stored code c stands for scale * value(c).  Element x is stored as the
 * nearest code (ties to the even mantissa, magnitudes beyond 448 saturate to
 * 448) of x / scale, the division correctly rounded in fp32.
 *
 *   k_new, v_new   device, [num_tokens, num_kv_heads, head_dim], src_dtype
 *                  (PKV_F32 or PKV_BF16).
 *   k_cache, v_cache  device uint8 [num_blocks, block_size, num_kv_heads,
 *                  head_dim].
 *   k_scale, v_scale  finite, > 0.
 *   num_kv_heads * head_dim must be a multiple of 16 (else
 *   PKV_ERR_UNSUPPORTED).  slot_mapping, error_flag and the rest as pkv_write.
 */
pkv_status pkv_write_e4m3(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                          int64_t num_tokens, void* k_cache, void* v_cache, int64_t num_blocks,
                          int block_size, int num_kv_heads, int head_dim, pkv_dtype src_dtype,
                          float k_scale, float v_scale, int32_t* error_flag, void* stream);

/*
 * pkv_write_e2m1 - pkv_write into a 4-bit E2M1 cache.
 *
 * "Model execution", section "Where it breaks": quantised KV caches are a
 * backend feature; the pages fix no 4-bit format.  This library's: a stored
 * element stands for t * value(s) * value(c), with t the cache tensor's fp32
 * scale (k_scale or v_scale), s an E4M3 code for 16 consecutive elements of a
 * token's head row, and c an E2M1 code (sign, 2 exponent bits with bias 1, 1
 * mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6).  For 16 elements x:
 *   y = x / t,  s = E4M3(max |y| / 6),  c = E2M1(y / value(s)),
 * every division correctly rounded in fp32, every code the nearest one (ties
 * to even) with magnitudes beyond the largest (448 and 6) saturating; s = 0
 * gives codes 0, and a NaN among the 16 gives s the NaN code and codes 0.
 *
 * Each cache is [num_blocks, num_kv_heads, 9 * head_dim] bytes.  The page of one
 * (block, KV head) holds its 16 tokens' rows of head_dim / 2 code bytes (element
 * 2 i in the low nibble of byte i, 2 i + 1 in the high one), then its 16 tokens'
 * rows of head_dim / 16 scale bytes: 4.5 bits an element.
 *
 *   k_new, v_new   device, [num_tokens, num_kv_heads, head_dim], src_dtype
 *                  (PKV_F32 or PKV_BF16).
 *   k_cache, v_cache  device, as above, 16-byte aligned.
 *   k_scale, v_scale  finite, > 0.
 *   head_dim 64 or 128 (else PKV_ERR_UNSUPPORTED).  slot_mapping, error_flag and
 *   the rest as pkv_write; two tokens naming the same slot leave its contents
 *   unspecified (codes and scales may be of different tokens).
 */
pkv_status pkv_write_e2m1(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                          int64_t num_tokens, void* k_cache, void* v_cache, int64_t num_blocks,
                          int block_size, int num_kv_heads, int head_dim, pkv_dtype src_dtype,
                          float k_scale, float v_scale, int32_t* error_flag, void* stream);

/*
 * pkv_read_e2m1 - the rows at the given slots of an E2M1 cache, widened.
 *
 * The inverse of pkv_write_e2m1, for moving a request's context to another
 * cache or engine: row i of k_out (v_out) becomes the values of slot
 * slot_mapping[i], t * (value(s) * value(c)) rounded to fp32 and then to
 * out_dtype.  A slot may be named any number of times.
 *   slot_mapping   device int64 [num_rows]; rows with a negative slot keep
 *                  their contents, and so do rows with a slot >= num_blocks *
 *                  block_size, flagged PKV_FLAG_BAD_SLOT.
 *   k_out, v_out   device, [num_rows, num_kv_heads, head_dim], out_dtype
 *                  (PKV_F32 or PKV_BF16); not overlapping the caches.
 *   The rest as pkv_write_e2m1.  num_rows == 0 is a no-op returning PKV_OK.
 */
pkv_status pkv_read_e2m1(const void* k_cache, const void* v_cache, const int64_t* slot_mapping,
                         int64_t num_rows, void* k_out, void* v_out, int64_t num_blocks,
                         int block_size, int num_kv_heads, int head_dim, pkv_dtype out_dtype,
                         float k_scale, float v_scale, int32_t* error_flag, void* stream);

/* Rows of a tensor [num_tokens, heads, dim] with dense elements: strides in
 * elements, each a multiple of 16 bytes and >= 0.  A stride whose extent is 1 is
 * not used. */
typedef struct {
    void* data;
    int64_t token_stride, head_stride;
} pkv_rows;

/*
 * pkv_rotation - how a step's queries and keys are turned by their positions.
 *
 * "Model execution", section "Flattening a step": the runner's positions name each
 * new token's place in its request.  Pair i (0 <= i < rotary_dim / 2) of a head's
 * leading rotary_dim elements, elements i and i + rotary_dim / 2, or with interleaved
 * != 0 elements 2 i and 2 i + 1, (a, b) becomes
 *   (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[i],
 * in fp32, rounded once.  The angle is reduced modulo a turn in 64-bit fractions of
 * one: t is off by 2^-53 of itself, |position| 2^-61 radians and 2^-22 radians at most.
 * With several axes (time, height, width of a picture's patch) a token has a
 * position for each; the first sections[0] pairs go by axis 0, the next
 * sections[1] by axis 1, and so on.
 *   positions   device int64 [num_axes, num_tokens], any values.
 *   inv_freq    device fp32 [rotary_dim / 2], radians a position, finite.
 *   rotary_dim  a multiple of 16 (of 32 for E2M1 caches), 16 .. min(head_dim, 1024).
 *   num_axes    1..4; sections: >= 0, their sum rotary_dim / 2 (not looked at for
 *               one axis).
 */
typedef struct {
    const int64_t* positions;
    const float* inv_freq;
    int rotary_dim;
    int interleaved;
    int num_axes;
    int sections[4];
} pkv_rotation;

/*
 * pkv_rotate_write - turn a step's queries and keys, and store the keys and values.
 *
 * pkv_write with the rotation applied on the way: q_out[t, h] = turned q[t, h]
 * for every token, and at slot slot_mapping[t] the turned k_new[t] and v_new[t].
 * The rows may be parts of one tensor (a projection's output): strides are given.
 *   q, q_out       [num_tokens, num_q_heads, head_dim], dtype; q_out may be q (the
 *                  same pointer and strides) and overlaps nothing else, nor its own
 *                  rows one another.  Both NULL
 *                  with num_q_heads == 0: keys only.
 *   k_new, v_new   [num_tokens, num_kv_heads, head_dim], dtype.
 *   head_dim       a multiple of 16.
 * A padding token's q (negative slot) is turned too.  Everything else as pkv_write: two
 * tokens naming the same slot leave its contents unspecified, here and in the forms below.
 */
pkv_status pkv_rotate_write(const pkv_rotation* rotation, const pkv_rows* q,
                            const pkv_rows* q_out, const pkv_rows* k_new, const pkv_rows* v_new,
                            const int64_t* slot_mapping, int64_t num_tokens, void* k_cache,
                            void* v_cache, int64_t num_blocks, int block_size, int num_q_heads,
                            int num_kv_heads, int head_dim, pkv_dtype dtype, int32_t* error_flag,
                            void* stream);

/* pkv_rotate_write_e4m3 - the same into E4M3 caches (pkv_write_e4m3): the codes are
 * of the turned fp32 keys, not of a narrower copy. */
pkv_status pkv_rotate_write_e4m3(const pkv_rotation* rotation, const pkv_rows* q,
                                 const pkv_rows* q_out, const pkv_rows* k_new,
                                 const pkv_rows* v_new, const int64_t* slot_mapping,
                                 int64_t num_tokens, void* k_cache, void* v_cache,
                                 int64_t num_blocks, int block_size, int num_q_heads,
                                 int num_kv_heads, int head_dim, pkv_dtype src_dtype,
                                 float k_scale, float v_scale, int32_t* error_flag, void* stream);

/* pkv_rotate_write_e2m1 - the same into E2M1 caches (pkv_write_e2m1; head_dim 64 or
 * 128), quantised from the turned fp32 keys. */
pkv_status pkv_rotate_write_e2m1(const pkv_rotation* rotation, const pkv_rows* q,
                                 const pkv_rows* q_out, const pkv_rows* k_new,
                                 const pkv_rows* v_new, const int64_t* slot_mapping,
                                 int64_t num_tokens, void* k_cache, void* v_cache,
                                 int64_t num_blocks, int block_size, int num_q_heads,
                                 int num_kv_heads, int head_dim, pkv_dtype src_dtype,
                                 float k_scale, float v_scale, int32_t* error_flag, void* stream);

/*
 * Latent caches.
 *
 * In latent attention all heads of a token share one cached row: a latent vector c
 * of PKV_LATENT_DIM elements, from which a head's key and value expand by its own
 * matrices, k_h = U_h c and v_h = W_h c, and PKV_ROPE_DIM further key elements r that
 * carry the position.  A latent cache is one tensor [num_blocks, block_size,
 * PKV_LATENT_DIM + PKV_ROPE_DIM] of bf16 rows [c | r] ("Inside the engine ...", section
 * "Attention over a block table, not a contiguous tensor": the same 16-token blocks).
 * A head's score of a query (n_h, p_h) is n_h . U_h c + p_h . r, which is
 * [U_h^T n_h | p_h] . [c | r]: with U_h^T n_h taken into the query (absorbed), every
 * head attends the cached rows themselves, and W_h applies to sum_j softmax_j c_j.
 */
#define PKV_LATENT_DIM 512
#define PKV_ROPE_DIM 64
#define PKV_NOPE_DIM 128        /* expanded heads: the key's own part, and the value */

/*
 * pkv_write_latent - store each new token's latent row, its key part turned.
 *
 *   c_new     bf16 [num_tokens, PKV_LATENT_DIM], stored as it is (head_stride unused).
 *   k_rope    bf16 [num_tokens, PKV_ROPE_DIM], stored turned (head_stride unused).
 *   q_rope    bf16 [num_tokens, num_q_heads, PKV_ROPE_DIM]: the queries' positional
 *             part, turned into q_out (which may be q_rope), for example the last
 *             elements of the absorbed queries.  Both NULL with num_q_heads == 0.
 *   rotation  rotary_dim PKV_ROPE_DIM.
 *   cache     device bf16 [num_blocks, block_size, PKV_LATENT_DIM + PKV_ROPE_DIM].
 * slot_mapping, error_flag and the rest as pkv_write.
 */
pkv_status pkv_write_latent(const pkv_rotation* rotation, const pkv_rows* c_new,
                            const pkv_rows* k_rope, const pkv_rows* q_rope,
                            const pkv_rows* q_out, const int64_t* slot_mapping,
                            int64_t num_tokens, void* cache, int64_t num_blocks, int block_size,
                            int num_q_heads, int32_t* error_flag, void* stream);

/*
 * pkv_latent_workspace_bytes - device workspace pkv_latent_attention_varlen needs on
 * device `device`, whatever the batch: the fp32 partials of two 64-row tiles for each
 * of its SMs, and where they belong.  0 for an invalid device.
 */
size_t pkv_latent_workspace_bytes(int device);

/*
 * pkv_latent_attention_varlen - attention in the absorbed form over a latent cache.
 *
 *   out[t, h, :] = sum_j softmax_j(softmax_scale * q[t, h, :] . row_j) row_j[: 512]
 * for the batch that pkv_attention_varlen describes, all heads over one row a key.
 * Any number of new tokens: tiles of 64 (token, head) rows on tcgen05 tensor cores, P
 * rounded to bf16 for its product.  The batch's key tiles are dealt out evenly over
 * the SMs ("Prefill has a full grid; decode at batch 1 has almost none": any split
 * leaves the result unchanged), a request's tiles that several SMs took merged by a
 * second kernel.
 *   q            device bf16 [num_tokens, num_q_heads, 576].
 *   cache        device bf16 [num_blocks, 16, 576].
 *   out          device bf16 [num_tokens, num_q_heads, 512].
 *   lse_out      device fp32 [num_tokens, num_q_heads] or NULL, as pkv_attention_varlen.
 *   softmax_scale  finite, > 0 (else PKV_ERR_UNSUPPORTED).
 *   workspace    >= pkv_latent_workspace_bytes(device) bytes, 256-byte aligned, of any
 *                contents; calls that may overlap on the GPU need one each.
 * What a row does not see never reaches it.  A row that sees a NaN or +inf score is NaN.  A
 * score of -inf weighs 0: where such a key holds an infinity, that element of the rows that
 * see it is NaN (0 times it); a row with no other scores is 0 elsewhere, its log-sum-exp
 * -inf.  Sums of weighted values are fp32, and tensor cores cut them off: with all weights and
 * signs alike an element is short by 1e-4 of itself where an SM takes 2^18 keys of a request,
 * 2e-3 for 2^20, 1.5e-2 for 2^22.  num_q_heads <= 4096, num_seqs <= 65535, num_tokens *
 * num_q_heads and num_blocks * 16 < 2^31 (else PKV_ERR_UNSUPPORTED); a context is at most 2^30
 * keys.  The rest as pkv_attention_varlen.
 */
pkv_status pkv_latent_attention_varlen(const void* q, const void* cache, void* out,
                                       float* lse_out, const int32_t* query_start_loc,
                                       const int32_t* seq_lens, const int32_t* block_table,
                                       int max_blocks_per_seq, int num_seqs, int64_t num_tokens,
                                       int max_query_len, int max_seq_len, int num_q_heads,
                                       int block_size, float softmax_scale, int causal,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* error_flag, int64_t num_blocks, void* stream);

/*
 * pkv_expanded_attention_varlen - attention in the expanded form.
 *
 * For requests of many new tokens, whose expanded keys and values cost less than
 * scores of 576 elements: keys [k[j, h] | k_rope[j]] of 128 + 64 elements,
 *   out[t, h, :] = sum_j softmax_j(softmax_scale * q[t, h, :] . key_j) v[j, h, :].
 * Keys and values are contiguous, not paged: request r has rows key_start_loc[r] ..
 * key_start_loc[r + 1] - 1 of them, m of them, and n new tokens; with causal != 0
 * its new token i sees keys 0 .. m - n + i (none where that is negative), otherwise
 * all m.  A row that sees no key has output 0 and log-sum-exp -inf.
 *   q        bf16 [num_tokens, num_q_heads, 192], dense.
 *   k, v     bf16 [num_keys, num_q_heads, 128]; strides given, > 0.
 *   k_rope   bf16 [num_keys, 64] (head_stride unused); not looked at, nor k and v,
 *            with num_keys == 0.
 *   out      bf16 [num_tokens, num_q_heads, 128], dense.
 *   lse_out  fp32 [num_tokens, num_q_heads] or NULL.
 *   query_start_loc, key_start_loc  device int32 [num_seqs + 1], nondecreasing, [0] =
 *            0, the last <= num_tokens, num_keys (PKV_FLAG_BAD_LENGTHS).
 *   max_query_len, max_key_len  host, >= every n and every m (PKV_FLAG_BAD_LENGTHS).
 *   softmax_scale  finite, > 0 (else PKV_ERR_UNSUPPORTED).
 * Runs on tcgen05 tensor cores, P rounded to bf16 for its product.  What rows other than
 * a request's own keys hold never reaches its rows, nor a later key one that does not see
 * it; infinities and NaN that a row sees reach it (an infinity whose weight rounds to 0 as
 * itself or as a NaN).  Where query_start_loc decreases, any row may be left unwritten.  Sums
 * are cut off as in the absorbed form, over all of a request's keys.  num_q_heads <= 4096,
 * num_seqs <= 65535, num_tokens * num_q_heads < 2^31 and num_keys <= 2^30 (else
 * PKV_ERR_UNSUPPORTED).
 */
pkv_status pkv_expanded_attention_varlen(const void* q, const pkv_rows* k,
                                         const pkv_rows* k_rope, const pkv_rows* v, void* out,
                                         float* lse_out, const int32_t* query_start_loc,
                                         const int32_t* key_start_loc, int num_seqs,
                                         int64_t num_tokens, int64_t num_keys, int max_query_len,
                                         int max_key_len, int num_q_heads, float softmax_scale,
                                         int causal, int32_t* error_flag, void* stream);

/*
 * pkv_stage_inputs - copy a step's packed inputs into device memory.
 *
 * "Inside the engine: kernels, CUDA graphs and the life of a request",
 * section on CUDA graphs (a captured step runs on fixed buffers, so each
 * step's inputs are copied into them first), and "Model execution", section
 * "Flattening a step" (the step's inputs are copied to the device
 * asynchronously; nothing waits for them on the host).  One kernel copies
 * nbytes from src to dst with the device's own loads: src may be pinned host
 * memory mapped into the device's address space (the loads cross the host
 * link) or device memory.  The kernel lets the next kernel on the stream
 * launch at once, and that kernel's dependency wait returns only after the
 * copy is complete, so a step's attention kernels overlap their set-up with
 * the transfer.  It starts copying after earlier work on the stream ends.
 *
 *   dst     device memory, 16-byte aligned, nbytes long.
 *   src     device-accessible memory, 16-byte aligned, nbytes long, not
 *           overlapping dst.
 *   nbytes  a multiple of 16 (else PKV_ERR_INVALID_ARG); 0 is a no-op.
 * Returns PKV_OK, PKV_ERR_INVALID_ARG (null or misaligned pointer, bad size)
 * or PKV_ERR_CUDA (launch failure).
 */
pkv_status pkv_stage_inputs(void* dst, const void* src, int64_t nbytes, void* stream);

/*
 * pkv_num_splits - how many KV splits the decode path should use.
 *
 * "Inside the engine ...", section "Prefill has a full grid; decode at batch 1
 * has almost none": split the KV axis when there are too few query rows to
 * fill the GPU; at high batch the grid is already full and the split is
 * turned off.  With U = num_seqs x num_kv_heads x row tiles of decode work
 * units and C the decode CTAs device `device` holds at once (SM count x
 * resident CTAs per SM), T = floor(7 C / 8): max(1, floor(T / U)), so one
 * wave of split CTAs leaves some SMs free for the combine kernel and the next
 * launch to start early (1 once the grid is nearly full);
 * never fewer than 8 blocks (128 keys) per split nor more than 64 splits.
 * Returns 0 for invalid arguments or device.
 */
int pkv_num_splits(int num_seqs, int max_query_len, int max_seq_len, int num_q_heads,
                   int num_kv_heads, int head_dim, int device);

/*
 * pkv_num_splits_e2m1 - the same for pkv_attention_varlen_e2m1, whose tiles hold
 * 8 rows (two CTAs fit an SM) or 16 (one).  A request has G query heads to a KV
 * head x max_query_len rows (1 token where max_query_len > PKV_DECODE_MAX_QLEN),
 * B blocks of max_seq_len; tiles of 16 rows are taken where it has more than 8 and
 * num_seqs x num_kv_heads x its tiles x max(1, B / 32) exceeds the SMs.  With U
 * units as above, s = min(B / 8, 7/8 SMs / U); where that leaves a split more than 64
 * blocks, s = min(CTA slots / U, max(s, B / 32)); at most 64, and 1 where the
 * split would not save B (s - 1) / s >= 48 blocks.  Returns 0 for invalid
 * arguments or device.
 */
int pkv_num_splits_e2m1(int num_seqs, int max_query_len, int max_seq_len, int num_q_heads,
                        int num_kv_heads, int head_dim, int device);

/*
 * pkv_workspace_bytes - device workspace pkv_attention_varlen needs.
 *
 * Holds the split-KV partials of the decode path: for every split, request,
 * decode row (< PKV_DECODE_MAX_QLEN) and query head, an fp32 partial output
 * [head_dim] and its log-sum-exp.  0 when num_splits <= 1.
 */
size_t pkv_workspace_bytes(int num_seqs, int num_q_heads, int head_dim, int num_splits);

/*
 * pkv_attention_varlen - attention of a flat varlen batch over the paged cache.
 *
 * For request r (0 <= r < num_seqs), n = query_start_loc[r+1] -
 * query_start_loc[r] new tokens occupy rows query_start_loc[r]..+n-1 of q and
 * out, and L = seq_lens[r] is its context after this step (its new tokens
 * already written, e.g. by pkv_write).  New token i is at position
 * p = L - n + i; with causal != 0 it attends keys 0..p, otherwise all L keys.
 * Key j of request r is cache row block_table[r * max_blocks_per_seq + j/16]
 * * 16 + j % 16, kv head h / (num_q_heads / num_kv_heads) for query head h.
 *   out[t, h, :] = sum_j softmax_j(softmax_scale * q[t,h,:] . k_j) v_j
 * computed as an online softmax over key tiles ("Never materialise the TxT
 * matrix"); requests with n <= PKV_DECODE_MAX_QLEN take the split-KV decode
 * kernel (partials merged by a log-sum-exp combine kernel when num_splits >
 * 1), longer ones the tiled prefill kernel: on tensor cores for bf16 at
 * head_dim 64 or 128 (two query heads of a KV head per CTA, or with an odd
 * GQA group two query tiles of one head; an E4M3 cache through
 * pkv_attention_varlen_e4m3 at head_dim 128), else on the decode kernel's
 * CUDA-core 16-row tiles.
 *
 *   q, out            device [num_tokens, num_q_heads, head_dim], dtype.
 *   lse_out           device fp32 [num_tokens, num_q_heads] or NULL: natural-log
 *                     log-sum-exp of each row's scaled scores (-inf if the row
 *                     sees no key).
 *   k_cache, v_cache  device [num_blocks, 16, num_kv_heads, head_dim], dtype.
 *   query_start_loc   device int32 [num_seqs + 1], nondecreasing, [0] = 0,
 *                     [num_seqs] <= num_tokens (rows of q/out past it, such
 *                     as a captured graph's padding rows, are neither read
 *                     nor written).
 *   seq_lens          device int32 [num_seqs].
 *   block_table       device int32 [num_seqs, max_blocks_per_seq].
 *   max_query_len     host: >= every n (bounds the prefill grid).
 *   max_seq_len       host: >= every L, <= 16 * max_blocks_per_seq (sizes the
 *                     split heuristic and the pre-launch L2 warm-up; a larger
 *                     value returns PKV_ERR_INVALID_ARG).  A seq_len beyond the
 *                     table row is flagged on the device (PKV_FLAG_BAD_LENGTHS).
 *   num_splits        0 = pkv_num_splits(...); else 1..64.
 *   workspace         device, >= pkv_workspace_bytes(num_seqs, num_q_heads,
 *                     head_dim, splits) bytes, 256-byte aligned; may be NULL
 *                     when that is 0.  Contents need no initialisation.
 * Rows of requests with n == 0 are absent; a request with L == 0 and n == 0
 * is a no-op.  Returns PKV_OK once the kernels are enqueued.
 */
pkv_status pkv_attention_varlen(const void* q, const void* k_cache, const void* v_cache,
                                void* out, float* lse_out, const int32_t* query_start_loc,
                                const int32_t* seq_lens, const int32_t* block_table,
                                int max_blocks_per_seq, int num_seqs, int64_t num_tokens,
                                int max_query_len, int max_seq_len, int num_q_heads,
                                int num_kv_heads, int head_dim, int block_size,
                                float softmax_scale, int causal, int num_splits,
                                void* workspace, size_t workspace_bytes, int32_t* error_flag,
                                int64_t num_blocks, pkv_dtype dtype, void* stream);

/*
 * pkv_write_attention_varlen - pkv_write then pkv_attention_varlen, as one
 * call.
 *
 * The same two steps ("Model execution", section "Flattening a step": the
 * new tokens' K/V go to their slots, then attention reads the cache).  When
 * every request is decode-class (max_query_len <= PKV_DECODE_MAX_QLEN) the
 * write rides in the decode kernel: each CTA stores the new-token rows it is
 * about to read (a bounded barrier orders the stores before its TMA loads of
 * them), so the step is one launch fewer.  Otherwise pkv_write runs first.
 *   k_new, v_new, slot_mapping: as pkv_write (q's dtype).  The other
 *   arguments as pkv_attention_varlen.  On the fused path only the tokens of
 *   rows below query_start_loc[num_seqs] are stored (padding rows carry slot
 *   -1 anyway); a slot past the cache is skipped and flagged
 *   PKV_FLAG_BAD_SLOT.  The cache contents after the call are those of the
 *   two separate calls.
 */
pkv_status pkv_write_attention_varlen(
    const void* k_new, const void* v_new, const int64_t* slot_mapping, const void* q,
    void* k_cache, void* v_cache, void* out, float* lse_out, const int32_t* query_start_loc,
    const int32_t* seq_lens, const int32_t* block_table, int max_blocks_per_seq, int num_seqs,
    int64_t num_tokens, int max_query_len, int max_seq_len, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float softmax_scale, int causal, int num_splits,
    void* workspace, size_t workspace_bytes, int32_t* error_flag, int64_t num_blocks,
    pkv_dtype dtype, void* stream);

/*
 * pkv_attention_varlen_window - pkv_attention_varlen with a sliding window.
 *
 * "Anatomy of a serving engine", section "Where it breaks": sliding-window
 * attention is a variant some backends support; the pages give no
 * definition.  Reading taken: with window W > 0 the new token at position
 * p = L - n + i sees only keys j with p - W < j (the W most recent
 * positions, itself included), on top of the causal limit j <= p (or j < L
 * with causal == 0).  window == 0 is pkv_attention_varlen exactly, and so is
 * any window >= max_seq_len (it excludes no key; the call runs as window 0).  Key
 * blocks wholly below a tile's window start are not read, and the automatic
 * split count is sized for a context of window + PKV_DECODE_MAX_QLEN keys.
 * Windows shorter than 128 keys run every request on the split-KV kernel's
 * CUDA-core tiles (fp32 P) instead of the tensor-core prefill.
 *   window  >= 0 (negative: PKV_ERR_INVALID_ARG).
 * Everything else as pkv_attention_varlen.
 */
pkv_status pkv_attention_varlen_window(const void* q, const void* k_cache, const void* v_cache,
                                       void* out, float* lse_out,
                                       const int32_t* query_start_loc, const int32_t* seq_lens,
                                       const int32_t* block_table, int max_blocks_per_seq,
                                       int num_seqs, int64_t num_tokens, int max_query_len,
                                       int max_seq_len, int num_q_heads, int num_kv_heads,
                                       int head_dim, int block_size, float softmax_scale,
                                       int causal, int window, int num_splits, void* workspace,
                                       size_t workspace_bytes, int32_t* error_flag,
                                       int64_t num_blocks, pkv_dtype dtype, void* stream);

/*
 * pkv_attention_varlen_e4m3 - pkv_attention_varlen over an E4M3 cache.
 *
 * The cache format of pkv_write_e4m3: key j stands for k_scale * value(code),
 * value j for v_scale * value(code), so
 *   out[t, h, :] = v_scale * sum_j softmax_j(softmax_scale * k_scale *
 *                  q[t,h,:] . value(K code_j)) value(V code_j)
 * (lse_out: the natural-log log-sum-exp of those scaled scores).  At head_dim
 * 128 the contractions run on tensor cores with fp32 accumulation and P
 * rounded to f16 for P.V.  V codes are widened exactly to f16.  K codes are
 * widened too, with q scaled by a power of two into f16, in split decode
 * launches without a window (the latency-bound form, which fetches each
 * split's first block speculatively) and in tiles of 16 rows; otherwise they
 * enter E4M3 MMAs as they are, against each q row scaled by a power of two
 * and split into two E4M3 terms (exact for every element within 2^9 of
 * the row's largest).  That is the decode kernel's mma.sync tiles for decode
 * rows; longer requests take the tcgen05 prefill tiles (codes widened in
 * shared memory, each q row rewritten as f16 scaled so its largest magnitude
 * lies in [2^14, 2^15)).  At head_dim 64 the codes are widened to fp32 in
 * registers on CUDA cores.
 *   q, out            device bf16 [num_tokens, num_q_heads, head_dim].
 *   k_cache, v_cache  device uint8 [num_blocks, 16, num_kv_heads, head_dim].
 *   k_scale, v_scale  finite, > 0 (else PKV_ERR_INVALID_ARG).
 * Everything else as pkv_attention_varlen, workspace included: requests with
 * n > PKV_DECODE_MAX_QLEN take the tensor-core prefill where the bf16 call's
 * would at head_dim 128 (a positive softmax_scale, no window below 128 keys),
 * else the decode kernel's CUDA-core tiles.
 */
pkv_status pkv_attention_varlen_e4m3(const void* q, const void* k_cache, const void* v_cache,
                                     void* out, float* lse_out, const int32_t* query_start_loc,
                                     const int32_t* seq_lens, const int32_t* block_table,
                                     int max_blocks_per_seq, int num_seqs, int64_t num_tokens,
                                     int max_query_len, int max_seq_len, int num_q_heads,
                                     int num_kv_heads, int head_dim, int block_size,
                                     float softmax_scale, float k_scale, float v_scale, int causal,
                                     int num_splits, void* workspace, size_t workspace_bytes,
                                     int32_t* error_flag, int64_t num_blocks, void* stream);

/*
 * pkv_attention_varlen_e4m3_window - pkv_attention_varlen_e4m3 with a sliding
 * window: the row at position p keeps keys j with p - window < j, on top of
 * the causal limit, as pkv_attention_varlen_window.
 *   window  >= 0 (0: no window; negative: PKV_ERR_INVALID_ARG).
 * Everything else as pkv_attention_varlen_e4m3.
 */
pkv_status pkv_attention_varlen_e4m3_window(
    const void* q, const void* k_cache, const void* v_cache, void* out, float* lse_out,
    const int32_t* query_start_loc, const int32_t* seq_lens, const int32_t* block_table,
    int max_blocks_per_seq, int num_seqs, int64_t num_tokens, int max_query_len, int max_seq_len,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, float softmax_scale,
    float k_scale, float v_scale, int causal, int window, int num_splits, void* workspace,
    size_t workspace_bytes, int32_t* error_flag, int64_t num_blocks, void* stream);

/*
 * pkv_write_attention_varlen_e4m3 - pkv_write_e4m3 then
 * pkv_attention_varlen_e4m3, as one call: the write rides in the decode
 * kernel (quantising bf16 rows with k_scale / v_scale as pkv_write_e4m3
 * does) when every request is decode-class, as for
 * pkv_write_attention_varlen.  k_new, v_new: bf16 [num_tokens,
 * num_kv_heads, head_dim].  Other arguments as pkv_attention_varlen_e4m3.
 */
pkv_status pkv_write_attention_varlen_e4m3(
    const void* k_new, const void* v_new, const int64_t* slot_mapping, const void* q,
    void* k_cache, void* v_cache, void* out, float* lse_out, const int32_t* query_start_loc,
    const int32_t* seq_lens, const int32_t* block_table, int max_blocks_per_seq, int num_seqs,
    int64_t num_tokens, int max_query_len, int max_seq_len, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float softmax_scale, float k_scale, float v_scale, int causal,
    int num_splits, void* workspace, size_t workspace_bytes, int32_t* error_flag,
    int64_t num_blocks, void* stream);

/*
 * pkv_attention_varlen_e2m1 - pkv_attention_varlen over an E2M1 cache.
 *
 * The cache format of pkv_write_e2m1; with K and V the products value(s) *
 * value(c) of key j,
 *   out[t, h, :] = v_scale * sum_j softmax_j(softmax_scale * k_scale *
 *                  q[t,h,:] . K_j) V_j
 * (lse_out: the natural-log log-sum-exp of those scaled scores).  The products
 * are widened exactly to f16; each q row enters as f16 scaled by a power of two
 * (its largest magnitude in [2^14, 2^15): exact for every element within 2^31
 * of it); both contractions run on tensor cores with fp32 accumulation, P
 * rounded to f16 for P.V (decode tiles divide by the sum of the rounded P, prefill
 * tiles by the sum of P before rounding: within 2^-11 of one another).  A row that
 * sees a NaN score has a NaN output and log-sum-exp at any num_splits; one that
 * sees a NaN V scale, NaN in its 16 dims alone.  Requests with n > PKV_DECODE_MAX_QLEN take the
 * tcgen05 prefill tiles (pages widened in shared memory) at a positive
 * softmax_scale without a window below 128 keys, else the decode kernel's 16-row
 * tiles; PKV_ERR_UNSUPPORTED for more than 65535 KV heads, on those tiles for
 * more than 524280 rows (query heads of a KV head x max_query_len) a request, and
 * for more than 1048560 decode rows (x min(max_query_len, PKV_DECODE_MAX_QLEN)).
 *   q, out            device bf16 [num_tokens, num_q_heads, head_dim].
 *   k_cache, v_cache  device, [num_blocks, num_kv_heads, 9 * head_dim] bytes.
 *   k_scale, v_scale  finite, > 0 (else PKV_ERR_INVALID_ARG).
 *   window            0: none; > 0: the row at position p keeps keys j with
 *                     p - window < j, on top of the causal limit, as
 *                     pkv_attention_varlen_window; < 0: PKV_ERR_INVALID_ARG.
 *   num_splits        0 = pkv_num_splits_e2m1(...) (with a window, for a context
 *                     of window + PKV_DECODE_MAX_QLEN keys); else 1..64.
 * What cache slots hold that a row may not see (behind a context, after its
 * position, before its window) never reaches the row, NaN scales included.
 * Everything else as pkv_attention_varlen, workspace included.
 */
pkv_status pkv_attention_varlen_e2m1(const void* q, const void* k_cache, const void* v_cache,
                                     void* out, float* lse_out, const int32_t* query_start_loc,
                                     const int32_t* seq_lens, const int32_t* block_table,
                                     int max_blocks_per_seq, int num_seqs, int64_t num_tokens,
                                     int max_query_len, int max_seq_len, int num_q_heads,
                                     int num_kv_heads, int head_dim, int block_size,
                                     float softmax_scale, float k_scale, float v_scale, int causal,
                                     int window, int num_splits, void* workspace,
                                     size_t workspace_bytes, int32_t* error_flag,
                                     int64_t num_blocks, void* stream);

/*
 * pkv_write_attention_varlen_e2m1 - pkv_write_e2m1 (bf16 rows) then
 * pkv_attention_varlen_e2m1, as one call: every argument is checked before
 * anything is enqueued, and the write rides in the decode kernel when every
 * request is decode-class, as for pkv_write_attention_varlen (there, the rows
 * of tokens at or behind query_start_loc[num_seqs], and of requests flagged
 * PKV_FLAG_BAD_LENGTHS, are not stored).
 */
pkv_status pkv_write_attention_varlen_e2m1(
    const void* k_new, const void* v_new, const int64_t* slot_mapping, const void* q,
    void* k_cache, void* v_cache, void* out, float* lse_out, const int32_t* query_start_loc,
    const int32_t* seq_lens, const int32_t* block_table, int max_blocks_per_seq, int num_seqs,
    int64_t num_tokens, int max_query_len, int max_seq_len, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float softmax_scale, float k_scale, float v_scale, int causal,
    int window, int num_splits, void* workspace, size_t workspace_bytes, int32_t* error_flag,
    int64_t num_blocks, void* stream);

/*
 * pkv_attention_varlen_noalloc - pkv_attention_varlen without a caller
 * workspace.
 *
 * The pages have no counterpart to this entry point; it exists for callers
 * that cannot allocate device memory (for example a plain C host program
 * whose device memory is owned by another runtime's caching allocator, or a
 * path that must never block in cudaMalloc/cudaFree).  The split-KV partials
 * live in a fixed 8 MiB array compiled into the library (held on every GPU
 * that loads it until the process exits); the call allocates nothing.
 *   Arguments are those of pkv_attention_varlen minus the workspace.  With
 *   num_splits == 0 the automatic split count is lowered until its partials
 *   (pkv_workspace_bytes) fit in 8 MiB; an explicit num_splits whose partials
 *   exceed 8 MiB returns PKV_ERR_WORKSPACE and enqueues nothing.
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current): make it before any
 *   stream capture.  Host threads may make first calls concurrently (the
 *   cached address is atomic).  All calls on a device share the array, so
 *   calls whose kernels overlap on the GPU race; serialise them.
 */
pkv_status pkv_attention_varlen_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                        void* out, float* lse_out,
                                        const int32_t* query_start_loc, const int32_t* seq_lens,
                                        const int32_t* block_table, int max_blocks_per_seq,
                                        int num_seqs, int64_t num_tokens, int max_query_len,
                                        int max_seq_len, int num_q_heads, int num_kv_heads,
                                        int head_dim, int block_size, float softmax_scale,
                                        int causal, int num_splits, int32_t* error_flag,
                                        int64_t num_blocks, pkv_dtype dtype, void* stream);

/*
 * Shared-prefix (cascade) attention.
 *
 * "Anatomy of a serving engine", section "Capacity belongs to the KV cache
 * manager": paged blocks let requests share the blocks of a common prefix.
 * Here every request of the batch starts with the same shared_blocks blocks
 * (P = 16 * shared_blocks keys, named by shared_block_table) followed by its
 * own suffix_lens[r] keys (suffix_block_table row r); its context is
 * L = P + suffix_lens[r] and its n new tokens are the last n of them, all in
 * its own part (n <= suffix_lens[r], else PKV_FLAG_BAD_LENGTHS).  The result
 * is that of pkv_attention_varlen (causal) with the table shared ++ own.
 * It is computed as the key axis split in two ("Inside the engine ...",
 * section "Prefill has a full grid; decode at batch 1 has almost none": a
 * split of the keys changes nothing about the result): every row of the
 * batch over the prefix at once (all prefix keys are visible to every new
 * row; the prefix is read from HBM once for all requests, split
 * prefix_splits ways over the key axis), each request over its own keys,
 * and a log-sum-exp merge of the prefix_splits + 1 partials per row.  The
 * prefix pass runs on the tensor cores for bf16 at head_dim 64 or 128 (E4M3
 * caches at 128, pkv_cascade_attention_e4m3) with an even GQA group that
 * divides 128 (each 128-row tile holds 128 / group tokens with their whole
 * group, so one K/V tile feeds every head of the KV head) and a positive
 * softmax_scale, else on the split-KV kernel's CUDA-core tiles; the own-key
 * pass runs on the decode kernel and the merge on CUDA cores.
 */

/* pkv_cascade_splits - prefix splits for num_tokens rows over shared_blocks
 * blocks: max(1, min(floor(T / U), cap, 63)) with T = floor(7 x SMs / 8).
 * Tensor-core prefix pass (bf16, head_dim 64 or 128, even GQA group dividing
 * 128): U = num_kv_heads x ceil(group x num_tokens / 256) row tiles, cap =
 * ceil(shared_blocks / 32) - each split at least four 128-key tiles (fewer
 * leave the pass short of its pipelined steady state).  CUDA-core pass
 * (otherwise): U = num_kv_heads x ceil(group x num_tokens / 16), cap =
 * floor(shared_blocks / 8).  0 when shared_blocks == 0; -1 for invalid
 * arguments or device. */
int pkv_cascade_splits(int64_t num_tokens, int shared_blocks, int num_q_heads, int num_kv_heads,
                       int head_dim, pkv_dtype dtype, int device);

/* pkv_cascade_workspace_bytes - device workspace pkv_cascade_attention needs:
 * fp32 partial outputs [prefix_splits + 1][num_tokens][num_q_heads][head_dim]
 * and their log-sum-exps, each 256-byte aligned. */
size_t pkv_cascade_workspace_bytes(int64_t num_tokens, int num_q_heads, int head_dim,
                                   int prefix_splits);

/*
 * pkv_cascade_attention - attention of a batch sharing a block-aligned prefix.
 *
 *   q, out, lse_out, query_start_loc, num_seqs, num_tokens, max_query_len,
 *   heads, head_dim, block_size, softmax_scale, error_flag, num_blocks,
 *   dtype, stream: as pkv_attention_varlen.
 *   suffix_lens         device int32 [num_seqs]: keys after the prefix.
 *   suffix_block_table  device int32 [num_seqs, max_blocks_per_seq]: the
 *                       blocks of those keys.
 *   shared_block_table  device int32 [shared_blocks] (NULL when 0 blocks).
 *   max_suffix_len      host, >= every suffix_lens[r] and <= 16 *
 *                       max_blocks_per_seq (else PKV_ERR_INVALID_ARG).
 *   prefix_splits       0 = pkv_cascade_splits(...); else 1..63.
 *   workspace           device, >= pkv_cascade_workspace_bytes(num_tokens,
 *                       num_q_heads, head_dim, splits), 256-byte aligned
 *                       (splits = 0 when shared_blocks == 0).
 * Rows of out past query_start_loc[num_seqs] are not written (the prefix
 * pass reads every q row below num_tokens).
 */
pkv_status pkv_cascade_attention(const void* q, const void* k_cache, const void* v_cache,
                                 void* out, float* lse_out, const int32_t* query_start_loc,
                                 const int32_t* suffix_lens, const int32_t* suffix_block_table,
                                 int max_blocks_per_seq, const int32_t* shared_block_table,
                                 int shared_blocks, int num_seqs, int64_t num_tokens,
                                 int max_query_len, int max_suffix_len, int num_q_heads,
                                 int num_kv_heads, int head_dim, int block_size,
                                 float softmax_scale, int prefix_splits, void* workspace,
                                 size_t workspace_bytes, int32_t* error_flag, int64_t num_blocks,
                                 pkv_dtype dtype, void* stream);

/*
 * pkv_cascade_attention_e4m3 - pkv_cascade_attention over an E4M3 cache (the
 * format of pkv_write_e4m3; k_scale, v_scale finite and > 0, else
 * PKV_ERR_INVALID_ARG).  q and out are bf16.  At head_dim 128 the prefix
 * pass runs on the tensor-core prefill tiles where the bf16 call's would
 * (even GQA group dividing 128, positive softmax_scale; codes widened to f16,
 * q rows scaled to f16 by powers of two) and prefix_splits 0 takes
 * pkv_cascade_splits(..., PKV_BF16, ...); otherwise it runs on the split-KV
 * kernel's CUDA-core tiles and takes pkv_cascade_splits(..., PKV_F32, ...).
 * The own-key pass runs on the decode kernel (tensor cores at head_dim 128).
 * Everything else as pkv_cascade_attention.
 */
pkv_status pkv_cascade_attention_e4m3(
    const void* q, const void* k_cache, const void* v_cache, void* out, float* lse_out,
    const int32_t* query_start_loc, const int32_t* suffix_lens, const int32_t* suffix_block_table,
    int max_blocks_per_seq, const int32_t* shared_block_table, int shared_blocks, int num_seqs,
    int64_t num_tokens, int max_query_len, int max_suffix_len, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, float softmax_scale, float k_scale, float v_scale,
    int prefix_splits, void* workspace, size_t workspace_bytes, int32_t* error_flag,
    int64_t num_blocks, void* stream);

/*
 * pkv_build_metadata - the flat-batch metadata of one step, on the host.
 *
 * "Model execution", section "Flattening a step": the scheduled tokens of all
 * requests form one flat batch; query_start_loc holds the cumulative token
 * offsets, seq_lens the context after this step (computed + scheduled),
 * block_table each request's physical blocks, and slot_mapping the slot
 * block_id * block_size + offset of new token k of request r, which sits at
 * position computed[r] + k.  Host memory only; no CUDA call.
 *   computed, scheduled  host int32 [num_seqs], >= 0.
 *   block_offsets        host int32 [num_seqs + 1], [0] = 0, nondecreasing:
 *                        request r's blocks are block_ids[block_offsets[r] ..
 *                        block_offsets[r + 1]), at least ceil((computed +
 *                        scheduled) / block_size) of them, ids >= 0.
 *   max_blocks_per_seq   width of block_table, >= every request's block count.
 *   num_tokens           must equal the sum of scheduled.
 *   Outputs (host, caller-allocated): query_start_loc int32 [num_seqs + 1],
 *   seq_lens int32 [num_seqs], block_table int32 [num_seqs,
 *   max_blocks_per_seq] (unused entries 0), slot_mapping int64 [num_tokens],
 *   positions int64 [num_tokens] or NULL, max_query_len / max_seq_len host
 *   int32 or NULL.
 * Every argument is checked before anything is written; a violation returns
 * PKV_ERR_INVALID_ARG and writes nothing.
 */
pkv_status pkv_build_metadata(int num_seqs, const int32_t* computed, const int32_t* scheduled,
                              const int32_t* block_offsets, const int32_t* block_ids,
                              int block_size, int max_blocks_per_seq, int64_t num_tokens,
                              int32_t* query_start_loc, int32_t* seq_lens, int32_t* block_table,
                              int64_t* slot_mapping, int64_t* positions, int32_t* max_query_len,
                              int32_t* max_seq_len);

/* Static, human-readable name of a status code. */
const char* pkv_status_string(pkv_status status);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
