/*
 * sq.h -- C ABI of libsq: the fused quantized gated delta-rule decode step
 * over a per-request pool of low-bit recurrent states, for AMD MI355X (gfx950).
 *
 * Sources (cited by title and section):
 *   [P1] "K1 論文詳解" (k1-news, paper of 2026-10-09), STEPQuant article,
 *        sections 背景 (background), 方法 (method), 實驗結果 (results).
 *   [P5] "线性注意力状态量化难题:Qwen状态池70并发就超模型权重" (aitest123),
 *        sections 直接量化为什么会翻车, 时间维度, 空间维度, 工程落地.
 *
 * What one decode step computes, per request n (owning slot p = slot_ids[n])
 * and head h, on that head's d_k x d_v state S (rows = key dims, columns =
 * value dims, [P5] 空间维度):
 *     S^ = decode(tile(p, h))                   stored codes -> real state
 *     u  = S^T k
 *     S' = alpha S^ + beta k (v - alpha u)^T    = alpha (I - beta k k^T) S^ + beta k v^T
 *     o  = S'^T q                                readout, before requantization
 *     tile(p, h) = encode(S')                    requantize + repack, in place
 * The update is the gated delta rule ([P5] opening and 时间维度: decay by the
 * gate, correction along the current key); every step reads, updates,
 * requantizes and stores the state ([P5] 直接量化为什么会翻车).
 *
 * STATE FORMAT (public; the CPU reference implements it independently)
 *   head_bits[h] selects the storage of head h:
 *     4, 6, 8  integer codes q in [-Q, Q], Q = 2^(b-1) - 1 ([P5]
 *              直接量化为什么会翻车: 4/6/8-bit integers), stored as the
 *              unsigned field q + 2^(b-1);
 *     16       FP16 "pivot" head, IEEE binary16, unquantized ([P1] 方法;
 *              [P5] 时间维度: the riskiest heads stay FP16);
 *     32       FP32 state, unquantized (the full-precision baseline path);
 *     144      (SQ_BITS_BF16) bfloat16 state, unquantized, 16-bit fields: a
 *              16-bit baseline beside the FP32 state, not a format of the
 *              pages; S' is rounded to bfloat16 (half to even).
 *   Dequantization uses a per-key-row factor times a per-value-column factor
 *   ([P5] 空间维度; [P1] 方法): S^_ij = q_ij * s_ij, s_ij = fl32(r_i * c_j).
 *   Requantization: q = clamp(rne(S'_ij / s_ij), -Q, Q) (round half to even).
 *   FP16 pivots round S' to binary16 (half to even).
 *   Tile layout: element (i, j) is field number
 *       n = 16 * ((i/4) * (d_v/4) + j/4) + 4 * (j%4) + (i%4)
 *   (4x4 blocks in block-row order; inside a block the four rows of a column
 *   are consecutive), and field n occupies bits [n*w, n*w + w) of the tile
 *   read as a little-endian bit stream, w = head_bits[h] (16 for
 *   SQ_BITS_BF16).  So 4-bit codes sit
 *   two per byte and 6-bit codes four per three bytes; a tile is
 *   d_k*d_v*w/8 bytes.  A slot's slab holds heads 0..H-1 in order, each tile
 *   starting on a 256-byte boundary; slot p's slab starts at p * slab_bytes.
 *
 * CONVENTIONS
 *   - Every function returns an sq_status (int); nothing throws across the ABI.
 *   - Host-checkable argument errors are reported before any HIP call is made.
 *   - Device pointers are borrowed: the caller allocates and frees them (for
 *     example as torch tensors).  The library owns only the sq_pool object and
 *     the small device tables it allocates in sq_pool_alloc.
 *   - All device work is enqueued on the caller's stream (a hipStream_t passed
 *     as void*, NULL = the null stream); no call synchronizes.  Results are
 *     visible after the caller synchronizes that stream.  Calls that touch the
 *     same pool must be ordered on one stream.
 *   - A pool lives on the device that was current at sq_pool_alloc.  Calls
 *     that enqueue work on it must be made with that device current (else
 *     SQ_ERR_INVALID, nothing enqueued); sq_pool_free switches to it itself.
 *     Calls without a pool (sq_prefill, sq_block_tables, sq_kv_append,
 *     sq_paged_attention) run on the current device, which must be the one
 *     their buffers and stream belong to; this is not checked.
 *   - A slot must not appear twice in one slot_ids batch: two workgroups would
 *     update the same tile (undefined result).  The step does not check slot
 *     ids on the device; sq_check_slots does, as a separate call, and the
 *     SQ_CHECK switch below makes every call check them on the host.
 *   - Non-finite inputs (alpha, beta, q, k, v, scales) are a caller error.  The
 *     result is defined on the updated value as the kernel evaluates it: a
 *     NaN quotient S'/s becomes code 0, +-Inf the nearest bound +-Q; FP16,
 *     BF16 and FP32 heads store the non-finite value.  The pages say nothing
 *     of non-finite values; this rule is a reading.  A NaN or infinite gate,
 *     write strength, key or value element gives the same stored result
 *     in any evaluation order; an infinite gate does not (its codes are
 *     then unspecified within [-Q, Q]).  A non-finite query only reaches the
 *     readout o.  Whenever a stored value comes from a non-finite one, the
 *     pool's sticky flag is set (sq_pool_last_device_error).  The d = 128
 *     code-tile kernel takes that decision on the update's factors (the
 *     gate, beta k_i / r_i, (v_j - alpha u_j) / c_j), the others on each
 *     value; the two agree unless finite factors overflow fp32 in their
 *     product, which takes step sizes near the bottom of the fp32 range.
 *   - d_k and d_v must be multiples of 4 and at most 256; d_k = d_v = 128 takes
 *     the tuned kernels, other shapes a plain one.
 *
 * SWITCHES (environment variables, read once per pool by sq_pool_alloc; a
 * pool keeps what it read)
 *   SQ_CHECK   set and not "0": every call that takes slot ids (store, load,
 *              the steps, readout) first copies the ids to the
 *              host, synchronizing the caller's stream, and returns
 *              SQ_ERR_INVALID before any kernel is enqueued if an id is
 *              outside [0, n_slots) or, for the calls that write the pool
 *              (store and the steps), appears twice.  A debugging aid: it
 *              costs a synchronization per call and cannot be used under
 *              graph capture.
 *   SQ_KERNEL  unset, empty or "tuned": d_k = d_v = 128 takes the tuned
 *              kernels.  "generic": every shape takes the plain per-width
 *              kernels, so that the tuned ones can be checked against a second
 *              implementation on the same data.  Any other value makes
 *              sq_pool_alloc return SQ_ERR_INVALID (before any HIP call).
 */
#ifndef SQ_H
#define SQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sq_pool sq_pool; /* opaque handle */

#define SQ_BITS_BF16 144 /* head_bits value of a bfloat16 state */

typedef enum {
    SQ_OK = 0,
    SQ_ERR_INVALID = -1,     /* null pointer, bad size, misaligned pointer, buffer too small */
    SQ_ERR_UNSUPPORTED = -2, /* head_bits not in {4,6,8,16,32,144}, or d_k/d_v not supported */
    SQ_ERR_HIP = -3,         /* a HIP runtime call or kernel launch failed */
    SQ_ERR_NOMEM = -4,       /* host or device allocation of the pool's tables failed */
    SQ_ERR_DEVICE = -5       /* sq_pool_last_device_error: a kernel met a non-finite value */
} sq_status;

typedef enum {
    SQ_F32 = 0, /* IEEE binary32 */
    SQ_BF16 = 1 /* bfloat16, upcast exactly to fp32 on load */
} sq_dtype;

typedef struct {
    int32_t n_slots;          /* number of resident request states (slots), >= 1 */
    int32_t n_heads;          /* recurrent heads per request, >= 1 */
    int32_t d_k, d_v;         /* state rows (key dims) and columns (value dims) */
    const uint8_t *head_bits; /* HOST [n_heads], each in {4, 6, 8, 16, 32, 144}; copied */
    const float *row_scale;   /* DEVICE fp32, r_i > 0: [n_heads][d_k], or with a slot stride
                                 S the factors of slot p, head h at row_scale + (p*S + h)*d_k;
                                 borrowed, read by every call; entries of unquantized heads
                                 are ignored */
    const float *col_scale;   /* DEVICE fp32, c_j > 0: [n_heads][d_v], or at
                                 col_scale + (p*S + h)*d_v; as row_scale */
    int64_t scale_slot_stride;/* S: 0 = one set of factors per head, shared by every slot;
                                 else S >= n_heads and every slot has its own factors
                                 ([P5] 空间维度: each row and each column of a state matrix
                                 has its own factor); the arrays then hold n_slots*S vectors */
    void *state;              /* DEVICE, 256-byte aligned, >= sq_pool_bytes(...) bytes,
                                 laid out as described above; borrowed */
    uint64_t state_bytes;     /* size of the state buffer in bytes */
} sq_pool_desc;

/* Bytes the state buffer needs for this shape: n_slots * slab_bytes.  One
 * resident state per request slot ([P1] 背景; [P5] opening: the pool grows
 * with concurrency), each head stored at its own width ([P5] 时间维度).
 * Returns 0 if any argument is invalid or unsupported.  Host only. */
uint64_t sq_pool_bytes(int32_t n_slots, int32_t n_heads, int32_t d_k, int32_t d_v,
                       const uint8_t *head_bits);

/* Validate desc, compute the tile offsets and upload them (and the per-width
 * head lists) to a small device table: the per-request state pool ([P1] 背景;
 * [P5] opening) with per-head widths and FP16 pivots ([P5] 时间维度) and
 * row x column factors ([P5] 空间维度).  On success *out receives a handle to
 * release with sq_pool_free.  Errors: SQ_ERR_INVALID (null desc/out/pointers,
 * n_slots or n_heads < 1, state not 256-byte aligned, scales not 16-byte
 * aligned, state_bytes too small, 0 < scale_slot_stride < n_heads, an
 * SQ_KERNEL value that names no kernel family), SQ_ERR_UNSUPPORTED (bits, d_k,
 * d_v), SQ_ERR_NOMEM, SQ_ERR_HIP.
 * Synchronous (uploads with a blocking copy). */
int sq_pool_alloc(const sq_pool_desc *desc, sq_pool **out);

/* Release the handle and its device table (not the borrowed buffers).
 * NULL is a no-op.  The caller must ensure no enqueued work still uses it. */
void sq_pool_free(sq_pool *pool);

/* Byte offset and size of tile (slot, head) inside the state buffer.
 * Host only; SQ_ERR_INVALID for a null pool/out pointer or out-of-range ids. */
int sq_pool_tile_offset(const sq_pool *pool, int32_t slot, int32_t head, uint64_t *offset,
                        uint64_t *bytes);

/* Quantize-and-store: encode fp32 states S (DEVICE, [n_req][n_heads][d_k][d_v],
 * row-major) into the tiles of slots slot_ids[0..n_req) (DEVICE int32), with
 * the quantizer and layout above (the hand-off of a state computed elsewhere,
 * e.g. at prefill).  n_req == 0 is a no-op.  Asynchronous on `stream`.
 * Errors as for sq_decode_step (S must be 16-byte aligned). */
int sq_pool_store(sq_pool *pool, const int32_t *slot_ids, int32_t n_req, const float *S,
                  void *stream);

/* Load-and-dequantize, the inverse of sq_pool_store: write the states of slots
 * slot_ids[0..n_req) (DEVICE int32) as fp32 S[n_req][n_heads][d_k][d_v]
 * (DEVICE, row-major, 16-byte aligned).  Each element is the stored value
 * rounded once to fp32: fl32(q * fl32(r_i c_j)) for codes, the binary16 value
 * for pivots, the stored value for FP32 heads.  The pool is not modified.
 * n_req == 0 is a no-op.  Asynchronous on `stream`.  (Calibration,
 * checkpoint export, inspection.)  Errors as for sq_pool_store. */
int sq_pool_load(const sq_pool *pool, const int32_t *slot_ids, int32_t n_req, float *S,
                 void *stream);

/* One fused decode step for a batch of n_req requests (see the top of this
 * file).  All pointers DEVICE, row-major:
 *   slot_ids int32 [n_req], each in [0, n_slots), no duplicates;
 *   q, k     [n_req][n_heads][d_k] of qkv_dtype (sq_dtype);
 *   v        [n_req][n_heads][d_v] of qkv_dtype;
 *   alpha, beta fp32 [n_req][n_heads] (gate in (0, 1], write strength in [0, 1]);
 *   o        fp32 [n_req][n_heads][d_v], written with S'^T q; may be NULL.
 * q/k/v/o must be 16-byte aligned.  The pool's tiles are updated in place.
 * n_req == 0 is a no-op.  Asynchronous on `stream`.
 * Errors: SQ_ERR_INVALID (null pool or required pointer, n_req < 0 or
 * > n_slots, qkv_dtype not an sq_dtype, misaligned pointer, another device
 * current), SQ_ERR_UNSUPPORTED (n_req * n_heads tiles exceed one launch
 * grid), SQ_ERR_HIP (a launch failed).  Device data (slot values, alpha,
 * beta, q/k/v) is not validated; see sq_check_slots for slot ids, and the
 * SQ_CHECK switch, under which an id out of range or repeated is
 * SQ_ERR_INVALID (the load and the readout accept repeated ids). */
int sq_decode_step(sq_pool *pool, const int32_t *slot_ids, int32_t n_req, const void *q,
                   const void *k, const void *v, int32_t qkv_dtype, const float *alpha,
                   const float *beta, float *o, void *stream);

/* The same step with a per-key-channel gate, for the second model family
 * ([P5] 直接量化为什么会翻车 names its gate KDA; the pages give no formula).
 * Reading taken: the gate is a vector alpha in (0, 1]^{d_k} that decays each
 * key row of the state before the delta correction,
 *     T  = diag(alpha) S^,   u = T^T k
 *     S' = T + beta k (v - u)^T  = (I - beta k k^T) diag(alpha) S^ + beta k v^T
 *     o  = S'^T q,           tile = encode(S')
 * which is sq_decode_step when all d_k entries of alpha are equal.  Arguments
 * as for sq_decode_step except
 *   alpha    fp32 [n_req][n_heads][d_k], DEVICE, 16-byte aligned.
 * Same errors; n_req == 0 is a no-op.  Asynchronous on `stream`. */
int sq_decode_step_kda(sq_pool *pool, const int32_t *slot_ids, int32_t n_req, const void *q,
                       const void *k, const void *v, int32_t qkv_dtype, const float *alpha,
                       const float *beta, float *o, void *stream);

/* The decode step without the delta correction, for recurrent layers that only
 * decay and write:
 *     S' = alpha S^ + beta k v^T,   o = S'^T q,   tile = encode(S')
 * Arguments, errors and formats as for sq_decode_step (alpha and beta fp32
 * [n_req][n_heads]).  n_req == 0 is a no-op.  Asynchronous on `stream`. */
int sq_decode_step_linear(sq_pool *pool, const int32_t *slot_ids, int32_t n_req, const void *q,
                          const void *k, const void *v, int32_t qkv_dtype, const float *alpha,
                          const float *beta, float *o, void *stream);

/* ------------------------------------------------------------------ prompts
 *
 * The prompt form of the recurrent layers: every token of n_seq sequences
 * through the state, for a state computed where the decode steps will go on
 * from it (pass S to sq_pool_store).  Sequence s is the packed tokens
 * [cu_seqlens[s], cu_seqlens[s + 1]); per token t and head h
 *     SQ_RULE_DELTA    S_t = alpha_t (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T
 *     SQ_RULE_LINEAR   S_t = alpha_t S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t
 * from S0 (or zero).  States, gates, sums and the products that feed a state
 * are fp32 or better; o is rounded once to its type. */
typedef enum {
    SQ_RULE_DELTA = 0, /* the rule of sq_decode_step */
    SQ_RULE_LINEAR = 1 /* the rule of sq_decode_step_linear */
} sq_rule;

typedef struct {
    int32_t n_seq;             /* sequences, >= 0 */
    int32_t n_tokens;          /* packed tokens of all sequences, 0 to 2^31 - 65 */
    int32_t n_heads;           /* value (and state) heads, >= 1 */
    int32_t n_k_heads;         /* query/key heads, a divisor of n_heads: head h
                                  reads query/key head h / (n_heads / n_k_heads) */
    int32_t d_k, d_v;          /* multiples of 4, at most 256 */
    int32_t dtype;             /* sq_dtype of q, k, v and o */
    int32_t rule;              /* sq_rule */
    const void *q, *k;         /* DEVICE [n_tokens][n_k_heads][d_k] */
    const void *v;             /* DEVICE [n_tokens][n_heads][d_v] */
    int64_t q_stride, k_stride, v_stride; /* elements between tokens (heads are
                                  contiguous inside a token), so that q, k and v
                                  may be parts of one wider buffer */
    const float *alpha, *beta; /* DEVICE fp32 [n_tokens][n_heads]: gate in [0, 1], write strength */
    const int32_t *cu_seqlens; /* DEVICE int32 [n_seq + 1], from 0 to n_tokens, never falling
                                  (equal neighbours are an empty sequence: S = S0) */
    const float *S0;           /* DEVICE fp32 [n_seq][n_heads][d_k][d_v], or NULL for zero */
    void *o;                   /* DEVICE [n_tokens][n_heads][d_v] of dtype */
    float *S;                  /* DEVICE fp32 [n_seq][n_heads][d_k][d_v], or NULL; may equal S0 */
    void *workspace;           /* DEVICE, 256-byte aligned, sq_prefill_workspace bytes; may be
                                  NULL where that is 0 */
    uint64_t workspace_bytes;
} sq_prefill_desc;

/* Bytes of workspace that sq_prefill needs for these sizes (0 if none, or if
 * an argument is invalid).  It grows with n_seq, n_tokens and n_heads: one
 * made for the largest call serves the smaller ones.  Host only. */
uint64_t sq_prefill_workspace(int32_t n_seq, int32_t n_tokens, int32_t n_heads, int32_t d_k,
                              int32_t d_v, int32_t dtype, int32_t rule);

/* Run the prompt form (above).  n_seq == 0 is a no-op; with n_tokens == 0, S
 * receives S0 (or zero).  Asynchronous on `stream`; the workspace is in use until
 * the call's work is done.  cu_seqlens is read on the device only: values
 * outside [0, n_tokens] are held to that range, nothing outside the buffers
 * is touched, but tokens that it assigns to two sequences, or to none, have
 * undefined outputs.  bfloat16 with d_k = d_v = 128, strides in multiples of
 * 8 elements (at most 2^23), 16-byte aligned q, k, v, o and more than 12 tokens a
 * sequence on average takes the chunked matrix kernel,
 * everything else a token-by-token one.  (So a long prompt goes ten times faster in
 * a call of its own than among many sequences of a token or two.)  o, S and the
 * workspace must not overlap the inputs, but S may be S0.  Non-finite inputs are a caller error:
 * they reach the outputs of their own sequence only, but in the chunked kernel
 * also those of earlier tokens of the same 64.  Errors: SQ_ERR_INVALID (null
 * or misaligned pointer, bad size, stride or enum, workspace too small),
 * SQ_ERR_UNSUPPORTED (d_k or d_v, n_tokens, or more tiles than one launch grid),
 * SQ_ERR_HIP. */
int sq_prefill(const sq_prefill_desc *desc, void *stream);

/* ------------------------------------------------------------- paged cache
 *
 * A key-value cache in pages of page_size tokens, for the softmax-attention
 * layers of a hybrid model.  Token position x of a request lies in page
 * block_table[request][x / page_size] at place x % page_size; its slot is
 * page * page_size + place.  FORMAT (public): keys
 *     k [n_pages][n_kv_heads][page_size][head_dim]
 * and values transposed inside the page,
 *     v [n_pages][n_kv_heads][head_dim][page_size]
 * (the order in which attention's second product takes them).  Pages may lie
 * anywhere in the pool and hold anything past a request's last token. */
typedef struct {
    void *k, *v;         /* DEVICE, 16-byte aligned; borrowed */
    int32_t n_pages;     /* >= 1 */
    int32_t page_size;   /* 16, 32, 64, 128 or 256 tokens */
    int32_t n_kv_heads;  /* >= 1 */
    int32_t head_dim;    /* 32, 64, 96, 128, 192 or 256 */
    int32_t dtype;       /* sq_dtype of the cache, and of the q, k, v, o that go with it */
} sq_kv_cache;

/* Block tables and slot maps of one step from the requests' lengths.  Request
 * i has ctx_lens[i] cached tokens and gets new_lens[i] more (both DEVICE int32
 * [n_req]); with P = page_size it holds ceil(ctx / P) pages, listed at the
 * start of its row, and needs ceil((ctx + new) / P).  All outputs DEVICE:
 *   block_table int32 [n_req][table_stride]: the missing pages are appended
 *               to each row, taken from free_pages (int32 [n_free]) in request
 *               order: request 0 takes the first ones; other entries stay;
 *   seq_lens    int32 [n_req]: ctx + new;
 *   cu_new      int32 [n_req + 1]: exclusive sums of new_lens (the cu_seqlens
 *               of sq_prefill);
 *   cu_pages    int32 [n_req + 1]: exclusive sums of the pages taken; the last
 *               entry is how many entries of free_pages are used up;
 *   slot_map    int64 [n_slots]: the slot of every new token, requests packed
 *               in order; entries after the last token are -1 (n_slots may
 *               be any capacity, for instance that of a captured graph);
 *   result      int32 [1]: 0, or a sum of 1 (a negative length, or more than
 *               2^31 - 1 tokens: the request is taken as empty), 2 (n_free
 *               pages are not enough), 4 (a row needs more than table_stride
 *               entries), 8 (n_slots is less than the new tokens).  Pages that
 *               are not to be had get -1 entries, their tokens slot -1.
 * Nothing is kept between calls.  n_req == 0 writes the two zero sums.
 * seq_lens, cu_new and cu_pages must not overlap the inputs.
 * Errors: SQ_ERR_INVALID (null or misaligned pointer, negative size, n_slots
 * above 2^31 - 1), SQ_ERR_UNSUPPORTED (page_size), SQ_ERR_HIP.  Asynchronous
 * on `stream`. */
int sq_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int32_t n_req,
                    int32_t page_size, const int32_t *free_pages, int32_t n_free,
                    int32_t *block_table, int64_t table_stride, int32_t *seq_lens, int32_t *cu_new,
                    int32_t *cu_pages, int64_t *slot_map, int64_t n_slots, int32_t *result,
                    void *stream);

/* Write the keys and values of n_tok tokens into the cache at slot_map[t]
 * (DEVICE int64 [n_tok]); a slot that is negative or past the cache is
 * skipped, and no slot may appear twice.  k, v: DEVICE
 * [n_tok][n_kv_heads][head_dim] of the cache's type, 16-byte aligned, tokens
 * k_stride / v_stride elements apart (a multiple of 16 bytes).  n_tok == 0 is a
 * no-op.  `cache` is a HOST struct, read during the call.
 * Errors: SQ_ERR_INVALID, SQ_ERR_UNSUPPORTED (page_size, head_dim, too many
 * tokens for a launch grid), SQ_ERR_HIP.  Asynchronous on `stream`. */
int sq_kv_append(const sq_kv_cache *cache, const void *k, const void *v, int64_t k_stride,
                 int64_t v_stride, const int64_t *slot_map, int32_t n_tok, void *stream);

/* Bytes of workspace for sq_paged_attention with at most n_req requests of at
 * most max_len tokens and any window (0 if none, or if an argument is
 * invalid).  Host only. */
uint64_t sq_paged_attention_workspace(const sq_kv_cache *cache, int32_t n_req, int32_t n_heads,
                                      int32_t max_len);

/* Attention of one new token per request over its cached tokens (the new
 * token's own key and value appended before):
 *     o[r][h] = sum_x p_x v_x,  p = softmax over x of scale q[r][h] . k_x,
 * x over the request's last `window` tokens (0: all) of seq_lens[r], query
 * head h reading key-value head h / (n_heads / n_kv_heads).
 *   q   DEVICE [n_req][n_heads][head_dim] of the cache's type, requests
 *       q_stride elements apart (a multiple of 16 bytes);
 *   block_table, seq_lens  DEVICE int32, as sq_block_tables writes them;
 *   max_len   HOST upper bound of seq_lens (it sets how the context is split
 *       over workgroups); a longer request is cut to its first max_len tokens,
 *       and to the table_stride * page_size tokens of its row (the smaller of the
 *       two at most 2^30);
 *   o   DEVICE [n_req][n_heads][head_dim] of the cache's type;
 *   lse DEVICE fp32 [n_req][n_heads], or NULL: log sum exp(scale q . k_x).
 * A request without tokens gets o = 0 and lse = -inf.  Table entries outside
 * the cache are read as absent tokens.  Keys and values past seq_lens are not
 * used, whatever they hold.  Sums and the softmax are fp32.  A query or key that
 * is not finite, or a score past the fp32 range, gives NaN in o and lse of the
 * heads that meet it, except that scores of -inf beside finite ones weigh
 * nothing; a value that is not finite makes its column of o not finite.  n_req == 0 is a
 * no-op.  Errors: SQ_ERR_INVALID (null or misaligned pointer, bad size,
 * workspace too small), SQ_ERR_UNSUPPORTED (page_size, head_dim, launch grid, more
 * than 2^30 tokens), SQ_ERR_HIP.  Asynchronous on `stream`; the workspace is in use until the
 * call's work is done. */
int sq_paged_attention(const sq_kv_cache *cache, const void *q, int64_t q_stride, int32_t n_req,
                       int32_t n_heads, const int32_t *block_table, int64_t table_stride,
                       const int32_t *seq_lens, int32_t max_len, float scale, int32_t window,
                       void *o, float *lse, void *workspace, uint64_t workspace_bytes, void *stream);

/* Readout without update ([P5] 空间维度: the head's output is the query read
 * out of the state): o = S^T q from the stored state (dequantized), for
 * slots slot_ids[0..n_req).  q: DEVICE [n_req][n_heads][d_k] of q_dtype;
 * o: DEVICE fp32 [n_req][n_heads][d_v].  Does not modify the pool.  n_req == 0
 * is a no-op.  Asynchronous on `stream`.  Errors as for sq_decode_step (q and
 * o required, 16-byte aligned). */
int sq_readout(const sq_pool *pool, const int32_t *slot_ids, int32_t n_req, const void *q,
               int32_t q_dtype, float *o, void *stream);

/* Device-side check of a batch's slot ids, for callers that cannot vouch for
 * them (the step does not check them; a repeated id makes two workgroups
 * update one tile).  Each request owns one resident state ([P1] 背景, [P5]
 * opening), so a valid batch names distinct slots in [0, n_slots).
 * Writes to *result (DEVICE int32, 4-byte aligned) 0 if the batch is valid,
 * otherwise a bit set: 1 = some id outside [0, n_slots), 2 = some id repeated.
 * slot_ids: DEVICE int32 [n_req]; n_req == 0 writes 0.  Uses per-slot stamps
 * and a generation counter in the pool's device table (no host state), so the
 * call can be captured in a HIP graph and replayed; calls on one pool must be
 * stream-ordered.
 * Errors: SQ_ERR_INVALID (null pool/result, negative n_req, misaligned
 * result), SQ_ERR_HIP.  Asynchronous on `stream`: read *result after
 * synchronizing it. */
int sq_check_slots(sq_pool *pool, const int32_t *slot_ids, int32_t n_req, int32_t *result,
                   void *stream);

/* The slot check of sq_check_slots for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation): it needs no pool, and keeps its per-slot stamps and
 * generation counter in a fixed array inside the library (one per GPU, about
 * 256 KB, held until the process ends) instead of a pool's table.  Nothing is
 * allocated, by this call or by anything it calls.
 * slot_ids: DEVICE int32 [n_req], checked against [0, n_slots); *result
 * (DEVICE int32, 4-byte aligned) receives 0, or 1 (an id out of range) | 2
 * (an id repeated), as for sq_check_slots.  n_slots must be at most
 * SQ_CHECK_NOALLOC_MAX_SLOTS.  n_req == 0 writes 0.
 * All calls on one GPU share that GPU's array: calls made on one GPU must not
 * overlap in time (order them on one stream), or their results race.
 * Errors: SQ_ERR_INVALID (null result, negative n_req, n_slots < 1, null
 * slot_ids with n_req > 0, misaligned result), SQ_ERR_UNSUPPORTED (n_slots
 * above the limit), SQ_ERR_HIP.  Asynchronous on `stream`. */
#define SQ_CHECK_NOALLOC_MAX_SLOTS 65536
int sq_check_slots_noalloc(const int32_t *slot_ids, int32_t n_req, int32_t n_slots, int32_t *result,
                           void *stream);

/* Read and clear the pool's sticky device flag.  The steps (scalar gate,
 * per-channel gate, plain decay) and the store set it when an updated value (the quotient S'/s for
 * codes, S' for unquantized heads) is not finite, which only non-finite or
 * huge inputs cause; the stored result then follows the rule above (NaN ->
 * code 0, +-Inf -> +-Q).  Synchronizes `stream` first (host-blocking).
 * Returns SQ_OK if no such value was met since the pool was made or the flag
 * last read, SQ_ERR_DEVICE if one was; SQ_ERR_INVALID (null pool, another
 * device current), SQ_ERR_HIP. */
int sq_pool_last_device_error(sq_pool *pool, void *stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char *sq_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SQ_H */
