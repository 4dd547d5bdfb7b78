/*
 * gqa_q8.h -- an 8-bit KV cache: rows quantised as they are written, read back as bf16, and the
 * attention of one new token a sequence over it (libgqa_decode.so).
 *
 * A cache row is one slot and KV head, 128 values, of K and of V each: 128 codes of 8 bits and one
 * binary32 scale; it stands for code * scale.  The codes are e4m3 (4 exponent and 3 mantissa
 * bits, largest level Q = 448) or int8 (Q = 127).  A row x is kept as
 *   scale = max |x| / Q, rounded to binary32;
 *   code  = the level next to the exact quotient x / scale, ties to the even one, at most Q in size.
 * A row of zeros has scale 0 and codes 0; a row with a value that is not finite has scale NaN and
 * codes 0, so that it reads as NaN throughout.
 *
 * Layouts are those of the bf16 caches (gqa_prefill.h) with 128 bytes in a row's place, the scales
 * beside them: paged, [num_cache_blocks, 64, H_kv, 128] codes and [num_cache_blocks, 64, H_kv]
 * scales, with a page table [B, ceil(max_seq_len / 64)]; or contiguous, [B, max_seq_len, H_kv, 128] and [B,
 * max_seq_len, H_kv].  The page calls (gqa_pages.h) move these pools where rows are multiples of 16
 * bytes: the codes' always, the scales' where H_kv is a multiple of 4.
 *
 * Keys are stored as they come: normalise and rotate them first (gqa_rope_append with the packed
 * rows as one sequence of a contiguous cache does so in one pass).
 *
 * Conventions are those of gqa_decode.h (bf16 as 16-bit storage, bf16 tensors and codes 16-byte
 * aligned, int32 and scales 4-byte aligned, asynchronous on `stream`, argument errors before any
 * launch, device-side index errors as GQA_DEVERR_* bits).  Nothing is allocated; no state is kept
 * between calls besides the kernels' one-time configuration per device (make a first call before
 * capturing a graph).  Kernels are launched with programmatic stream serialization but read and
 * write nothing before the preceding kernel has completed, and the last kernel of a call never
 * lets the next one start early.
 */
#ifndef GQA_Q8_H_
#define GQA_Q8_H_

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_Q8_E4M3 0
#define GQA_Q8_INT8 1

/* Shapes and layout of one call. */
typedef struct gqa_q8_desc {
    int batch;            /* B, 1..GQA_MAX_BATCH */
    int num_q_heads;      /* H_q: gqa_q8_attn only (H_q % H_kv == 0 and G = H_q / H_kv <= 16) */
    int num_kv_heads;     /* H_kv */
    int head_dim;         /* d; must be 128 */
    int format;           /* GQA_Q8_E4M3 or GQA_Q8_INT8 */
    int num_tokens;       /* N, rows of the packed tensors: gqa_q8_append and gqa_q8_read only (>= 1) */
    int block_size;       /* 64: paged cache; 0: contiguous (as gqa_prefill_desc_t) */
    int max_seq_len;      /* per-sequence capacity in tokens */
    int num_cache_blocks; /* paged: 64-token blocks in each cache pool (>= 1); else ignored */
    int device;           /* CUDA device ordinal the call runs on */
    int k_stride;         /* elements between the rows of consecutive tokens of the packed k and v: */
    int v_stride;         /*   0 for dense (H_kv * 128), else a multiple of 8 >= H_kv * 128 */
} gqa_q8_desc_t;

/*
 * gqa_q8_append -- quantise and store new rows, of any number of tokens a sequence.
 *   k, v       [N, H_kv, 128] bf16 device   the tokens of all sequences, one sequence behind the
 *              other; a token's heads are dense, consecutive tokens *_stride elements apart
 *   k_codes, v_codes, k_scale, v_scale, page_table   the cache
 *   offsets    [B + 1] int32 device, ascending, 0 <= offsets[0], offsets[B] <= N: rows offsets[b] ..
 *              offsets[b + 1] - 1 are sequence b's (none where the two are equal; other rows are
 *              not used); NULL: N = B, one row a sequence
 *   slot_start [B] int32 device   slot of the sequence's first row
 *   device_errors   optional device pointer to a uint32 the kernel ORs GQA_DEVERR_* bits into.  A
 *              sequence whose offsets descend or pass N, or whose last slot is beyond max_seq_len
 *              (GQA_DEVERR_SEQLEN), or with a negative slot_start (GQA_DEVERR_POSITION), stores
 *              nothing; a page id outside the pool (GQA_DEVERR_PAGE) stores nothing for the tokens
 *              there.  Where offsets descend anywhere, rows of other sequences may be left out too (a row's
 *              sequence is found by bisection); a row that is stored is stored where it belongs.
 * Every slot written must belong to its sequence alone (no shared page: gqa_pages.h).
 * Errors: GQA_ERR_INVALID_ARG (NULL or misaligned tensors, page_table given for a contiguous cache
 * or missing for a paged one, bad sizes, strides or format, NULL offsets with N != B),
 * GQA_ERR_UNSUPPORTED (head_dim != 128, block_size other than 0 or 64, more than 2^31 - 1 cache rows or rows
 * N H_kv), GQA_ERR_CUDA.
 */
gqa_status_t gqa_q8_append(const gqa_q8_desc_t *desc, const void *k, const void *v, void *k_codes, void *v_codes,
                           float *k_scale, float *v_scale, const int32_t *page_table, const int32_t *offsets,
                           const int32_t *slot_start, uint32_t *device_errors, void *stream);

/*
 * gqa_q8_read -- rows of the cache as bf16 (code * scale, rounded to binary32 and then to bf16), packed.
 *   k_codes, v_codes, k_scale, v_scale, page_table   the cache; read only
 *   offsets, slot_start   as in gqa_q8_append: row offsets[b] + i receives slot slot_start[b] + i of
 *              sequence b; slot_start NULL for 0
 *   k_out, v_out   [N, H_kv, 128] bf16 device, strides as k and v above; rows that belong to no
 *              sequence are left as they were.  Must not overlap any input.
 *   device_errors   as in gqa_q8_append, with "reads nothing" (the rows are left as they were) in
 *              place of "stores nothing"; a page id outside the pool gives zeros.
 * Errors: as gqa_q8_append.
 */
gqa_status_t gqa_q8_read(const gqa_q8_desc_t *desc, const void *k_codes, const void *v_codes, const float *k_scale,
                         const float *v_scale, const int32_t *page_table, const int32_t *offsets,
                         const int32_t *slot_start, void *k_out, void *v_out, uint32_t *device_errors, void *stream);

/*
 * gqa_q8_workspace_bytes -- size of the workspace gqa_q8_attn needs for a geometry on its device, into
 * *bytes (num_tokens and the strides are not used).  Errors: those of gqa_q8_attn's geometry
 * checks; GQA_ERR_CUDA.
 */
gqa_status_t gqa_q8_workspace_bytes(const gqa_q8_desc_t *desc, size_t *bytes);

/*
 * gqa_q8_attn -- attention of one new token a sequence over the cache, its own slot included.
 *   q          [B, H_q, 128] bf16 device, dense   rotated queries
 *   k_codes, v_codes, k_scale, v_scale, page_table   the cache; read only
 *   seq_lens   [B] int32 device   slots 0 .. seq_lens[b] - 1 are attended to; 0 <= seq_lens[b] <= max_seq_len
 *   out        [B, H_q, 128] bf16 device   softmax over these slots of q . K / sqrt(128), applied to V;
 *              zeros for a sequence without slots (or a head whose every score is -infinity).  Must
 *              not overlap any input.
 *   workspace  device memory of gqa_q8_workspace_bytes bytes, 256-byte aligned; its contents need not be
 *              set and are not kept.  Calls that may overlap (different streams, two graphs
 *              replayed at once) need one each.
 *   device_errors   optional device pointer to a uint32.  A seq_lens[b] outside [0, max_seq_len]
 *              (GQA_DEVERR_SEQLEN) gives zeros; a page id outside the pool (GQA_DEVERR_PAGE) reads
 *              that page as zeros.
 * Slots from seq_lens[b] on have no effect whatever they hold.  A scale that is not finite, or an e4m3
 * code that is no number, makes what depends on it infinite or NaN.  A weight times its V scale is kept
 * to 2^-11 of itself, 2^-33 of the head's largest such product or 2^-182, whichever is most; a weight below 2^-118
 * of the head's largest may count as 0.  The rounding of the result does not depend on timing: the same
 * inputs give the same bits.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_UNSUPPORTED (as gqa_q8_append; also H_q % H_kv != 0, H_q / H_kv >
 * 16, B (ceil(max_seq_len / 16) + 24) or max(B, 640) H_q above 2^31 - 1), GQA_ERR_CUDA.
 */
gqa_status_t gqa_q8_attn(const gqa_q8_desc_t *desc, const void *q, const void *k_codes, const void *v_codes,
                         const float *k_scale, const float *v_scale, const int32_t *page_table,
                         const int32_t *seq_lens, void *out, void *workspace, uint32_t *device_errors, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_Q8_H_ */
