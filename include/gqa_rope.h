/*
 * gqa_rope.h -- QK RMSNorm, rotary embedding and KV append as a call of its own
 * (libgqa_decode.so), in the layouts and scalings that the decode step and the prefill
 * chunk do not have.
 *
 * gqa_decode_attn and gqa_prefill_attn rotate the whole 128-dim head in the half-split
 * layout, unscaled, and store a token at the slot of its position.  Here
 *   - the pairs are (i, i + r/2) (half) or (2i, 2i + 1) (interleaved), i < r/2;
 *   - only the first r = rotary_dim dims rotate, the others pass (after the norm);
 *   - the pairs' frequencies may be scaled for contexts longer than those trained on;
 *   - the position of a token and the cache slot it is stored at are separate, as a tree of
 *     drafted tokens needs (gqa_tree.h): siblings share a position but not a slot.
 * The cache it fills is read by gqa_tree_attn (single tokens included), and, where the
 * rotary embedding is the unscaled full-width half-split one, by the decode step and
 * prefill: the key rows are then the same bits that those append.  gqa_prefill_attn rotates by
 * itself, so a prompt with another embedding attends by gqa_tree_attn, GQA_MAX_TREE tokens at a time with a
 * chain's masks.
 *
 * For token t of sequence b, every head row x of q and k, with w its norm weights:
 *   y    = x / sqrt(mean(x^2) + eps) * w          (y = x where no weights are given)
 *   z_i  = m (y_i cos a - y_j sin a),  z_j = m (y_j cos a + y_i sin a),  a = p f_i
 * for each pair (i, j) of index i, p = positions[b][t], m the magnitude; z = y in the dims
 * from r on.  z is rounded once to bf16; for keys, which stay in the cache, the rounding is
 * that of the exact value (as in the decode step); queries are computed in binary32.  Where a
 * row is normalised, mean(x^2) + eps has to lie between 2^-100 and 2^120: |x| below about 10^18, and
 * from an eps of 10^-30 on no row is too small.  A row outside it (with a smaller eps: a zero row, or
 * |x| below about 10^-15) gets values of no meaning, NaN and infinities among them, and no other
 * row does.
 *
 * Conventions are those of gqa_decode.h (bf16 as 16-bit storage, row-major device tensors,
 * asynchronous on `stream`, argument errors before any launch, device-side index errors as
 * GQA_DEVERR_* bits).  Nothing is allocated.  Between calls a host thread keeps what follows from the
 * fields of the last gqa_rope_t it used (never from a CUSTOM one, whose table is read at every
 * call), and a device the kernels' one-time configuration (make a first call before capturing a graph);
 * calls on different streams may overlap.  The kernel is launched with programmatic stream
 * serialization but reads and writes nothing before the preceding kernel has completed,
 * and never lets the next one start early.
 */
#ifndef GQA_ROPE_H_
#define GQA_ROPE_H_

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Pair layouts. */
#define GQA_ROPE_HALF 0        /* (i, i + r/2) */
#define GQA_ROPE_INTERLEAVED 1 /* (2i, 2i + 1) */

/* Frequency scalings; f_i = theta^(-2i/r) is the unscaled frequency of pair i. */
#define GQA_ROPE_NONE 0
#define GQA_ROPE_LINEAR 1 /* f_i / factor (position interpolation) */
#define GQA_ROPE_BANDED 2 /* by the pair's wavelength 2 pi / f_i: kept where it is below
                             original_max_len / high_freq_factor, divided by factor where it is
                             above original_max_len / low_freq_factor, a linear mix (in the
                             number of periods in original_max_len) in between */
#define GQA_ROPE_YARN 3   /* YaRN ("YaRN: Efficient Context Window Extension of Large Language
                             Models", section 3.2): f_i and f_i / factor mixed by a ramp over i
                             from floor(d(beta_fast)) to ceil(d(beta_slow)),
                             d(b) = r ln(original_max_len / (2 pi b)) / (2 ln theta) */
#define GQA_ROPE_CUSTOM 4 /* freqs[i], i < r/2 (for example a table with a factor per pair) */

typedef struct gqa_rope {
    int layout;             /* GQA_ROPE_HALF or GQA_ROPE_INTERLEAVED */
    int rotary_dim;         /* r: a multiple of 8, 8 .. 128 */
    int scaling;            /* GQA_ROPE_NONE .. GQA_ROPE_CUSTOM */
    int original_max_len;   /* BANDED, YARN: the trained length (>= 1) */
    float theta;            /* base (> 0; YARN: > 1); not used by CUSTOM */
    float factor;           /* LINEAR, BANDED, YARN: > 0 (YARN: >= 1) */
    float low_freq_factor;  /* BANDED: > 0 */
    float high_freq_factor; /* BANDED: > low_freq_factor */
    float beta_fast;        /* YARN: > beta_slow */
    float beta_slow;        /* YARN: > 0 */
    float magnitude;        /* m; 0 takes the scaling's own: 0.1 ln(factor) + 1 for YARN, else 1 */
    const double *freqs;    /* CUSTOM: host array [r/2], finite; else not used */
} gqa_rope_t;

/*
 * gqa_rope_freqs -- the frequencies and the magnitude a gqa_rope_t stands for (host,
 * synchronous, no device work).
 *   freqs [r/2] receives f_i after scaling; magnitude receives m; either may be NULL.
 * Errors: GQA_ERR_INVALID_ARG (NULL rope, a field outside the ranges above, a frequency beyond
 * 65536 in size).
 */
gqa_status_t gqa_rope_freqs(const gqa_rope_t *rope, double *freqs, double *magnitude);

/* Shapes and layout of one call. */
typedef struct gqa_rope_desc {
    int batch;            /* B, 1..GQA_MAX_BATCH */
    int num_q_heads;      /* H_q */
    int num_kv_heads;     /* H_kv; H_q % H_kv == 0 and H_q / H_kv <= 16 */
    int head_dim;         /* d; must be 128 */
    int num_tokens;       /* T: tokens of a sequence in this call, 1 <= T <= max_seq_len */
    int block_size;       /* 64: paged cache; 0: contiguous (as gqa_prefill_desc_t) */
    int max_seq_len;      /* per-sequence capacity in tokens */
    int num_cache_blocks; /* paged: 64-token blocks in each cache pool (>= 1); else ignored */
    int device;           /* CUDA device ordinal the call runs on */
    int q_stride;         /* elements between the rows of consecutive tokens of q, k and v: */
    int k_stride;         /*   0 for dense (H * 128), else a multiple of 8 >= H * 128, as in */
    int v_stride;         /*   one [B * T, (H_q + 2 H_kv) * 128] projection that holds all three */
} gqa_rope_desc_t;

/*
 * gqa_rope_append -- norm, rotate and store the new tokens.
 *   q, k, v    [B, T, H, 128] bf16 device, H = H_q for q and H_kv for k and v; a token's heads are
 *              dense, consecutive tokens are *_stride elements apart
 *   k_cache, v_cache, page_table   as in gqa_prefill_attn; the rows of the slots
 *              slot_start[b] + t are written
 *   slot_start [B] int32 device   slot of the sequence's first token
 *   positions  [B, T] int32 device   p >= 0, the rotary position of each token; NULL for
 *              slot_start[b] + t
 *   counts     [B] int32 device   tokens of each sequence, 0 <= counts[b] <= T; NULL for T.
 *              Rows t >= counts[b] of q, k, v and positions are not used, those of q_out not
 *              written, and nothing is stored for them.
 *   q_norm_w, k_norm_w   [128] bf16 device, or NULL for no norm on q / on k
 *   rope       the rotary embedding (read during the call only)
 *   eps        RMSNorm epsilon (>= 0)
 *   q_out      [B, T, H_q, 128] bf16 device, dense; may be q itself when q is dense, else must not
 *              overlap any input
 *   device_errors   optional device pointer to a uint32 the kernel ORs GQA_DEVERR_* bits into.
 *              A count outside [0, T] or a last slot beyond max_seq_len (GQA_DEVERR_SEQLEN) or
 *              a negative slot_start (GQA_DEVERR_POSITION) stores nothing of that sequence and
 *              gives zeros in all its T rows of q_out; a negative position does so for its token; a page id
 *              outside the pool (GQA_DEVERR_PAGE) stores nothing for the tokens there.
 * Every slot written must belong to its sequence alone (no shared page: gqa_pages.h).
 * Errors: GQA_ERR_INVALID_ARG (NULL or misaligned tensor -- 16 bytes for bf16, 4 for int32 --,
 * page_table given for a contiguous cache or missing for a paged one, bad sizes, strides,
 * rope fields or eps), GQA_ERR_UNSUPPORTED (head_dim != 128, H_q % H_kv != 0, H_q / H_kv > 16,
 * block_size other than 0 or 64, more than 2^31 - 1 cache rows or tokens, (H_q + 2 H_kv) x 256 B
 * above 200 KiB), GQA_ERR_CUDA.
 */
gqa_status_t gqa_rope_append(const gqa_rope_desc_t *desc, const void *q, const void *k, const void *v,
                             void *k_cache, void *v_cache, const int32_t *page_table,
                             const int32_t *slot_start, const int32_t *positions, const int32_t *counts,
                             const void *q_norm_w, const void *k_norm_w, const gqa_rope_t *rope, float eps,
                             void *q_out, uint32_t *device_errors, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_ROPE_H_ */
