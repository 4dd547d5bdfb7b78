/*
 * gqa_packed.h -- attention over prompts of different lengths, packed one behind the other
 * (libgqa_decode.so).
 *
 * The queries of B sequences lie in one [N_q, H_q, 128] tensor, their keys and values in [N_k, H_kv, 128]
 * tensors, without padding.  Sequence b has n_b queries and m_b keys.  The two end at the same token:
 * query i stands at position i + m_b - n_b and sees, if causal, the keys j <= i + m_b - n_b (none where
 * that is negative), else all m_b.  With m_b = n_b that is a whole prompt; with m_b > n_b the chunk of a
 * prompt that goes on over a prefix (rows that gqa_q8_read has brought back from a cache, for one).
 *
 * Conventions are those of gqa_decode.h (bf16 as 16-bit storage, bf16 tensors 16-byte and int32 ones
 * 4-byte aligned, asynchronous on `stream`, argument errors before any launch, device-side index
 * errors as GQA_DEVERR_* bits).  Nothing is allocated, no workspace is needed and no state is kept between
 * calls besides the kernel's one-time configuration per device (make a first call before capturing
 * a graph).  The kernel is launched with programmatic stream serialization but reads and writes nothing
 * before the preceding kernel has completed, and never lets the next one start early.
 */
#ifndef GQA_PACKED_H_
#define GQA_PACKED_H_

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Shapes and layout of one call. */
typedef struct gqa_packed_desc {
    int batch;        /* B, 1..GQA_MAX_BATCH */
    int num_q_heads;  /* H_q */
    int num_kv_heads; /* H_kv; H_q % H_kv == 0 and G = H_q / H_kv <= 16 */
    int head_dim;     /* d; must be 128 */
    int num_queries;  /* N_q >= 1 */
    int num_keys;     /* N_k, 1..2^26 */
    int causal;       /* non-zero: the mask above; 0: every query sees all its sequence's keys */
    int device;       /* CUDA device ordinal the call runs on */
    int q_stride;     /* elements between the rows of consecutive tokens of q, k and v: */
    int k_stride;     /*   0 for dense (H * 128), else a multiple of 8 >= H * 128, as in one */
    int v_stride;     /*   [N, (H_q + 2 H_kv) * 128] projection that holds all three */
} gqa_packed_desc_t;

/*
 * gqa_packed_attn -- softmax(q . K / sqrt(128)) V over each sequence's own keys.
 *   q          [N_q, H_q, 128] bf16 device   rotated queries; a token's heads are dense
 *   k, v       [N_k, H_kv, 128] bf16 device   query head h reads KV head h / G
 *   q_offsets  [B + 1] int32 device, ascending, 0 <= q_offsets[0], q_offsets[B] <= N_q: rows q_offsets[b] ..
 *              q_offsets[b + 1] - 1 are sequence b's queries
 *   k_offsets  [B + 1] int32 device, likewise over N_k; NULL for q_offsets
 *   out        [N_q, H_q, 128] bf16 device, dense; zeros for a query that sees no key (or whose
 *              every score is -infinity); rows that belong to no sequence are left as they were.  Must
 *              not overlap any input.
 *   device_errors   optional device pointer to a uint32.  A sequence whose q_offsets descend, are negative or
 *              pass N_q (GQA_DEVERR_SEQLEN) is left out: its rows stay as they were; one whose k_offsets
 *              do (GQA_DEVERR_SEQLEN) counts as one without keys.
 * Keys and values that a query does not see have no effect on it whatever they hold (NaN and infinities
 * included).  A value that is not finite makes that dim of every query that sees it infinite or NaN, however
 * small its weight, unless the query's every score is -infinity.  The weights are rounded to bf16 (by at most 2^-8 of
 * each) before V is multiplied, where gqa_prefill_attn and gqa_tree_attn keep 16 bits of them: with N(0, 1) inputs the
 * result is off by 1.9e-3 to 2.3e-3 of itself in the 2-norm, 1.65e-3 there (the rounding of the output alone).
 * Scores are meant to be at most 2^29 in size (beyond, 2^ the rounding of the row's maximum leaves the range of the
 * weights), values at most 2^119 / m_b (they are added in binary32 under weights of up to 2^8).  The rounding of the
 * result does not depend on timing or on the other sequences of the batch: the same inputs give the same bits.
 * Errors: GQA_ERR_INVALID_ARG (NULL or misaligned tensors, bad sizes or strides), GQA_ERR_UNSUPPORTED
 * (head_dim != 128, H_q % H_kv != 0, H_q / H_kv > 16, more than 2^31 - 1 rows N_q H_q or N_k H_kv, more than 2^26
 * keys), GQA_ERR_CUDA.
 */
gqa_status_t gqa_packed_attn(const gqa_packed_desc_t *desc, const void *q, const void *k, const void *v,
                             const int32_t *q_offsets, const int32_t *k_offsets, void *out, uint32_t *device_errors,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PACKED_H_ */
