/*
 * gqa_tree.h -- attention for a tree of drafted tokens over a KV cache (libgqa_decode.so).
 *
 * Speculative decoding verifies several drafted continuations of a sequence at once: n <= T
 * nodes, each a token whose parent is an earlier node or the context.  A node attends to the
 * whole cached context and to its own ancestors and itself, not to its siblings.  Its rotary
 * position is context length + depth, its cache slot context length + node index; the keys
 * and values of the nodes are stored by gqa_rope_append (gqa_rope.h) before the attention
 * reads them.  One node a sequence is the decode step's attention, a chain is a causal chunk.
 *
 * Conventions are those of gqa_decode.h (bf16 as 16-bit storage, dense row-major device
 * tensors, bf16 tensors 16-byte aligned, int32 ones 4-byte and masks 8-byte aligned,
 * asynchronous on `stream`, argument errors before any launch, device-side index errors as
 * GQA_DEVERR_* bits).  Nothing is allocated; no state is kept between calls besides the
 * kernels' one-time configuration per device (make a first call before capturing a graph).  Scratch memory is the caller's `workspace`:
 * calls that may overlap (different streams, two graphs replayed at once) need one each.
 * Kernels are launched with programmatic stream serialization but read and write nothing
 * before the preceding kernel has completed, and the last kernel of a call never lets the
 * next one start early.
 */
#ifndef GQA_TREE_H_
#define GQA_TREE_H_

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GQA_MAX_TREE 256 /* nodes of a sequence */

/*
 * gqa_tree_prepare -- the nodes' masks and positions from their parents, once a step.
 *   batch, tree_len  B (1..GQA_MAX_BATCH) and T (1..GQA_MAX_TREE)
 *   parents   [B, T] int32 device   parent node of node t, -1 <= parents[b][t] < t (-1: the
 *             node continues the context)
 *   ctx_lens  [B] int32 device   c_b >= 0: cached tokens before the tree
 *   counts    [B] int32 device   nodes of each sequence, 0 <= counts[b] <= T; NULL for T
 *   mask      [B, T, ceil(T/64)] uint64 device   bit u % 64 of word u / 64: node t sees node u
 *             (its ancestors and itself)
 *   positions [B, T] int32 device   c_b + depth (a node whose parent is -1 has depth 0)
 *   device_errors   optional device pointer to a uint32: a parent outside its range
 *             (GQA_DEVERR_POSITION) counts as -1; a count outside [0, T] or a negative c_b, or
 *             a position that would pass 2^31 - 1 (GQA_DEVERR_SEQLEN) leaves the sequence's
 *             rows as they were.
 * Rows t >= counts[b] of parents are not read and of mask and positions not written.
 * Errors: GQA_ERR_INVALID_ARG (sizes, NULL or misaligned tensors, device), GQA_ERR_CUDA.
 */
gqa_status_t gqa_tree_prepare(int batch, int tree_len, const int32_t *parents, const int32_t *ctx_lens,
                              const int32_t *counts, uint64_t *mask, int32_t *positions, int device,
                              uint32_t *device_errors, void *stream);

/* Shapes and layout of one attention call. */
typedef struct gqa_tree_desc {
    int batch;            /* B, 1..GQA_MAX_BATCH */
    int num_q_heads;      /* H_q */
    int num_kv_heads;     /* H_kv; H_q % H_kv == 0 and G = H_q / H_kv <= 16 */
    int head_dim;         /* d; must be 128 */
    int tree_len;         /* T: nodes of a sequence at most, 1..GQA_MAX_TREE, <= max_seq_len */
    int block_size;       /* 64: paged cache; 0: contiguous (as gqa_prefill_desc_t) */
    int max_seq_len;      /* per-sequence capacity in tokens */
    int num_cache_blocks; /* paged: 64-token blocks in each cache pool (>= 1); else ignored */
    int device;           /* CUDA device ordinal the call runs on */
} gqa_tree_desc_t;

/*
 * gqa_tree_workspace_bytes -- size of the workspace gqa_tree_attn needs for a geometry on
 * its device, into *bytes.  Errors: those of gqa_tree_attn's geometry checks; GQA_ERR_CUDA.
 */
gqa_status_t gqa_tree_workspace_bytes(const gqa_tree_desc_t *desc, size_t *bytes);

/*
 * gqa_tree_attn -- attention of the tree's nodes.
 *   q          [B, T, H_q, d] bf16 device   rotated queries
 *   k_cache, v_cache, page_table   as in gqa_prefill_attn; read only
 *   ctx_lens   [B] int32 device   c_b: slots 0 .. c_b - 1 are seen by every node
 *   counts     [B] int32 device   n_b nodes, at slots c_b .. c_b + n_b - 1; 0 <= n_b <= T; NULL for T
 *   mask       [B, T, ceil(T/64)] uint64 device   as gqa_tree_prepare writes it; any pattern is
 *              allowed (bits from n_b on are ignored)
 *   out        [B, T, H_q, d] bf16 device   softmax over the seen keys of q . K / sqrt(d), applied to
 *              V; zeros for a node that sees no key (or whose every score is -infinity); rows t >= n_b
 *              are left as they were.  Must not overlap any input.
 *   workspace  device memory of gqa_tree_workspace_bytes bytes, 256-byte aligned; its contents need
 *              not be set and are not kept
 *   device_errors   optional device pointer to a uint32.  c_b < 0 (GQA_DEVERR_POSITION), n_b
 *              outside [0, T] or c_b + n_b > max_seq_len (GQA_DEVERR_SEQLEN) gives zeros in all T
 *              rows of the sequence; a page id outside the pool (GQA_DEVERR_PAGE) reads that page as zeros.
 * Keys and values that a node does not see have no effect on it whatever they hold (NaN and
 * infinities included), nor do slots from c_b + n_b on.  A value of the context that is not finite
 * makes that dim of every node infinite or NaN, one of a node that dim of every node that sees it, however
 * small its weight.  The rounding of the result does not
 * depend on timing: the same inputs give the same bits.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_UNSUPPORTED (as gqa_prefill_attn; also B (ceil(max_seq_len/64)
 * + 7) or B H_kv ceil(T / floor(128 / G)) above 2^31 - 1), GQA_ERR_CUDA.
 */
gqa_status_t gqa_tree_attn(const gqa_tree_desc_t *desc, const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *page_table, const int32_t *ctx_lens, const int32_t *counts,
                           const uint64_t *mask, void *out, void *workspace, uint32_t *device_errors,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_TREE_H_ */
