/*
 * gqa_pages.h -- the pages of a paged KV cache: sharing, growing, shrinking, copying
 * (libgqa_decode.so).
 *
 * A page is 64 token slots of every pool (the K and V pools of each layer, or the index and
 * scale pools of a 4-bit cache with H_kv a multiple of 4, since a token's scales are 4 H_kv bytes and
 * rows are moved 16 bytes at a time: all share one page table).  The state, device memory of the
 * caller's, is
 *   ref_counts [num_blocks] int32         how many sequences hold each page; 0 = free
 *   page_table [B, max_blocks] int32      pages of each sequence, -1 where it has none
 *   seq_lens   [B] int32                  tokens of each sequence; it holds ceil(L/64) pages
 * started as zeros, -1 and zeros.  gqa_pages_fork lets a sequence share another's pages;
 * gqa_pages_resize grows and shrinks sequences (a shared page that would be written to is
 * replaced by a copy of its own); gqa_pages_copy copies the pages it lists in every pool;
 * gqa_cache_keep_rows moves the tokens to keep (accepted drafts, or what an eviction leaves)
 * to the front.  Everything runs on the device, on `stream`, and can be captured in a graph.
 *
 * Results do not depend on timing: pages are taken lowest id first, in the order of the
 * sequences and of their pages.  Conventions are those of gqa_decode.h; int32 tensors 4-byte
 * aligned; nothing is allocated and no state is kept (the first call of each kind on a device
 * loads its kernel: make it before capturing a graph).  Kernels are launched with
 * programmatic stream serialization but read and write nothing before the preceding kernel
 * has completed, and never let the next one start early.
 */
#ifndef GQA_PAGES_H_
#define GQA_PAGES_H_

#include "gqa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the device error word besides gqa_decode.h's. */
#define GQA_DEVERR_NOPAGE 0x20u   /* not enough free pages: the call changed nothing */
#define GQA_DEVERR_CONFLICT 0x40u /* the same sequence or page named twice where it may not be */

#define GQA_MAX_POOLS 256
#define GQA_MAX_PAGE_PAIRS 4096

/* One pool of a cache: rows of row_bytes bytes (one token slot, every head). */
typedef struct gqa_pool {
    void *base;         /* device memory, 16-byte aligned */
    long long row_bytes; /* a multiple of 16, 16 .. 2^20 */
} gqa_pool_t;

/* Shape of the page state. */
typedef struct gqa_pages_desc {
    int batch;      /* B sequences, 1..GQA_MAX_BATCH */
    int max_blocks; /* entries of a sequence's page-table row (>= 1; B * max_blocks < 2^31) */
    int num_blocks; /* pages of the pool, 1 .. 2^25 - 1 */
    int device;     /* CUDA device ordinal the call runs on */
} gqa_pages_desc_t;

/*
 * gqa_pages_fork -- sequence dst[i] becomes another holder of the pages of src[i], for
 * i < num_pairs (1..GQA_MAX_BATCH): its table row and length become those of src, and each
 * page's count goes up by one.  Nothing is copied; a shared last page is split when either grows.
 *   src, dst [num_pairs] int32 device   src[i] < 0: the pair is not used
 * A pair is skipped, with a bit in device_errors, when an index is outside [0, B) or dst has
 * pages of its own (length != 0) or the source's length does not fit its row or its row names
 * a page outside the pool or a free one
 * (GQA_DEVERR_POSITION, _SEQLEN, _PAGE), and when dst is src, is an
 * earlier pair's dst, or is the src of any pair (GQA_DEVERR_CONFLICT).
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_UNSUPPORTED, GQA_ERR_CUDA.
 */
gqa_status_t gqa_pages_fork(const gqa_pages_desc_t *desc, int32_t *ref_counts, int32_t *page_table,
                            int32_t *seq_lens, const int32_t *src, const int32_t *dst, int num_pairs,
                            uint32_t *device_errors, void *stream);

/*
 * gqa_pages_resize -- sets the sequences' lengths to new_lens (negative: leave as it is; 0 gives
 * up every page).  Shrinking drops the pages past the new length (their counts go down, the
 * table entries become -1).  Growing adds free pages; and where the sequence's last page is
 * partly filled and held by another sequence too, so that the next token would be written to
 * a shared page, the sequence gets a page of its own instead: cow_src[b], cow_dst[b] name the
 * pair to copy (gqa_pages_copy) before it is written.  Pages that this call frees can be taken
 * by it, except a page given up by such a split.  When every holder of a page grows at once,
 * the last of them (by index) keeps it.
 *   new_lens [B] int32 device
 *   cow_src, cow_dst [B] int32 device   written: the pages to copy, or -1
 * If there are too few free pages, nothing changes and GQA_DEVERR_NOPAGE is set (cow_* are all -1):
 * the sequences must not be written to then, a last page that they share has not been split.  Where
 * nobody can look at the error word in between (a captured step), seq_lens less the lengths before the
 * call is what each sequence was granted, 0 where it could not grow: as the counts of
 * gqa_tree_prepare, gqa_rope_append and gqa_tree_attn, and as the limit of gqa_cache_keep_rows', it
 * keeps the step from touching a slot that the sequence has not got.  A
 * sequence whose length or new length is beyond its row (GQA_DEVERR_SEQLEN) or
 * whose table names a page outside the pool or a free one, where the call needs it
 * (GQA_DEVERR_PAGE), is left as it is.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_CUDA.
 */
gqa_status_t gqa_pages_resize(const gqa_pages_desc_t *desc, int32_t *ref_counts, int32_t *page_table,
                              int32_t *seq_lens, const int32_t *new_lens, int32_t *cow_src, int32_t *cow_dst,
                              uint32_t *device_errors, void *stream);

/*
 * gqa_pages_copy -- page dst[i] := page src[i] in every pool, for i < num_pairs
 * (1..GQA_MAX_PAGE_PAIRS).
 *   pools      host array [num_pools] (1..GQA_MAX_POOLS), read during the call only; pools must not
 *              overlap (their rows would be moved twice), here and in gqa_cache_keep_rows
 *   num_blocks pages of each pool (its size is num_blocks * 64 * row_bytes)
 *   src, dst   [num_pairs] int32 device   src[i] < 0: the pair is not used
 * A pair with a page outside the pool (GQA_DEVERR_PAGE), or whose dst is an earlier used pair's dst or
 * any other used pair's src (GQA_DEVERR_CONFLICT: the order would decide), copies nothing.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_CUDA.
 */
gqa_status_t gqa_pages_copy(const gqa_pool_t *pools, int num_pools, int num_blocks, const int32_t *src,
                            const int32_t *dst, int num_pairs, int device, uint32_t *device_errors, void *stream);

/* Shape of a gqa_cache_keep_rows call. */
typedef struct gqa_keep_desc {
    int batch;       /* B, 1..GQA_MAX_BATCH */
    int max_keep;    /* N: entries of a sequence's list (1..max_seq_len, at most 2^30) */
    int max_seq_len; /* per-sequence capacity in tokens (>= 1) */
    int block_size;  /* 64: paged pools; 0: contiguous pools of B * max_seq_len rows */
    int num_blocks;  /* paged: pages of each pool (>= 1); else ignored */
    int device;      /* CUDA device ordinal the call runs on */
} gqa_keep_desc_t;

/*
 * gqa_cache_keep_rows -- in every pool, the row of slot start[b] + keep[b][i] moves to slot
 * start[b] + i, for i < counts[b]: the accepted path of a draft tree (ascending node indices)
 * becomes the sequence's next tokens, or an eviction's survivors become contiguous.
 *   page_table [B, ceil(max_seq_len/64)] int32 device, or NULL when contiguous
 *   start      [B] int32 device   first slot the list refers to (>= 0)
 *   keep       [B, max_keep] int32 device   strictly ascending, >= 0, start + keep < max_seq_len
 *   counts     [B] int32 device   0 <= counts[b] <= max_keep (entries from there on are not read)
 * A sequence whose list breaks these rules (GQA_DEVERR_POSITION; GQA_DEVERR_SEQLEN for
 * counts) or has a page outside the pool in its way (GQA_DEVERR_PAGE) moves nothing.  The slots
 * written must belong to the sequence alone (gqa_pages_resize sees to that for slots it grew).
 * Rows keep their contents: rotary positions are those they were stored with.
 * Errors: GQA_ERR_INVALID_ARG, GQA_ERR_UNSUPPORTED (block_size, more than 2^31 - 1 rows, max_keep), GQA_ERR_CUDA.
 */
gqa_status_t gqa_cache_keep_rows(const gqa_keep_desc_t *desc, const gqa_pool_t *pools, int num_pools,
                                 const int32_t *page_table, const int32_t *start, const int32_t *keep,
                                 const int32_t *counts, uint32_t *device_errors, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_PAGES_H_ */
