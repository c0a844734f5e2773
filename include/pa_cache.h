/*
 * pa_cache.h -- the paged cache between decode steps: pages handed out to the
 * sequences of a step (block tables, slot map, positions, the pool of free
 * pages), and the step's keys and values stored into the cache.  With pa_decode
 * or pa_diff_decode (pa_decode.h) after them they make one step of serving:
 *
 *     pa_build_tables  lengths            -> block tables, slots, new lengths
 *                      (so metadata_ready stays 0 in the decode of that stream)
 *     pa_append_kv     keys, values       -> cache pages, through the slots
 *     pa_decode        query, cache       -> out
 *
 * The pages of the reference keep the block table and the cache as inputs
 * (block_tables and key_cache / value_cache of paged_attention_v2_pytorch in
 * "paged_attention_v2_pytorch.py -- BI-V100 PagedAttention V2 implementation");
 * they have no counterpart of these entry points.  The conventions of
 * pa_decode.h hold here too: device pointers owned by the caller, asynchronous
 * on `stream`, nothing allocated, host-visible errors returned before anything
 * is launched, data-dependent ones reported in `dev_error`.
 */
#ifndef PA_CACHE_H
#define PA_CACHE_H

#include "pa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A step of the batch: sequence s holds seq_lens[s] tokens in
 * own = ceil(seq_lens[s] / 16) pages, the first `own` entries of its row of
 * block_tables.  keep = keep_lens[s] of its tokens stay (all of them without
 * keep_lens; fewer after rejected drafts; 0 for a sequence that has ended), and
 * n = query_start[s+1] - query_start[s] tokens follow them (one without
 * query_start).  Then, with want = ceil((keep + n) / 16):
 *     new_seq_lens[s]        = keep + n
 *     want > own: entries [own, want) of its row get the next free pages,
 *     want < own: the pages of entries [want, own) go back to the pool (the
 *                 entries stay as they are),
 *     row t = query_start[s] + i is its token at positions[t] = keep + i, and
 *     slots[t] = 16 * block_tables[s][positions[t] / 16] + positions[t] % 16.
 * The pool is a ring of num_blocks entries: its `count` free pages are
 * free_ring[(head + k) % num_blocks], k < count, with pool_state = {head,
 * count}.  Pages are taken from the front in the order of the sequences (and of
 * each one's pages) and put back behind the last one in the same order, so the
 * result does not depend on the run; pages put back are there for the next call.
 * Rows of slots behind query_start[num_seqs] get -1 (which pa_append_kv skips)
 * and position 0: a batch may be padded to a fixed number of rows.
 *
 * All or nothing.  When a length is out of range (PA_DEVERR_SEQ_LEN:
 * seq_lens[s] outside [0, max_seq_len], keep_lens[s] outside [0, seq_lens[s]],
 * keep + n above max_seq_len, offsets that fall or pass num_tokens), the pool
 * has fewer pages than the step needs, or its state cannot be (PA_DEVERR_POOL),
 * nothing is taken or put back: new_seq_lens and new_pool_state are copies of
 * seq_lens and pool_state, and every slot is -1.  A page id outside
 * [0, num_blocks) is written to the table as it is, its tokens' slots are -1 and
 * PA_DEVERR_BLOCK_ID is set.  Each page belongs to one sequence or the ring
 * (shared pages would be put back twice); this is not checked.
 */
typedef struct pa_tables_args {
    int32_t* block_tables;      /* [num_seqs][max_blocks_per_seq], updated in place */
    const int32_t* seq_lens;    /* [num_seqs] */
    const int32_t* keep_lens;   /* [num_seqs] or NULL */
    const int32_t* query_start; /* [num_seqs + 1] or NULL */
    int32_t* free_ring;         /* [num_blocks], updated in place */
    const int32_t* pool_state;  /* [2] head, count */
    int32_t* slots;             /* [num_tokens] */
    int32_t* positions;         /* [num_tokens] or NULL */
    int32_t* new_seq_lens;      /* [num_seqs]; may be seq_lens itself */
    int32_t* new_pool_state;    /* [2]; may be pool_state itself */
    int32_t num_seqs;           /* at most 2^30 */
    int32_t num_tokens;         /* rows of slots and positions, at most 2^30; >= num_seqs without query_start */
    int32_t num_blocks;         /* pages of the cache, below 2^27 (slots are int32) */
    int32_t block_size;         /* must be PA_BLOCK_SIZE */
    int32_t max_seq_len;        /* upper bound of the lengths before and after */
    int32_t max_blocks_per_seq; /* row stride of block_tables, >= ceil(max_seq_len / block_size) */
    int32_t* dev_error;         /* optional: PA_DEVERR_* bits */
    /* Optional [1] int32, zero before the first call and left at zero by each:
     * with it a call of many rows runs on many CTAs, the last of which writes
     * the new lengths and pool state; without it on one CTA (2.1 million rows: 8.6 us
     * with it, 429 without).  Calls that share it must not overlap on the GPU. */
    int32_t* done_counter;
} pa_tables_args;

/* num_seqs == 0 only marks every row of slots as padding. */
pa_status pa_build_tables(const pa_tables_args* args, void* stream);

/*
 * Stores the key and value rows of a step's tokens: token t goes to the slot
 * slots[t] = 16 * block + offset of both caches,
 *     K(block, head, offset) = key[t][head],   V(block, head, offset) = value[t][head],
 * divided by k_scale or v_scale (the quotient rounded to fp32) and rounded to the
 * nearest fp8 value (half to even; beyond the largest finite value, that value; a NaN
 * stays one) when kv_dtype is fp8, and otherwise copied bit by bit.  A negative slot is skipped (padding); one past
 * the cache is skipped and reported (PA_DEVERR_SLOT).  The slots of a call are
 * distinct (of a slot given twice each element is that of one of its rows).
 * Slots that no row names keep their bytes.
 *
 * Keys and values have head counts and sizes of their own: num_kv_heads of
 * head_size for pa_decode, twice the heads for the keys and twice the size for
 * the values of a differential cache (pa_diff_decode).
 */
typedef struct pa_append_args {
    const void* key;    /* token t, head h at key + (t * key_stride + h * key_head_stride) elements of dtype */
    const void* value;  /* likewise; both and all four strides 16-byte aligned */
    void* key_cache;    /* layouts of pa_layout; 16-byte aligned */
    void* value_cache;
    const int32_t* slots; /* [num_tokens] */
    int64_t key_stride, key_head_stride, value_stride, value_head_stride; /* elements */
    int32_t num_tokens;  /* at most 2^30 */
    int32_t num_key_heads, key_head_size;     /* head sizes: 64, 128 or 256 */
    int32_t num_value_heads, value_head_size;
    int32_t num_blocks;  /* pages in each cache, below 2^27 */
    int32_t block_size;  /* must be PA_BLOCK_SIZE */
    int32_t dtype;       /* pa_dtype of key and value */
    int32_t layout;      /* pa_layout */
    int32_t kv_dtype;    /* pa_kv_dtype of the caches */
    float k_scale, v_scale; /* fp8 caches; values <= 0 mean 1.0, a reciprocal beyond fp32 is refused */
    int32_t* dev_error;  /* optional: PA_DEVERR_* bits */
} pa_append_args;

/* num_tokens == 0 is a no-op. */
pa_status pa_append_kv(const pa_append_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_CACHE_H */
