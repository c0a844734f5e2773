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
 * 4-bit caches (PA_KV_FP4_E2M1, 16-bit rows of 64 or 128, NHD): of each 16 successive
 * elements x of a row, with g = k_scale or v_scale,
 *     scale = e4m3(max|x| / (6 g)),   code = e2m1(x / (g scale)),
 * the real quotients rounded once, half to even, beyond the largest value: that value
 * (an infinity too).  A scale that comes out zero makes all 16 codes zero; a NaN among the
 * elements makes the scale NaN and the codes zero.  (Of a slot given twice, the codes of an
 * element and its scale may be of different rows.)
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
    int32_t num_key_heads, key_head_size;     /* head sizes: 64, 128 or 256 (4-bit: not 256) */
    int32_t num_value_heads, value_head_size;
    int32_t num_blocks;  /* pages in each cache, below 2^27 */
    int32_t block_size;  /* must be PA_BLOCK_SIZE */
    int32_t dtype;       /* pa_dtype of key and value */
    int32_t layout;      /* pa_layout */
    int32_t kv_dtype;    /* pa_kv_dtype of the caches */
    float k_scale, v_scale; /* fp8 and 4-bit caches; values <= 0 mean 1.0, a reciprocal beyond fp32 is refused */
    int32_t* dev_error;  /* optional: PA_DEVERR_* bits */
} pa_append_args;

/* num_tokens == 0 is a no-op. */
pa_status pa_append_kv(const pa_append_args* args, void* stream);

/*
 * A cache that is short of room: the tokens that attention has used least go.  Between two
 * decode steps,
 *     pa_add_weights     query, keys, statistics of the decode -> a score of every token
 *     pa_select_tokens   scores, budgets                       -> which tokens stay
 *     pa_compact_kv      those                                 -> cache pages without the others
 *     pa_build_tables    with keep_lens = the new lengths: their pages go back to the pool
 * Scores are fp32, [num_blocks][num_kv_heads][16]: a page of them for every page of the
 * cache, found through the same block tables, and each kv head keeps tokens of its own.
 */

/*
 * Adds to the score of every token the attention weights that it had in a decode:
 *     scores(t, kv head) = decay * scores(t, kv head) + sum over the kv head's query heads h and
 *                          the sequence's query tokens of softmax(z)(t),
 * with the logits z of pa_decode (scale, softcap, alibi_slopes, sliding_window,
 * query_start as there).  exp_sums and max_logits are the statistics that pa_decode left in
 * PA_MODE_V2 for the same arguments, in the same shapes (v1, which PA_MODE_AUTO may run, leaves the
 * workspace as it was: what an earlier call left there would be taken).  The tokens of this step, the
 * last query_start[s+1] - query_start[s] of the sequence (without query_start the last one),
 * are set to their weights and not added to, so a slot's former score does not matter; decay 0
 * sets every token (the scores of a prompt, by its last tokens).  Tokens outside the window
 * only fade (with decay 1 pages before every row's window are not looked at).  Sums are fp32, in an order that does not depend on the run.  Places behind a
 * sequence's end keep their scores; a page whose block id is out of range is skipped
 * (PA_DEVERR_BLOCK_ID).  Each page belongs to one sequence: two that share one would both write
 * its scores.  num_kv_heads pages of keys of one block are less than 2^31 bytes.
 *
 * With alibi_slopes set relative_max in both calls.  Without it max_logits hold slope * position, and what
 * their rounding to fp32 has lost is a factor on all weights of a row: off by up to 2^-23 * slope *
 * seq_len (slope 0.8: 1e-4 at 1000 tokens, 1e-2 at 100000).
 */
typedef struct pa_weights_args {
    float* scores;               /* [num_blocks][num_kv_heads][16], updated in place */
    const void* query;           /* [rows][num_heads][head_size], dtype; 16-byte aligned */
    const void* key_cache;       /* as pa_decode */
    const int32_t* block_tables; /* [num_seqs][max_blocks_per_seq] */
    const int32_t* seq_lens;     /* [num_seqs], in [0, max_seq_len]; this step's tokens among them */
    const float* exp_sums;       /* [rows][num_heads][pa_max_num_partitions(max_seq_len)] */
    const float* max_logits;
    const float* alibi_slopes;   /* [num_heads] or NULL */
    const int32_t* query_start;  /* [num_seqs + 1] or NULL */
    int32_t* dev_error;          /* optional: PA_DEVERR_* bits */
    int32_t num_seqs;
    int32_t num_heads, num_kv_heads; /* max_query_len * (num_heads / num_kv_heads) <= 16 */
    int32_t head_size;           /* 64 or 128 */
    int32_t num_blocks;
    int32_t block_size;          /* must be PA_BLOCK_SIZE */
    int32_t max_seq_len;         /* as the decode had it, at most 2^30 */
    int32_t max_blocks_per_seq;
    int32_t num_query_tokens, max_query_len; /* with query_start */
    int32_t sliding_window;      /* as pa_decode: 0 = off */
    int32_t dtype;               /* pa_dtype of the query */
    int32_t layout;              /* pa_layout */
    int32_t kv_dtype;            /* pa_kv_dtype */
    float scale, softcap, k_scale;
    float decay;                 /* >= 0; 1: plain sums */
    int32_t relative_max;        /* as the decode had it */
} pa_weights_args;

/* num_seqs == 0 or max_seq_len == 0 is a no-op. */
pa_status pa_add_weights(const pa_weights_args* args, void* stream);

/*
 * The tokens that stay: of the n = seq_lens[s] tokens of sequence s, for each kv head,
 * new_seq_lens[s] = min(n, budgets[s]) of them, namely the last `recent`, the first `sink`
 * (both as far as the budget goes, the last ones first) and of the others those with the
 * largest scores (of equal ones the lower position; a NaN counts as less than any number).
 * kept[s][kv head][i], i < new_seq_lens[s], are their positions in ascending order; places behind
 * stay as they were.  n <= budgets[s]: all of them.  A length or budget outside its range is
 * clamped and reported (PA_DEVERR_SEQ_LEN); the scores of a page whose block id is out of
 * range (PA_DEVERR_BLOCK_ID) count as NaN.
 */
typedef struct pa_select_args {
    int32_t* kept;               /* [num_seqs][num_kv_heads][max_budget] */
    int32_t* new_seq_lens;       /* [num_seqs] */
    const float* scores;         /* [num_blocks][num_kv_heads][16]; 16-byte aligned */
    const int32_t* block_tables; /* [num_seqs][max_blocks_per_seq] */
    const int32_t* seq_lens;     /* [num_seqs], in [0, max_seq_len]; not new_seq_lens itself */
    const int32_t* budgets;      /* [num_seqs], in [0, max_budget] */
    int32_t* dev_error;          /* optional: PA_DEVERR_* bits */
    int32_t num_seqs, num_kv_heads, num_blocks;
    int32_t block_size;          /* must be PA_BLOCK_SIZE */
    int32_t max_seq_len;         /* at most 2^30 */
    int32_t max_blocks_per_seq;
    int32_t max_budget;          /* at most 2^30 */
    int32_t sink, recent;        /* >= 0 */
} pa_select_args;

/* num_seqs == 0 is a no-op. */
pa_status pa_select_tokens(const pa_select_args* args, void* stream);

/*
 * Moves the tokens kept[s][kv head][i], i < new_seq_lens[s], to position i of their sequence, in the
 * pages that it has: keys, values and scores, in place and bit by bit.  The positions of a row
 * ascend strictly, so that kept[i] >= i and nothing is overwritten before it has moved; an
 * entry that does not (or whose page is out of range: PA_DEVERR_BLOCK_ID) is not moved
 * (PA_DEVERR_SLOT), and what its place and its row's later ones then hold is some token's old
 * or new contents.  Slots from new_seq_lens[s] on keep their bytes.  The block tables are not
 * changed: pages that no token is left in go back with pa_build_tables (keep_lens =
 * new_seq_lens).
 *
 * Caches as in pa_append_kv; num_key_heads and num_value_heads are multiples of
 * num_kv_heads, whose row of `kept` key head h follows: h / (num_key_heads / num_kv_heads), and
 * value heads likewise (differential caches: two key heads to each value head).
 */
typedef struct pa_compact_args {
    void* key_cache;             /* 16-byte aligned */
    void* value_cache;
    float* scores;               /* [num_blocks][num_kv_heads][16] or NULL */
    const int32_t* block_tables; /* [num_seqs][max_blocks_per_seq] */
    const int32_t* kept;         /* [num_seqs][num_kv_heads][max_budget] */
    const int32_t* new_seq_lens; /* [num_seqs], in [0, max_budget] */
    int32_t* dev_error;          /* optional: PA_DEVERR_* bits */
    int32_t num_seqs, num_kv_heads, max_budget; /* max_budget at most 2^30 */
    int32_t num_key_heads, key_head_size; /* head sizes: 64, 128 or 256 (4-bit: not 256) */
    int32_t num_value_heads, value_head_size;
    int32_t num_blocks;          /* below 2^27 */
    int32_t block_size;          /* must be PA_BLOCK_SIZE */
    int32_t max_blocks_per_seq;  /* max_budget <= 16 * max_blocks_per_seq */
    int32_t dtype;               /* pa_dtype of the caches with kv_dtype PA_KV_SAME */
    int32_t layout;              /* pa_layout */
    int32_t kv_dtype;            /* pa_kv_dtype */
} pa_compact_args;

/* num_seqs == 0 or max_budget == 0 is a no-op. */
pa_status pa_compact_kv(const pa_compact_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* PA_CACHE_H */
