/*
 * atlas_evict.h -- a K/V cache kept under a budget of keys per (sequence, kv head) by
 * dropping the keys that received the least attention.
 *
 * Three calls, each useful alone:
 *   atlas_kv_weights   adds the attention weight that each cached key received from the
 *                      given query rows to a running total per (sequence, kv head, key);
 *   atlas_kv_select    picks the keys that stay: the first and the most recent ones
 *                      always, the others by their total;
 *   atlas_kv_compact   moves the kept rows of K and V together, in the sequence's own
 *                      pages or into fresh ones.
 * After them the sequence has new_lens[b] cached keys in their old order, and the
 * attention calls of atlas_attn.h run on it as on any cache (keys carry their rotary
 * positions, so a key's slot may differ from its token's position; new tokens are
 * written with atlas_kv_append_rope, which takes positions apart from slots).
 *
 * Which keys go is decided for each kv head by itself; all heads of a sequence keep
 * equally many, so one seq_lens entry and one page table serve them.
 *
 * Sources: the CFR-Atlas README ("What CFR-Atlas is") bounds resident K/V by bytes and
 * is exact because pages come back; the pages have no counterpart that drops keys for
 * good.  An evicted cache is an approximation its user chose.
 *
 * Layouts, ownership, asynchrony and errors are those of atlas_attn.h: device pointers
 * owned by the caller, everything enqueued on `stream`, host checks before anything is
 * launched, data-dependent problems as ATLAS_DEV_* bits in *status_word.  What a call writes
 * may not overlap what it reads, or another of its outputs, but where a call says so.
 */
#ifndef ATLAS_EVICT_H
#define ATLAS_EVICT_H

#include "atlas_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Arguments of atlas_kv_weights beyond its pointer / size list. */
typedef struct {
    int32_t batch;
    int32_t max_pages_per_seq;
    int32_t num_pages;
    int32_t q_len;             /* query rows per head; batch * n_q_heads * q_len < 2^31 - 1 */
    atlas_dtype dtype;         /* of q and the K pool */
    float *weights;            /* [batch][n_kv_heads][row_tokens]; 4-byte aligned */
    int32_t row_tokens;        /* floats per (sequence, kv head): at least the longest seq_len */
    int32_t accumulate;        /* 1: add to weights; 0: overwrite them */
    const int32_t *q_lens;     /* optional device [batch]: ragged query counts, as in atlas_launch */
    int32_t window;            /* as the attention call that made lse */
    float softcap;
    void *workspace;           /* device scratch, >= atlas_kv_weights_workspace_size() bytes */
    size_t workspace_bytes;
    uint32_t *status_word;
    void *stream;
    int32_t sm_count;          /* as in atlas_launch */
} atlas_weights;

/*
 * atlas_kv_weights: for b < batch, kv head g and key t < seq_lens[b],
 *   weights[b][g][t] (+)= sum over the q heads h of group g and the query rows i that see
 *                         key t of  exp(s - lse[b][h][i]),
 * where s is the scaled (and soft-capped) score of row i and key t, lse what the
 * attention call with the same q, scale, window, softcap and q_lens returned, and "sees"
 * is the suffix rule of atlas_attn.h: the rows are the last q_len (or q_lens[b])
 * positions of the sequence.  With sinks the lse includes them and the weights of a row
 * sum to less than 1.  Decode (q_len 1), the last rows of a prompt as observers, and a
 * whole prompt (q_len = seq_len) are the same call.  Sums and exponentials are float32;
 * the sum's order depends only on the call's sizes.  A row whose lse is -inf saw nothing
 * and adds nothing.  Keys t >= seq_lens[b] are not touched.  A bad seq_len or q_len
 * (seq_len < rows, > max_pages_per_seq * page_tokens or > row_tokens) sets
 * ATLAS_DEV_BAD_SEQLEN and a page id outside [0, num_pages) ATLAS_DEV_BAD_PAGE; the
 * weights of that sequence (of the keys on that page) are left as they were.
 * ATLAS_DEV_TIMEOUT leaves the keys concerned NaN.  Infinities and NaN in K are not
 * scanned for and stay with their key: its weight is exp of its scores (0, infinite or
 * NaN), or NaN in float32 calls with more than two rows per (sequence, kv head), whose
 * scores are sums of tf32 parts; other keys' weights do not depend on it, a key that no
 * row sees gets 0 whatever it holds, and atlas_kv_select counts NaN as -inf.
 * Supported sizes and types are those of the attention calls.
 */
atlas_status atlas_kv_weights(const void *q, const void *k_pages, const int32_t *page_table,
                              const int32_t *seq_lens, const float *lse, int32_t n_q_heads,
                              int32_t n_kv_heads, int32_t head_dim, int32_t page_tokens,
                              float scale, const atlas_weights *W);

/* Bytes of workspace the call needs (0 if none; SIZE_MAX if the arguments are invalid);
 * reads the sizes of *W and ignores its pointers. */
size_t atlas_kv_weights_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t page_tokens, const atlas_weights *W);

/* Arguments of atlas_kv_select beyond its pointer / size list. */
typedef struct {
    int32_t batch;
    int32_t row_tokens;        /* floats per row of weights: at least the longest seq_len */
    int32_t budget;            /* keys to keep, >= 1 */
    int32_t keep_first;        /* the first keep_first keys always stay, */
    int32_t keep_recent;       /* and the last keep_recent; together at most budget */
    int32_t kept_row_tokens;   /* floats per row of kept_weights: 0 (budget of them) or at least
                                  budget, with room for the keys that are to come */
    int32_t *kept;             /* [batch][n_kv_heads][budget], written */
    int32_t *new_lens;         /* [batch], written: min(seq_lens[b], budget) */
    float *kept_weights;       /* optional [batch][n_kv_heads][kept_row_tokens], written: the
                                  totals of the kept keys */
    uint32_t *status_word;
    void *stream;
} atlas_select;

/*
 * atlas_kv_select: for each (sequence, kv head), the keys that stay: all of them when
 * seq_lens[b] <= budget; else the first keep_first, the last keep_recent, and of those
 * between the ones with the largest weights, equal weights by the lower index (-0 equals
 * 0; a NaN counts as -inf).  kept holds their indices in ascending order, then -1 up to
 * the budget; kept_weights the totals, then 0 to the row's end: the weights that
 * atlas_kv_weights goes on adding to after atlas_kv_compact, if its rows (row_tokens there)
 * have room for the longest seq_len to come.  A seq_len below 0 or above row_tokens
 * sets ATLAS_DEV_BAD_SEQLEN and counts as 0.  kept, new_lens and kept_weights that overlap
 * weights, seq_lens (lengths updated in place) or one another are ATLAS_ERR_INVALID_ARG:
 * all of a row's CTAs read them while others write.
 */
atlas_status atlas_kv_select(const float *weights, const int32_t *seq_lens, int32_t n_kv_heads,
                             const atlas_select *S);

/* Arguments of atlas_kv_compact beyond its pointer / size list. */
typedef struct {
    int32_t batch;
    int32_t max_pages_per_seq; /* row length of page_table */
    int32_t num_pages;
    int32_t max_kept;          /* row length of kept */
    atlas_dtype kv_dtype;
    const int32_t *new_page_table; /* device [batch][new_max_pages]: the pages of the compacted
                                  sequences; NULL: their own, in place */
    int32_t new_max_pages;     /* row length of new_page_table */
    uint32_t *status_word;
    void *stream;
} atlas_compact;

/*
 * atlas_kv_compact: rows of both pools move, for b < batch, kv head g, j < new_lens[b]:
 *   row j of the compacted sequence = row kept[b][g][j] of the sequence
 * with rows found through the page tables.  kept: [batch][n_kv_heads][max_kept]; rows
 * from new_lens[b] on are not written, nor are other pages.
 *   In place (new_page_table NULL): each kept row must be strictly ascending (as
 *     atlas_kv_select writes it), and the pages of the batch's sequences must not be
 *     shared with one another or with anyone who still needs them.  The pools must be two
 *     (overlapping ones are ATLAS_ERR_INVALID_ARG: each would move the other's rows).
 *     Rows move in order, on at most 16 CTAs per (sequence, kv head): one long sequence of
 *     few heads is faster into fresh pages.
 *   Into fresh pages: all different, and none of them a page that page_table's sequences
 *     use; kept rows may be in any order and repeat.  Shared pages (a common prefix) stay intact.
 * An index outside the sequence's table (in place: also one below its own j) or a
 * new_lens[b] that does not fit sets ATLAS_DEV_BAD_SEQLEN, a bad page id
 * ATLAS_DEV_BAD_PAGE; the rows concerned are skipped.
 */
atlas_status atlas_kv_compact(void *k_pages, void *v_pages, const int32_t *page_table,
                              const int32_t *kept, const int32_t *new_lens, int32_t n_kv_heads,
                              int32_t head_dim, int32_t page_tokens, const atlas_compact *C);

#ifdef __cplusplus
}
#endif

#endif /* ATLAS_EVICT_H */
