/*
 * atlas_pages.h -- page tables made on the device from the sequences' lengths.
 *
 * Every attention call and append takes a page_table; this call makes it.  The pages that
 * nobody holds stand in a ring on the device, and each step's call gives every sequence the
 * pages that its length needs: new tokens of a running request or a prompt that comes take
 * pages, a request that ends, drafted tokens that were not accepted and a cache that
 * atlas_kv_select cut give theirs back.  Lengths may be results of the device (the new_lens of
 * a cut): nothing is read on the host, and a captured step replays with whatever they are.
 *
 * Sources: the CFR-Atlas README, "Minimal integration", reaches K/V through pages of a fixed
 * size per (layer, kv head, token range) and leaves their bookkeeping to the backend.
 *
 * Layouts, ownership, asynchrony and errors are those of atlas_attn.h; arrays are 4-byte
 * aligned.
 */
#ifndef ATLAS_PAGES_H
#define ATLAS_PAGES_H

#include "atlas_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A further bit of *status_word: pages ran out, and some sequence kept what it had. */
#define ATLAS_DEV_NO_PAGES 8u

/* Arguments of atlas_kv_resize beyond its pointer / size list. */
typedef struct {
    int32_t batch;             /* batch * max_pages_per_seq and batch * max_new < 2^31 */
    int32_t max_pages_per_seq; /* row length of page_table */
    int32_t num_pages;         /* pages in each pool: entries of free_pages; times page_tokens
                                  < 2^31 */
    int32_t max_new;           /* row length of slots; 0: no slots wanted */
    const int32_t *n_new;      /* optional device [batch]: each sequence's new tokens, the last
                                  n_new[b] of its seq_lens[b], at most max_new; NULL: max_new of
                                  them, or all where it has fewer.  Read for slots only */
    int32_t *slots;            /* optional device [batch][max_new], written */
    uint32_t *status_word;
    void *stream;
} atlas_resize;

/*
 * atlas_kv_resize: sequence b shall hold ceil(seq_lens[b] / page_tokens) pages.  Where
 * n_pages[b] is less, it takes pages from the front of the ring, in the order of the batch,
 * into page_table[b][n_pages[b]], ...; where it is more, the pages behind go to the end of the
 * ring, in the order of the batch and of the row, and their entries become -1.  Pages given
 * back may be taken from the next call on.  n_pages and free_state then say what holds; entries
 * that nobody took or gave back keep their values.
 *   free_pages   device [num_pages], the ring: free_state[1] free pages from entry
 *                free_state[0] on (modulo num_pages).  At first: all page ids, state {0,
 *                num_pages}, n_pages all 0.
 *   slots        slots[b][i] = page_table[b][t / page_tokens] * page_tokens + t % page_tokens for
 *                the i-th new token, t = seq_lens[b] - n_new[b] + i: its place in a pool seen as
 *                [num_pages * page_tokens] tokens; -1 for i >= n_new[b], and for a sequence
 *                whose new tokens have no room.
 * When the ring has too few pages, sequences are served in order as long as all that they and
 * those before them lack fits; the others that lack pages keep what they have and
 * ATLAS_DEV_NO_PAGES is set.  A seq_len below 0 or above max_pages_per_seq * page_tokens, an
 * n_pages out of range, or an n_new below 0 or above max_new or seq_lens[b] sets
 * ATLAS_DEV_BAD_SEQLEN and leaves that sequence as it is.  A free_state out of range, or more
 * pages given back than the ring has room for, sets ATLAS_DEV_BAD_PAGE and moves nothing at
 * all; every slot is -1 then.  A page id outside [0, num_pages) that is taken, given back or asked for a slot sets
 * ATLAS_DEV_BAD_PAGE; ids are passed on as they are, and such a slot is -1.
 * page_table, n_pages, free_pages, free_state and slots are written and may not overlap one
 * another or what is read (ATLAS_ERR_INVALID_ARG).
 */
atlas_status atlas_kv_resize(int32_t *page_table, int32_t *n_pages, const int32_t *seq_lens,
                             int32_t *free_pages, int32_t *free_state, int32_t page_tokens,
                             const atlas_resize *Z);

#ifdef __cplusplus
}
#endif

#endif /* ATLAS_PAGES_H */
