/*
 * atlas_shared.h -- attention of a batch whose sequences share prefixes.
 *
 * Requests that begin with the same tokens (a system prompt, a document, the examples of a
 * task) need the prefix's K/V once.  Here it has pages and a table row of its own, and each
 * sequence has its own cache behind it, a page table and a length as any sequence of
 * atlas_attn.h: appends, atlas_kv_weights and the cut of a cache work on that as they stand
 * (slots start at 0 behind the prefix; rotary positions go on from it, and the calls that
 * rotate take positions apart from slots).  One call attends to both parts, and reads a
 * prefix once for all the sequences that share it, not once for each.
 *
 * Sources: CFR-Atlas README, "Core contract": exact pages folded into one online-softmax
 * state give the full-K/V result, in whatever parts and order they are folded; the CPUAttn
 * README, "Operator model", joins parts of the key axis by a structured merge.  The pages
 * have no entry point for a prefix of several sequences.
 *
 * Layouts, ownership, asynchrony and errors are those of atlas_attn.h.
 */
#ifndef ATLAS_SHARED_H
#define ATLAS_SHARED_H

#include "atlas_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Test-only bits of atlas_launch.debug_flags: prefixes on the split kernels, in one launch with the
 * sequences' own keys (at most 16 rows to a sequence and kv head), or on the tensor-core ones. */
#define ATLAS_DEBUG_SHARED_SPLIT 4u
#define ATLAS_DEBUG_SHARED_TC 8u
/* ... (with it) bf16 sequences in tiles of their own, over the prefix and their own keys. */
#define ATLAS_DEBUG_SHARED_WHOLE 16u

/* The shared prefixes of a call: group n is the neighbouring sequences group_starts[n] <= b <
 * group_starts[n + 1], and their prefix the first prefix_lens[n] keys of prefix_table[n]. */
typedef struct {
    const int32_t *prefix_table; /* device [n_groups][max_prefix_pages], pages of the same pools;
                                    entries past a prefix's last page are never read */
    const int32_t *prefix_lens;  /* device [n_groups], each 0 (no prefix) .. max_prefix_pages *
                                    page_tokens; any length, whole pages or not */
    const int32_t *group_starts; /* device [n_groups + 1], ascending (an empty group repeats its
                                    start), from 0 or more to batch or less; sequences in no
                                    group have no prefix */
    int32_t n_groups;            /* 1 .. batch */
    int32_t max_prefix_pages;    /* row length of prefix_table, >= 1 */
} atlas_shared;

/*
 * atlas_attn_shared: for sequence b of group n, q head h of kv head g, row i < q_len (or
 * q_lens[b]),
 *   out[b][h][i] = sum_j exp(s_j - M) v_j / sum_j exp(s_j - M),  lse[b][h][i] = M + ln sum_j exp(s_j - M)
 * where j runs over all prefix_lens[n] keys of the prefix and over the sequence's own keys
 * t <= seq_lens[b] - q_len + i (the suffix rule of atlas_attn.h: the rows are the last q_len
 * positions of its own cache, page_table[b] and seq_lens[b], which do not count the prefix).
 * It is what atlas_attn_suffix returns for the two parts in one cache, to rounding.  q_len is 1
 * for a decode step.  Softcap, sinks (counted once), ragged q_lens and sm_count are those of
 * atlas_launch; its three events are recorded before the splits, after them and after the
 * merge.  split_tokens fixes the splits of the own keys and of prefixes on the split kernels; on
 * the bf16 tensor-core kernels, which cut a prefix where the SMs' shares end, it bounds the parts
 * of a prefix instead (max_prefix_pages * page_tokens / split_tokens + 2).  A window is
 * ATLAS_ERR_INVALID_ARG (it would cut the prefix off), a phase other than ATLAS_PHASE_ALL or a
 * chunk_range ATLAS_ERR_UNSUPPORTED.  out, lse and the workspace may not overlap one another, q
 * or the pools (ATLAS_ERR_INVALID_ARG).
 * A call whose partial states would take more than 512 MB runs in parts of neighbouring sequences, one
 * after the other in the same workspace (event 1: before the last part's merge); a single sequence of
 * very many rows may need more.  Refused as ATLAS_ERR_UNSUPPORTED, beside what atlas_attn_suffix
 * refuses: a sequence alone of more than 65535 tiles of 128 rows whose own keys are split, and one (or
 * its prefix) of more than 2^31 / 11 pairs of a 256-row tile and a 128-key block of its tables.
 * The same call on the same arrays gives the same bits.  On the split kernels a sequence's bits
 * depend on its own group alone (and on the sizes that the call is planned from); on the bf16
 * tensor-core kernels also on the other groups and lengths of the batch and on sm_count, which
 * decide where the shares of the SMs end.
 * On the device: group_starts out of order or out of range set ATLAS_DEV_BAD_SEQLEN and leave
 * every row NaN; a prefix length out of range does so for its group, a bad seq_len or q_len
 * for its sequence; a page id outside the pool sets ATLAS_DEV_BAD_PAGE and leaves the rows
 * that read it NaN.
 * Infinities and NaN in K and V are not scanned for and propagate to the rows that see them: a NaN
 * score, or one of +inf, makes its row NaN (in fp32 on the tensor cores any infinite key element does,
 * to all rows of its group and kv head), a score of -inf has no weight, and a value that is NaN or
 * infinite makes its element NaN or infinite.  A sink that is NaN or +inf makes its head's rows NaN.
 * Precision: the split kernels are those of atlas_attn_decode (bf16 weights as two bf16 parts,
 * fp32 products for fp32).  The bf16 tensor-core kernels take the weights as two bf16 parts for up
 * to 16 rows to a sequence and kv head (decode steps, drafted rows), as atlas_attn_decode and
 * atlas_attn_suffix do there: a step is as exact however many others share its prompt.  For more
 * rows they do so where the tiles have 128 rows (at most 128 to a kv head of a group, on average, or
 * of a sequence whose rows have tiles of their own), where the second part costs nothing, or where
 * few keys carry a row, and take one part elsewhere, as atlas_attn_suffix and atlas_attn_prefill do.
 * The fp32 one takes three tf32 products for each, within the 1e-5 of the largest value that holds
 * for all fp32 calls: 7e-7 to 1e-6 off in the root mean square (atlas_attn_suffix 2e-6), where the
 * split kernels are 2e-7 to 3e-7.
 */
atlas_status atlas_attn_shared(const void *q, const void *k_pages, const void *v_pages,
                               const int32_t *page_table, const int32_t *seq_lens,
                               int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                               int32_t page_tokens, float scale, const atlas_shared *S,
                               const atlas_launch *L);

/* Bytes of device workspace the call needs; reads the sizes of *S and *L (split_tokens, sm_count and
 * debug_flags among them), ignores their pointers.  SIZE_MAX if the call would be refused. */
size_t atlas_attn_shared_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        int32_t page_tokens, const atlas_shared *S,
                                        const atlas_launch *L);

#ifdef __cplusplus
}
#endif

#endif /* ATLAS_SHARED_H */
