// internal.h -- parameter blocks and launchers shared by the host entry points
// (atlas_attn.cu) and the kernel translation units.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "atlas_attn.h"

namespace atlas {

// Whether every pointer can be read as 32-bit words (a null one can).
inline bool aligned4(std::initializer_list<const void *> pointers) {
    uintptr_t bits = 0;
    for (const void *p : pointers) bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 3u) == 0;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A bounded wait gives up after this long and reports ATLAS_DEV_TIMEOUT.
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// Keys per pipeline stage of the split-KV kernels.
constexpr int kSplitBlockTokens = 64;

// Query tiles whose rows see fewer keys than this use a hi + lo split of P:
// with few keys (or a peaked softmax) a single bf16 rounding of P moves the
// output by up to 2^-8 |v| (bf16 keeps 8 significant bits).  Scores sharper than
// unit-variance inputs at scale 1/sqrt(D) (|scale| sqrt(D) above kHiLoScale) use
// the split on every tile.  Elsewhere the kernel decides per block (fmha_tc.cu).
constexpr int kHiLoBelow = 512;
constexpr float kHiLoScale = 1.25f;
inline int hilo_below(float scale, int D) {
    return fabsf(scale) * sqrtf((float)D) > kHiLoScale ? INT32_MAX : kHiLoBelow;
}

// Balanced split geometry of the tensor-core path: a context of L keys is cut into
// n = ceil(L / chunk) splits of round_up(ceil(L / n), 128) keys (the last one
// shorter), split s covering keys [s * size, (s + 1) * size).  The kernels and the
// merge derive it from seq_lens alike.
__host__ __device__ inline int balanced_split(int L, int chunk) {
    const int Lc = L < 1 ? 1 : L;
    const int n = (Lc + chunk - 1) / chunk;
    const int per = (Lc + n - 1) / n;
    return (per + 127) / 128 * 128;
}
// Largest batch whose splits the tensor-core kernels order longest-first (each CTA
// ranks the batch's sequences itself).
constexpr int kTcOrderMaxSeqs = 128;

// Everything the split-KV kernels (bf16 mma.sync and f32) and the merge need.
// "Columns" are the query rows one (sequence, kv head) owns: column n is q head
// g = n / q_len of the group and query row i = n % q_len.
struct SplitParams {
    const void *q;              // [B][Hq][q_len][D]
    const void *k_pages;        // f32 path reads the pools directly
    const void *v_pages;
    const int32_t *page_table;  // [B][max_pages]
    const int32_t *seq_lens;    // [B]
    int32_t B, Hq, Hkv, G, D, P, q_len, max_pages, num_pages;
    int32_t chunk;              // keys per split (multiple of 64)
    int32_t n_chunks;           // splits per (sequence, kv head): ceil(max_pages*P / chunk)
    int32_t col_tiles;          // ceil(G*q_len / columns per CTA)
    int32_t require_full;       // prefill: seq_len must equal q_len
    // Keys one query row sees more than the row before it: 1 (causal), or 0 for cross
    // attention, whose rows all see the seq_len encoder states (possibly none).
    int32_t row_step;
    float scale_log2;           // scale * log2(e)
    int32_t window;             // > 0: keys pos - window < t <= pos only
    float softcap_log2;         // > 0: s2 = softcap_log2 * tanh(raw * softcap_inv)
    float softcap_inv;          // scale / softcap
    const int32_t *q_lens;      // [B] ragged query rows (<= q_len) or null
    const int32_t *chunk_range; // [B][2] splits [lo, hi) this launch computes, or null (all)
    float *ws_acc;              // [B*Hq*q_len][n_chunks][D]   unnormalised accumulators
    float *ws_ml;               // [B*Hq*q_len][n_chunks][2]   (m in log2 units, l)
    uint32_t *status;           // may be null
    uint32_t debug_flags;
    // Direct mode (bf16): one split covers the whole context; the split kernel
    // writes the output rows itself (no workspace, no merge).
    int32_t direct;
    // Cluster mode (f32): the n_chunks (<= 8) splits of one (sequence, kv head,
    // column tile) run as one thread-block cluster and merge through distributed
    // shared memory; rank 0 writes the output rows (no workspace, no merge launch).
    int32_t cluster;
    void *out;
    int32_t out_bf16;
    float *lse;
    const float *sinks;         // [Hq] natural-log logits or null (direct mode only)
};

// The split-KV kernels' call with shared prefixes in the same launch (shared_prefix.cu): CTAs
// below own_items are the sequences' own splits, the others take the prefixes'.
struct SharedSplitParams : SplitParams {
    const int32_t *prefix_table;  // [n_groups][max_prefix_pages]
    const int32_t *prefix_lens;   // [n_groups]
    const int32_t *group_starts;  // [n_groups + 1]
    int32_t n_groups, max_prefix_pages;
    int32_t pre_chunk, n_pre;     // keys per split, splits of the longest prefix
    int32_t own_items;            // n_chunks * Hkv * col_tiles * B
    int32_t cols;                 // columns per CTA: bf16 8 or 16, fp32 4, 8 or 16
    float *pre_acc, *pre_ml;      // as SharedMergeParams
    const int32_t *order;         // the own items' sequences, longest first, or null (the batch's)
    int32_t after_prefix;         // 1: a dependent of the prefixes' launch (own items alone)
};

// A call's kernels (atlas_attn.cu); the entry points are this and a kind.
atlas_status run_attention(atlas_kind kind, const void *q, const void *k_pages, const void *v_pages,
                           const int32_t *page_table, const int32_t *seq_lens, int32_t Hq,
                           int32_t Hkv, int32_t D, int32_t P, float scale, const atlas_launch *L);

struct MergeParams {
    const int32_t *seq_lens;
    int32_t B, Hq, D, q_len, max_pages, P, chunk, n_chunks, require_full;
    int32_t balanced;           // splits of balanced_split(seq_len, chunk) keys
    int32_t row_step;           // 1 causal, 0 cross attention (as in SplitParams)
    int32_t window;             // splits below a row's window hold nothing for it
    const float *sinks;         // [Hq] natural-log logits or null: one more state (m, 1, 0)
    const int32_t *q_lens;      // [B] ragged query rows or null; padding rows untouched
    const float *ws_acc;
    const float *ws_ml;
    void *out;
    int32_t out_bf16;
    float *lse;
    int32_t sms;            // SM count: sizes the warps per row
    int32_t warps_per_row;  // set by launch_merge
};

// A CTA's piece of a tile.
struct SharedSeg {
    int unit, hkv, row0;   // the tile's first row (of the unit's, in one kv head)
    int rows;              // the unit's rows
    int blk0, nb;          // blocks [blk0, blk0 + nb) of the tile
    int state;             // index of its partial state; -1: the tile is not cut
    int len, own;          // keys of the prefix, own keys that the tile's rows see at most
    int group;             // whose prefix (-1: none)
};

// A tile over whole keys (st.whole) that is cut first behind the CTA that it begins in: its rows,
// and the CTAs that have blocks of it (0: none is).
struct SharedCut {
    int unit, hkv, row0, rows, states;
};

// The tiles of a call with shared prefixes on the tensor cores, cut evenly among CTAs
// (shared_prefix.cuh).  Arrays in the workspace, written by the plan kernel.
struct SharedStream {
    // by the host
    const int32_t *prefix_table, *prefix_lens, *group_starts;
    int32_t n_groups, max_prefix_pages;
    int32_t whole;       // 0: units are groups, their prefixes alone; 1: units are sequences,
                         // their prefix and their own keys
    int32_t units;       // n_groups or batch
    int32_t tile_rows;   // rows of a CTA's tiles: 128 or 256
    int32_t max_items;   // (tile, key range) pieces of one CTA at most
    int32_t max_states;  // CTAs that a tile may be cut among at most (whole 0)
    int32_t sms;
    // by the plan kernel
    int32_t *head;       // [2]: a CTA's length of the line, and all of it
    int32_t *first;      // [units + 1] where the units begin
    int32_t *head_cost;  // [units] length of one kv head's tiles
    int32_t *blocks;     // [units] blocks of a tile; -1: out of range, its rows are NaN
    int32_t *weight;     // [units] blocks that a tile counts for (short ones count for more)
    int32_t *rows;       // [units] rows of one kv head
    int32_t *group;      // [batch] the sequence's group, or -1
    int32_t *before;     // [batch + 1] rows of one kv head of the sequences before
    int32_t *list;       // ragged groups: [batch * G * q_len] the rows (of kv head 0), or null
    SharedSeg *segs;     // [CTAs][max_items] the CTAs' pieces,
    int32_t *counts;     // [CTAs] and how many
    SharedCut *cuts;     // whole: [CTAs] the tile that is cut behind each
    int32_t *order;      // [batch] the sequences, those of most own keys first
    int32_t *info;       // [batch][8]: what the merge wants to know of a sequence (SeqInfo)
    int32_t wait_first;  // 1: wait for the grid before at the start, 0: at the end (the plan's is
                         // done by then)
    float own_rate;      // bytes a microsecond that an SM takes of the own keys' splits, which run
                         // beside the tiles; 0: nothing runs beside them
};
// SharedStream::info, for the place of a row's tile in the line.
struct SeqInfo {
    int32_t blocks;      // of a tile; 0: no prefix; -1: out of range, the rows are NaN
    int32_t row0;        // rows of the group before it: row f = row0 + q head * query rows + row
    int32_t rows, first, head_cost, weight, per, pad;
};

// The same with the splits of the sequence's shared prefix (shared_prefix.cu) as further
// states of each row.
struct SharedMergeParams : MergeParams {
    const int32_t *group_starts;  // [n_groups + 1]
    const int32_t *prefix_lens;   // [n_groups]
    int32_t n_groups, max_prefix;
    int32_t pre_chunk, n_pre;     // keys per split, splits of the longest prefix (pre_chunk 0:
                                  // the tiles of st, n_pre states at most)
    const float *pre_acc;         // [B*Hq*q_len][n_pre][D]
    const float *pre_ml;          // [B*Hq*q_len][n_pre][2]
    int32_t G;
    SharedStream st;
};

// A bit of atlas_launch.debug_flags for the library's own calls: TcParams::nearest.
constexpr uint32_t kNearestProducts = 1u << 31;

// Tensor-core (tcgen05 / TMEM) path for many query rows per (sequence, kv head):
// 128-row query tiles x 128-key blocks (bf16) or 64-key blocks (fp32 as 3 x tf32),
// head_dim 64 or 128.  Either writes the
// normalised output directly (one CTA per tile, all its keys) or, when there are
// too few tiles to fill the GPU, split partials in the SplitParams layout.
struct TcParams {
    const int32_t *page_table;
    const int32_t *seq_lens;
    int32_t B, Hq, Hkv, G, D, P, q_len, max_pages, num_pages;
    int32_t tiles_per_unit;   // ceil(G * q_len / 128)
    int32_t tiles_per_head;   // q_len / 128 when q_len % 128 == 0 (heavy-first order), else 0
    int32_t split;            // 1: write split partials; 0: write the output
    int32_t chunk, n_chunks;  // split geometry (chunk a multiple of 128)
    int32_t balanced;         // split mode: balanced splits in longest-first order
                              // (tc_order.cuh); the grid's CTAs are work items
    int32_t require_full;
    int32_t row_step;         // 1 causal, 0 cross attention (as in SplitParams)
    int32_t hilo_below;       // tiles whose rows see fewer keys use a hi+lo split of P
    int32_t negate_scores;    // scale < 0: S = -Q K^T with |scale| (keeps the max exact)
    float scale_log2;         // |scale| * log2(e)
    int32_t window;           // > 0: keys pos - window < t <= pos only
    float softcap_log2;       // > 0: s2 = softcap_log2 * tanh(raw * softcap_inv)
    float softcap_inv;        // |scale| / softcap
    const float *sinks;       // [Hq] or null (direct mode folds it into the epilogue)
    const int32_t *q_lens;    // [B] ragged query rows (<= q_len) or null
    const int32_t *chunk_range;  // split mode: [B][2] splits [lo, hi) to compute, or null
    void *out;
    int32_t out_bf16;
    float *lse;
    float *ws_acc, *ws_ml;
    uint32_t *status;
    int32_t sms;         // SM count (sizes the persistent prefill grid)
    // Prefixes shared by groups of sequences.  fp32 (split mode): page_table, seq_lens and
    // max_pages are the prefixes', one row for each group, the tiles' rows those of all of a
    // group's sequences; bf16: the tiles of st.
    const int32_t *group_starts;  // [n_groups + 1] first sequences, or null
    int32_t n_groups;
    const void *q;                // read row by row there (no tensor map)
    SharedStream st;
    int32_t nearest;              // fp32: the more exact form of the products
};

// Paged KV append (kv_append.cu).
struct AppendParams {
    const void *k_new, *v_new;  // [B][Hkv][max_new][D]
    void *k_pages, *v_pages;    // [num_pages][Hkv][P][D]
    const int32_t *page_table, *seq_lens, *n_new;
    int32_t B, Hkv, max_new, P, max_pages, num_pages, row_bytes;
    uint32_t *status;
};
cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream);

cudaError_t launch_fmha_tc(const TcParams &p, const CUtensorMap &tmQ, const CUtensorMap &tmK,
                           const CUtensorMap &tmV, cudaStream_t stream);
// The tiles of p.st (bf16; with st.whole the call's output, else partial states and a
// dependent of the launch before), or the splits of shared prefixes, `ctas` of them at most.
// Borders of n_groups groups of B sequences among the n from b0 on.
cudaError_t launch_shared_starts(const int32_t *starts, int32_t *mine, int n_groups, int B, int b0, int n,
                                 cudaStream_t stream);
// p.st's arrays, one CTA; and the output rows of the tiles that are cut (st.whole).
cudaError_t launch_shared_plan(const TcParams &p, cudaStream_t stream);
cudaError_t launch_shared_cut_merge(const TcParams &p, int64_t ctas, cudaStream_t stream);
int shared_tc_items(int tiles);  // st.max_items for that many tiles of 128 rows to a CTA
cudaError_t launch_shared_tc(const TcParams &p, int64_t ctas, const CUtensorMap &tmK,
                             const CUtensorMap &tmV, cudaStream_t stream);
cudaError_t launch_shared_tc_f32(const TcParams &p, int64_t ctas, const CUtensorMap &tmK,
                                 const CUtensorMap &tmV, cudaStream_t stream);
// The same for fp32 q/K/V: three tf32 products per fp32 product (fmha_tc_f32.cu).
cudaError_t launch_fmha_tc_f32(const TcParams &p, const CUtensorMap &tmQ, const CUtensorMap &tmK,
                               const CUtensorMap &tmV, cudaStream_t stream);

// TMA view of a bf16 (or fp32) tensor with D elements per row: `rows` rows; boxes of
// one 128-byte row slab (64 bf16 or 32 fp32 elements) x box_rows rows with 128-byte
// swizzling.
atlas_status encode_rows_map(CUtensorMap *map, const void *base, int64_t rows, int32_t D,
                             int32_t box_rows, bool f32 = false);

// Columns handled by one CTA of the bf16 split kernel.
int split_bf16_cols_per_cta(int G, int q_len);

cudaError_t launch_split_bf16(const SplitParams &p, const CUtensorMap &tmK, const CUtensorMap &tmV,
                              cudaStream_t stream);
// fp32 with few columns: 4, 8 or 16 columns per CTA by G x q_len.
int split_f32_cols_per_cta(int G, int q_len);
cudaError_t launch_split_f32(const SplitParams &p, cudaStream_t stream);
// `ctas`: the own items and the most that the prefixes may be.
cudaError_t launch_shared_split_bf16(const SharedSplitParams &p, int64_t ctas, const CUtensorMap &tmK,
                                     const CUtensorMap &tmV, cudaStream_t stream);
cudaError_t launch_shared_split_f32(const SharedSplitParams &p, int64_t ctas, cudaStream_t stream);
// Tensor map of a page pool for the bf16 split kernel.
atlas_status encode_pool_map(CUtensorMap *map, const void *pool, int32_t num_pages, int32_t Hkv,
                             int32_t P, int32_t D);
cudaError_t launch_merge(const MergeParams &p, cudaStream_t stream);
cudaError_t launch_shared_merge(const SharedMergeParams &p, cudaStream_t stream);

// Multiprocessor count of the current device (cached per device); 152 (one
// GB300) when no device is visible.
int device_sm_count();

// The split plan of a call: which kernel path, split geometry and workspace.  A
// pure function of the call's sizes and the SM count (atlas_launch.sm_count, else
// device_sm_count()).
enum class Path { SplitBF16, SplitF32, TensorCore, TensorCoreF32 };

struct Plan {
    Path path;
    int direct;   // bf16 split kernel: one split, output written directly
    int cluster;  // f32 split kernel: splits merged inside one thread-block cluster
    int balanced; // tensor-core split mode: equal splits per sequence, longest first
    int chunk, n_chunks, col_tiles, G;
    int tc_split, tiles_per_unit, tiles_per_head;
    size_t acc_bytes, ml_offset, ws_bytes;
};

atlas_status make_plan(atlas_kind kind, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                       const atlas_launch *L, Plan *plan);

}  // namespace atlas
