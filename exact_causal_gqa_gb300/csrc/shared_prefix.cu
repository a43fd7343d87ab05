// shared_prefix.cu -- attention of a batch whose sequences share prefixes
// (include/atlas_shared.h): checks, the plan, and the launches.
//
// A row's softmax runs over two sets of keys, its sequence's own and its group's prefix.  Each
// set is cut into splits whose partial states (m, l, acc) go to the workspace, and one merge
// joins a row's states of both kinds.  Two ways to the prefixes' states:
//   split kernels: the own splits and those of the prefixes are CTAs of one launch of the
//     decode kernels (split_kv.cu).  A CTA has up to 16 of a group's rows, so a prefix is read
//     once for each 16 rows, from L2 for all but the first;
//   tensor cores: the tensor-core kernels take the prefixes with 128 or 256 of a group's rows
//     to a CTA (shared_prefix.cuh).  The own splits, on the split kernels or the tensor cores by
//     a sequence's rows and keys, are a launch of their own beside that one: the second of the two
//     is a dependent of the first, whose results it does not need, and its CTAs take the SMs as
//     those of the first leave them.
// bf16 sequences whose rows fill tiles by themselves have little use for a gather (whole_pays).
// Their tiles walk the prefix's blocks and go on with the sequence's own, in one launch, and write
// the output; only tiles that a cut between two CTAs goes through are merged.
// A batch whose states would take too much memory runs in parts (kMostBytes).
#include "internal.h"
#include "atlas_shared.h"
#include "shared_prefix.cuh"

#include <limits.h>
#include <math.h>
#include <algorithm>

namespace atlas {
namespace {

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SMs to plan for (a number that no device has is cut to what the plan's sums have room for).
int planned_sms(const atlas_launch *L) {
    return std::min(L->sm_count > 0 ? L->sm_count : device_sm_count(), 1 << 14);
}

struct Range {
    const void *at;
    size_t bytes;
};
bool meet(const Range &a, const Range &b) {
    const char *x = static_cast<const char *>(a.at), *y = static_cast<const char *>(b.at);
    return x && y && x < y + b.bytes && y < x + a.bytes;
}

struct SharedPlan {
    Plan own;
    bool few;              // at most 16 rows to a sequence and kv head: the decode kernels' calls
    bool split;            // the split kernels, in one launch
    bool whole, stream;    // bf16 on the tensor cores: whole tiles, or the prefixes' (both: stream)
    int tiles;             // tensor cores: query tiles to a CTA; split kernels: columns
    int chunk, n_pre;      // keys per prefix split, splits of the longest prefix (stream: states
                           // of a tile at most)
    int64_t ctas;          // most (group, kv head, split, rows of a CTA) items, or CTAs
    size_t acc_at, ml_at;  // the prefixes' states in the workspace (whole: the cut tiles')
    size_t plan_at;        // stream: its arrays
    size_t bytes;
    // The whole call: neighbouring sequences in parts of so many (the last has what is left), each
    // with the groups' borders among them in the workspace.
    int32_t part, parts;
    bool sparing;          // own keys in no more splits than fill the SMs
    size_t starts_at;
};

// States of a call at most, in bytes.  A batch that needs more runs in parts, one after the other, in
// the same workspace.  A part has some 10^5 rows of states and takes a millisecond or more, its
// launches, its end and another pass over the prefixes some 40 us: 1200 sequences of 4 rows in 40
// groups behind 4096 keys 928 -> 975 us in two parts, 64 of 300 rows behind 32768 9.0 -> 9.1 ms in five.
constexpr size_t kMostBytes = (size_t)512 << 20;

// CTAs of a wave of the split kernels, in hundredths of the SMs, and a CTA's keys at least.
constexpr int64_t kSplitWave = 200, kSplitWaveF32 = 300, kMinSplit = 128, kMinSplitF32 = 64;

// Keys of the own splits beside the tiles.
int64_t own_split(int64_t max_ctx) {
    const int64_t splits = (max_ctx + 4095) / 4096;
    return round_up((max_ctx + splits - 1) / splits, 64);
}

// Bytes a microsecond that the split kernels of 8 and of 16 columns take on one SM, when not all
// SMs ask for memory.
constexpr float kOwnRate = 70e3f, kOwnRateWide = 50e3f;

// Whether the split kernels take less time: the prefixes once for each CTA's rows, against the
// plan's launch, a longer start, and the prefixes once.  In fp32 the own keys count too: beside
// prefixes of more than 4 rows they are taken 8 columns wide, where 4 would do.
// Fitted to 56 measured sizes in bf16 and 20 in fp32: bf16, 32 / 8 heads of 128, one prefix, split
// kernels and tensor cores: 8 sequences behind 1024 keys 17 and 27 us, behind 32768 53 and 54; 16
// behind 8192 42 and 33; 32 behind 8192 67 and 35; 64 behind 1024 39 and 33, behind 32768 309 and 82;
// heads of 64, 64 in 4 groups behind 4096 43 and 33.  fp32: 8 behind 1024 23 and 42, behind 8192 73
// and 50; heads of 64, 32 in 4 groups behind 2000 61 and 43.
bool split_pays(double prefix_bytes, int64_t tiles, double flops, double own_bytes, bool own_twice, bool f32) {
    // bytes and floating point operations a microsecond
    if (!f32)
        return (double)tiles * prefix_bytes / 6e6 <= 13.0 + std::max(prefix_bytes / 5e6, flops / 9e8);
    const double tc = 28.0 + std::max(prefix_bytes / 2.7e6, flops / 1.2e8) + own_bytes / 6e6;
    return 10.0 + ((double)tiles * prefix_bytes + own_bytes * (own_twice ? 1.3 : 1.0)) / 3.6e6 <= tc;
}

// Rows and own keys of a sequence up to which the own keys of more than 16 rows are splits of the
// decode kernels (a CTA for each 16 rows) all the same: 64 sequences of 32 rows, up to 120 keys 73
// us and 79 on the tensor cores, up to 1000 103 and 107, up to 2500 148 and 134; of 48 rows 107 and
// 97 with 120.
constexpr int64_t kOwnSplitRows = 32, kOwnSplitKeys = 1024;

// Whether tiles over whole keys take less time than the prefixes' tiles, which the rows of a group's
// sequences fill, beside the own ones: a block of a prefix 2.0 us for 256 rows, and 1.1 where a
// sequence's (or a group's) end in the first half, against 9.5 for each own tile of 128 rows on the
// tensor cores, which has a launch, a start and states to itself there, or 2.6 where the own keys are
// splits.  Fitted to 98 sizes of 20 to 264 rows, prefixes of 300 to 16000 keys and 100 or 800 own ones
// (32 / 8 heads of 128), of which few lose more than 6 %; whole tiles and others, 100 own keys: 128
// sequences behind 1500 keys, 264 rows 424 and 536 us, 64 rows 180 and 177, 20 rows 178 and 103; 16
// behind 16000 keys, 264 rows 368 and 294.  Behind 16000 keys with 800 own ones, 80 rows: 2 sequences
// with a group each 53 and 65 us, 16 with a group each 179 and 187, 32 in 4 groups 318 and 207.
// Of `tiles` in all: where one is cut among more than 16 CTAs, of two blocks each at least, the merge of
// its states, one after the other, takes longer than is saved: a sequence of 80 rows and one kv head
// behind 32768 keys 99 us for 31, behind 8192 43 for 29; of 8 kv heads 65 for 72, and 41 for 33.
bool whole_pays(int64_t rows, int64_t group_rows, int64_t max_prefix, int64_t max_ctx, int64_t tiles, int64_t sms,
                bool own_splits) {
    if (std::min(sms / tiles, (max_prefix + max_ctx) / 256) > 16) return false;
    auto block = [](int64_t n) {  // of the tiles of n rows
        const int64_t pairs = n / 256 + (n % 256 > 128), single = n % 256 > 0 && n % 256 <= 128;
        return 2.0 * (double)pairs + 1.1 * (double)single;
    };
    const double more = block(rows) - block(group_rows) * (double)rows / (double)group_rows;
    return (double)((max_prefix + 127) / 128) * more <=
           (own_splits ? 2.6 : 9.5) * (double)((rows + 127) / 128);
}

// The plan of a part: L is its launch, `groups` the groups that it has, on average.  `sparing`: own
// keys in no more splits than fill the SMs.
atlas_status plan_part(int32_t Hq, int32_t Hkv, int32_t D, int32_t P, const atlas_shared *S,
                       const atlas_launch *L, int32_t groups, bool sparing, SharedPlan *plan) {
    if (L->window != 0) return ATLAS_ERR_INVALID_ARG;
    if (L->phase != ATLAS_PHASE_ALL || L->chunk_range) return ATLAS_ERR_UNSUPPORTED;
    if (L->split_tokens < 0 || L->split_tokens % kSplitBlockTokens != 0) return ATLAS_ERR_INVALID_ARG;
    // The call's checks, and its kernels without prefixes.  (No splits: what those may be too many
    // for counts only where they are launched.)
    atlas_launch own = *L;
    own.split_tokens = 0;
    own.debug_flags |= ATLAS_DEBUG_TC_DIRECT;
    atlas_status st = make_plan(ATLAS_KIND_SUFFIX, Hq, Hkv, D, P, &own, &plan->own);
    if (st != ATLAS_OK) return st;
    own.split_tokens = L->split_tokens;
    own.debug_flags = L->debug_flags & ~ATLAS_DEBUG_TC_DIRECT;
    own.phase = ATLAS_PHASE_CHUNKS;  // partial states only, whatever the sizes
    if (S->max_prefix_pages < 1) return ATLAS_ERR_INVALID_ARG;
    const int64_t max_prefix = (int64_t)S->max_prefix_pages * P;
    if (max_prefix > INT32_MAX / 2) return ATLAS_ERR_INVALID_ARG;

    const int64_t sms = planned_sms(L);
    const int G = Hq / Hkv;
    const int64_t rows = (int64_t)L->batch * G * L->q_len;  // of one kv head, all groups
    const int64_t group_rows = (rows + groups - 1) / groups;
    const bool f32 = L->kv_dtype == ATLAS_F32;
    const bool few = plan->few = plan->own.path == Path::SplitBF16 || plan->own.path == Path::SplitF32;
    const int cols = f32 ? (group_rows <= 4 ? 4 : 8) : group_rows <= 8 ? 8 : 16;
    const double bytes = 2.0 * groups * max_prefix * Hkv * D * (f32 ? 4 : 2);
    const int64_t seq_rows = (int64_t)G * L->q_len, max_ctx = (int64_t)L->max_pages_per_seq * P;
    // (own keys: half of the most there may be)
    plan->split = few && split_pays(bytes, (group_rows + cols - 1) / cols, 4.0 * D * rows * Hkv * max_prefix,
                                    (double)L->batch * Hkv * max_ctx * D * (f32 ? 4 : 2),
                                    cols == 8 && seq_rows <= 4, f32);
    if (few && (L->debug_flags & ATLAS_DEBUG_SHARED_SPLIT)) plan->split = true;
    if (L->debug_flags & ATLAS_DEBUG_SHARED_TC) plan->split = false;
    plan->stream = !f32 && !plan->split;
    const bool own_splits = seq_rows <= kOwnSplitRows && max_ctx <= kOwnSplitKeys;
    plan->whole = plan->stream && !few && L->split_tokens == 0 &&
                  whole_pays(seq_rows, group_rows, max_prefix, max_ctx, L->batch * Hkv * ((seq_rows + 255) / 256), sms,
                             own_splits);
    if (L->debug_flags & ATLAS_DEBUG_SHARED_TC) plan->whole = false;
    if (L->debug_flags & ATLAS_DEBUG_SHARED_WHOLE) plan->whole = plan->stream;
    if (plan->stream && !plan->whole && few && L->split_tokens == 0 &&
        (int64_t)L->batch * Hkv * plan->own.col_tiles >= 2 * sms)
        // The own splits run beside the tiles, the longest first: where there are enough
        // sequences they are best left whole (up to 4096 keys).
        own.split_tokens = (int32_t)own_split(max_ctx);
    if (plan->whole) {
        plan->own.ws_bytes = 0;  // (no states but those of cut tiles)
    } else if (plan->stream && !few && L->split_tokens == 0 && own_splits) {
        const int64_t out = (int64_t)L->batch * Hq * L->q_len;
        plan->own.path = Path::SplitBF16;
        plan->own.col_tiles = (int)((seq_rows + 15) / 16);
        plan->own.chunk = (int)own_split(max_ctx);
        plan->own.n_chunks = (int)((max_ctx + plan->own.chunk - 1) / plan->own.chunk);
        plan->own.acc_bytes = (size_t)out * plan->own.n_chunks * D * sizeof(float);
        plan->own.ml_offset = (size_t)round_up((int64_t)plan->own.acc_bytes, 256);
        plan->own.ws_bytes = plan->own.ml_offset + (size_t)out * plan->own.n_chunks * 2 * sizeof(float);
    } else {
        if (sparing && !few && L->split_tokens == 0) {
            const int64_t tiles = (int64_t)L->batch * Hkv * ((seq_rows + 127) / 128);
            const int64_t splits = (6 * sms + tiles - 1) / tiles;
            own.split_tokens = (int32_t)round_up(std::max<int64_t>((max_ctx + splits - 1) / splits, 1024), 128);
        }
        st = make_plan(ATLAS_KIND_SUFFIX, Hq, Hkv, D, P, &own, &plan->own);
        if (st != ATLAS_OK) return st;
    }
    const bool own_cols =
        !plan->whole && (plan->own.path == Path::SplitBF16 || plan->own.path == Path::SplitF32);
    if (own_cols && (int64_t)plan->own.n_chunks * Hkv * plan->own.col_tiles * L->batch >= INT32_MAX)
        return ATLAS_ERR_UNSUPPORTED;  // (the own splits' CTAs)
    const int64_t tile_of = plan->whole ? seq_rows : group_rows;
    plan->tiles = plan->split ? cols : !f32 && tile_of > 128 ? 2 : 1;
    // CTAs of one split: a group's last may be partly filled
    const int64_t cta_rows = plan->split ? cols : 128 * plan->tiles;
    const int64_t units = (plan->whole ? L->batch * ((seq_rows + cta_rows - 1) / cta_rows)
                                       : rows / cta_rows + std::min(S->n_groups, L->batch)) * Hkv;
    const int64_t likely = std::max<int64_t>((rows + cta_rows - 1) / cta_rows, groups) * Hkv;
    const int64_t out_rows = (int64_t)L->batch * Hq * L->q_len;
    plan->acc_at = plan->whole ? 0 : (size_t)round_up((int64_t)plan->own.ws_bytes, 256);
    if (plan->stream) {
        // At most this many states of a tile: what the likely number of tiles leaves to each,
        // and some more where groups are uneven.
        const int64_t blocks = (max_prefix + 127) / 128 +
                               (plan->whole ? (max_ctx + 127) / 128 : 0);
        if (L->split_tokens > 0) plan->n_pre = (int)((max_prefix + L->split_tokens - 1) / L->split_tokens + 2);
        else plan->n_pre = (int)std::min<int64_t>(blocks / 4 + 3, sms / likely + 6);
        plan->chunk = 0;
        // (short tiles that count as more blocks make for more CTAs than SMs)
        plan->ctas = sms + units / 10 + 2;
        // Places in the line have 32 bits.  Short tiles count for more, so that a share has few enough
        // pieces: with a = blocks + 5 at most to a tile, a share is at most 28 such tiles of 7 a block
        // (three quarters of a CTA's pieces), and a tile counts for at least 9/8 of a share over 4 * 38
        // blocks, 1.46 a: no more than that for any tile, and one for rounding.
        const double line = (double)units * kPairCost * (1.5 * (double)(blocks + kWholeTileBlocks) + 2.0);
        if (line + 1e6 >= INT32_MAX) return ATLAS_ERR_UNSUPPORTED;
        const int64_t states = plan->whole ? plan->ctas * 2 * cta_rows : out_rows * plan->n_pre;
        plan->ml_at = plan->acc_at + (size_t)round_up(states * D * 4, 256);
        plan->plan_at = plan->ml_at + (size_t)round_up(states * 8, 256);
        const int64_t n = plan->whole ? L->batch : S->n_groups;
        const int64_t segs = 1 + shared_tc_items(plan->tiles) * (int64_t)(sizeof(SharedSeg) / 4) +
                             (int64_t)(sizeof(SharedCut) / 4);
        plan->bytes = plan->plan_at + 4 * (size_t)(11 * (int64_t)L->batch + 1 + 2 + 5 * n + 1 +
                                                   plan->ctas * segs + (plan->whole ? 0 : rows));
        return ATLAS_OK;
    }
    int64_t chunk = plan->split ? L->split_tokens : round_up(L->split_tokens, 128);
    if (chunk == 0 && plan->split) {
        // One wave of CTAs, all with as many keys: the own keys (half of the most there may be)
        // and the prefixes' for each CTA's rows, on the CTAs that are resident.
        const int64_t own_units = (int64_t)L->batch * Hkv * ((G * L->q_len + cols - 1) / cols);
        const int64_t slots = sms * (f32 ? kSplitWaveF32 : kSplitWave) / 100;
        const int64_t keys = own_units * max_ctx / 2 + likely * max_prefix;
        chunk = round_up((keys + slots - 1) / slots, 64);
        chunk = std::min<int64_t>(std::max<int64_t>(chunk, f32 ? kMinSplitF32 : kMinSplit), 2560);
        own.split_tokens = (int32_t)chunk;
        if (make_plan(ATLAS_KIND_SUFFIX, Hq, Hkv, D, P, &own, &plan->own) != ATLAS_OK)
            return ATLAS_ERR_UNSUPPORTED;
        plan->acc_at = (size_t)round_up((int64_t)plan->own.ws_bytes, 256);
    } else if (chunk == 0) {
        const int64_t splits = std::max<int64_t>(1, sms * 3 / likely);
        chunk = std::max<int64_t>(512, round_up((max_prefix + splits - 1) / splits, 128));
    }
    chunk = std::min(chunk, round_up(max_prefix, plan->split ? 64 : 128));
    plan->chunk = (int)chunk;
    plan->n_pre = (int)((max_prefix + chunk - 1) / chunk);
    plan->ctas = units * plan->n_pre;
    if (plan->split) {
        plan->own.col_tiles = (G * L->q_len + cols - 1) / cols;
        plan->ctas += (int64_t)plan->own.n_chunks * Hkv * plan->own.col_tiles * L->batch;
    }
    if (plan->ctas >= INT32_MAX) return ATLAS_ERR_UNSUPPORTED;
    plan->ml_at = plan->acc_at + (size_t)round_up(out_rows * plan->n_pre * D * 4, 256);
    plan->bytes = plan->ml_at + (size_t)out_rows * plan->n_pre * 8;
    return ATLAS_OK;
}

// Groups of a part of n of B sequences, on average.
int32_t part_groups(int64_t n_groups, int64_t n, int64_t B) { return (int32_t)((n_groups * n + B - 1) / B); }

// The whole call's plan, that of its first part; `bytes` is what the call needs.
atlas_status shared_plan(int32_t Hq, int32_t Hkv, int32_t D, int32_t P, const atlas_shared *S,
                         const atlas_launch *L, SharedPlan *plan) {
    if (!S || !L || L->batch < 1 || S->n_groups < 1 || S->n_groups > L->batch) return ATLAS_ERR_INVALID_ARG;
    const int64_t B = L->batch;
    atlas_launch part = *L;
    for (bool sparing = false;; sparing = true) {
        // (parts of equal sizes)
        const int64_t parts = (B + part.batch - 1) / part.batch, last = B - (parts - 1) * part.batch;
        SharedPlan rest;
        rest.bytes = 0;
        atlas_launch behind = part;
        behind.batch = (int32_t)last;
        atlas_status st = plan_part(Hq, Hkv, D, P, S, &part, part_groups(S->n_groups, part.batch, B), sparing, plan);
        if (st == ATLAS_OK && last != part.batch)
            st = plan_part(Hq, Hkv, D, P, S, &behind, part_groups(S->n_groups, last, B), sparing, &rest);
        if (st == ATLAS_ERR_INVALID_ARG) return st;
        if (st == ATLAS_OK) {
            plan->sparing = sparing;
            plan->part = part.batch;
            plan->parts = (int32_t)parts;
            if (parts > 1) {
                plan->starts_at = (size_t)round_up((int64_t)std::max(plan->bytes, rest.bytes), 256);
                plan->bytes = plan->starts_at + 4 * ((size_t)S->n_groups + 1);
            }
            if (plan->bytes <= kMostBytes || (part.batch == 1 && sparing)) return ATLAS_OK;
        } else if (part.batch == 1 && sparing) {
            return st;
        }
        if (!sparing) continue;  // (fewer splits first)
        int64_t size = part.batch / 2;
        if (st == ATLAS_OK)
            size = std::min((int64_t)((double)part.batch * (double)kMostBytes / (double)plan->bytes),
                            (int64_t)part.batch * 7 / 8);
        size = std::max<int64_t>(size, 1);
        const int64_t fewer = (B + size - 1) / size;
        part.batch = (int32_t)((B + fewer - 1) / fewer);
    }
}

// The own splits and the prefixes' in one launch; or (order given) the own ones alone, behind
// the launch of the prefixes and in that order.
cudaError_t launch_split(const SharedPlan &plan, const void *q, const void *k_pages,
                         const void *v_pages, const int32_t *page_table, const int32_t *seq_lens,
                         int32_t Hq, int32_t Hkv, int32_t D, int32_t P, float scale,
                         const atlas_shared *S, const atlas_launch *L, float *pre_acc,
                         float *pre_ml, const int32_t *order = nullptr) {
    SharedSplitParams p{};
    p.q = q;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.B = L->batch;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.D = D;
    p.P = P;
    p.q_len = L->q_len;
    p.max_pages = L->max_pages_per_seq;
    p.num_pages = L->num_pages;
    p.chunk = plan.own.chunk;
    p.n_chunks = plan.own.n_chunks;
    p.col_tiles = plan.own.col_tiles;
    p.row_step = 1;
    p.scale_log2 = scale * kLog2e;
    p.softcap_log2 = L->softcap > 0.f ? L->softcap * kLog2e : 0.f;
    p.softcap_inv = L->softcap > 0.f ? scale / L->softcap : 0.f;
    p.q_lens = L->q_lens;
    p.ws_acc = static_cast<float *>(L->workspace);
    p.ws_ml = reinterpret_cast<float *>(static_cast<char *>(L->workspace) + plan.own.ml_offset);
    p.status = L->status_word;
    p.debug_flags = L->debug_flags;
    p.prefix_table = S->prefix_table;
    p.prefix_lens = S->prefix_lens;
    p.group_starts = S->group_starts;
    p.n_groups = S->n_groups;
    p.max_prefix_pages = S->max_prefix_pages;
    p.pre_chunk = plan.chunk;
    p.n_pre = plan.n_pre;
    p.own_items = plan.own.n_chunks * Hkv * plan.own.col_tiles * L->batch;
    p.cols = order ? split_bf16_cols_per_cta(p.G, p.q_len) : plan.tiles;
    p.order = order;
    p.after_prefix = order != nullptr;
    const int64_t ctas = order ? p.own_items : plan.ctas;
    p.pre_acc = pre_acc;
    p.pre_ml = pre_ml;
    cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
    if (L->kv_dtype == ATLAS_F32) return launch_shared_split_f32(p, ctas, stream);
    CUtensorMap tmK, tmV;
    if (encode_pool_map(&tmK, k_pages, L->num_pages, Hkv, P, D) != ATLAS_OK ||
        encode_pool_map(&tmV, v_pages, L->num_pages, Hkv, P, D) != ATLAS_OK)
        return cudaErrorUnknown;
    return launch_shared_split_bf16(p, ctas, tmK, tmV, stream);
}

// The tensor-core kernels' view of a call.
atlas_status tc_params(const SharedPlan &plan, const void *q, const void *k_pages,
                       const void *v_pages, int32_t Hq, int32_t Hkv, int32_t D, int32_t P,
                       float scale, const atlas_launch *L, float *acc, float *ml, TcParams *tp,
                       CUtensorMap *tmK, CUtensorMap *tmV) {
    const bool f32 = L->kv_dtype == ATLAS_F32;
    const int bn = f32 ? 64 : 128;  // keys per block of the kernel
    atlas_status st = encode_rows_map(tmK, k_pages, (int64_t)L->num_pages * Hkv * P, D, std::min(P, bn), f32);
    if (st == ATLAS_OK)
        st = encode_rows_map(tmV, v_pages, (int64_t)L->num_pages * Hkv * P, D, std::min(P, bn), f32);
    tp->B = L->batch;
    tp->Hq = Hq;
    tp->Hkv = Hkv;
    tp->G = Hq / Hkv;
    tp->D = D;
    tp->P = P;
    tp->q_len = L->q_len;
    tp->num_pages = L->num_pages;
    tp->split = 1;
    tp->row_step = 1;
    tp->chunk = plan.chunk;
    tp->n_chunks = plan.n_pre;
    // bf16 weights in two parts wherever the call without prefixes, on the split kernels, takes them
    // so (64 sequences behind 32768 keys 107 -> 110 us, 192 of 4 rows in 7 groups 227 -> 243), and
    // where the second part costs nothing.  The tiles of more rows are those of atlas_attn_suffix
    // (16 prompts of 256 rows behind 8192 keys take 357 us, with two parts throughout 424).
    tp->hilo_below = plan.few || plan.tiles == 1 ? INT32_MAX : hilo_below(scale, D);
    tp->negate_scores = scale < 0.f;
    tp->scale_log2 = fabsf(scale) * kLog2e;
    tp->softcap_log2 = L->softcap > 0.f ? L->softcap * kLog2e : 0.f;
    tp->softcap_inv = L->softcap > 0.f ? fabsf(scale) / L->softcap : 0.f;
    tp->sinks = L->sinks;
    tp->q_lens = L->q_lens;
    tp->out = L->out;
    tp->out_bf16 = L->out_dtype == ATLAS_BF16;
    tp->lse = L->lse;
    tp->ws_acc = acc;
    tp->ws_ml = ml;
    tp->status = L->status_word;
    tp->q = q;
    return st;
}

// The arrays of a stream, in the workspace.
SharedStream stream_arrays(const SharedPlan &plan, int32_t G, const atlas_shared *S, const atlas_launch *L) {
    SharedStream st{};
    st.prefix_table = S->prefix_table;
    st.prefix_lens = S->prefix_lens;
    st.group_starts = S->group_starts;
    st.n_groups = S->n_groups;
    st.max_prefix_pages = S->max_prefix_pages;
    st.whole = plan.whole;
    st.units = plan.whole ? L->batch : S->n_groups;
    st.tile_rows = 128 * plan.tiles;
    st.max_items = shared_tc_items(plan.tiles);
    st.max_states = plan.n_pre;
    st.sms = planned_sms(L);
    int32_t *at = reinterpret_cast<int32_t *>(static_cast<char *>(L->workspace) + plan.plan_at);
    auto take = [&](int64_t n) {
        int32_t *x = at;
        at += n;
        return x;
    };
    st.info = take(8 * (int64_t)L->batch);  // (16-byte loads: first)
    st.head = take(2);
    st.first = take(st.units + 1);
    st.head_cost = take(st.units);
    st.blocks = take(st.units);
    st.weight = take(st.units);
    st.rows = take(st.units);
    st.group = take(L->batch);
    st.before = take(L->batch + 1);
    st.order = take(L->batch);
    st.counts = take(plan.ctas);
    st.segs = reinterpret_cast<SharedSeg *>(take(plan.ctas * st.max_items * (int64_t)(sizeof(SharedSeg) / 4)));
    st.cuts = reinterpret_cast<SharedCut *>(take(plan.ctas * (int64_t)(sizeof(SharedCut) / 4)));
    st.list = !plan.whole && L->q_lens ? take((int64_t)L->batch * G * L->q_len) : nullptr;
    return st;
}

// The own splits, then the prefixes' on the tensor cores.
atlas_status launch_tc(const SharedPlan &plan, const void *q, const void *k_pages,
                       const void *v_pages, const int32_t *page_table, const int32_t *seq_lens,
                       int32_t Hq, int32_t Hkv, int32_t D, int32_t P, float scale,
                       const atlas_shared *S, const atlas_launch *L, float *pre_acc, float *pre_ml) {
    CUtensorMap tmK, tmV;
    TcParams tp{};
    atlas_status st = tc_params(plan, q, k_pages, v_pages, Hq, Hkv, D, P, scale, L, pre_acc, pre_ml,
                                &tp, &tmK, &tmV);
    if (st != ATLAS_OK) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
    if (plan.stream) {
        const bool beside = plan.own.path == Path::SplitBF16;
        tp.st = stream_arrays(plan, Hq / Hkv, S, L);
        tp.st.wait_first = beside;
        tp.st.own_rate = !beside ? 0.f : Hq / Hkv * L->q_len <= 8 ? kOwnRate : kOwnRateWide / plan.own.col_tiles;
        tp.seq_lens = seq_lens;
        tp.max_pages = L->max_pages_per_seq;
        if (launch_shared_plan(tp, stream) != cudaSuccess) return ATLAS_ERR_CUDA;
        if (beside) {
            // The prefixes' CTAs, which take equally long, then the own splits, the longest
            // first: the SMs that the former leave are filled to the end.
            return launch_shared_tc(tp, plan.ctas, tmK, tmV, stream) == cudaSuccess &&
                           launch_split(plan, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P,
                                        scale, S, L, pre_acc, pre_ml, tp.st.order) == cudaSuccess
                       ? ATLAS_OK
                       : ATLAS_ERR_CUDA;
        }
    }
    atlas_launch own = *L;
    own.phase = ATLAS_PHASE_CHUNKS;
    own.split_tokens = plan.own.chunk;
    own.debug_flags = (own.debug_flags & ~ATLAS_DEBUG_TC_DIRECT) | kNearestProducts;
    own.events = nullptr;
    own.workspace_bytes = plan.own.ws_bytes;
    st = run_attention(ATLAS_KIND_SUFFIX, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P,
                       scale, &own);
    if (st != ATLAS_OK) return st;
    if (plan.stream) return launch_shared_tc(tp, plan.ctas, tmK, tmV, stream) == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
    tp.page_table = S->prefix_table;
    tp.seq_lens = S->prefix_lens;
    tp.max_pages = S->max_prefix_pages;
    tp.group_starts = S->group_starts;
    tp.n_groups = S->n_groups;
    return launch_shared_tc_f32(tp, plan.ctas, tmK, tmV, stream) == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

// Whole tiles: the prefixes and the sequences' own keys, the output, and the merge of what is cut.
atlas_status launch_whole(const SharedPlan &plan, const void *q, const void *k_pages,
                          const void *v_pages, const int32_t *page_table, const int32_t *seq_lens,
                          int32_t Hq, int32_t Hkv, int32_t D, int32_t P, float scale,
                          const atlas_shared *S, const atlas_launch *L, float *acc, float *ml,
                          cudaEvent_t between) {
    CUtensorMap tmK, tmV;
    TcParams tp{};
    const atlas_status st = tc_params(plan, q, k_pages, v_pages, Hq, Hkv, D, P, scale, L, acc, ml, &tp,
                                      &tmK, &tmV);
    if (st != ATLAS_OK) return st;
    tp.page_table = page_table;
    tp.seq_lens = seq_lens;
    tp.max_pages = L->max_pages_per_seq;
    tp.st = stream_arrays(plan, Hq / Hkv, S, L);
    tp.st.wait_first = 1;
    cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
    if (launch_shared_plan(tp, stream) != cudaSuccess ||
        launch_shared_tc(tp, plan.ctas, tmK, tmV, stream) != cudaSuccess ||
        (between && cudaEventRecord(between, stream) != cudaSuccess) ||
        launch_shared_cut_merge(tp, plan.ctas, stream) != cudaSuccess)
        return ATLAS_ERR_CUDA;
    return ATLAS_OK;
}

// All launches of a part; `between` is recorded before the merge.
atlas_status launch_part(const SharedPlan &plan, const void *q, const void *k_pages, const void *v_pages,
                         const int32_t *page_table, const int32_t *seq_lens, int32_t Hq, int32_t Hkv, int32_t D,
                         int32_t P, float scale, const atlas_shared *S, const atlas_launch *L, cudaEvent_t between) {
    cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
    float *pre_acc = reinterpret_cast<float *>(static_cast<char *>(L->workspace) + plan.acc_at);
    float *pre_ml = reinterpret_cast<float *>(static_cast<char *>(L->workspace) + plan.ml_at);
    if (plan.whole) {
        return launch_whole(plan, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P, scale, S, L,
                            pre_acc, pre_ml, between);
    }
    if (plan.split) {
        if (launch_split(plan, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P, scale, S, L,
                         pre_acc, pre_ml) != cudaSuccess)
            return ATLAS_ERR_CUDA;
    } else {
        const atlas_status st = launch_tc(plan, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P, scale, S, L,
                                          pre_acc, pre_ml);
        if (st != ATLAS_OK) return st;
    }
    if (between && cudaEventRecord(between, stream) != cudaSuccess) return ATLAS_ERR_CUDA;

    SharedMergeParams mp{};
    mp.seq_lens = seq_lens;
    mp.B = L->batch;
    mp.Hq = Hq;
    mp.D = D;
    mp.q_len = L->q_len;
    mp.max_pages = L->max_pages_per_seq;
    mp.P = P;
    mp.chunk = plan.own.chunk;
    mp.n_chunks = plan.own.n_chunks;
    mp.row_step = 1;
    mp.sinks = L->sinks;
    mp.q_lens = L->q_lens;
    mp.ws_acc = static_cast<float *>(L->workspace);
    mp.ws_ml = reinterpret_cast<float *>(static_cast<char *>(L->workspace) + plan.own.ml_offset);
    mp.out = L->out;
    mp.out_bf16 = L->out_dtype == ATLAS_BF16;
    mp.lse = L->lse;
    mp.sms = planned_sms(L);
    mp.group_starts = S->group_starts;
    mp.prefix_lens = S->prefix_lens;
    mp.n_groups = S->n_groups;
    mp.max_prefix = S->max_prefix_pages * P;
    mp.pre_chunk = plan.chunk;
    mp.n_pre = plan.n_pre;
    mp.pre_acc = pre_acc;
    mp.pre_ml = pre_ml;
    mp.G = Hq / Hkv;
    if (plan.stream) mp.st = stream_arrays(plan, mp.G, S, L);
    return launch_shared_merge(mp, stream) == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace
}  // namespace atlas

extern "C" size_t atlas_attn_shared_workspace_size(int32_t n_q_heads, int32_t n_kv_heads,
                                                   int32_t head_dim, int32_t page_tokens,
                                                   const atlas_shared *S, const atlas_launch *L) {
    atlas::SharedPlan plan;
    return atlas::shared_plan(n_q_heads, n_kv_heads, head_dim, page_tokens, S, L, &plan) == ATLAS_OK
               ? plan.bytes
               : SIZE_MAX;
}

extern "C" atlas_status atlas_attn_shared(const void *q, const void *k_pages, const void *v_pages,
                                          const int32_t *page_table, const int32_t *seq_lens,
                                          int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                          int32_t page_tokens, float scale, const atlas_shared *S,
                                          const atlas_launch *L) {
    using namespace atlas;
    // (the whole call's checks come before its first launch)
    if (!q || !k_pages || !v_pages || !page_table || !seq_lens || !S || !L || !S->prefix_table ||
        !S->prefix_lens || !S->group_starts || !L->out)
        return ATLAS_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(L->out) ||
        !aligned16(L->workspace) ||
        !aligned4({page_table, seq_lens, S->prefix_table, S->prefix_lens, S->group_starts, L->lse,
                   L->sinks, L->q_lens, L->status_word}))
        return ATLAS_ERR_INVALID_ARG;
    if (!(fabsf(scale) < INFINITY) || !(L->softcap >= 0.f) || L->softcap == INFINITY)
        return ATLAS_ERR_INVALID_ARG;
    const int32_t Hq = n_q_heads, Hkv = n_kv_heads, D = head_dim, P = page_tokens;
    SharedPlan plan;
    atlas_status st = shared_plan(Hq, Hkv, D, P, S, L, &plan);
    if (st != ATLAS_OK) return st;
    if (!L->workspace || L->workspace_bytes < plan.bytes) return ATLAS_ERR_WORKSPACE;
    // What is written, and what else there is: tiles read their queries while others are done.
    const size_t rows = (size_t)L->batch * Hq * L->q_len, size = L->kv_dtype == ATLAS_F32 ? 4 : 2;
    const size_t pool = (size_t)L->num_pages * Hkv * P * D * size;
    const Range all[] = {{L->out, rows * D * (L->out_dtype == ATLAS_F32 ? 4 : 2)}, {L->lse, rows * 4},
                         {L->workspace, plan.bytes}, {q, rows * D * size}, {k_pages, pool}, {v_pages, pool}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 6; ++j)
            if (meet(all[i], all[j])) return ATLAS_ERR_INVALID_ARG;
    cudaStream_t stream = static_cast<cudaStream_t>(L->stream);
    cudaEvent_t ev[3] = {nullptr, nullptr, nullptr};
    if (L->events)
        for (int i = 0; i < 3; ++i) ev[i] = static_cast<cudaEvent_t>(L->events[i]);

    (void)cudaGetLastError();
    if (ev[0] && cudaEventRecord(ev[0], stream) != cudaSuccess) return ATLAS_ERR_CUDA;
    if (plan.parts == 1) {
        st = launch_part(plan, q, k_pages, v_pages, page_table, seq_lens, Hq, Hkv, D, P, scale, S, L, ev[1]);
        if (st != ATLAS_OK) return st;
    }
    for (int64_t b0 = 0; plan.parts > 1 && b0 < L->batch; b0 += plan.part) {
        const int32_t n = (int32_t)std::min<int64_t>(plan.part, L->batch - b0);
        const size_t row0 = (size_t)b0 * Hq * L->q_len;
        atlas_launch part = *L;
        part.batch = n;
        part.out = static_cast<char *>(L->out) + row0 * D * (L->out_dtype == ATLAS_F32 ? 4 : 2);
        if (L->lse) part.lse = L->lse + row0;
        if (L->q_lens) part.q_lens = L->q_lens + b0;
        int32_t *const starts = reinterpret_cast<int32_t *>(static_cast<char *>(L->workspace) + plan.starts_at);
        atlas_shared groups = *S;
        groups.group_starts = starts;
        SharedPlan own;
        st = plan_part(Hq, Hkv, D, P, S, &part, part_groups(S->n_groups, n, L->batch), plan.sparing, &own);
        if (st != ATLAS_OK) return st;
        if (launch_shared_starts(S->group_starts, starts, S->n_groups, L->batch, (int)b0, n, stream) != cudaSuccess)
            return ATLAS_ERR_CUDA;
        st = launch_part(own, static_cast<const char *>(q) + row0 * D * size, k_pages, v_pages,
                         page_table + b0 * L->max_pages_per_seq, seq_lens + b0, Hq, Hkv, D, P, scale,
                         &groups, &part, b0 + n == L->batch ? ev[1] : nullptr);
        if (st != ATLAS_OK) return st;
    }
    if (ev[2] && cudaEventRecord(ev[2], stream) != cudaSuccess) return ATLAS_ERR_CUDA;
    return ATLAS_OK;
}
