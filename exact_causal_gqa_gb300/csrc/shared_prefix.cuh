// shared_prefix.cuh -- work items and rows of prefixes that groups of sequences share.
//
// A prefix's keys are seen by every row of every sequence of its group, so the rows of one
// kv head -- (sequence, q head of the kv head, query row), in that order -- form one long
// list that is cut into tiles: a tile's rows may belong to many sequences, and each K/V block
// is read once for all of them.  Group sizes and prefix lengths are known on the device alone.
//
// The split kernels (tiles of 4 to 16 rows) and the fp32 tensor-core kernel (128) have items
// (group, kv head, split of the prefix, tile), tiles fastest, so that the CTAs which read the
// same keys run side by side and all but the first find them in L2.  Each CTA counts the items
// of all groups, one lane for each, and finds its own; the grid covers the most that the call's
// sizes allow, and the CTAs behind the last item leave.  The bf16 tensor-core kernel (128 or 256)
// has its items from a plan: below.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace atlas {

struct SharedItem {
    int group, hkv, split, tile;  // group < 0: no item for this CTA; tile: the CTA's rows
    int seq0, seqs, len;          // the group's sequences and its prefix's keys
};

// What the items are counted from.
struct SharedGroups {
    const int32_t *starts, *lens;  // [n + 1], [n]
    int n, B, max_len;
    int rows, cta_rows;            // rows of a sequence (G * q_len), and of a CTA
    int chunk, Hkv;
    uint32_t *status;
};

// All threads of the CTA call this (it synchronises the CTA); `scratch`: 7 ints of shared
// memory.  Item 0 reports groups that are out of range; they have no items.
__device__ inline SharedItem shared_item(const SharedGroups &p, int item, int *scratch) {
    if (threadIdx.x < 32) {
        const int lane = (int)threadIdx.x;
        if (lane == 0) scratch[0] = -1;
        __syncwarp();
        int64_t base = 0;  // items of the groups before these (64 bits: starts out of order repeat)
        bool bad = false;
        for (int n0 = 0; n0 < p.n; n0 += 32) {
            const int n = n0 + lane;
            int seq0 = 0, seqs = 0, len = 0, ctas = 0, items = 0;
            if (n < p.n) {
                seq0 = p.starts[n];
                const int end = p.starts[n + 1];
                len = p.lens[n];
                if (seq0 < 0 || end < seq0 || end > p.B || len < 0 || len > p.max_len) {
                    bad = true;
                } else {
                    seqs = end - seq0;
                    ctas = (int)(((int64_t)seqs * p.rows + p.cta_rows - 1) / p.cta_rows);
                    items = ctas * (int)(((int64_t)len + p.chunk - 1) / p.chunk) * p.Hkv;
                }
            }
            int64_t upto = items;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += x;
            }
            const int64_t first = base + upto - items;
            if (item >= first && item < first + items) {
                const int at = (int)(item - first);
                const int rest = at / ctas;
                const int splits = items / (ctas * p.Hkv);
                scratch[0] = n;
                scratch[1] = rest / splits;
                scratch[2] = rest % splits;
                scratch[3] = at % ctas;
                scratch[4] = seq0;
                scratch[5] = seqs;
                scratch[6] = len;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
            if (base > item && item > 0) break;
        }
        if (bad && item == 0 && p.status) atomicOr(p.status, ATLAS_DEV_BAD_SEQLEN);
    }
    __syncthreads();
    return {scratch[0], scratch[1], scratch[2], scratch[3], scratch[4], scratch[5], scratch[6]};
}

// Output row of tile row f of a group whose first sequence is seq0.
template <typename Params>
__device__ __forceinline__ int64_t shared_row(const Params &p, int seq0, int hkv, int f) {
    const int per = p.G * p.q_len, s = f / per;
    return ((int64_t)(seq0 + s) * p.Hq + (int64_t)hkv * p.G) * p.q_len + (f - s * per);
}

// Whether tile row f is a query: inside the group, and not padding of a ragged sequence.
template <typename Params>
__device__ __forceinline__ bool shared_real(const Params &p, int seq0, int rows, int f) {
    if (f >= rows) return false;
    const int per = p.G * p.q_len, s = f / per;
    return !p.q_lens || (f - s * per) % p.q_len < p.q_lens[seq0 + s];
}

// ---------------------------------------------------------------- evenly cut tiles (bf16)
// A unit -- a group with its prefix (st.whole 0), or a sequence with its prefix and its own keys
// (1) -- has tiles of st.tile_rows rows for each kv head, and a tile has 128-key blocks: the
// prefix's, the last of them perhaps in part, then the sequence's own.  The blocks of all tiles
// stand in one line, tile after tile, each as long as it takes; CTA x has those that begin in
// [x n, (x + 1) n) of it, n chosen so that every SM gets one CTA: whatever the lengths, all end
// together.  A tile that is cut leaves partial states of its rows, one for each CTA that has
// blocks of it.
//
// Lengths on the line, measured: a block of a 256-row tile (a pair of MMA tiles) 2.0 us, of one
// whose rows end in its first half 1.1 us, and what a tile takes besides (its queries, the first
// products, the epilogue) about two blocks, or with own keys, whose last blocks are masked, five: 47
// prompts of 256 rows with 256 to 1587 own keys behind 355 take 407, 380, 378 and 376 us with 2, 4, 5
// and 6, 64 steps behind 32768 as long with 2 as with 5.
constexpr int kPairCost = 7, kSingleCost = 4, kTileBlocks = 2, kWholeTileBlocks = 5;

// Length of a tile's block.
__device__ __forceinline__ int block_cost(const SharedStream &st, int tile, int rows) {
    return st.tile_rows == 256 && rows - tile * 256 > 128 ? kPairCost : kSingleCost;
}

// Own keys (with st.whole) that a tile's rows see at most: rows are q heads times query rows.
__device__ __forceinline__ int tile_own_keys(int seq_len, int qn, int row0, int row_end) {
    const int last = row_end - 1;  // (the tile's last row)
    const int i = last / qn != row0 / qn ? qn - 1 : last % qn;
    return seq_len - qn + i + 1;
}

struct SharedTile {
    int tile, first, cost, end;  // where it begins in the line, the length of its blocks, its end
};

// The first of a tile's blocks that begins at the place or behind it.
__device__ __forceinline__ int block_from(const SharedTile &t, int place) {
    return (max(place - t.first, 0) + t.cost - 1) / t.cost;
}

// Output row of row f of a unit.
template <typename Params>
__device__ __forceinline__ int64_t unit_row(const Params &p, int unit, int hkv, int f) {
    const SharedStream &st = p.st;
    if (st.whole) {
        const int qn = p.q_lens ? p.q_lens[unit] : p.q_len, g = f / qn;
        return ((int64_t)unit * p.Hq + hkv * p.G + g) * p.q_len + (f - g * qn);
    }
    const int seq0 = st.group_starts[unit];
    if (st.list) return (int64_t)st.list[st.before[seq0] + f] + (int64_t)hkv * p.G * p.q_len;
    return shared_row(p, seq0, hkv, f);
}

// A launch that may start as soon as every CTA of the grid before it in the stream has
// started or ended.
template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t stream, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace atlas
