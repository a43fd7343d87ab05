// kv_evict.cu -- the keys that stay under a budget (atlas_kv_select) and the pages with
// only those keys left (atlas_kv_compact).
//
// Selection.  One thread-block cluster per (sequence, kv head), its CTAs sharing the row:
// each maps its part of the weights to order-preserving 32-bit keys in shared memory (read
// from memory once), and three digits of 11, 11 and 10 bits, from the top, narrow the k-th
// largest key down exactly: a histogram of the digit over the keys that match the digits
// found so far, summed over the cluster through distributed shared memory, tells which bin
// the k-th largest lies in and how many are still wanted there.  What equals the last key
// is taken by lowest index, so the set never depends on timing, and positions in the
// ascending output are counts of kept keys before (ballots in a warp, sums over warps and
// CTAs).  Memory: 4 bytes per key in, 8 per kept key out; bound by latency: a load, four
// cluster barriers, and per digit a pass over the keys in shared memory and a scan.
//
// Compaction.  Rows of head_dim elements move between page slots, 16 bytes per thread and
// step.  Into fresh pages every row is independent.  In place, row j takes row kept[j] >= j:
// a row may only be overwritten once it has been read.  Rows are taken in ascending order
// in chunks, and since a chunk's sources lie at or behind its own destinations, it is
// enough that a chunk is read completely (a CTA barrier) before it is written: later
// chunks' sources lie behind it, earlier ones have been read.  No CTA waits on another:
// each owns a 64-byte wide strip of one (sequence, kv head, K or V) from end to end, with
// seven chunks in flight (cp.async) ahead of the one it writes, and their page ids and
// indices read one and two chunks before that.
#include "internal.h"
#include "ptx.cuh"

#include "atlas_evict.h"

#include <math.h>

namespace atlas {
namespace {

__device__ __forceinline__ void record(uint32_t *status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

// ---------------------------------------------------------------- selection
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCtas = 8;    // the portable cluster size
constexpr int kSelKeys = 8192;    // keys of a CTA, while there are fewer than 8 of them
constexpr int kBins = 2 * kSelThreads;
constexpr int kSelCache = 200 * 1024;

struct SelectParams {
    const float *weights;
    const int32_t *seq_lens;
    int32_t Hkv, row_tokens, budget, first, recent;
    int32_t *kept, *new_lens;
    float *kept_weights;
    uint32_t *status;
};

// Larger weight, larger key; -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (isnan(w)) w = -INFINITY;
    if (w == 0.f) w = 0.f;
    const uint32_t u = __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The 32-bit words that CTA `rank` of the cluster holds where this CTA holds *local.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t *local, int rank) {
    uint32_t addr, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 ld_cluster2(const uint32_t *local, int rank) {
    uint32_t addr;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}

// grid (CTAs of a row's cluster, Hkv, B).  CACHED: the row's keys stay in shared memory;
// else (rows too long for that) each pass reads the weights again.
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads, 1) select_kernel(const SelectParams p) {
    extern __shared__ uint32_t cached[];
    __shared__ __align__(8) uint32_t hist[2][kBins];
    __shared__ uint32_t found[2];                 // digit, keys above it
    __shared__ uint32_t warp_sum[kSelWarps];
    __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ uint32_t cta_gt, cta_eq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x, g = blockIdx.y, b = blockIdx.z;
    const int all = ctas * kSelThreads, me = rank * kSelThreads + tid;
    int L = p.seq_lens[b];
    if (L < 0 || L > p.row_tokens) {
        if (me == 0 && g == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        L = 0;
    }
    const int n = min(L, p.budget);
    if (me == 0 && g == 0) p.new_lens[b] = n;
    const int64_t row = (int64_t)b * p.Hkv + g;
    const float *w = p.weights + row * p.row_tokens;
    int32_t *kept = p.kept + row * p.budget;
    float *kept_w = p.kept_weights ? p.kept_weights + row * p.budget : nullptr;
    // Keys that stay whatever their weight: all of them, or the first and the recent ones.
    const bool whole = L <= p.budget;
    const int lo = whole ? L : p.first, hi = whole ? L : L - p.recent;
    uint32_t want = (uint32_t)(n - lo - (L - hi));  // of the keys in [lo, hi)
    const int seg = (hi - lo + ctas - 1) / ctas;
    const int s0 = min(hi, lo + rank * seg), len = want == 0 ? 0 : min(hi, s0 + seg) - s0;
    if (CACHED) {
#pragma unroll 8
        for (int i = tid; i < len; i += kSelThreads) cached[i] = order_key(w[s0 + i]);
    }
    for (int j = n + me; j < p.budget; j += all) {
        kept[j] = -1;
        if (kept_w) kept_w[j] = 0.f;
    }
    for (int j = me; j < lo + (L - hi); j += all) {
        const int t = j < lo ? j : hi + (j - lo);
        const int at = j < lo ? j : n - (L - hi) + (j - lo);
        kept[at] = t;
        if (kept_w) kept_w[at] = w[t];
    }
    if (want == 0) return;  // the whole cluster alike
    auto key_of = [&](int i) { return CACHED ? cached[i] : order_key(w[s0 + i]); };

    uint32_t prefix = 0;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        const uint32_t mask = d == 2 ? 1023u : 2047u;
        const uint32_t known = d == 0 ? 0u : ~0u << (d == 1 ? 21 : 10);  // the digits found
        uint32_t *h = hist[d & 1];
        h[tid] = h[tid + kSelThreads] = 0u;
        __syncthreads();
        for (int i0 = 0; i0 < len; i0 += kSelThreads) {
            const int i = i0 + tid;
            uint32_t bin = kBins;  // no vote
            if (i < len) {
                const uint32_t k = key_of(i);
                if (((k ^ prefix) & known) == 0u) bin = (k >> shift) & mask;
            }
            // Equal keys all fall into one bin: a warp that agrees adds once.
            const uint32_t votes = __ballot_sync(0xffffffffu, bin < kBins);
            if (votes == 0u) continue;
            const uint32_t one = __shfl_sync(0xffffffffu, bin, __ffs(votes) - 1);
            if (__ballot_sync(0xffffffffu, bin == one) == votes) {
                if (lane == 0) atomicAdd(&h[one], (uint32_t)__popc(votes));
            } else if (bin < kBins) {
                atomicAdd(&h[bin], 1u);
            }
        }
        cluster_barrier();
        // Thread l owns bins 2047 - 2l and 2046 - 2l: a scan over threads goes from the top.
        uint32_t first = 0, second = 0;
#pragma unroll 8
        for (int r = 0; r < ctas; ++r) {
            const uint2 v = ld_cluster2(&h[kBins - 2 - 2 * tid], r);
            first += v.y;
            second += v.x;
        }
        uint32_t above = first + second;  // inclusive over the warp's lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
            if (lane >= o) above += v;
        }
        if (lane == 31) warp_sum[warp] = above;
        __syncthreads();
        above += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u) - (first + second);
        if (above < want && above + first + second >= want) {  // exactly one thread
            const bool top = above + first >= want;
            found[0] = (uint32_t)(kBins - 1 - 2 * tid - (top ? 0 : 1));
            found[1] = above + (top ? 0u : first);
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want -= found[1];
        // (found and warp_sum are written again only after the next cluster barrier; this
        // digit's histogram only after the one after that, when every CTA has read it)
    }
    // Keys above `prefix` stay, and the first `want` equal to it.  A warp takes a
    // contiguous part, 32 keys at a time in order.
    const int part = ((len + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int w0 = min(len, warp * part), w1 = min(len, w0 + part);
    uint32_t gt = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key_of(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t a = __reduce_add_sync(0xffffffffu, warp_gt[lane]);
        const uint32_t c = __reduce_add_sync(0xffffffffu, warp_eq[lane]);
        if (lane == 0) {
            cta_gt = a;
            cta_eq = c;
        }
    }
    cluster_barrier();
    // kept keys before this warp's: earlier CTAs (lanes 0..7 read one each), earlier warps
    uint32_t gt_before = lane < warp ? warp_gt[lane] : 0u, eq_before = lane < warp ? warp_eq[lane] : 0u;
    if (lane < rank) {
        gt_before += ld_cluster(&cta_gt, lane);
        eq_before += ld_cluster(&cta_eq, lane);
    }
    gt_before = __reduce_add_sync(0xffffffffu, gt_before);
    eq_before = __reduce_add_sync(0xffffffffu, eq_before);
    uint32_t at = (uint32_t)lo + gt_before + min(want, eq_before);
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? key_of(i) : 0u;
        const uint32_t eqs = __ballot_sync(0xffffffffu, i < w1 && k == prefix);
        const bool keep = i < w1 && (k > prefix || (k == prefix &&
                                                    eq_before + __popc(eqs & below) < want));
        const uint32_t keeps = __ballot_sync(0xffffffffu, keep);
        if (keep) {
            const uint32_t j = at + __popc(keeps & below);
            kept[j] = s0 + i;
            if (kept_w) kept_w[j] = w[s0 + i];
        }
        at += __popc(keeps);
        eq_before += __popc(eqs);
    }
    cluster_barrier();  // no CTA leaves while another may still read its counts
}

// ---------------------------------------------------------------- compaction
struct CompactParams {
    void *k_pages, *v_pages;
    const int32_t *page_table, *new_table, *kept, *new_lens;
    int32_t Hkv, P, max_pages, new_max_pages, num_pages, max_kept;
    int32_t vec;       // 16-byte pieces per row: 8, 16 or 32
    int32_t lg_piece;  // log2 of the pieces of a row that one CTA moves
    uint32_t *status;
};

// Which strip of which pool this CTA moves, and the rows of its sequence.
struct Strip {
    uint4 *pool;
    const int32_t *src_table, *dst_table, *kept;
    int n, piece;  // rows of the compacted sequence; this thread's piece of each
    bool tells;    // this thread reports what is wrong with its rows
};

__device__ __forceinline__ bool strip_of(const CompactParams &p, Strip &s) {
    const int strips = p.vec >> p.lg_piece;
    const int b = blockIdx.z;
    int y = blockIdx.y;
    const int strip = y % strips;
    y /= strips;
    const int g = y % p.Hkv, kv = y / p.Hkv;
    const int in_strip = (int)threadIdx.x & ((1 << p.lg_piece) - 1);
    s.piece = (strip << p.lg_piece) + in_strip;
    s.tells = kv == 0 && s.piece == 0;
    s.pool = static_cast<uint4 *>(kv ? p.v_pages : p.k_pages) + (int64_t)g * p.P * p.vec;
    s.kept = p.kept + ((int64_t)b * p.Hkv + g) * p.max_kept;
    s.src_table = p.page_table + (int64_t)b * p.max_pages;
    s.dst_table = p.new_table ? p.new_table + (int64_t)b * p.new_max_pages : s.src_table;
    s.n = p.new_lens[b];
    const int64_t room = (int64_t)(p.new_table ? p.new_max_pages : p.max_pages) * p.P;
    if (s.n < 0 || s.n > p.max_kept || s.n > room) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return false;
    }
    return s.n > 0;
}

// Row `t` of a sequence in 16-byte units of its pool, from its page id.
__device__ __forceinline__ int64_t slot_of(const CompactParams &p, int page, int t) {
    return ((int64_t)page * p.Hkv * p.P + (t & (p.P - 1))) * p.vec;
}

constexpr int kMoveThreads = 256, kMoveRows = 4;

// Fresh pages: a CTA moves kMoveRows rows per thread, all loads before the first store.
__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const CompactParams p) {
    Strip s;
    if (!strip_of(p, s)) return;
    const int lp = 31 - __clz(p.P);
    const int per = kMoveThreads >> p.lg_piece;
    const int j0 = (int)blockIdx.x * per * kMoveRows + ((int)threadIdx.x >> p.lg_piece);
    uint4 x[kMoveRows];
    int64_t dst[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
        dst[u] = -1;
        const int j = j0 + u * per;
        if (j >= s.n) continue;
        const int t = s.kept[j];
        uint32_t bad = 0;
        if (t < 0 || (int64_t)t >= (int64_t)p.max_pages * p.P) {
            bad = ATLAS_DEV_BAD_SEQLEN;
        } else {
            const int a = s.src_table[t >> lp], z = s.dst_table[j >> lp];
            if (a < 0 || a >= p.num_pages || z < 0 || z >= p.num_pages) {
                bad = ATLAS_DEV_BAD_PAGE;
            } else {
                x[u] = s.pool[slot_of(p, a, t) + s.piece];
                dst[u] = slot_of(p, z, j) + s.piece;
            }
        }
        if (bad && s.tells) record(p.status, bad);
    }
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
        if (dst[u] >= 0) s.pool[dst[u]] = x[u];
}

// In place: one CTA per strip walks the rows in order, kShiftRows rows per thread and
// chunk, each thread copying its own pieces through its own slots of a ring.
constexpr int kShiftThreads = 512, kShiftRows = 2, kShiftStages = 8;
constexpr int kShiftSmem = kShiftStages * kShiftRows * kShiftThreads * 16;

__global__ void __launch_bounds__(kShiftThreads, 1) compact_shift_kernel(const CompactParams p) {
    extern __shared__ __align__(16) uint4 ring[];  // [stage][row][thread]
    Strip s;
    if (!strip_of(p, s)) return;
    constexpr int R = kShiftRows, S = kShiftStages;
    const int lp = 31 - __clz(p.P);
    const int per = kShiftThreads >> p.lg_piece;
    const int r = (int)threadIdx.x >> p.lg_piece;
    const int64_t ctx = (int64_t)p.max_pages * p.P;
    const int64_t chunks = (s.n + (int64_t)per * R - 1) / (per * R);
    auto row = [&](int64_t c, int u) { return c * (per * R) + u * per + r; };
    // The index of a row (unchecked; -1: no such row), and the page ids of an index and of
    // a row: each only used a chunk later.
    auto index = [&](int64_t c, int (&t)[R]) {
#pragma unroll
        for (int u = 0; u < R; ++u) t[u] = row(c, u) < s.n ? s.kept[row(c, u)] : -1;
    };
    auto source = [&](int64_t c, int (&t)[R], int (&a)[R]) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (row(c, u) < s.n && (t[u] < row(c, u) || t[u] >= ctx)) {
                if (s.tells) record(p.status, ATLAS_DEV_BAD_SEQLEN);
                t[u] = -1;
            }
            a[u] = t[u] >= 0 ? s.src_table[t[u] >> lp] : 0;
        }
    };
    auto target = [&](int64_t c, int (&z)[R]) {
#pragma unroll
        for (int u = 0; u < R; ++u) z[u] = row(c, u) < s.n ? s.dst_table[row(c, u) >> lp] : -1;
    };
    uint32_t moving = 0;  // bit (chunk % S) * R + u: that row is in the ring
    auto load = [&](int64_t c, const int (&t)[R], const int (&a)[R]) {
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const uint32_t bit = 1u << ((int)(c % S) * R + u);
            moving &= ~bit;
            if (t[u] < 0) continue;
            if (a[u] < 0 || a[u] >= p.num_pages) {
                if (s.tells) record(p.status, ATLAS_DEV_BAD_PAGE);
                continue;
            }
            if (t[u] == row(c, u)) continue;  // it is where it belongs
            moving |= bit;
            cp_async16(smem_u32(ring + ((int)(c % S) * R + u) * kShiftThreads + threadIdx.x),
                       s.pool + slot_of(p, a[u], t[u]) + s.piece, 16);
        }
        cp_async_commit();
    };
    // Chunks 0 .. S - 2 are on their way before the first is written.
    int t0[R], t1[R], a0[R], z0[R];
    index(0, t0);
    index(1, t1);
    source(0, t0, a0);
#pragma unroll 1
    for (int64_t c = 0; c < S - 1; ++c) {
        load(c, t0, a0);
#pragma unroll
        for (int u = 0; u < R; ++u) t0[u] = t1[u];
        source(c + 1, t0, a0);
        index(c + 2, t1);
    }
    target(0, z0);
#pragma unroll 1
    for (int64_t c = 0; c < chunks; ++c) {
        load(c + S - 1, t0, a0);
        int z1[R];
        target(c + 1, z1);
#pragma unroll
        for (int u = 0; u < R; ++u) t0[u] = t1[u];
        source(c + S, t0, a0);
        index(c + S + 1, t1);
        cp_async_wait<S - 1>();
        __syncthreads();  // every thread has chunk c (and all before it) in the ring
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int at = (int)(c % S) * R + u;
            if ((moving >> at) & 1u) {
                if (z0[u] >= 0 && z0[u] < p.num_pages)
                    s.pool[slot_of(p, z0[u], (int)row(c, u)) + s.piece] = ring[at * kShiftThreads + threadIdx.x];
                else if (s.tells)
                    record(p.status, ATLAS_DEV_BAD_PAGE);
            }
            z0[u] = z1[u];
        }
    }
    cp_async_wait<0>();
}

}  // namespace
}  // namespace atlas

extern "C" {

atlas_status atlas_kv_select(const float *weights, const int32_t *seq_lens, int32_t n_kv_heads,
                             const atlas_select *S) {
    using namespace atlas;
    if (!weights || !seq_lens || !S || !S->kept || !S->new_lens) return ATLAS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(S->kept) |
         reinterpret_cast<uintptr_t>(S->kept_weights)) & 3u)
        return ATLAS_ERR_INVALID_ARG;
    if (S->batch < 1 || S->batch > 65535 || n_kv_heads < 1 || n_kv_heads > 65535 ||
        S->row_tokens < 1 || S->row_tokens > INT32_MAX / 2 || S->budget < 1 ||
        S->budget > INT32_MAX / 2 || S->keep_first < 0 || S->keep_recent < 0 ||
        (int64_t)S->keep_first + S->keep_recent > S->budget)
        return ATLAS_ERR_INVALID_ARG;
    SelectParams p{};
    p.weights = weights;
    p.seq_lens = seq_lens;
    p.Hkv = n_kv_heads;
    p.row_tokens = S->row_tokens;
    p.budget = S->budget;
    p.first = S->keep_first;
    p.recent = S->keep_recent;
    p.kept = S->kept;
    p.new_lens = S->new_lens;
    p.kept_weights = S->kept_weights;
    p.status = S->status_word;
    int ctas = 1;
    while (ctas < kSelMaxCtas && (int64_t)ctas * kSelKeys < p.row_tokens) ctas *= 2;
    const int64_t bytes = ((int64_t)p.row_tokens + ctas - 1) / ctas * 4;
    const bool cached = bytes <= kSelCache;
    auto kern = cached ? select_kernel<true> : select_kernel<false>;
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATLAS_ERR_CUDA;
    if (dev >= 64 || !configured[dev]) {
        if (cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSelCache) != cudaSuccess)
            return ATLAS_ERR_CUDA;
        if (dev < 64) configured[dev] = 1;
    }
    (void)cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)n_kv_heads, (unsigned)S->batch);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.dynamicSmemBytes = cached ? (size_t)bytes : 0;
    cfg.stream = static_cast<cudaStream_t>(S->stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

atlas_status atlas_kv_compact(void *k_pages, void *v_pages, const int32_t *page_table,
                              const int32_t *kept, const int32_t *new_lens, int32_t n_kv_heads,
                              int32_t head_dim, int32_t page_tokens, const atlas_compact *C) {
    using namespace atlas;
    if (!k_pages || !v_pages || !page_table || !kept || !new_lens || !C) return ATLAS_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15u)
        return ATLAS_ERR_INVALID_ARG;
    if (C->batch < 1 || C->batch > 65535 || C->max_pages_per_seq < 1 || C->num_pages < 1 ||
        C->max_kept < 1 || n_kv_heads < 1 || n_kv_heads > 4095 ||
        (C->new_page_table && C->new_max_pages < 1) ||
        (int64_t)C->max_pages_per_seq * page_tokens > INT32_MAX / 2 || C->max_kept > INT32_MAX / 2)
        return ATLAS_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return ATLAS_ERR_UNSUPPORTED;
    if (page_tokens < 1 || page_tokens > 128 || (page_tokens & (page_tokens - 1)))
        return ATLAS_ERR_UNSUPPORTED;
    if (C->kv_dtype != ATLAS_F32 && C->kv_dtype != ATLAS_BF16) return ATLAS_ERR_UNSUPPORTED;
    CompactParams p{};
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.new_table = C->new_page_table;
    p.kept = kept;
    p.new_lens = new_lens;
    p.Hkv = n_kv_heads;
    p.P = page_tokens;
    p.max_pages = C->max_pages_per_seq;
    p.new_max_pages = C->new_max_pages;
    p.num_pages = C->num_pages;
    p.max_kept = C->max_kept;
    p.vec = head_dim * (C->kv_dtype == ATLAS_BF16 ? 2 : 4) / 16;
    p.status = C->status_word;
    const cudaStream_t stream = static_cast<cudaStream_t>(C->stream);
    (void)cudaGetLastError();
    if (p.new_table) {
        p.lg_piece = p.vec == 8 ? 3 : p.vec == 16 ? 4 : 5;  // whole rows
        const int rows = (kMoveThreads >> p.lg_piece) * kMoveRows;
        const dim3 grid((unsigned)((p.max_kept + rows - 1) / rows), (unsigned)(2 * n_kv_heads),
                        (unsigned)C->batch);
        compact_move_kernel<<<grid, kMoveThreads, 0, stream>>>(p);
    } else {
        static int configured[64] = {0};
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return ATLAS_ERR_CUDA;
        if (dev >= 64 || !configured[dev]) {
            if (cudaFuncSetAttribute(compact_shift_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kShiftSmem) != cudaSuccess)
                return ATLAS_ERR_CUDA;
            if (dev < 64) configured[dev] = 1;
        }
        p.lg_piece = 2;  // 64-byte strips
        const dim3 grid(1, (unsigned)(2 * n_kv_heads * (p.vec >> 2)), (unsigned)C->batch);
        compact_shift_kernel<<<grid, kShiftThreads, kShiftSmem, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
