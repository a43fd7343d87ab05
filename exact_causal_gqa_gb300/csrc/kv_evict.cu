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
// CTAs).  Memory: 4 bytes per key in, 8 per kept key out, 1 to 2 us of bytes for long rows.
// Two rows of 600 keys take 6.3 us: a load, four cluster barriers, three scans.  What long
// rows take beyond that grows with the keys of a CTA, each of which five passes look at (one
// from memory, four in shared memory): 8 x 8 rows of up to 32768 keys (16384 a CTA), 4096
// kept, 18.5 us; one sequence's 8 rows of 131072 keys (64 CTAs, the rest of the GPU idle),
// half kept, 23 us.
//
// Compaction.  Rows of head_dim elements move between page slots, 16 bytes per thread and
// step.  Into fresh pages every row is independent.  In place, row j takes row kept[j] >= j:
// a row may only be overwritten once it has been read.  Rows are taken in ascending order
// in chunks, and since a chunk's sources lie at or behind its own destinations, it is
// enough that a chunk is read completely (a CTA barrier) before it is written: later
// chunks' sources lie behind it, earlier ones have been read.  A thread-block cluster
// shares the rows of one (sequence, kv head, K or V): its barrier stands between reading a
// chunk and writing it, arrived at one chunk ahead, with four chunks in flight (cp.async);
// indices and page tables come through shared memory, so that nothing but the data's own
// latency is in the loop.
// Times: 65536 of 131072 rows of 8 heads of 128 bf16 (537 MB read and written) take 89 us
// into fresh pages, 6.0 TB/s of DRAM traffic, and 116 to 119 in place: the order costs the
// rest, the clusters going through their chunks in step (64 bf16: 52 and 95 us, 128 fp32: 165
// and 199).  4096 rows of 8 sequences x 8 heads of 128 bf16 into fresh pages: 44 us.  Variants
// in place: strips of 64 bytes a warp 382, a cp.async ring per CTA 199, clusters of 8 with
// releasing arrivals 240, relaxed 160, four pieces a thread 121, four stages 116.
#include "internal.h"
#include "ptx.cuh"

#include "atlas_evict.h"

#include <math.h>

namespace atlas {
namespace {

__device__ __forceinline__ void record(uint32_t *status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

// Whether `n` bytes from a and `m` bytes from b have any in common.
bool overlap(const void *a, uint64_t n, const void *b, uint64_t m) {
    const uint64_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
}

// ---------------------------------------------------------------- selection
constexpr int kSelMaxCtas = 8;    // the portable cluster size
constexpr int kSelKeys = 8192;    // keys of a CTA, while fewer than 8 CTAs share a row
// Rows of at most kSelSmallKeys keys take smaller CTAs, for the same latency or less and more
// rows at once: 512 threads (8 rows of 1500 keys 7.9 -> 6.7 us, 256 of 4096 16.9 -> 11.6), and
// 256 when the rows are more than two for each SM (1024 rows of 600 / 2000 / 4000 keys 46 / 49 /
// 54 us with 1024 threads, 26 / 28 / 35 with 512, 17 / 21 / 29 with 256; but 8 rows of 4096 8.7,
// 8.4 and 10.4).
constexpr int kSelSmallKeys = 4096;
constexpr int kBins = 2048;
constexpr int kSelCache = 200 * 1024;
constexpr int kSelAhead = 8;

struct SelectParams {
    const float *weights;
    const int32_t *seq_lens;
    int32_t Hkv, row_tokens, budget, first, recent;
    int32_t *kept, *new_lens;
    float *kept_weights;
    int32_t kept_row;  // floats per row of it, budget or more
    uint32_t *status;
};

// Larger weight, larger key; -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (isnan(w)) w = -INFINITY;
    if (w == 0.f) w = 0.f;
    const uint32_t u = __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float key_weight(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// Orders nothing, so it does not wait for earlier writes to be performed.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
    cluster_arrive();
    cluster_wait();
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
template <bool CACHED, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) select_kernel(const SelectParams p) {
    constexpr int kWarps = kThreads / 32, kOwn = kBins / kThreads;  // bins of a thread
    extern __shared__ __align__(16) uint32_t cached[];
    __shared__ __align__(8) uint32_t hist[2][kBins];
    __shared__ uint32_t found[2];                 // digit, keys above it
    __shared__ uint32_t warp_sum[kWarps];
    __shared__ uint32_t warp_gt[kWarps], warp_eq[kWarps];
    __shared__ uint32_t cta_gt, cta_eq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, ctas = gridDim.x, g = blockIdx.y, b = blockIdx.z;
    const int all = ctas * kThreads, me = rank * kThreads + tid;
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
    float *kept_w = p.kept_weights ? p.kept_weights + row * p.kept_row : nullptr;
    // Keys that stay whatever their weight: all of them, or the first and the recent ones.
    const bool whole = L <= p.budget;
    const int lo = whole ? L : p.first, hi = whole ? L : L - p.recent;
    uint32_t want = (uint32_t)(n - lo - (L - hi));  // of the keys in [lo, hi)
    const int seg = (hi - lo + ctas - 1) / ctas;
    const int s0 = min(hi, lo + rank * seg), len = want == 0 ? 0 : min(hi, s0 + seg) - s0;
    // The entries that no weight decides.  Written last: the cluster barrier before would
    // wait for them to reach L2.
    auto fixed = [&] {
        for (int j = n + me; j < p.budget; j += all) kept[j] = -1;
        if (kept_w)
            for (int j = n + me; j < p.kept_row; j += all) kept_w[j] = 0.f;
        for (int j = me; j < lo + (L - hi); j += all) {
            const int t = j < lo ? j : hi + (j - lo);
            const int at = j < lo ? j : n - (L - hi) + (j - lo);
            kept[at] = t;
            if (kept_w) kept_w[at] = w[t];
        }
    };
    if (want == 0) {  // the whole cluster alike
        fixed();
        return;
    }
    // Keys i .. i + 3 (i a multiple of 4); past the end 0, which `in` tells apart.
    auto keys_of = [&](int i, bool (&in)[4]) {
        uint4 k = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 4; ++e) in[e] = i + e < len;
        if (CACHED) {
            if (in[0]) k = *reinterpret_cast<const uint4 *>(cached + i);
        } else {
            if (in[0]) k.x = order_key(w[s0 + i]);
            if (in[1]) k.y = order_key(w[s0 + i + 1]);
            if (in[2]) k.z = order_key(w[s0 + i + 2]);
            if (in[3]) k.w = order_key(w[s0 + i + 3]);
        }
        return k;
    };

    uint32_t prefix = 0;
#pragma unroll 1
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        uint32_t *h = hist[d & 1];
#pragma unroll
        for (int e = 0; e < kOwn; ++e) h[tid + e * kThreads] = 0u;
        __syncthreads();
        if (d == 0) {
            // Every key votes, on its way into shared memory, kSelAhead loads of a thread at
            // a time.  Equal weights all fall into one bin: a warp that agrees adds once.
            for (int i0 = 0; i0 < len; i0 += kSelAhead * kThreads) {
                float v[kSelAhead];
#pragma unroll
                for (int e = 0; e < kSelAhead; ++e) {
                    const int i = i0 + e * kThreads + tid;
                    v[e] = i < len ? w[s0 + i] : 0.f;
                }
#pragma unroll
                for (int e = 0; e < kSelAhead; ++e) {
                    const int i = i0 + e * kThreads + tid;
                    if (i0 + e * kThreads >= len) break;
                    const uint32_t k = order_key(v[e]);
                    if (CACHED && i < len) cached[i] = k;
                    int same;
                    __match_all_sync(0xffffffffu, i < len ? k >> shift : (uint32_t)kBins, &same);
                    if (i < len && (!same || lane == 0)) atomicAdd(&h[k >> shift], same ? 32u : 1u);
                }
            }
        } else {
            // Few keys match the digits found, or (many equal weights) whole warps do.
            const uint32_t known = ~0u << (d == 1 ? 21 : 10), mask = d == 1 ? 2047u : 1023u;
            for (int i0 = 0; i0 < len; i0 += 4 * kThreads) {
                bool in[4];
                const uint4 k4 = keys_of(i0 + 4 * tid, in);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
                bool any = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    in[e] = in[e] && ((k[e] ^ prefix) & known) == 0u;
                    any |= in[e];
                }
                if (!__any_sync(0xffffffffu, any)) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t bin = (k[e] >> shift) & mask;
                    int same = 0;
                    if (__all_sync(0xffffffffu, in[e])) __match_all_sync(0xffffffffu, bin, &same);
                    if (in[e] && (!same || lane == 0)) atomicAdd(&h[bin], same ? 32u : 1u);
                }
            }
        }
        cluster_barrier();
        // Thread l owns the kOwn bins down from 2047 - kOwn l: a scan over threads goes from
        // the top.
        uint32_t own[kOwn], sum = 0;  // from the highest bin down
#pragma unroll
        for (int e = 0; e < kOwn; ++e) own[e] = 0;
#pragma unroll (kOwn == 2 ? 8 : 2)
        for (int r = 0; r < ctas; ++r)
#pragma unroll
            for (int e = 0; e < kOwn; e += 2) {
                const uint2 v = ld_cluster2(&h[kBins - 2 - e - kOwn * tid], r);
                own[e] += v.y;
                own[e + 1] += v.x;
            }
#pragma unroll
        for (int e = 0; e < kOwn; ++e) sum += own[e];
        uint32_t above = sum;  // inclusive over the warp's lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
            if (lane >= o) above += v;
        }
        if (lane == 31) warp_sum[warp] = above;
        __syncthreads();
        above += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0u) - sum;
        if (above < want && above + sum >= want) {  // exactly one thread
            int e = 0;
#pragma unroll
            for (int k = 0; k < kOwn - 1; ++k)
                if (e == k && above + own[k] < want) {
                    above += own[k];
                    ++e;
                }
            found[0] = (uint32_t)(kBins - 1 - kOwn * tid - e);
            found[1] = above;
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want -= found[1];
        // (found and warp_sum are written again only after the next cluster barrier; this
        // digit's histogram only after the one after that, when every CTA has read it)
    }
    // Keys above `prefix` stay, and the first `want` equal to it.  A warp takes a
    // contiguous part, 128 keys at a time, four consecutive ones to a lane.
    const int part = ((len + kWarps - 1) / kWarps + 127) / 128 * 128;
    const int w0 = min(len, warp * part), w1 = min(len, w0 + part);
    uint32_t gt = 0, eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 128) {
        bool in[4];
        const uint4 k = keys_of(i0 + 4 * lane, in);
        gt += (in[0] && k.x > prefix) + (in[1] && k.y > prefix) + (in[2] && k.z > prefix) +
              (in[3] && k.w > prefix);
        eq += (in[0] && k.x == prefix) + (in[1] && k.y == prefix) + (in[2] && k.z == prefix) +
              (in[3] && k.w == prefix);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t a = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_gt[lane] : 0u);
        const uint32_t c = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_eq[lane] : 0u);
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
    cluster_arrive_relaxed();  // this thread has read what it needs of the others
    uint32_t at = (uint32_t)lo + gt_before + min(want, eq_before);
    // Sum of v <= 4 over the lanes before this one, and the warp's total, bit by bit.
    const uint32_t below = (1u << lane) - 1u;
    auto lanes_before = [&](uint32_t v, uint32_t &total) {
        const uint32_t b0 = __ballot_sync(0xffffffffu, v & 1), b1 = __ballot_sync(0xffffffffu, v & 2),
                       b2 = __ballot_sync(0xffffffffu, v & 4);
        total = __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
        return (uint32_t)(__popc(b0 & below) + 2 * __popc(b1 & below) + 4 * __popc(b2 & below));
    };
    for (int i0 = w0; i0 < w1; i0 += 128) {
        const int i = i0 + 4 * lane;
        bool in[4];
        const uint4 k4 = keys_of(i, in);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        bool same[4], keep[4];
        uint32_t equals = 0, count = 0, total;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            same[e] = in[e] && k[e] == prefix;
            equals += same[e];
        }
        if (__any_sync(0xffffffffu, equals != 0)) {  // ties, by index
            uint32_t rank_eq = eq_before + lanes_before(equals, total);
            eq_before += total;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (same[e]) same[e] = rank_eq++ < want;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            keep[e] = same[e] || (in[e] && k[e] > prefix);
            count += keep[e];
        }
        uint32_t j = at + lanes_before(count, total);
        at += total;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!keep[e]) continue;
            kept[j] = s0 + i + e;
            if (kept_w) {
                // the weight from its key, without another trip to memory, but for the
                // keys that two weights share (0 and -0; NaN and -inf)
                const float v = key_weight(k[e]);
                kept_w[j] = v == 0.f || v == -INFINITY ? w[s0 + i + e] : v;
            }
            ++j;
        }
    }
    fixed();
    cluster_wait();  // no CTA leaves while another may still read its counts
}

// ---------------------------------------------------------------- compaction
struct CompactParams {
    void *k_pages, *v_pages;
    const int32_t *page_table, *new_table, *kept, *new_lens;
    int32_t Hkv, P, max_pages, new_max_pages, num_pages, max_kept;
    int32_t vec;       // 16-byte pieces per row: 8, 16 or 32
    int32_t lg_piece;  // log2 of it
    uint32_t *status;
};

// The rows that this CTA moves: those of one kv head in one pool of one sequence.
struct Strip {
    uint4 *pool;
    const int32_t *src_table, *dst_table, *kept;
    int n;  // rows of the compacted sequence
};

// grid (.., 2 Hkv, B); false: nothing to move.
__device__ __forceinline__ bool strip_of(const CompactParams &p, Strip &s) {
    const int b = blockIdx.z, g = (int)blockIdx.y % p.Hkv, kv = (int)blockIdx.y / p.Hkv;
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

constexpr int kMoveThreads = 256, kMovePieces = 4, kMoveRows = 2;

// Fresh pages: a thread moves kMovePieces pieces of kMoveRows rows, all loads before the
// first store.
__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const CompactParams p) {
    Strip s;
    if (!strip_of(p, s)) return;
    const int lp = 31 - __clz(p.P), lg = p.lg_piece - 2;  // threads per row: vec / 4
    const int per = kMoveThreads >> lg;
    const int in_row = (int)threadIdx.x & ((1 << lg) - 1);
    const int j0 = (int)blockIdx.x * per * kMoveRows + ((int)threadIdx.x >> lg);
    uint4 x[kMoveRows][kMovePieces];
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
                const uint4 *src = s.pool + slot_of(p, a, t) + in_row;
#pragma unroll
                for (int k = 0; k < kMovePieces; ++k) x[u][k] = src[k << lg];
                dst[u] = slot_of(p, z, j) + in_row;
            }
        }
        if (bad && in_row == 0 && blockIdx.y < (unsigned)p.Hkv) record(p.status, bad);
    }
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
        if (dst[u] >= 0) {
#pragma unroll
            for (int k = 0; k < kMovePieces; ++k) s.pool[dst[u] + (k << lg)] = x[u][k];
        }
}

// In place.  grid (CTAs of a cluster, 2 Hkv, B): the cluster takes one row per group of
// vec / 4 threads and CTA at a time, in order; each thread copies its own four pieces of a
// row through its own slots of a ring (with a row's index, page and address worked out for
// every piece, the instructions took longer than the copies).
constexpr int kShiftThreads = 256, kShiftPieces = 4, kShiftStages = 4;
constexpr int kShiftPer = 16;                                   // chunks whose indices come together
constexpr int kShiftBatch = kShiftPer * kShiftThreads / 2;      // groups of 2 threads or more
constexpr int kShiftPages = 4096;                               // page ids kept in shared memory
constexpr int kShiftRing = kShiftStages * kShiftPieces * kShiftThreads * 16;
constexpr int kShiftSmem = kShiftRing + 2 * kShiftBatch * 4 + kShiftPages * 4;
static_assert(2 * (kShiftSmem + 1024) <= 233472, "two CTAs share an SM");

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kShiftThreads, 2) compact_shift_kernel(const CompactParams p) {
    extern __shared__ __align__(16) uint4 ring[];  // [stage][piece][thread]
    int32_t *kept = reinterpret_cast<int32_t *>(ring + kShiftRing / 16);  // [2][kShiftBatch]
    int32_t *ids = kept + 2 * kShiftBatch;
    Strip s;
    if (!strip_of(p, s)) return;  // the whole cluster alike
    constexpr int N = kShiftPieces, S = kShiftStages;
    const int tid = threadIdx.x;
    const int lp = 31 - __clz(p.P);
    const int lg = p.lg_piece - 2;                       // threads per row: vec / 4
    const int mine = kShiftThreads >> lg, step = mine * (int)gridDim.x;  // rows of a chunk
    const int group = tid >> lg, in_row = tid & ((1 << lg) - 1);
    const int first = (int)blockIdx.x * mine;
    const int ctx = p.max_pages * p.P;                   // below 2^30 (host)
    const int chunks = (s.n + step - 1) / step;
    const bool tells = blockIdx.y < (unsigned)p.Hkv && in_row == 0;
    // Page ids from shared memory, or (tables too long for that) from memory.
    const int32_t *table = s.src_table;
    if (p.max_pages <= kShiftPages) {
        for (int i = tid; i < p.max_pages; i += kShiftThreads) cp_async4(smem_u32(ids + i), table + i);
        table = ids;
    }
    auto fetch = [&](int batch) {  // this CTA's indices of chunks [batch * kShiftPer, + kShiftPer)
        for (int i = tid; i < kShiftPer * mine; i += kShiftThreads) {
            const int64_t j = (int64_t)(batch * kShiftPer + i / mine) * step + first + i % mine;
            if (j < s.n) cp_async4(smem_u32(kept + (batch & 1) * kShiftBatch + i), s.kept + j);
        }
    };
    uint32_t moving = 0;  // bit `slot`: that row is in the ring
    // Sends for chunk c, into slot c % S of the ring.
    auto load = [&](int c, int slot) {
        moving &= ~(1u << slot);
        const int64_t j = (int64_t)c * step + first + group;
        const int t = j < s.n ? kept[(c / kShiftPer & 1) * kShiftBatch + c % kShiftPer * mine + group] : 0;
        if (j < s.n && t != j) {  // (t == j: it is where it belongs)
            if (t < j || t >= ctx) {
                if (tells) record(p.status, ATLAS_DEV_BAD_SEQLEN);
            } else {
                const int a = table[t >> lp], z = table[(int)j >> lp];
                if (a < 0 || a >= p.num_pages || z < 0 || z >= p.num_pages) {
                    if (tells) record(p.status, ATLAS_DEV_BAD_PAGE);
                } else {
                    moving |= 1u << slot;
                    const uint4 *src = s.pool + slot_of(p, a, t) + in_row;
                    const uint32_t dst = smem_u32(ring + slot * N * kShiftThreads + tid);
#pragma unroll
                    for (int k = 0; k < N; ++k)
                        cp_async16(dst + k * kShiftThreads * 16, src + (k << lg), 16);
                }
            }
        }
        cp_async_commit();
    };
    fetch(0);
    fetch(1);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    // Chunks 0 .. S - 2 are on their way before the first is written.
#pragma unroll 1
    for (int c = 0; c < S - 1; ++c) load(c, c);
    cp_async_wait<S - 2>();
    // The barrier only has to keep writes behind reads, never reads behind writes: a row is
    // read once, before any chunk that writes it.  Arrivals are relaxed, so that they do not
    // wait for the writes of the chunk before (a release did, for most of the kernel's time).
    // The memory model orders nothing across a relaxed arrival; what is relied on is that a
    // thread arrives only after cp.async.wait_group has told it that its data lie in shared
    // memory, where no later write to their source can reach them, and that no thread passes
    // the barrier, to issue such a write, before all have arrived.
    cluster_arrive_relaxed();  // this thread has read chunk 0
    int slot = 0, ahead = S - 1;  // the slots of chunks c and c + S - 1
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        // Where batch k of the indices begins, its fetch (kShiftPer chunks ago, long waited
        // for by each thread) becomes visible to the CTA, every thread is done with batch
        // k - 1, and batch k + 1 can be fetched over it.
        const int next = c + S - 1;
        if (next % kShiftPer == 0) {
            __syncthreads();
            fetch(next / kShiftPer + 1);
        }
        load(next, ahead);
        cp_async_wait<S - 2>();  // chunk c + 1 is in the ring
        cluster_wait();          // the whole cluster has read chunk c
        cluster_arrive_relaxed();
        if ((moving >> slot) & 1u) {
            const int j = c * step + first + group;
            uint4 *dst = s.pool + slot_of(p, table[j >> lp], j) + in_row;
            const uint4 *src = ring + slot * N * kShiftThreads + tid;
#pragma unroll
            for (int k = 0; k < N; ++k) dst[k << lg] = src[k * kShiftThreads];
        }
        slot = slot + 1 == S ? 0 : slot + 1;
        ahead = ahead + 1 == S ? 0 : ahead + 1;
    }
    cluster_wait();
    cp_async_wait<0>();
}

}  // namespace
}  // namespace atlas

extern "C" {

atlas_status atlas_kv_select(const float *weights, const int32_t *seq_lens, int32_t n_kv_heads,
                             const atlas_select *S) {
    using namespace atlas;
    if (!weights || !seq_lens || !S || !S->kept || !S->new_lens) return ATLAS_ERR_INVALID_ARG;
    if (!aligned4({weights, seq_lens, S->kept, S->new_lens, S->kept_weights, S->status_word}))
        return ATLAS_ERR_INVALID_ARG;
    if (S->batch < 1 || S->batch > 65535 || n_kv_heads < 1 || n_kv_heads > 65535 ||
        S->row_tokens < 1 || S->row_tokens > INT32_MAX / 2 || S->budget < 1 ||
        S->budget > INT32_MAX / 2 || S->keep_first < 0 || S->keep_recent < 0 ||
        (int64_t)S->keep_first + S->keep_recent > S->budget)
        return ATLAS_ERR_INVALID_ARG;
    const int32_t kept_row = S->kept_row_tokens == 0 ? S->budget : S->kept_row_tokens;
    if (kept_row < S->budget || kept_row > INT32_MAX / 2) return ATLAS_ERR_INVALID_ARG;
    // CTAs write lengths and kept keys while others still read the lengths and the totals: a
    // CTA that read a shortened length would leave the cluster barriers of its row.
    const uint64_t rows_bytes = 4ull * S->batch * n_kv_heads, lens_bytes = 4ull * S->batch;
    const struct {
        const void *at;
        uint64_t bytes;
    } outputs[] = {{S->new_lens, lens_bytes},
                   {S->kept, rows_bytes * S->budget},
                   {S->kept_weights, S->kept_weights ? rows_bytes * kept_row : 0}};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outputs[i].at, outputs[i].bytes, seq_lens, lens_bytes) ||
            overlap(outputs[i].at, outputs[i].bytes, weights, rows_bytes * S->row_tokens))
            return ATLAS_ERR_INVALID_ARG;
        for (int k = 0; k < i; ++k)
            if (overlap(outputs[i].at, outputs[i].bytes, outputs[k].at, outputs[k].bytes))
                return ATLAS_ERR_INVALID_ARG;
    }
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
    p.kept_row = kept_row;
    p.status = S->status_word;
    // More CTAs per row as long as one wave holds them all.
    const int64_t rows = (int64_t)S->batch * n_kv_heads;
    int ctas = 1;
    while (ctas < kSelMaxCtas && (int64_t)ctas * kSelKeys < p.row_tokens &&
           (rows * ctas * 2 <= device_sm_count() || (int64_t)ctas * kSelCache / 4 < p.row_tokens))
        ctas *= 2;
    const int64_t bytes = (((int64_t)p.row_tokens + ctas - 1) / ctas + 3) / 4 * 16;
    const bool cached = bytes <= kSelCache;
    const int threads = ctas > 1 || p.row_tokens > kSelSmallKeys  ? 1024
                        : rows > 2 * (int64_t)device_sm_count() ? 256
                                                                : 512;
    auto kern = threads == 256   ? select_kernel<true, 256>
                : threads == 512 ? select_kernel<true, 512>
                : cached         ? select_kernel<true, 1024>
                                 : select_kernel<false, 1024>;
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATLAS_ERR_CUDA;
    if (dev >= 64 || !configured[dev]) {
        if (cudaFuncSetAttribute(select_kernel<true, 1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSelCache) != cudaSuccess)
            return ATLAS_ERR_CUDA;
        if (dev < 64) configured[dev] = 1;
    }
    (void)cudaGetLastError();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)n_kv_heads, (unsigned)S->batch);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
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
    if (((reinterpret_cast<uintptr_t>(k_pages) | reinterpret_cast<uintptr_t>(v_pages)) & 15u) ||
        !aligned4({page_table, kept, new_lens, C->new_page_table, C->status_word}))
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
    const uint64_t pool = (uint64_t)C->num_pages * n_kv_heads * page_tokens * head_dim *
                          (C->kv_dtype == ATLAS_BF16 ? 2 : 4);
    if (!C->new_page_table && overlap(k_pages, pool, v_pages, pool)) return ATLAS_ERR_INVALID_ARG;
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
    p.lg_piece = p.vec == 8 ? 3 : p.vec == 16 ? 4 : 5;
    if (p.new_table) {
        const int rows = (kMoveThreads >> (p.lg_piece - 2)) * kMoveRows;
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
        // As many CTAs per (sequence, kv head, pool) as fit at once (two to an SM, a few SMs
        // lost to whole clusters), up to a cluster's 8 and to the rows there are.
        const int64_t units = 2 * (int64_t)n_kv_heads * C->batch;
        const int rows = kShiftThreads >> (p.lg_piece - 2);
        int ctas = 1;
        while (ctas < 8 && units * ctas * 2 <= (int64_t)device_sm_count() * 15 / 8 &&
               (int64_t)ctas * rows < p.max_kept)
            ctas *= 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas, (unsigned)(2 * n_kv_heads), (unsigned)C->batch);
        cfg.blockDim = dim3(kShiftThreads, 1, 1);
        cfg.dynamicSmemBytes = kShiftSmem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, compact_shift_kernel, p) != cudaSuccess) return ATLAS_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
