// kv_evict.cu -- the keys that stay under a budget (atlas_kv_select) and the pages with
// only those keys left (atlas_kv_compact).
//
// Selection.  One thread-block cluster per (sequence, kv head), its CTAs sharing the row:
// each maps its part of the weights to order-preserving 32-bit keys in shared memory (read
// from memory once), and four 8-bit digits, from the top, narrow the k-th largest key down
// exactly: a histogram of the digit over the keys that match the digits found so far,
// summed over the cluster through distributed shared memory, tells which bin the k-th
// largest lies in and how many are still wanted there.  What equals the last key is taken
// by lowest index, so the set never depends on timing, and positions in the ascending
// output are counts of kept keys before (ballots in a warp, sums over warps and CTAs).
// Memory: 4 bytes per key in, 8 per kept key out; bound by latency, five cluster barriers.
//
// Compaction.  Rows of head_dim elements move between page slots, 16 bytes per thread and
// step.  Into fresh pages every row is independent.  In place, row j takes row kept[j] >= j:
// a row may only be overwritten once it has been read.  Rows are taken in ascending order
// in chunks, and since a chunk's sources lie at or behind its own destinations, it is
// enough that a chunk is read completely (a CTA barrier) before it is written: later
// chunks' sources lie behind it, earlier ones have been read.  No CTA waits on another:
// each owns a 64-byte wide strip of one (sequence, kv head, K or V) from end to end, reads
// one chunk ahead (and page ids and indices two and three ahead), so a step costs one
// memory latency.
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
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMaxCtas = 8;  // the portable cluster size

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

// The 32-bit word that CTA `rank` of the cluster holds where this CTA holds *local.
__device__ __forceinline__ uint32_t ld_cluster(const uint32_t *local, int rank) {
    uint32_t addr, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// grid (CTAs of a row's cluster, Hkv, B).  CACHED: the row's keys stay in shared memory;
// else (rows too long for that) each pass reads the weights again.
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    extern __shared__ uint32_t cached[];
    __shared__ uint32_t hist[2][256];
    __shared__ uint32_t found[2];                 // digit, keys above it
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
    for (int j = n + me; j < p.budget; j += all) {
        kept[j] = -1;
        if (kept_w) kept_w[j] = 0.f;
    }
    // Keys that stay whatever their weight: all of them, or the first and the recent ones.
    const bool whole = L <= p.budget;
    const int lo = whole ? L : p.first, hi = whole ? L : L - p.recent;
    for (int j = me; j < lo + (L - hi); j += all) {
        const int t = j < lo ? j : hi + (j - lo);
        const int at = j < lo ? j : n - (L - hi) + (j - lo);
        kept[at] = t;
        if (kept_w) kept_w[at] = w[t];
    }
    uint32_t want = (uint32_t)(n - lo - (L - hi));  // of the keys in [lo, hi)
    if (want == 0) return;                          // the whole cluster alike

    const int seg = (hi - lo + ctas - 1) / ctas;
    const int s0 = min(hi, lo + rank * seg), len = min(hi, s0 + seg) - s0;
    if (CACHED)
        for (int i = tid; i < len; i += kSelThreads) cached[i] = order_key(w[s0 + i]);
    auto key_of = [&](int i) { return CACHED ? cached[i] : order_key(w[s0 + i]); };

    uint32_t prefix = 0;
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
        const int shift = 24 - 8 * d;
        uint32_t *h = hist[d & 1];
        for (int i = tid; i < 256; i += kSelThreads) h[i] = 0u;
        __syncthreads();
        for (int i0 = 0; i0 < len; i0 += kSelThreads) {
            const int i = i0 + tid;
            uint32_t bin = 256;  // no vote
            if (i < len) {
                const uint32_t k = key_of(i);
                if (d == 0 || ((k ^ prefix) >> (shift + 8)) == 0u) bin = (k >> shift) & 255u;
            }
            // one addition per distinct digit of the warp: the top digits are nearly all
            // alike, and 32 additions to one word would go one after another
            const uint32_t peers = __match_any_sync(0xffffffffu, bin);
            if (bin < 256 && lane == __ffs(peers) - 1) atomicAdd(&h[bin], (uint32_t)__popc(peers));
        }
        cluster_barrier();
        if (warp == 0) {
            // lane l: bins 255 - 8l .. 248 - 8l, from the top
            uint32_t cnt[8], sum = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cnt[e] = 0;
                for (int r = 0; r < ctas; ++r) cnt[e] += ld_cluster(&h[255 - 8 * lane - e], r);
                sum += cnt[e];
            }
            uint32_t above = sum;  // inclusive scan over lanes, then exclusive
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += v;
            }
            above -= sum;
            if (above < want && above + sum >= want) {  // exactly one lane
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (above < want && above + cnt[e] >= want) {
                        found[0] = 255u - 8u * lane - e;
                        found[1] = above;
                    }
                    above += cnt[e];
                }
            }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want -= found[1];
        // (found is written again only after the next cluster barrier; this digit's
        // histogram only after the one after that, when every CTA has read it)
    }
    // Keys above `prefix` stay, and the first `want` equal to it.  A warp takes a
    // contiguous part, 32 keys at a time in order.
    const int part = ((len + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int w0 = min(len, warp * part), w1 = min(len, w0 + part);
    uint32_t gt = 0, eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? key_of(i) : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i < w1 && k > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i < w1 && k == prefix));
    }
    if (lane == 0) {
        warp_gt[warp] = gt;
        warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t a = 0, c = 0;
        for (int k = 0; k < kSelWarps; ++k) {
            a += warp_gt[k];
            c += warp_eq[k];
        }
        cta_gt = a;
        cta_eq = c;
    }
    cluster_barrier();
    uint32_t gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        gt_before += ld_cluster(&cta_gt, r);
        eq_before += ld_cluster(&cta_eq, r);
    }
    for (int k = 0; k < warp; ++k) {
        gt_before += warp_gt[k];
        eq_before += warp_eq[k];
    }
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

constexpr int kShiftThreads = 512, kShiftRows = 4;

// In place: one CTA per strip walks the rows in order, a chunk at a time.
__global__ void __launch_bounds__(kShiftThreads) compact_shift_kernel(const CompactParams p) {
    Strip s;
    if (!strip_of(p, s)) return;
    const int lp = 31 - __clz(p.P);
    const int per = kShiftThreads >> p.lg_piece;
    const int chunk = per * kShiftRows;
    const int r = (int)threadIdx.x >> p.lg_piece;
    const int64_t ctx = (int64_t)p.max_pages * p.P;
    // Index of row u of chunk c (-1: no such row), and the page ids of an index and of
    // its destination; both are only used a step later.
    auto index = [&](int64_t c, int (&t)[kShiftRows]) {
#pragma unroll
        for (int u = 0; u < kShiftRows; ++u) {
            const int64_t j = c * chunk + u * per + r;
            t[u] = j < s.n ? s.kept[j] : -1;
            if (j < s.n && (t[u] < j || t[u] >= ctx)) {
                if (s.tells) record(p.status, ATLAS_DEV_BAD_SEQLEN);
                t[u] = -1;
            }
        }
    };
    auto pages = [&](int64_t c, const int (&t)[kShiftRows], int (&a)[kShiftRows], int (&z)[kShiftRows]) {
#pragma unroll
        for (int u = 0; u < kShiftRows; ++u) {
            const int64_t j = c * chunk + u * per + r;
            a[u] = t[u] >= 0 ? s.src_table[t[u] >> lp] : 0;
            z[u] = t[u] >= 0 ? s.dst_table[j >> lp] : 0;
        }
    };
    // Loads chunk c; dst -1 where nothing moves (no row, a bad page, a row already there).
    auto load = [&](int64_t c, const int (&t)[kShiftRows], const int (&a)[kShiftRows],
                    const int (&z)[kShiftRows], uint4 (&x)[kShiftRows], int64_t (&dst)[kShiftRows]) {
#pragma unroll
        for (int u = 0; u < kShiftRows; ++u) {
            const int64_t j = c * chunk + u * per + r;
            dst[u] = -1;
            if (t[u] < 0) continue;
            if (a[u] < 0 || a[u] >= p.num_pages || z[u] < 0 || z[u] >= p.num_pages) {
                if (s.tells) record(p.status, ATLAS_DEV_BAD_PAGE);
                continue;
            }
            if (t[u] == j) continue;
            x[u] = s.pool[slot_of(p, a[u], t[u]) + s.piece];
            dst[u] = slot_of(p, z[u], (int)j) + s.piece;
        }
    };
    const int64_t chunks = (s.n + chunk - 1) / chunk;
    int t1[kShiftRows], t2[kShiftRows], a1[kShiftRows], z1[kShiftRows];
    uint4 cur[kShiftRows], nxt[kShiftRows];
    int64_t dst[kShiftRows], dst_nxt[kShiftRows];
    index(0, t1);
    index(1, t2);
    pages(0, t1, a1, z1);
    load(0, t1, a1, z1, cur, dst);
    pages(1, t2, a1, z1);
#pragma unroll
    for (int u = 0; u < kShiftRows; ++u) t1[u] = t2[u];
    index(2, t2);
    for (int64_t c = 0; c < chunks; ++c) {
        load(c + 1, t1, a1, z1, nxt, dst_nxt);
        pages(c + 2, t2, a1, z1);
#pragma unroll
        for (int u = 0; u < kShiftRows; ++u) t1[u] = t2[u];
        index(c + 3, t2);
        __syncthreads();  // every thread has read chunk c
#pragma unroll
        for (int u = 0; u < kShiftRows; ++u) {
            if (dst[u] >= 0) s.pool[dst[u]] = cur[u];
            cur[u] = nxt[u];
            dst[u] = dst_nxt[u];
        }
    }
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
    // CTAs per row: up to 8 of about 4096 keys each.
    int ctas = 1;
    while (ctas < kSelMaxCtas && (int64_t)ctas * 4096 < p.row_tokens) ctas *= 2;
    const int64_t bytes = ((int64_t)p.row_tokens + ctas - 1) / ctas * 4;
    const bool cached = bytes <= 200 * 1024;
    auto kern = cached ? select_kernel<true> : select_kernel<false>;
    static int configured[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ATLAS_ERR_CUDA;
    if (dev >= 64 || !configured[dev]) {
        if (cudaFuncSetAttribute(select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 200 * 1024) != cudaSuccess)
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
        p.lg_piece = 2;  // 64-byte strips
        const dim3 grid(1, (unsigned)(2 * n_kv_heads * (p.vec >> 2)), (unsigned)C->batch);
        compact_shift_kernel<<<grid, kShiftThreads, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
