// kv_resize.cu -- page tables made on the device from the sequences' lengths
// (include/atlas_pages.h): each sequence takes the pages that it lacks from a ring of free
// ones, or gives back those that it has too many of.
//
// The mathematics.  want = ceil(len / P), n what a sequence holds, need = max(0, want - n),
// back = max(0, n - want).  The pages that a sequence takes are the `need` ring entries behind
// those of the sequences before it, and what it gives back goes behind what they give, at the
// ring's end: exclusive sums of need and back over the batch, so the outcome is that of one
// sequence after the other, whatever runs when.  The ring has room for every page, so what is
// written behind its end never meets what is read at its front.
//
// A call reads n_pages and the ring's state, and hands their new values on to the next call in
// the same places, so these are written after the last read of them.  Calls of moderate size
// are one cluster of CTAs with a barrier before those writes; large ones a grid on all SMs and
// a single CTA after it.  Every CTA works the sums out for itself, kThreads sequences a round,
// one to a thread; then a round's moves are one list, cut evenly among all threads, which find
// the sequence of a list entry in the sums by bisection.
//
// What bounds it: latencies -- the launch, the sums' barriers, a move's dependent loads, of which
// a thread has kAtOnce in flight.  A call where 32 sequences gain or lose a page or two takes 4.2 us,
// one where half of 256 sequences of up to 8192 pages arrive or leave (0.5 million moves) 9.9.
#include "internal.h"
#include "atlas_pages.h"
#include "ptx.cuh"

namespace atlas {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterCtas = 8;  // the portable cluster size
// Entries of table and slots up to which a call is one cluster (what it moves is known on the
// device alone).  Cluster and grid: 2^16 entries, few moves 4.2 and 5.3 us, half of the batch
// arriving 6.4 and 5.6; 2^17 entries 4.4 and 5.6, 8.9 and 5.8; 2^18 4.4 and 5.6, 14.6 and 6.0.  Most
// steps move little.
constexpr int64_t kOneLaunch = 1 << 17;

struct ResizeParams {
    int32_t *table, *n_pages, *ring, *state;
    const int32_t *lens, *n_new;
    int32_t *slots;
    int32_t B, max_pages, num_pages, P, max_new;
    uint32_t *status;
};

// One sequence's part in the call.
struct Move {
    int n, want;  // pages it holds, pages it shall hold
    int len, fresh;
    bool bad;     // out of range: left as it is
    __device__ int need() const { return max(0, want - n); }
    __device__ int back() const { return max(0, n - want); }
};

__device__ __forceinline__ Move move_of(const ResizeParams &p, int b) {
    Move m{0, 0, 0, 0, false};
    if (b >= p.B) return m;
    m.len = p.lens[b];
    m.n = p.n_pages[b];
    m.fresh = p.max_new == 0 ? 0 : p.n_new ? p.n_new[b] : min(p.max_new, max(m.len, 0));
    m.bad = m.len < 0 || m.len > p.max_pages * p.P || m.n < 0 || m.n > p.max_pages || m.fresh < 0 ||
            m.fresh > p.max_new || m.fresh > m.len;
    m.want = m.bad ? m.n : (m.len + p.P - 1) / p.P;
    return m;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\t"
        "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Inclusive sums of need (low half) and back (high half) over the CTA's threads, and the totals.
// (Each is below 2^31, as batch * max_pages is, so the halves do not meet.)
__device__ __forceinline__ uint64_t scan(uint64_t x, uint64_t &total) {
    __shared__ uint64_t sums[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint64_t a = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += a;
    }
    __syncthreads();  // (the sums of the scan before this one have been read)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    uint64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return x + before;
}

__device__ __forceinline__ int largest(int x) {
    __shared__ int most;
    __syncthreads();
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    x = __reduce_max_sync(0xffffffffu, x);
    if (threadIdx.x % 32 == 0) atomicMax(&most, x);
    __syncthreads();
    return most;
}

struct Totals {
    int need = 0, back = 0;  // sums over the rounds so far
    int taken = 0;           // pages taken by the sequences that are served
};

// One sequence's place in the sums.
struct Round {
    Move m;
    int need, back;  // inclusive sums over the batch
    int moves;       // inclusive sum of the round's moves
    int all;         // moves of the round
    bool lacks;      // its need does not fit
};

__device__ __forceinline__ Round take_round(const ResizeParams &p, int b, int count, Totals &t) {
    Round r;
    r.m = move_of(p, b);
    uint64_t total;
    const uint64_t upto = scan((uint64_t)r.m.need() | (uint64_t)r.m.back() << 32, total);
    const int need = (int)(uint32_t)upto, back = (int)(upto >> 32);
    r.need = t.need + need;
    r.back = t.back + back;
    r.lacks = r.m.need() > 0 && r.need > count;
    // Those that are served are the first ones: pages taken up to a sequence are its sum of needs
    // while that fits, then what the last one served left it at.
    int fits = (int)(uint32_t)total;
    if (t.need + fits > count) fits = largest(r.need <= count ? need : 0);
    r.moves = min(need, fits) + back;
    r.all = fits + (int)(total >> 32);
    t.need += (int)(uint32_t)total;
    t.back += (int)(total >> 32);
    t.taken += fits;
    return r;
}

__device__ __forceinline__ int wrapped(int64_t at, int num) {
    return (int)(at >= 2 * (int64_t)num ? at - 2 * (int64_t)num : at >= num ? at - num : at);
}

// Whether the ring's state is one, and has room for all that comes back.
__device__ bool ring_fits(const ResizeParams &p, int head, int count, int64_t back) {
    return head >= 0 && head < p.num_pages && count >= 0 && count <= p.num_pages &&
           back <= p.num_pages - count;
}
__device__ int64_t all_back(const ResizeParams &p) {
    int64_t back = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        uint64_t total;
        scan((uint64_t)move_of(p, b0 + (int)threadIdx.x).back(), total);
        back += (int64_t)total;
    }
    return back;
}

// The new n_pages and state (one CTA, after everyone's last read of the old ones).
__device__ void finish(const ResizeParams &p, int head, int count) {
    Totals t;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        const Round r = take_round(p, b, count, t);
        if (b < p.B && !r.lacks && r.m.n != r.m.want) p.n_pages[b] = r.m.want;
    }
    if (threadIdx.x == 0) {
        p.state[0] = wrapped((int64_t)head + t.taken, p.num_pages);
        p.state[1] = count - t.taken + t.back;
    }
}

constexpr int kAtOnce = 4;  // moves and slots of a thread whose loads are in flight together

template <bool ONE_LAUNCH>
__global__ void __launch_bounds__(kThreads) kv_resize_kernel(const ResizeParams p) {
    // The round's sequences: inclusive sums of their moves, pages held and wanted, where their
    // pages stand in the ring (behind those of the sequences before), lengths, new tokens.
    __shared__ int s_moves[kThreads], s_n[kThreads], s_want[kThreads], s_from[kThreads],
        s_len[kThreads], s_fresh[kThreads];
    if (!ONE_LAUNCH) allow_dependent_launch();
    const int threads = (int)(gridDim.x * kThreads), me = (int)(blockIdx.x * kThreads + threadIdx.x);
    const int tid = (int)threadIdx.x, lp = 31 - __clz(p.P);
    const int head = p.state[0], count = p.state[1];
    // (a batch of one round finds out below)
    bool fits = p.B <= kThreads || ring_fits(p, head, count, all_back(p));
    uint32_t flags = 0;
    Totals t;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const Round r = take_round(p, b0 + tid, count, t);
        if (p.B <= kThreads) fits = ring_fits(p, head, count, t.back);
        if (r.m.bad) flags |= ATLAS_DEV_BAD_SEQLEN;
        if (r.lacks && fits) flags |= ATLAS_DEV_NO_PAGES;
        const bool moves = fits && !r.lacks;
        s_moves[tid] = r.moves;
        s_n[tid] = r.m.n;
        s_want[tid] = moves ? r.m.want : r.m.n;
        s_from[tid] = r.m.need() ? r.need - r.m.need() : r.back - r.m.back();
        s_len[tid] = r.m.len;
        s_fresh[tid] = moves && !r.m.bad ? r.m.fresh : 0;
        __syncthreads();
        // (places in the lists in 64 bits: a list may have 2^31 - 1, and a step goes past its end)
        const int total = fits ? r.all : 0;
        for (int64_t e0 = me; e0 < total; e0 += threads * kAtOnce) {
            int32_t *from[kAtOnce], *to[kAtOnce];
            int id[kAtOnce];
            bool back[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (e0 + u * threads >= total) continue;
                const int e = (int)e0 + u * threads;
                int lo = 0, hi = kThreads - 1;  // the first sequence whose sum is above e
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (s_moves[mid] > e) hi = mid;
                    else lo = mid + 1;
                }
                const int k = e - (lo ? s_moves[lo - 1] : 0), n = s_n[lo], want = s_want[lo];
                int32_t *row = p.table + (int64_t)(b0 + lo) * p.max_pages;
                back[u] = want < n;
                if (back[u]) {
                    from[u] = row + want + k;
                    to[u] = p.ring + wrapped((int64_t)head + count + s_from[lo] + k, p.num_pages);
                } else {
                    from[u] = p.ring + wrapped((int64_t)head + s_from[lo] + k, p.num_pages);
                    to[u] = row + n + k;
                }
                id[u] = *from[u];
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (e0 + u * threads >= total) continue;
                *to[u] = id[u];
                if (back[u]) *from[u] = -1;
                if (id[u] < 0 || id[u] >= p.num_pages) flags |= ATLAS_DEV_BAD_PAGE;
            }
        }
        // The slots of new tokens: pages that were there from the table, those that are taken
        // now from the ring, so that nothing written in this call is read in it.
        const int slots = p.slots ? min(kThreads, p.B - b0) * p.max_new : 0;
        for (int64_t e0 = me; e0 < slots; e0 += threads * kAtOnce) {
            int id[kAtOnce], at[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                at[u] = -1;
                if (e0 + u * threads >= slots) continue;
                const int e = (int)e0 + u * threads;
                const int s = e / p.max_new, i = e - s * p.max_new;
                if (i >= s_fresh[s]) continue;
                at[u] = s_len[s] - s_fresh[s] + i;
                const int j = at[u] >> lp;
                id[u] = j < s_n[s] ? p.table[(int64_t)(b0 + s) * p.max_pages + j]
                                   : p.ring[wrapped((int64_t)head + s_from[s] + j - s_n[s], p.num_pages)];
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                if (e0 + u * threads >= slots) continue;
                int slot = -1;
                if (at[u] >= 0) {
                    if (id[u] < 0 || id[u] >= p.num_pages) flags |= ATLAS_DEV_BAD_PAGE;
                    else slot = id[u] * p.P + (at[u] & (p.P - 1));
                }
                p.slots[(int64_t)b0 * p.max_new + e0 + u * threads] = slot;
            }
        }
        if (b0 + kThreads < p.B) __syncthreads();  // the round's arrays are rewritten
    }
    if (!fits) flags |= ATLAS_DEV_BAD_PAGE;
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && threadIdx.x % 32 == 0 && p.status) atomicOr(p.status, flags);
    if (ONE_LAUNCH) {
        cluster_sync();
        if (blockIdx.x == 0 && fits) finish(p, head, count);
    }
}

__global__ void __launch_bounds__(kThreads) kv_resize_finish_kernel(const ResizeParams p) {
    wait_for_previous_grid();
    const int head = p.state[0], count = p.state[1];
    const int64_t back = all_back(p);
    __syncthreads();  // (every thread has read the state)
    if (ring_fits(p, head, count, back)) finish(p, head, count);
}

bool apart(const void *a, int64_t na, const void *b, int64_t nb) {
    const char *x = static_cast<const char *>(a), *y = static_cast<const char *>(b);
    return !a || !b || x + 4 * na <= y || y + 4 * nb <= x;
}

}  // namespace
}  // namespace atlas

extern "C" atlas_status atlas_kv_resize(int32_t *page_table, int32_t *n_pages,
                                        const int32_t *seq_lens, int32_t *free_pages,
                                        int32_t *free_state, int32_t page_tokens,
                                        const atlas_resize *Z) {
    using namespace atlas;
    if (!Z || !page_table || !n_pages || !seq_lens || !free_pages || !free_state)
        return ATLAS_ERR_INVALID_ARG;
    if (Z->batch < 1 || Z->max_pages_per_seq < 1 || Z->num_pages < 1 || Z->max_new < 0 ||
        (Z->max_new > 0 && !Z->slots))
        return ATLAS_ERR_INVALID_ARG;
    if (page_tokens < 1 || page_tokens > 128 || (page_tokens & (page_tokens - 1)))
        return ATLAS_ERR_UNSUPPORTED;
    const int64_t B = Z->batch, table = B * Z->max_pages_per_seq, slots = B * Z->max_new;
    if (table > INT32_MAX || slots > INT32_MAX || (int64_t)Z->num_pages * page_tokens > INT32_MAX ||
        (int64_t)Z->max_pages_per_seq * page_tokens > INT32_MAX / 2)
        return ATLAS_ERR_INVALID_ARG;
    if (!aligned4({page_table, n_pages, seq_lens, free_pages, free_state, Z->n_new, Z->slots,
                   Z->status_word}))
        return ATLAS_ERR_INVALID_ARG;
    const struct { const void *at; int64_t n; } all[] = {
        {page_table, table}, {n_pages, B}, {free_pages, Z->num_pages}, {free_state, 2},
        {Z->max_new ? Z->slots : nullptr, slots}, {Z->status_word, 1}, {seq_lens, B},
        {Z->max_new ? Z->n_new : nullptr, B}};
    for (int i = 0; i < 6; ++i)  // the first six are written
        for (int j = i + 1; j < 8; ++j)
            if (!apart(all[i].at, all[i].n, all[j].at, all[j].n)) return ATLAS_ERR_INVALID_ARG;

    ResizeParams p{};
    p.table = page_table;
    p.n_pages = n_pages;
    p.ring = free_pages;
    p.state = free_state;
    p.lens = seq_lens;
    p.n_new = Z->n_new;
    p.slots = Z->max_new ? Z->slots : nullptr;
    p.B = Z->batch;
    p.max_pages = Z->max_pages_per_seq;
    p.num_pages = Z->num_pages;
    p.P = page_tokens;
    p.max_new = Z->max_new;
    p.status = Z->status_word;
    const cudaStream_t stream = static_cast<cudaStream_t>(Z->stream);
    (void)cudaGetLastError();
    // What a call may have to move at most: the table, and the slots.
    const int64_t most = table + slots;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (most <= kOneLaunch) {
        const int ctas = most <= kThreads ? 1 : kClusterCtas;
        cfg.gridDim = dim3(ctas);
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        return cudaLaunchKernelEx(&cfg, kv_resize_kernel<true>, p) == cudaSuccess ? ATLAS_OK
                                                                                  : ATLAS_ERR_CUDA;
    }
    kv_resize_kernel<false><<<(unsigned)device_sm_count(), kThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return ATLAS_ERR_CUDA;
    cfg.gridDim = dim3(1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, kv_resize_finish_kernel, p) == cudaSuccess ? ATLAS_OK
                                                                               : ATLAS_ERR_CUDA;
}
