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
#include "internal.h"
#include "atlas_pages.h"
#include "ptx.cuh"

namespace atlas {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kClusterCtas = 8;  // the portable cluster size

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

// Inclusive sums of x over the CTA's threads, and the total (below 2^31: batch * max_pages is).
__device__ __forceinline__ int scan(int x, int &total) {
    __shared__ int sums[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int a = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += a;
    }
    __syncthreads();  // (the sums of the scan before this one have been read)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return x + before;
}

// The sums of one round of sequences.
struct Round {
    Move m;
    int need, back;    // inclusive sums over the batch
    bool lacks;        // its need does not fit
};

struct Totals {
    int need = 0, back = 0;  // sums over the rounds so far
    int taken = 0;           // pages taken by the sequences that are served
};

__device__ __forceinline__ Round take_round(const ResizeParams &p, int b, int count, Totals &t) {
    Round r;
    r.m = move_of(p, b);
    int need, back;
    r.need = t.need + scan(r.m.need(), need);
    r.back = t.back + scan(r.m.back(), back);
    r.lacks = r.m.need() > 0 && r.need > count;
    t.need += need;
    t.back += back;
    int served;
    scan(r.lacks ? 0 : r.m.need(), served);
    t.taken += served;
    return r;
}

__device__ __forceinline__ int wrapped(int64_t at, int num) {
    return (int)(at >= 2 * (int64_t)num ? at - 2 * (int64_t)num : at >= num ? at - num : at);
}

// Whether the ring's state is one, and has room for all that comes back.
__device__ bool ring_fits(const ResizeParams &p, int head, int count) {
    if (head < 0 || head >= p.num_pages || count < 0 || count > p.num_pages) return false;
    int64_t back = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        int total;
        scan(move_of(p, b0 + (int)threadIdx.x).back(), total);
        back += total;
    }
    return back <= p.num_pages - count;
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

template <bool ONE_LAUNCH>
__global__ void __launch_bounds__(kThreads) kv_resize_kernel(const ResizeParams p) {
    __shared__ int s_moves[kThreads];             // inclusive sums of the round's moves
    __shared__ int s_n[kThreads], s_want[kThreads], s_from[kThreads], s_len[kThreads], s_fresh[kThreads];
    if (!ONE_LAUNCH) allow_dependent_launch();
    const int threads = (int)(gridDim.x * kThreads), me = (int)(blockIdx.x * kThreads + threadIdx.x);
    const int head = p.state[0], count = p.state[1];
    const bool fits = ring_fits(p, head, count);
    uint32_t flags = fits ? 0u : ATLAS_DEV_BAD_PAGE;
    Totals t;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
        const int tid = (int)threadIdx.x;
        const Round r = take_round(p, b0 + tid, count, t);
        const bool moves = fits && !r.lacks;
        if (r.m.bad) flags |= ATLAS_DEV_BAD_SEQLEN;
        if (r.lacks && fits) flags |= ATLAS_DEV_NO_PAGES;
        int total;
        s_moves[tid] = scan(moves ? r.m.need() + r.m.back() : 0, total);
        s_n[tid] = r.m.n;
        s_want[tid] = moves ? r.m.want : r.m.n;
        // where its pages stand in the ring: behind those of the sequences before it
        s_from[tid] = r.m.need() ? r.need - r.m.need() : r.back - r.m.back();
        s_len[tid] = r.m.len;
        s_fresh[tid] = moves && !r.m.bad ? r.m.fresh : 0;
        __syncthreads();
        for (int e = me; e < total; e += threads) {
            int lo = 0, hi = kThreads - 1;  // the first sequence whose sum is above e
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                if (s_moves[mid] > e) hi = mid;
                else lo = mid + 1;
            }
            const int k = e - (lo ? s_moves[lo - 1] : 0), n = s_n[lo], want = s_want[lo];
            int32_t *row = p.table + (int64_t)(b0 + lo) * p.max_pages;
            int id;
            if (want > n) {
                id = p.ring[wrapped((int64_t)head + s_from[lo] + k, p.num_pages)];
                row[n + k] = id;
            } else {
                id = row[want + k];
                p.ring[wrapped((int64_t)head + count + s_from[lo] + k, p.num_pages)] = id;
                row[want + k] = -1;
            }
            if (id < 0 || id >= p.num_pages) flags |= ATLAS_DEV_BAD_PAGE;
        }
        // The slots of new tokens: pages that were there from the table, those that are taken
        // now from the ring, so that nothing written in this call is read in it.
        const int rows = min(kThreads, p.B - b0);
        if (p.slots) {
            for (int e = me; e < rows * p.max_new; e += threads) {
                const int s = e / p.max_new, i = e - s * p.max_new;
                int slot = -1;
                if (i < s_fresh[s]) {
                    const int at = s_len[s] - s_fresh[s] + i, j = at / p.P;
                    const int id = j < s_n[s] ? p.table[(int64_t)(b0 + s) * p.max_pages + j]
                                              : p.ring[wrapped((int64_t)head + s_from[s] + j - s_n[s],
                                                               p.num_pages)];
                    if (id < 0 || id >= p.num_pages) flags |= ATLAS_DEV_BAD_PAGE;
                    else slot = id * p.P + at % p.P;
                }
                p.slots[(int64_t)b0 * p.max_new + e] = slot;
            }
        }
        __syncthreads();  // the round's arrays are rewritten
    }
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
    if (ring_fits(p, head, count)) {
        __syncthreads();  // (every thread has read the state)
        finish(p, head, count);
    }
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
    if (most <= (int64_t)1 << 18) {
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
