// shared_stream.cu -- the line of blocks that a call with shared prefixes is cut into
// (shared_prefix.cuh): the plan kernel, which works it out on the device from the groups and
// lengths, and the merge of the tiles that the cuts go through.
#include "internal.h"
#include "ptx.cuh"
#include "shared_prefix.cuh"

#include <math.h>

namespace atlas {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kMinBlocks = 2;  // a CTA's share at least: below, its start outweighs it

// Inclusive sums of x over the CTA, and the total.
__device__ __forceinline__ int64_t plan_scan(int64_t x, int64_t &total) {
    __shared__ int64_t sums[kPlanThreads / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t a = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += a;
    }
    __syncthreads();  // (the sums of the scan before this one have been read)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return x + before;
}

// SMs for the tiles when the sequences' own splits run beside them, on the other SMs and in the
// end on all: the number for which both are done the soonest.  The tiles are bound by their
// products and the splits by memory, so that neither gains from all SMs: 64 sequences of up to
// 2048 own keys behind 32768 shared ones take 113 us with 152 CTAs of tiles, 99 with 96, 108 with
// 64.  Times measured: a pair's block 2.6 us beside the splits and a CTA's start and end 12;
// memory 6 MB a microsecond at most.
__device__ int ctas_beside(const TcParams &p, float line, float own_keys) {
    __shared__ unsigned long long best;
    if (threadIdx.x == 0) best = ~0ull;
    __syncthreads();
    const int sms = p.st.sms;
    for (int n = (int)threadIdx.x + 1; n <= sms; n += kPlanThreads) {
        const float tiles = 12.f + line * (2.6f / kPairCost) / (float)n;
        const float bytes = own_keys * (float)p.Hkv * (float)p.D * 4.f;
        const float beside = fminf(6e6f, (float)(sms - n) * p.st.own_rate);
        const float after = fminf(6e6f, (float)sms * p.st.own_rate);
        const float t = tiles + fmaxf(0.f, bytes - beside * tiles) / after;
        // (positive floats compare as integers; of equal times the larger number)
        atomicMin(&best, ((unsigned long long)__float_as_uint(t) << 32) | (unsigned)(sms - n));
    }
    __syncthreads();
    return sms - (int)(best & 0xffffffffu);
}

// One CTA, before the kernels that read what it writes: a few microseconds, the latency of the
// loads at its start and of the sums.  Batches of up to kPlanThreads sequences keep every array
// in shared memory on the way (longer ones in the workspace).
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const TcParams p) {
    allow_dependent_launch();
    constexpr int N = kPlanThreads;
    __shared__ int s_starts[N + 1], s_pre[N], s_len[N], s_before[N + 1], s_group[N], s_rows[N],
        s_blocks[N], s_weight[N], s_cost[N], s_first[N + 1];
    const SharedStream &st = p.st;
    const int tid = (int)threadIdx.x;
    const bool small = p.B <= N;  // (and as many groups at most)
    const int *const starts = small ? s_starts : st.group_starts;
    const int *const pre_lens = small ? s_pre : st.prefix_lens, *const lens = small ? s_len : p.seq_lens;
    int *const before = small ? s_before : st.before, *const group_of = small ? s_group : st.group;
    int *const rows_of = small ? s_rows : st.rows, *const blocks_of = small ? s_blocks : st.blocks;
    int *const weight_of = small ? s_weight : st.weight, *const cost_of = small ? s_cost : st.head_cost;
    int *const first_of = small ? s_first : st.first;
    const int max_prefix = st.max_prefix_pages * p.P, max_ctx = p.max_pages * p.P;

    bool wrong = false;
    for (int n = tid; n < st.n_groups; n += N) {
        const int a = st.group_starts[n], z = st.group_starts[n + 1];
        wrong |= a < 0 || z < a || z > p.B;
        if (small) {
            s_starts[n] = a;
            s_starts[n + 1] = z;  // (the same value from two threads)
            s_pre[n] = st.prefix_lens[n];
        }
    }
    int my_qn = 0, mine = 0;
    if (tid < p.B) {
        my_qn = p.q_lens ? p.q_lens[tid] : p.q_len;
        mine = p.seq_lens[tid];
        if (small) s_len[tid] = mine;
    }
    const bool bad = __syncthreads_or(wrong) != 0;
    uint32_t flags = bad ? ATLAS_DEV_BAD_SEQLEN : 0u;

    // sequences: their groups, and the rows before them
    int64_t carry = 0, own_keys = 0;
    for (int b0 = 0; b0 < p.B; b0 += N) {
        const int b = b0 + tid;
        int rows = 0, own = 0;
        if (b < p.B) {
            int group = -1;
            if (!bad) {
                int lo = -1, hi = st.n_groups - 1;  // the last group that starts at b or before
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (starts[mid] <= b) lo = mid;
                    else hi = mid - 1;
                }
                if (lo >= 0 && b < starts[lo + 1]) group = lo;
            }
            group_of[b] = group;
            const int qn = b0 == 0 ? my_qn : p.q_lens ? p.q_lens[b] : p.q_len;
            const int len = b0 == 0 ? mine : p.seq_lens[b];
            if (len > 0 && len <= max_ctx) own = len;
            bool good = qn >= 0 && qn <= p.q_len && !bad;
            if (st.whole) {
                const int pre = group >= 0 ? pre_lens[group] : 0;
                good = good && pre >= 0 && pre <= max_prefix && len >= qn && len <= max_ctx;
                blocks_of[b] = good ? (pre + 127) / 128 + (len + 127) / 128 : -1;
                if (!good) flags |= ATLAS_DEV_BAD_SEQLEN;
                rows_of[b] = good ? p.G * qn : 0;
            }
            rows = good ? p.G * qn : 0;
        }
        // (both sums in one scan: rows below 2^31, own keys below 2^31 a round)
        int64_t total;
        const int64_t upto = plan_scan((int64_t)rows << 32 | (uint32_t)own, total);
        if (b < p.B) before[b] = (int)(carry + (upto >> 32) - rows);
        carry += total >> 32;
        own_keys += (uint32_t)total;
    }
    if (tid == 0) before[p.B] = (int)carry;
    __syncthreads();

    // units: their rows and blocks, and what all of them have
    auto head_cost = [&](int rows, int nb) {  // tiles of one kv head, each counting as nb blocks
        if (st.tile_rows != 256) return (rows + 127) / 128 * kSingleCost * nb;
        const int last = rows % 256;
        return (rows / 256 * kPairCost + (last == 0 ? 0 : last <= 128 ? kSingleCost : kPairCost)) * nb;
    };
    __shared__ int s_most;
    if (tid == 0) s_most = 0;
    int64_t all = 0;
    for (int u0 = 0; u0 < st.units; u0 += N) {
        const int u = u0 + tid;
        int64_t length = 0;
        int nb = 0;
        if (u < st.units) {
            if (!st.whole) {
                const int len = pre_lens[u];
                const bool good = len >= 0 && len <= max_prefix && !bad;
                if (!good) flags |= ATLAS_DEV_BAD_SEQLEN;
                rows_of[u] = good ? before[starts[u + 1]] - before[starts[u]] : 0;
                blocks_of[u] = good ? (len + 127) / 128 : -1;
            }
            if (rows_of[u] > 0 && blocks_of[u] > 0) {
                nb = blocks_of[u];
                length = (int64_t)head_cost(rows_of[u], nb + kTileBlocks) * p.Hkv;
            }
        }
        nb = __reduce_max_sync(0xffffffffu, nb);
        int64_t total;
        plan_scan(length, total);
        if (tid % 32 == 0 && nb > 0) atomicMax(&s_most, nb);  // (zeroed before the scan's barriers)
        all += total;
    }
    __syncthreads();
    const int most = s_most;
    // A CTA's share: one CTA for each SM, few enough states of a tile, and few enough pieces of a
    // CTA, for which short tiles count as more blocks than they have.
    const int ctas = st.own_rate > 0.f ? ctas_beside(p, (float)all, (float)own_keys) : st.sms;
    int64_t per64 = (all + ctas - 1) / ctas;
    per64 = max(per64, (int64_t)kMinBlocks * kPairCost);
    per64 = max(per64, (int64_t)((most + st.max_states - 3) / (st.max_states - 2)) * kPairCost);
    const int per = (int)per64;
    const int least = (per + kSingleCost * (st.max_items - 2) - 1) / (kSingleCost * (st.max_items - 2));
    carry = 0;
    for (int u0 = 0; u0 < st.units; u0 += N) {
        const int u = u0 + tid;
        int64_t length = 0;
        if (u < st.units) {
            const bool some = rows_of[u] > 0 && blocks_of[u] > 0;
            const int nb = some ? max(blocks_of[u] + kTileBlocks, least) : 0;
            weight_of[u] = nb;
            cost_of[u] = some ? head_cost(rows_of[u], nb) : 1;
            length = some ? (int64_t)cost_of[u] * p.Hkv : 0;
        }
        int64_t total;
        const int64_t upto = plan_scan(length, total);
        if (u < st.units) first_of[u] = (int)(carry + upto - length);
        carry += total;
    }
    const int line = (int)carry;
    if (tid == 0) {
        first_of[st.units] = line;
        st.head[0] = per;
        st.head[1] = line;
        st.head[2] = bad;
    }
    if (flags && p.status) atomicOr(p.status, flags);
    __syncthreads();
    if (small) {  // what the kernels behind read
        for (int u = tid; u < st.units; u += N) {
            st.rows[u] = rows_of[u];
            st.blocks[u] = blocks_of[u];
            st.weight[u] = weight_of[u];
            st.head_cost[u] = cost_of[u];
            st.first[u] = first_of[u];
        }
        if (tid == 0) st.first[st.units] = line;
        if (tid < p.B) {
            st.before[tid] = before[tid];
            st.group[tid] = group_of[tid];
        }
        if (tid == 0) st.before[p.B] = before[p.B];
    }
    if (!st.whole) {
        for (int b = tid; b < p.B; b += N) {
            const int u = group_of[b];
            SeqInfo s{};
            if (bad) s.blocks = -1;
            else if (u >= 0) {
                s.blocks = blocks_of[u];
                s.row0 = before[b] - before[starts[u]];
                s.first = first_of[u];
                s.rows = rows_of[u];
                s.head_cost = cost_of[u];
                s.weight = weight_of[u];
                s.per = per;
            }
            reinterpret_cast<SeqInfo *>(st.info)[b] = s;
        }
        // The order of the sequences' own splits: the longest first, so that the CTAs left over
        // when the others are done are short ones.
        if (small) {
            if (tid < p.B) {
                int rank = 0;
#pragma unroll 8
                for (int k = 0; k < p.B; ++k) rank += lens[k] > mine || (lens[k] == mine && k < tid);
                st.order[rank] = tid;
            }
        } else {
            for (int b = tid; b < p.B; b += N) st.order[b] = b;
        }
    }
    // The CTAs' pieces, a CTA to a thread.
    for (int64_t x = tid; x * per < line; x += N) {
        const int end = (int)min((int64_t)line, (x + 1) * per);
        SharedSeg *const segs = st.segs + x * st.max_items;
        int n = 0, s = (int)x * per, lo = 0, hi = st.units - 1;
        while (lo < hi) {  // the last unit that begins at s or before and is not empty
            const int mid = (lo + hi + 1) / 2;
            if (first_of[mid] <= s) lo = mid;
            else hi = mid - 1;
        }
        int unit = lo;
        const int full = st.tile_rows == 256 ? kPairCost : kSingleCost;
        while (s < end && n < st.max_items) {
            while (s >= first_of[unit + 1]) ++unit;
            const int weight = weight_of[unit], rows = rows_of[unit];
            const int tiles = (rows + st.tile_rows - 1) / st.tile_rows;
            const int at = s - first_of[unit], hkv = at / cost_of[unit];
            const int tile = min((at - hkv * cost_of[unit]) / (full * weight), tiles - 1);
            SharedTile t{unit, hkv, tile, first_of[unit] + hkv * cost_of[unit] + tile * full * weight,
                         block_cost(st, tile, rows), 0};
            t.end = t.first + t.cost * weight;
            SharedSeg g;
            g.unit = unit;
            g.hkv = hkv;
            g.row0 = tile * st.tile_rows;
            g.rows = rows;
            g.group = st.whole ? group_of[unit] : unit;
            g.len = g.group >= 0 ? pre_lens[g.group] : 0;
            g.own = 0;
            if (st.whole)
                g.own = tile_own_keys(lens[unit], rows / p.G, g.row0, min(g.row0 + st.tile_rows, rows));
            const int nb = (g.len + 127) / 128 + (g.own + 127) / 128;
            g.blk0 = block_from(t, s);
            g.nb = min(block_from(t, min(end, t.end)), nb) - g.blk0;
            const int home = t.first / per;
            g.state = st.whole && home == (t.first + (nb - 1) * t.cost) / per ? -1 : (int)x - home;
            if (g.nb > 0) segs[n++] = g;
            s = t.end;
        }
        st.counts[x] = n;
    }

    // ragged groups: their rows one after the other, no padding between
    if (st.list && p.q_lens) {
        const int lane = tid % 32;
        for (int b = tid / 32; b < p.B; b += N / 32) {
            const int at = before[b], rows = before[b + 1] - at;
            const int qn = rows / p.G;
            for (int r = lane; r < rows; r += 32) {
                const int g = r / qn;
                st.list[at + r] = (b * p.Hq + g) * p.q_len + (r - g * qn);
            }
        }
    }
}

// The tiles that are cut (st.whole): the CTA's share of the rows of the tile that the line's
// cut before block x n goes through, if that is the tile's first cut; and NaN for the sequences
// that are out of range.
constexpr int kCutWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCutWarps * 32) shared_cut_merge_kernel(const TcParams p, int ctas) {
    constexpr int E = D / 32;  // (a lane's elements: one vector load)
    const SharedStream &st = p.st;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_for_previous_grid();
    auto put = [&](int64_t row, const float (&o)[E], float lse) {
        if (p.out_bf16) {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<uint32_t *>(out + e) = pack_bf16(o[e], o[e + 1]);
        } else {
            float *out = static_cast<float *>(p.out) + row * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<float2 *>(out + e) = make_float2(o[e], o[e + 1]);
        }
        if (lane == 0 && p.lse) p.lse[row] = lse;
    };
    if ((int)blockIdx.x >= ctas) {
        const int b = (int)blockIdx.x - ctas;
        if (st.blocks[b] >= 0) return;
        const float nan = __int_as_float(0x7fc00000);
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = nan;
        const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
        const int rows = qn >= 0 && qn <= p.q_len ? qn : p.q_len;
        for (int64_t r = (int64_t)blockIdx.y * kCutWarps + warp; r < (int64_t)p.Hq * p.q_len;
             r += (int64_t)gridDim.y * kCutWarps)
            if (r % p.q_len < rows) put((int64_t)b * p.Hq * p.q_len + r, o, nan);
        return;
    }
    const int per = st.head[0], x = (int)blockIdx.x + 1;
    if ((int64_t)x * per >= st.head[1]) return;
    const SharedTile t = tile_of(st, x * per);
    if (t.first / per != x - 1) return;  // not cut here first
    SharedSeg s;
    const int nb = tile_blocks(p, t, s);
    const int states = (t.first + (nb - 1) * t.cost) / per - (x - 1) + 1;
    const int f = s.row0 + (int)blockIdx.y * kCutWarps + warp;
    if (states < 2 || f >= s.rows) return;
    // the first state is that of a tile's start, the others those of their CTAs' first pieces
    auto slot = [&](int k) { return ((int64_t)(x - 1 + k) * 2 + (k == 0)) * st.tile_rows + f - s.row0; };
    const int64_t row = unit_row(p, t.unit, t.hkv, f);
    float M = p.sinks ? p.sinks[s.hkv * p.G + f / (s.rows / p.G)] * kLog2e : -INFINITY;
    bool has_nan = isnan(M);
    float sum = p.sinks ? 1.f : 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    // Lane k has the weight of state k, of 32 at a time; the accumulators' loads of a few states
    // are in flight together.
    for (int k0 = 0; k0 < states; k0 += 32) {
        const int k = k0 + lane;
        float m = -INFINITY, l = 0.f;
        if (k < states) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + slot(k) * 2);
            m = ml.x;
            l = ml.y;
        }
        has_nan |= __any_sync(0xffffffffu, isnan(m) || isnan(l));
        float top = l > 0.f ? m : -INFINITY;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = fmaxf(M, top);
        const float old = M == -INFINITY ? 0.f : ex2(M - top), w = l > 0.f ? ex2(m - top) : 0.f;
        M = top;
        float add = w * l;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) add += __shfl_xor_sync(0xffffffffu, add, d);
        sum = sum * old + add;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= old;
#pragma unroll 4
        for (int j = 0; j < min(32, states - k0); ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const float *at = p.ws_acc + slot(k0 + j) * D + lane * E;
            float a[E];
            if constexpr (E == 4) *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(at);
            else *reinterpret_cast<float2 *>(a) = *reinterpret_cast<const float2 *>(at);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(wj, a[e], o[e]);
        }
    }
    const float nan = __int_as_float(0x7fc00000);
    const bool none = has_nan || M == -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = none ? nan : o[e] / sum;
    put(row, o, none ? nan : kLn2 * (M + log2f(sum)));
}

}  // namespace

cudaError_t launch_shared_plan(const TcParams &p, cudaStream_t stream) {
    shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_shared_cut_merge(const TcParams &p, int64_t ctas, cudaStream_t stream) {
    const dim3 grid((unsigned)(ctas + p.B), (unsigned)(p.st.tile_rows / kCutWarps));
    return p.D == 128 ? launch_dependent(shared_cut_merge_kernel<128>, grid, dim3(kCutWarps * 32), 0,
                                         stream, p, (int)ctas)
                      : launch_dependent(shared_cut_merge_kernel<64>, grid, dim3(kCutWarps * 32), 0,
                                         stream, p, (int)ctas);
}

}  // namespace atlas
