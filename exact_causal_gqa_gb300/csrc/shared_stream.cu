// shared_stream.cu -- the line of blocks that a call with shared prefixes is cut into
// (shared_prefix.cuh): the plan kernel, which works it out on the device from the groups and
// lengths, and the merge of the tiles that the cuts go through.
#include "internal.h"
#include "ptx.cuh"
#include "shared_prefix.cuh"

#include <math.h>
#include <type_traits>

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
// 64 (weights in one part).  Times measured: a pair's block 2.6 us beside the splits and a CTA's start
// and end 12; memory 6 MB a microsecond at most.  (2.6 to 3.2 us lead to the same times within 2 %.)
__device__ int ctas_beside(const TcParams &p, float line, float own_keys) {
    __shared__ uint64_t best[kPlanThreads / 32];
    const int sms = p.st.sms;
    uint64_t mine = ~0ull;
    for (int n = (int)threadIdx.x + 1; n <= sms; n += kPlanThreads) {
        const float tiles = 12.f + line * (2.6f / kPairCost) / (float)n;
        const float bytes = own_keys * (float)p.Hkv * (float)p.D * 4.f;
        const float beside = fminf(6e6f, (float)(sms - n) * p.st.own_rate);
        const float after = fminf(6e6f, (float)sms * p.st.own_rate);
        const float t = tiles + fmaxf(0.f, bytes - beside * tiles) / after;
        // (positive floats compare as integers; of equal times the larger number)
        mine = min(mine, ((uint64_t)__float_as_uint(t) << 32) | (unsigned)(sms - n));
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) mine = min(mine, __shfl_xor_sync(0xffffffffu, mine, d));
    if (threadIdx.x % 32 == 0) best[threadIdx.x / 32] = mine;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) mine = min(mine, best[w]);
    return sms - (int)(mine & 0xffffffffu);
}

// One CTA, before the kernels that read what it writes: a few microseconds, the latency of the
// loads at its start and of the sums.  Batches of up to kPlanThreads sequences keep every array
// in shared memory on the way (longer ones in the workspace).
__global__ void __launch_bounds__(kPlanThreads) shared_plan_kernel(const TcParams p) {
    allow_dependent_launch();
    constexpr int N = kPlanThreads;
    __shared__ int s_starts[N + 1], s_pre[N], s_len[N], s_before[N + 1], s_group[N], s_rows[N],
        s_blocks[N], s_weight[N], s_cost[N], s_first[N + 1];
    __shared__ __align__(16) int s_key[N];  // the sequences' order: length, then place
    const SharedStream &st = p.st;
    const int tid = (int)threadIdx.x;
    const bool small = p.B <= N && st.n_groups <= N;
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
    static_assert(N == 1 << 9, "the keys' places");
    s_key[tid] = tid < p.B ? min(max(mine, 0), (1 << 22) - 1) << 9 | (N - 1 - tid) : -1;
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
            if (len > 0 && len <= max_ctx) own = min(len, 1 << 22);  // (an estimate's)
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
        // (both sums in one scan: rows below 2^31, own keys 512 * 2^22 a round at most)
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
    const int tile_blocks = st.whole ? kWholeTileBlocks : kTileBlocks;
    int64_t all = 0;
    int n_tiles = 0;
    for (int u0 = 0; u0 < st.units; u0 += N) {
        const int u = u0 + tid;
        int64_t length = 0, tiles = 0;
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
                length = (int64_t)head_cost(rows_of[u], nb + tile_blocks) * p.Hkv;
                tiles = (int64_t)((rows_of[u] + st.tile_rows - 1) / st.tile_rows) * p.Hkv;
            }
        }
        nb = __reduce_max_sync(0xffffffffu, nb);
        int64_t total;
        plan_scan(tiles << 36 | length, total);  // (lengths below 2^31 in all, tiles below 2^26)
        n_tiles += (int)(total >> 36);
        total &= (1ll << 36) - 1;
        if (tid % 32 == 0 && nb > 0) atomicMax(&s_most, nb);  // (zeroed before the scan's barriers)
        all += total;
    }
    __syncthreads();
    const int most = s_most;
    // A CTA's share: one CTA for each SM (two, three for very many tiles), few enough states of a
    // tile, and few enough pieces of a CTA, for which short tiles count as more blocks than they
    // have.  Shares grow by what that adds where an eighth is enough: a few CTAs more than SMs would
    // wait for one to end (120 prompts of 275 rows, up to 1792 own keys behind 355: 1913 us, not 1161).
    // Where it is not they stay as they are (210 behind 300: 1461 us, an eighth larger 1616).
    int ctas = st.own_rate > 0.f ? ctas_beside(p, (float)all, (float)own_keys) : st.sms;
    const int pieces = st.max_items - 2;
    ctas *= 1 + n_tiles / (ctas * (pieces * 3 / 4));
    int64_t per64 = (all + ctas - 1) / ctas;
    // (A share of n blocks' length, of a tile's longest kind; with st.whole a tile may have any
    // number of states, two places to a CTA.)
    const int longest = st.tile_rows == 256 ? kPairCost : kSingleCost;
    per64 = max(per64, (int64_t)kMinBlocks * longest);
    if (!st.whole) per64 = max(per64, (int64_t)((most + st.max_states - 3) / (st.max_states - 2)) * longest);
    int per = (int)per64;
    const int most_per = per + per / 8;
    auto least_blocks = [&](int rows) {  // of a unit's tiles, with a short one among them or without
        const bool pairs = st.tile_rows == 256 && (rows % 256 == 0 || rows % 256 > 128);
        const int blocks = (pairs ? kPairCost : kSingleCost) * pieces;
        return (most_per + blocks - 1) / blocks;
    };
    carry = 0;
    for (int u0 = 0; u0 < st.units; u0 += N) {
        const int u = u0 + tid;
        int64_t length = 0;
        if (u < st.units) {
            const bool some = rows_of[u] > 0 && blocks_of[u] > 0;
            const int nb = some ? max(blocks_of[u] + tile_blocks, least_blocks(rows_of[u])) : 0;
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
    if ((line + ctas - 1) / ctas <= most_per) per = max(per, (line + ctas - 1) / ctas);
    if (tid == 0) {
        first_of[st.units] = line;
        st.head[0] = per;
        st.head[1] = line;
    }
    if (flags && p.status) atomicOr(p.status, flags);
    __syncthreads();
    // What the kernels behind read, by three groups of warps side by side.
    constexpr int kSegThreads = 192, kInfoThreads = 128, kListThreads = N - kSegThreads - kInfoThreads;
    if (tid < kSegThreads) {
        // The CTAs' pieces, a CTA to a thread, and the tiles that begin in the CTA before and are cut.
        const int full = st.tile_rows == 256 ? kPairCost : kSingleCost;
        for (int64_t x = tid; x * per < line; x += kSegThreads) {
            const int begin = (int)(x * per), end = (int)min((int64_t)line, (x + 1) * per);
            SharedSeg *const segs = st.segs + x * st.max_items;
            int n = 0, s = begin, lo = 0, hi = st.units - 1;
            while (lo < hi) {  // the last unit that begins at s or before
                const int mid = (lo + hi + 1) / 2;
                if (first_of[mid] <= s) lo = mid;
                else hi = mid - 1;
            }
            SharedSeg g;
            SharedTile t;
            int tiles = 0, weight = 0;
            for (g.unit = lo - 1; s < end && n < st.max_items; s = t.end) {
                if (g.unit < lo || s >= first_of[g.unit + 1]) {  // a unit's first, or the CTA's
                    do ++g.unit;
                    while (s >= first_of[g.unit + 1]);
                    lo = g.unit;
                    weight = weight_of[g.unit];
                    g.rows = rows_of[g.unit];
                    tiles = (g.rows + st.tile_rows - 1) / st.tile_rows;
                    const int at = s - first_of[g.unit];
                    g.hkv = at / cost_of[g.unit];
                    t.tile = min((at - g.hkv * cost_of[g.unit]) / (full * weight), tiles - 1);
                    g.group = st.whole ? group_of[g.unit] : g.unit;
                    g.len = g.group >= 0 ? pre_lens[g.group] : 0;
                } else if (++t.tile == tiles) {
                    t.tile = 0;
                    ++g.hkv;
                }
                t.cost = block_cost(st, t.tile, g.rows);
                t.first = first_of[g.unit] + g.hkv * cost_of[g.unit] + t.tile * full * weight;
                t.end = t.first + t.cost * weight;
                g.row0 = t.tile * st.tile_rows;
                g.own = !st.whole ? 0
                                  : tile_own_keys(lens[g.unit], g.rows / p.G, g.row0,
                                                  min(g.row0 + st.tile_rows, g.rows));
                const int nb = (g.len + 127) / 128 + (g.own + 127) / 128;
                g.blk0 = block_from(t, s);
                g.nb = min(block_from(t, min(end, t.end)), nb) - g.blk0;
                const int home = t.first / per, last = (t.first + (nb - 1) * t.cost) / per;
                g.state = st.whole && home == last ? -1 : (int)x - home;
                if (st.whole && s == begin && x > 0) {
                    const bool cut = t.first < begin && home == x - 1 && last > home;
                    st.cuts[x - 1] = {g.unit, g.hkv, g.row0, g.rows, cut ? last - home + 1 : 0};
                }
                if (g.nb > 0) segs[n++] = g;
            }
            st.counts[x] = n;
        }
    } else if (tid < kSegThreads + kInfoThreads) {
        const int me = tid - kSegThreads;
        if (!small) {
            for (int b = me; b < p.B && !st.whole; b += kInfoThreads) st.order[b] = b;
        } else {
            // The order of the sequences' own splits: the longest first, so that the CTAs left
            // over when the others are done are short ones.
            for (int b = me; b < p.B && !st.whole; b += kInfoThreads) {
                const int mine = s_key[b];
                int rank = 0;
#pragma unroll 4
                for (int k = 0; k < p.B; k += 4) {
                    const int4 x = *reinterpret_cast<const int4 *>(s_key + k);
                    rank += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
                }
                st.order[rank] = b;
            }
            for (int b = me; b <= p.B; b += kInfoThreads) st.before[b] = before[b];
            for (int u = me; u < st.units && st.whole; u += kInfoThreads) st.blocks[u] = blocks_of[u];
        }
        for (int b = me; b < p.B && !st.whole; b += kInfoThreads) {
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
    } else if (st.list && p.q_lens) {
        // ragged groups: their rows one after the other, no padding between
        const int lane = tid % 32;
        for (int b = (tid - kSegThreads - kInfoThreads) / 32; b < p.B; b += kListThreads / 32) {
            const int at = before[b], rows = before[b + 1] - at;
            const int qn = rows / p.G;
            for (int r = lane; r < rows; r += 32) {
                const int g = r / qn;
                st.list[at + r] = (b * p.Hq + g) * p.q_len + (r - g * qn);
            }
        }
    }
}

// The tiles that are cut (st.whole): kCutRows rows a warp of the tile that the line is cut in
// before CTA blockIdx.x + 1, if that is the tile's first cut; and NaN for the sequences that are
// out of range.
constexpr int kCutWarps = 8, kCutRows = 4;

template <int D>
__global__ void __launch_bounds__(kCutWarps * 32) shared_cut_merge_kernel(const TcParams p, int ctas) {
    constexpr int E = D / 32;  // (a lane's elements: one vector load)
    using Part = std::conditional_t<E == 4, float4, float2>;
    const SharedStream &st = p.st;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_for_previous_grid();
    const float nan = __int_as_float(0x7fc00000);
    auto put = [&](int64_t row, const float *o, float lse) {
        if (p.out_bf16) {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<uint32_t *>(out + e) = pack_bf16(o[e], o[e + 1]);
        } else {
            *reinterpret_cast<Part *>(static_cast<float *>(p.out) + row * D + lane * E) =
                *reinterpret_cast<const Part *>(o);
        }
        if (lane == 0 && p.lse) p.lse[row] = lse;
    };
    if ((int)blockIdx.x >= ctas) {
        const int b = (int)blockIdx.x - ctas;
        if (st.blocks[b] >= 0) return;
        const float o[4] = {nan, nan, nan, nan};
        const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
        const int rows = qn >= 0 && qn <= p.q_len ? qn : p.q_len;
        for (int64_t r = (int64_t)blockIdx.y * kCutWarps + warp; r < (int64_t)p.Hq * p.q_len;
             r += (int64_t)gridDim.y * kCutWarps)
            if (r % p.q_len < rows) put((int64_t)b * p.Hq * p.q_len + r, o, nan);
        return;
    }
    const int x = (int)blockIdx.x;  // the CTA that the tile begins in
    const SharedCut cut = st.cuts[x];
    if (((int64_t)x + 1) * st.head[0] >= st.head[1] || cut.states < 2) return;
    const int f0 = cut.row0 + ((int)blockIdx.y * kCutWarps + warp) * kCutRows;
    if (f0 >= cut.rows) return;
    const int qn = cut.rows / p.G;
    float M[kCutRows], sum[kCutRows];
    __align__(16) float o[kCutRows][E];
    bool has_nan[kCutRows];
#pragma unroll
    for (int r = 0; r < kCutRows; ++r) {
        const int f = min(f0 + r, cut.rows - 1);  // (rows past the last are not stored)
        M[r] = p.sinks ? p.sinks[cut.hkv * p.G + f / qn] * kLog2e : -INFINITY;
        has_nan[r] = isnan(M[r]);
        sum[r] = p.sinks ? 1.f : 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    for (int k = 0; k < cut.states; ++k) {
        // the first state is that of a tile's start, the others those of their CTAs' first pieces
        const int64_t slot = ((int64_t)(x + k) * 2 + (k == 0)) * st.tile_rows + f0 - cut.row0;
        float2 ml[kCutRows];
        __align__(16) float a[kCutRows][E];
#pragma unroll
        for (int r = 0; r < kCutRows; ++r) {
            ml[r] = make_float2(0.f, 0.f);
            if (f0 + r >= cut.rows) continue;
            ml[r] = *reinterpret_cast<const float2 *>(p.ws_ml + (slot + r) * 2);
            *reinterpret_cast<Part *>(a[r]) =
                *reinterpret_cast<const Part *>(p.ws_acc + (slot + r) * D + lane * E);
        }
#pragma unroll
        for (int r = 0; r < kCutRows; ++r) {
            if (isnan(ml[r].x) || isnan(ml[r].y)) has_nan[r] = true;
            if (!(ml[r].y > 0.f)) continue;
            const float top = fmaxf(M[r], ml[r].x);
            const float old = M[r] == -INFINITY ? 0.f : ex2(M[r] - top), w = ex2(ml[r].x - top);
            sum[r] = fmaf(w, ml[r].y, sum[r] * old);
#pragma unroll
            for (int e = 0; e < E; ++e) o[r][e] = fmaf(w, a[r][e], o[r][e] * old);
            M[r] = top;
        }
    }
#pragma unroll
    for (int r = 0; r < kCutRows; ++r) {
        if (f0 + r >= cut.rows) break;
        const bool none = has_nan[r] || M[r] == -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = none ? nan : o[r][e] / sum[r];
        const int g = (f0 + r) / qn;
        put(((int64_t)cut.unit * p.Hq + cut.hkv * p.G + g) * p.q_len + (f0 + r - g * qn), o[r],
            none ? nan : kLn2 * (M[r] + log2f(sum[r])));
    }
}

// The groups' borders among sequences [b0, b0 + n): out of range wherever those of the batch are.
__global__ void __launch_bounds__(kPlanThreads) shared_starts_kernel(const int32_t *starts, int32_t *mine,
                                                                     int n_groups, int B, int b0, int n) {
    bool wrong = false;
    for (int i = (int)threadIdx.x; i < n_groups; i += kPlanThreads)
        wrong |= starts[i] < 0 || starts[i + 1] < starts[i] || starts[i + 1] > B;
    wrong = __syncthreads_or(wrong) != 0;
    for (int i = (int)threadIdx.x; i <= n_groups; i += kPlanThreads)
        mine[i] = wrong ? -1 : min(max(starts[i] - b0, 0), n);
}

}  // namespace

cudaError_t launch_shared_starts(const int32_t *starts, int32_t *mine, int n_groups, int B, int b0, int n,
                                 cudaStream_t stream) {
    shared_starts_kernel<<<1, kPlanThreads, 0, stream>>>(starts, mine, n_groups, B, b0, n);
    return cudaGetLastError();
}

cudaError_t launch_shared_plan(const TcParams &p, cudaStream_t stream) {
    shared_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_shared_cut_merge(const TcParams &p, int64_t ctas, cudaStream_t stream) {
    const dim3 grid((unsigned)(ctas + p.B), (unsigned)(p.st.tile_rows / (kCutWarps * kCutRows)));
    return p.D == 128 ? launch_dependent(shared_cut_merge_kernel<128>, grid, dim3(kCutWarps * 32), 0,
                                         stream, p, (int)ctas)
                      : launch_dependent(shared_cut_merge_kernel<64>, grid, dim3(kCutWarps * 32), 0,
                                         stream, p, (int)ctas);
}

}  // namespace atlas
