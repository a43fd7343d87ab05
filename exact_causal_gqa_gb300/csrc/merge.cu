// merge.cu -- structured log-sum-exp merge of split-KV partial states
// (CPUAttn README, "Operator model": split-K is offered only with a structured
// merge).  For one output row with splits s = 0..S-1 holding (m_s, l_s, acc_s),
// m in log2 units:
//   M = max_s m_s,  w_s = 2^(m_s - M),  o = sum_s w_s acc_s / sum_s w_s l_s,
//   lse = ln 2 * (M + log2 sum_s w_s l_s).
// W warps per row (W = 1, 2 or 4, chosen from the row count so that the grid
// holds enough warps): warp k of a row takes splits k, k + W, ...; its lanes split
// the head dimension.  Each warp keeps a running maximum (its sums are rescaled
// when a group of splits raises it), so a warp's share of up to kGroup splits
// costs one round trip to memory; with W > 1 the warps' states are combined the
// same way through shared memory.  S is derived on the device from seq_lens, so
// no host sync is needed.
// Launched as a programmatic dependent of the split kernel before it: its CTAs
// may start while that kernel's last CTAs still run, read their sequence's
// length, and wait (griddepcontrol.wait) before the first partial is read.
#include "internal.h"
#include "ptx.cuh"
#include "shared_prefix.cuh"

#include <math.h>
#include <type_traits>

namespace atlas {
namespace {

constexpr int kWarps = 4;  // warps per CTA: 4 / W rows
constexpr int kGroup = 8;  // splits of one warp whose loads are in flight together

// Splits of the prefix that sequence b's group shares (0 outside all groups), -1 if there is
// no telling: the prefix's length is out of range, or any group's borders are or descend.  All
// lanes of a warp call this with the same b; lane k looks at groups k, k + 32, ...
__device__ int prefix_splits(const SharedMergeParams &p, int b) {
    int splits = 0;
    for (int n0 = 0; n0 < p.n_groups; n0 += 32) {
        const int n = n0 + (int)(threadIdx.x % 32);
        bool mine = false, wrong = false;
        int s = 0;
        if (n < p.n_groups) {
            const int a = p.group_starts[n], z = p.group_starts[n + 1];
            wrong = a < 0 || z < a || z > p.B;
            mine = a <= b && b < z;
            if (mine) {
                const int len = p.prefix_lens[n];
                s = len < 0 || len > p.max_prefix ? -1 : (len + p.pre_chunk - 1) / p.pre_chunk;
            }
        }
        if (__any_sync(0xffffffffu, wrong)) return -1;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who != 0) splits = __shfl_sync(0xffffffffu, s, __ffs(who) - 1);
    }
    return splits;
}

// The same where the prefixes are tiles of the line that p.st says (shared_prefix.cuh): the
// states of the tile that row i of head h of sequence b is in.
__device__ int tile_states(const SharedMergeParams &p, int b, int h, int i, int qn) {
    // (read before the wait: the plan's grid is done, but not one that this grid waits for, so
    // past the L1)
    const int4 *const at = reinterpret_cast<const int4 *>(p.st.info) + 2 * b;
    int4 raw[2] = {__ldcg(at), __ldcg(at + 1)};
    SeqInfo s;
    static_assert(sizeof(s) == sizeof(raw), "");
    memcpy(&s, raw, sizeof(s));
    if (s.blocks <= 0 || i >= qn) return s.blocks < 0 ? -1 : 0;
    const int f = s.row0 + h % p.G * qn + i;
    const int tile = f / p.st.tile_rows, full = p.st.tile_rows == 256 ? kPairCost : kSingleCost;
    const int first = s.first + h / p.G * s.head_cost + tile * full * s.weight;
    const int last = first + (s.blocks - 1) * block_cost(p.st, tile, s.rows);
    return last / s.per - first / s.per + 1;
}

template <int D, typename Params>
__global__ void __launch_bounds__(kWarps * 32) merge_kernel(const Params p) {
    // a call with shared prefixes: their splits follow the sequence's own
    constexpr bool kShared = std::is_same<Params, SharedMergeParams>::value;
    constexpr int DPL = D / 32;
    const int warp = (int)(threadIdx.x / 32), lane = (int)(threadIdx.x % 32);
    const int W = p.warps_per_row;
    const int sub = warp % W;  // this warp's share of its row's splits
    // rows = B * Hq * q_len < 2^31 (the plan refuses larger calls): 32-bit index math
    const int row = (int)blockIdx.x * (kWarps / W) + warp / W;
    bool active = row < p.B * p.Hq * p.q_len;
    const int bh = active ? row / p.q_len : 0;  // b * Hq + h
    const int i = active ? row - bh * p.q_len : 0;
    const int b = bh / p.Hq;
    const int L = active ? p.seq_lens[b] : 0;
    const int qn = !active ? 0 : p.q_lens ? p.q_lens[b] : p.q_len;  // ragged: rows of b
    int n_pre = 0;
    if constexpr (kShared)
        n_pre = !active ? 0 : p.pre_chunk ? prefix_splits(p, b) : tile_states(p, b, bh - b * p.Hq, i, qn);
    const bool bad_len = qn < 0 || qn > p.q_len || L < p.row_step * qn || L > p.max_pages * p.P ||
                         (p.require_full && L != qn) || n_pre < 0;
    if (!bad_len && i >= qn) active = false;  // padding row: not a query, not written
    if (W == 1 && !active) {                  // (W > 1: every warp reaches the exchange)
        // (a grid of padding rows alone must not end before the splits: another part may follow)
        if (kShared) wait_for_previous_grid();
        return;
    }
    // the split kernel that wrote the partials has completed, its writes visible
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // This warp's state: running max M (log2 units), sum, acc slice, NaN seen.  A
    // sink is one more state (m = sink * log2 e, l = 1, acc = 0), held by warp 0.
    float M = -INFINITY, lsum = 0.f, acc[DPL];
#pragma unroll
    for (int j = 0; j < DPL; ++j) acc[j] = 0.f;
    bool has_nan = false;
    if (active && !bad_len) {
        const int visible = p.row_step ? L - qn + i + 1 : L;
        // splits holding this row's keys: [first, nsplit)
        const int chunk =
            p.balanced ? balanced_split(min(L, p.max_pages * p.P), p.chunk) : p.chunk;
        const int first = p.window > 0 ? max(0, visible - p.window) / chunk : 0;
        const int n_own = (visible + chunk - 1) / chunk;
        const int nsplit = n_own + n_pre;
        const float *ml = p.ws_ml + (int64_t)row * p.n_chunks * 2;
        if (p.sinks && sub == 0) {
            M = p.sinks[bh - b * p.Hq] * kLog2e;
            lsum = 1.f;
            has_nan = isnan(M);
        }
        const float *wa = p.ws_acc + (int64_t)row * p.n_chunks * D + lane * DPL;
        // state s of the row: its own splits, then the prefix's
        auto ml_of = [&](int s) -> const float * {
            if constexpr (kShared)
                if (s >= n_own) return p.pre_ml + ((int64_t)row * p.n_pre + s - n_own) * 2;
            return ml + 2 * s;
        };
        auto acc_of = [&](int s) -> const float * {
            if constexpr (kShared)
                if (s >= n_own)
                    return p.pre_acc + ((int64_t)row * p.n_pre + s - n_own) * D + lane * DPL;
            return wa + (int64_t)s * D;
        };
        // [kWarps][kGroup][32 lanes] x 16 bytes (D = 128): each lane's slice of a
        // split lands here, so no registers are held while the loads are in flight
        __shared__ __align__(16) uint8_t stage[D == 128 ? kWarps * kGroup * 512 : 16];
        const uint32_t my_stage = smem_u32(stage) + (uint32_t)(warp * kGroup * 512 + lane * 16);
        for (int s0 = first + sub; s0 < nsplit; s0 += kGroup * W) {
            float m[kGroup], l[kGroup], a[kGroup][DPL];
            if (DPL == 4) {
#pragma unroll
                for (int u = 0; u < kGroup; ++u)
                    if (s0 + u * W < nsplit)
                        cp_async16(my_stage + u * 512, acc_of(s0 + u * W), 16);
                cp_async_commit();
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                const int s = s0 + u * W;
                m[u] = -INFINITY;
                l[u] = 0.f;
#pragma unroll
                for (int j = 0; j < DPL; ++j) a[u][j] = 0.f;
                if (s < nsplit) {
                    m[u] = ml_of(s)[0];
                    l[u] = ml_of(s)[1];
                    if (DPL != 4) {
                        const float2 v = *reinterpret_cast<const float2 *>(acc_of(s));
                        a[u][0] = v.x;
                        a[u][1 % DPL] = v.y;
                    }
                }
            }
            if (DPL == 4) cp_async_wait<0>();
            float Mg = M;
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                if (isnan(m[u]) || isnan(l[u])) has_nan = true;
                else if (l[u] > 0.f) Mg = fmaxf(Mg, m[u]);
            }
            if (Mg > M) {  // M = -inf only while the sums are still zero
                const float r = ex2(M - Mg);
                lsum *= r;
#pragma unroll
                for (int j = 0; j < DPL; ++j) acc[j] *= r;
                M = Mg;
            }
#pragma unroll
            for (int u = 0; u < kGroup; ++u) {
                if (DPL == 4 && s0 + u * W < nsplit) {
                    const uint4 v = ld_shared_v4(my_stage + u * 512);
                    a[u][0] = __uint_as_float(v.x);
                    a[u][1 % DPL] = __uint_as_float(v.y);
                    a[u][2 % DPL] = __uint_as_float(v.z);
                    a[u][3 % DPL] = __uint_as_float(v.w);
                }
                const float w = l[u] > 0.f ? ex2(m[u] - M) : 0.f;
                lsum = fmaf(w, l[u], lsum);
#pragma unroll
                for (int j = 0; j < DPL; ++j) acc[j] = fmaf(w, a[u][j], acc[j]);
            }
        }
    }
    if (W > 1) {
        // The row's warps combine their states in warp order (sub 0 first).
        __shared__ float x_acc[kWarps][DPL][32];
        __shared__ float x_m[kWarps], x_l[kWarps];
        __shared__ int x_nan[kWarps];
#pragma unroll
        for (int j = 0; j < DPL; ++j) x_acc[warp][j][lane] = acc[j];
        if (lane == 0) {
            x_m[warp] = M;
            x_l[warp] = lsum;
            x_nan[warp] = has_nan;
        }
        __syncthreads();
        if (sub != 0 || !active) return;
        for (int k = 1; k < W; ++k) M = fmaxf(M, x_m[warp + k]);
        if (M > -INFINITY) {
            const float r0 = ex2(x_m[warp] - M);
            lsum *= r0;
#pragma unroll
            for (int j = 0; j < DPL; ++j) acc[j] *= r0;
            for (int k = 1; k < W; ++k) {
                const float r = ex2(x_m[warp + k] - M);  // 0 for a warp with no state
                lsum = fmaf(r, x_l[warp + k], lsum);
#pragma unroll
                for (int j = 0; j < DPL; ++j) acc[j] = fmaf(r, x_acc[warp + k][j][lane], acc[j]);
            }
        }
        for (int k = 1; k < W; ++k) has_nan |= x_nan[warp + k] != 0;
    }

    float o[DPL];
    float lse = __int_as_float(0x7fc00000);
    if (!bad_len && !has_nan && M == -INFINITY && p.row_step == 0 && L == 0) {
        // cross attention over no encoder states: nothing to weigh
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[j] = 0.f;
        lse = -INFINITY;
    } else if (bad_len || has_nan || M == -INFINITY) {
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[j] = __int_as_float(0x7fc00000);
    } else {
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[j] = acc[j] / lsum;
        lse = kLn2 * (M + log2f(lsum));
    }
    const int64_t off = (int64_t)row * D + lane * DPL;
    if (p.out_bf16) {
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + off;
        if (DPL == 4) {
            uint2 v;
            v.x = pack_bf16(o[0], o[1 % DPL]);
            v.y = pack_bf16(o[2 % DPL], o[3 % DPL]);
            *reinterpret_cast<uint2 *>(out) = v;
        } else {
            *reinterpret_cast<uint32_t *>(out) = pack_bf16(o[0], o[1 % DPL]);
        }
    } else {
        float *out = static_cast<float *>(p.out) + off;
        if (DPL == 4)
            *reinterpret_cast<float4 *>(out) =
                make_float4(o[0], o[1 % DPL], o[2 % DPL], o[3 % DPL]);
        else
            *reinterpret_cast<float2 *>(out) = make_float2(o[0], o[1 % DPL]);
    }
    if (p.lse && lane == 0) p.lse[row] = lse;
}

// The same for many rows, kRows neighbouring ones a warp and kAhead states of each in flight; a
// lane works out one row's places, whose divisions are most of what merge_kernel does for it.  A
// row's states are joined one after the other.  256 sequences of 32 rows in 8 groups: 85 us for the
// call, 88 with merge_kernel; 192 sequences of 1 to 4 x 32 rows 221 and 227 (four rows a warp 222;
// four for all the lanes' work done by each 229); 2048 rows of up to 20 states 108 and 103.
constexpr int kRowWarps = 4, kRows = 2, kAhead = 2;

template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) shared_rows_kernel(const SharedMergeParams p) {
    constexpr int E = D / 32;
    using Part = std::conditional_t<E == 4, float4, float2>;
    const int lane = (int)(threadIdx.x % 32);
    const int row0 = ((int)blockIdx.x * kRowWarps + (int)(threadIdx.x / 32)) * kRows;
    const int rows = p.B * p.Hq * p.q_len;
    // A lane works out one row's states (its divisions are most of the instructions): its own, and
    // all; -1: the row is NaN, -2: it is not written.
    int my_own, my_all, my_h;
    {
        const int row = min(row0 + lane % kRows, rows - 1), bh = row / p.q_len, i = row - bh * p.q_len;
        const int b = bh / p.Hq;
        my_h = bh - b * p.Hq;
        const int L = p.seq_lens[b], qn = p.q_lens ? p.q_lens[b] : p.q_len;
        int pre = 0;
        if (p.pre_chunk) {
            int last = -1, splits = 0;
            for (int r = 0; r < kRows; ++r) {
                const int of = __shfl_sync(0xffffffffu, b, r);
                if (of != last) splits = prefix_splits(p, of);
                last = of;
                if (lane % kRows == r) pre = splits;
            }
        } else {
            pre = tile_states(p, b, my_h, i, qn);
        }
        const bool bad = qn < 0 || qn > p.q_len || L < qn || L > p.max_pages * p.P || pre < 0;
        my_own = (L - qn + i + p.chunk) / p.chunk;
        my_all = row0 + lane % kRows >= rows ? -2 : bad ? -1 : i >= qn ? -2 : my_own + pre;
    }
    const int most = __reduce_max_sync(0xffffffffu, my_all);
    int own[kRows], all[kRows];
    float M[kRows], sum[kRows];
    __align__(16) float o[kRows][E];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        own[r] = __shfl_sync(0xffffffffu, my_own, r);
        all[r] = __shfl_sync(0xffffffffu, my_all, r);
        const int h = __shfl_sync(0xffffffffu, my_h, r);
        M[r] = -INFINITY;
        sum[r] = 0.f;
        if (p.sinks && all[r] >= 0) {
            M[r] = p.sinks[h] * kLog2e;
            sum[r] = 1.f;
            if (isnan(M[r])) all[r] = -1;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = 0.f;
    }
    wait_for_previous_grid();
    for (int s0 = 0; s0 < most; s0 += kAhead) {
        float2 ml[kAhead][kRows];
        __align__(16) float a[kAhead][kRows][E];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int s = s0 + u;
                ml[u][r] = make_float2(0.f, 0.f);
                if (s >= all[r]) continue;
                const int64_t row = row0 + r;
                const bool mine = s < own[r];
                const int64_t at = mine ? row * p.n_chunks + s : row * p.n_pre + s - own[r];
                ml[u][r] = *reinterpret_cast<const float2 *>((mine ? p.ws_ml : p.pre_ml) + at * 2);
                *reinterpret_cast<Part *>(a[u][r]) =
                    *reinterpret_cast<const Part *>((mine ? p.ws_acc : p.pre_acc) + at * D + lane * E);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (isnan(ml[u][r].x) || isnan(ml[u][r].y)) all[r] = -1;
                if (!(ml[u][r].y > 0.f)) continue;
                const float top = fmaxf(M[r], ml[u][r].x);
                const float old = M[r] == -INFINITY ? 0.f : ex2(M[r] - top), w = ex2(ml[u][r].x - top);
                sum[r] = fmaf(w, ml[u][r].y, sum[r] * old);
#pragma unroll
                for (int e = 0; e < E; ++e) o[r][e] = fmaf(w, a[u][r][e], o[r][e] * old);
                M[r] = top;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (all[r] == -2) continue;
        const bool none = all[r] < 0 || M[r] == -INFINITY;
        const int64_t row = row0 + r;
#pragma unroll
        for (int e = 0; e < E; ++e) o[r][e] = none ? __int_as_float(0x7fc00000) : o[r][e] / sum[r];
        if (p.out_bf16) {
            uint32_t two[E / 2];
#pragma unroll
            for (int e = 0; e < E; e += 2) two[e / 2] = pack_bf16(o[r][e], o[r][e + 1]);
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + row * D + lane * E;
            if constexpr (E == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(two[0], two[1]);
            else *reinterpret_cast<uint32_t *>(out) = two[0];
        } else {
            *reinterpret_cast<Part *>(static_cast<float *>(p.out) + row * D + lane * E) =
                *reinterpret_cast<const Part *>(o[r]);
        }
        if (p.lse && lane == 0)
            p.lse[row] = none ? __int_as_float(0x7fc00000) : kLn2 * (M[r] + log2f(sum[r]));
    }
}

}  // namespace

template <typename Params>
static cudaError_t launch(const Params &p, int states, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.B * p.Hq * p.q_len;
    if (rows >= INT32_MAX) return cudaErrorInvalidValue;  // make_plan refuses these
    // Several warps per row when the rows alone would leave most warp slots empty
    // and there are splits to share.
    Params q = p;
    const int64_t target = (int64_t)(p.sms > 0 ? p.sms : 1) * 16;
    q.warps_per_row = 1;
    while (q.warps_per_row < kWarps && rows * q.warps_per_row < target &&
           states >= 2 * q.warps_per_row)
        q.warps_per_row *= 2;
    const int64_t rows_per_cta = kWarps / q.warps_per_row;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + rows_per_cta - 1) / rows_per_cta), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.D == 128 ? cudaLaunchKernelEx(&cfg, merge_kernel<128, Params>, q)
                      : cudaLaunchKernelEx(&cfg, merge_kernel<64, Params>, q);
}

cudaError_t launch_merge(const MergeParams &p, cudaStream_t stream) {
    return launch(p, p.n_chunks, stream);
}

cudaError_t launch_shared_merge(const SharedMergeParams &p, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.B * p.Hq * p.q_len;
    if (rows >= (int64_t)(p.sms > 0 ? p.sms : 1) * 16) {  // (else several warps a row)
        const dim3 grid((unsigned)((rows + kRowWarps * kRows - 1) / (kRowWarps * kRows)));
        return p.D == 128 ? launch_dependent(shared_rows_kernel<128>, grid, dim3(kRowWarps * 32), 0, stream, p)
                          : launch_dependent(shared_rows_kernel<64>, grid, dim3(kRowWarps * 32), 0, stream, p);
    }
    return launch(p, p.n_chunks + p.n_pre, stream);
}

}  // namespace atlas
