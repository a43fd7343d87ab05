// kv_weights_tc.cuh -- what the tensor-core kernels of the attention weights (bf16, and
// fp32 as tf32 parts) share: the walk over query tiles, the columns' facts, and the sum of
// exponentials along a lane's TMEM columns.
#pragma once

#include "kv_weights.cuh"

namespace atlas {

constexpr int BT = 128;           // keys per tile
constexpr int kSlab = 128 * 128;  // one 64-element slab of a 128-row bf16 tile

__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort, kWaitLimitNs));
}

// Barrier `id` of `threads` threads (whole warps) of the CTA.
__device__ __forceinline__ void group_barrier(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Adds 2^(s2 + neg_lse2[c]) of NC columns of scores; with kMasked, of those columns c that
// key t is visible to (t < lim[c], and t >= lim[c] - window with a window).
template <int NC, bool kMasked, bool kCapped>
__device__ __forceinline__ void add_columns(const WeightsParams &p, const uint32_t (&s)[NC],
                                            const float *neg_lse2, const int *lim, int t,
                                            float2 (&sum)[2]) {
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    const int far = p.window > 0 ? t + p.window : INT32_MAX;
#pragma unroll
    for (int c = 0; c < NC; c += 4) {
        const float4 l4 = *reinterpret_cast<const float4 *>(neg_lse2 + c);
        float2 a = make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
        float2 b = make_float2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]));
        if (kCapped) {
            a = make_float2(score_log2(p, a.x) + l4.x, score_log2(p, a.y) + l4.y);
            b = make_float2(score_log2(p, b.x) + l4.z, score_log2(p, b.y) + l4.w);
        } else {
            a = ffma2(a, sc, make_float2(l4.x, l4.y));
            b = ffma2(b, sc, make_float2(l4.z, l4.w));
        }
        if (kMasked) {
            const int4 m = *reinterpret_cast<const int4 *>(lim + c);
            a.x = t < m.x && m.x <= far ? a.x : -INFINITY;
            a.y = t < m.y && m.y <= far ? a.y : -INFINITY;
            b.x = t < m.z && m.z <= far ? b.x : -INFINITY;
            b.y = t < m.w && m.w <= far ? b.y : -INFINITY;
        }
        sum[0] = fadd2(sum[0], make_float2(ex2(a.x), ex2(a.y)));
        sum[1] = fadd2(sum[1], make_float2(ex2(b.x), ex2(b.y)));
    }
}

// The common case (no cap, every column visible) on a path of its own: compares and
// selects computed and not used doubled the time of the prompt's kernel.
template <int NC>
__device__ __forceinline__ void add_weights(const WeightsParams &p, const uint32_t (&s)[NC],
                                            const float *neg_lse2, const int *lim, int t, bool masked,
                                            float2 (&sum)[2]) {
    const bool capped = p.softcap_log2 > 0.f;
    if (!masked && !capped) add_columns<NC, false, false>(p, s, neg_lse2, lim, t, sum);
    else if (!capped) add_columns<NC, true, false>(p, s, neg_lse2, lim, t, sum);
    else add_columns<NC, true, true>(p, s, neg_lse2, lim, t, sum);
}

// The query tiles first .. end - 1 of a (sequence, kv head) that have a row which sees a
// key of [kb, kb + keys), in order: rows 128 j .. 128 j + 127 of its G * q_len
// (q head, row) pairs, and the keys their real rows see.  The producer, the MMA warp and
// the warp that brings the columns each walk this list.
struct QueryTiles {
    const WeightsParams &p;
    const int L, qn, kb, keys, end;
    int j, i;              // tile, and its first row's place in its head
    int n = -1;            // tiles taken before this one: ring position and phase
    bool started = false;
    bool whole = false;    // every row is real
    int lim_min = 0, lim_max = 0;  // keys below: seen by the earliest / latest row

    __device__ __forceinline__ QueryTiles(const WeightsParams &p_, int L_, int qn_, int kb_,
                                          int keys_, int first, int end_)
        : p(p_), L(L_), qn(qn_), kb(kb_), keys(keys_), end(end_), j(first - 1),
          i((int)((int64_t)first * BT % p_.q_len)) {}

    // Moves on to the next tile of the list; false at its end.
    __device__ __forceinline__ bool next() {
        for (;;) {
            if (++j >= end) return false;
            if (started) {
                i += BT;
                if (i >= p.q_len) i = p.q_len >= BT ? i - p.q_len : i % p.q_len;
            }
            started = true;
            const int count = min(BT, p.G * p.q_len - j * BT);
            const bool spans = i + count > p.q_len;
            const int i0 = spans ? 0 : i;
            const int i1 = min(spans ? p.q_len : i + count, qn) - 1;
            if (i0 >= qn) continue;  // padding rows only
            whole = count == BT && (qn == p.q_len || (!spans && i + count <= qn));
            lim_min = L - qn + i0 + 1;
            lim_max = L - qn + i1 + 1;
            if (!seen(kb, keys)) continue;
            ++n;
            return true;
        }
    }
    __device__ __forceinline__ bool seen(int k0, int keys) const {
        return sees(p, lim_min, lim_max, k0, keys);
    }
};

// What the epilogue needs to know of a query tile, worked out once by the warp that
// brings its columns.
struct __align__(16) TileInfo {
    int lim_min, lim_max;  // as in QueryTiles
    int whole, stop;       // stop: no tile, the list has ended
};

// The warp that brings a query tile's columns: the negated lse in log2 units and the limits
// of its 128 rows, and the tile's facts, into slot n % S of a ring (full[s] is arrived at
// once, empty[s] waited on), then `stops` slots that say the list has ended.  Returns
// whether it got through.
template <int S>
__device__ __forceinline__ bool bring_columns(const WeightsParams &p, QueryTiles &q, int64_t row0,
                                              uint8_t *smem, int off_lse, int off_lim, int off_info,
                                              uint32_t full0, uint32_t empty0, int stops,
                                              volatile int *abort_flag) {
    const int lane = threadIdx.x & 31;
    int left = stops;
    for (int n = 0; left > 0; ++n) {
        const bool more = left == stops && q.next();
        const int s = n % S;
        float v[4];
        int m[4];
        if (more) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int f = q.j * BT + e * 32 + lane;
                const int i = f % p.q_len;
                const bool real = f < p.G * p.q_len && i < q.qn;
                v[e] = real ? -lse_log2(p.lse[row0 + f]) : -INFINITY;
                m[e] = real ? q.L - q.qn + i + 1 : 0;
            }
        } else {
            --left;
        }
        if (n >= S && !wait_warp(empty0 + 8u * s, ((n / S) - 1) & 1, abort_flag)) {
            if (lane == 0) *abort_flag = 1;
            return false;
        }
        if (more) {
            float *nlse = reinterpret_cast<float *>(smem + off_lse) + s * BT;
            int *lim = reinterpret_cast<int *>(smem + off_lim) + s * BT;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                nlse[e * 32 + lane] = v[e];
                lim[e * 32 + lane] = m[e];
            }
        }
        if (lane == 0)
            reinterpret_cast<TileInfo *>(smem + off_info)[s] =
                TileInfo{q.lim_min, q.lim_max, q.whole, !more};
        __syncwarp();
        if (lane == 0) mbar_arrive(full0 + 8u * s);
    }
    return true;
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device, once per device.
inline cudaError_t configure_smem(const void *kern, int bytes, int (&done)[64]) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev < 64 && done[dev]) return cudaSuccess;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && dev < 64) done[dev] = 1;
    return err;
}

// The parts' sums of each key, in order (p.n_parts > 1).
cudaError_t launch_weights_join(const WeightsParams &p, cudaStream_t stream);

}  // namespace atlas
