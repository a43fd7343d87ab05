// kv_weights.cu -- the attention weight each cached key received: for key t of
// (sequence, kv head),
//   w[t] (+)= sum over columns c that see t of 2^(s2(t, c) - lse2(c)),
// a column being one (q head of the group, query row) pair, s2 its score with key t and
// lse2 the row's log-sum-exp that the attention call returned, both in log2 units.  No
// softmax state is needed -- lse normalises every row -- and K is read once.
//
// bf16 runs on the tensor cores (kv_weights_tc.cu); this file has the entry point and
// fp32.
//
// weights_warp_kernel, at most 8 columns (decode): K is read once, straight into registers,
//   and its bytes are the bound.  A warp takes 8 keys at a time, a lane D / 32 elements of
//   each; the 8 x NC partial dot products are added across the lanes by halving -- each
//   step sends half of a lane's values to the lane that keeps them, one shuffle per score
//   in all -- which leaves every score in one lane, and the columns' weights are added over
//   neighbouring lanes.  8 sequences of 16384 keys, 8 kv heads of 128: 106 us, 5.1 TB/s
//   with 4 columns, 90 us for half the bytes with 8 (3.0 TB/s, bound by latency at two
//   CTAs an SM; 4 keys a warp are slower: 120 and 117 us).
// weights_ffma_kernel, more columns: a CTA owns 128 keys of one (sequence, kv head), held in
//   shared memory, and walks the columns in tiles of NC that one of its keys is visible to.
//   A thread forms 4 keys x NC / 8 columns of scores as whole dot products (packed fp32
//   pairs), exponentiates them and keeps one sum per key; the 8 lanes that share a key add
//   up at the end.  Bound by shared-memory reads (12 of 16 bytes per 128 products):
//   28-33 TFLOP/s.
#include "kv_weights.cuh"

namespace atlas {
namespace {

constexpr int kKeys = 128;  // keys of a CTA

template <int D, int NC>
struct FfmaLayout {
    static constexpr int KS = D + 4;  // padded row stride (floats): conflict-free 16-byte reads
    static constexpr int kBytes = (kKeys + NC) * KS * 4;
};

template <int D, int NC>
__global__ void __launch_bounds__(256, 2) weights_ffma_kernel(const WeightsParams p) {
    using Lay = FfmaLayout<D, NC>;
    constexpr int KS = Lay::KS, CPT = NC / 8;  // columns per thread
    extern __shared__ __align__(16) float smem_f[];
    __shared__ float col_lse[NC];
    __shared__ int col_lim[NC], col_lo[NC];
    float *sK = smem_f, *sQ = smem_f + kKeys * KS;
    const int b = blockIdx.z, hkv = blockIdx.y, kb = (int)blockIdx.x * kKeys;
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    if (kb >= L) return;
    const int lp = 31 - __clz(p.P);
    const int nkeys = min(kKeys, L - kb);
    // the K block; keys past the end or on a bad page stay zero
    for (int i = threadIdx.x; i < kKeys * (D / 4); i += 256) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nkeys) {
            const int t = kb + r;
            const int page = p.page_table[(int64_t)b * p.max_pages + (t >> lp)];
            if (page >= 0 && page < p.num_pages) {
                const int64_t row = ((int64_t)page * p.Hkv + hkv) * p.P + (t & (p.P - 1));
                x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.k_pages) + row * D + d);
            } else if (d == 0) {
                record(p.status, ATLAS_DEV_BAD_PAGE);
            }
        }
        *reinterpret_cast<float4 *>(sK + r * KS + d) = x;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cg = lane & 7, kg = warp * 4 + (lane >> 3);  // keys kg + 32 r, columns cg + 8 c
    const int ncols = p.G * p.q_len;
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < ncols; c0 += NC) {
        // A tile none of whose rows is real or sees a key of this CTA is passed over.
        const int i0 = c0 % p.q_len, count = min(NC, ncols - c0);
        const bool spans = i0 + count > p.q_len;
        const int lim_min = L - qn + (spans ? 0 : i0) + 1;
        const int lim_max = L - qn + min(spans ? p.q_len : i0 + count, qn);
        if ((spans ? 0 : i0) >= qn || !sees(p, lim_min, lim_max, kb, nkeys)) continue;
        __syncthreads();
        if (threadIdx.x < NC) {
            const int f = c0 + (int)threadIdx.x;
            const int i = f % p.q_len;
            const bool real = f < ncols && i < qn;
            const int visible = L - qn + i + 1;
            col_lse[threadIdx.x] = real ? lse_log2(p.lse[row0 + f]) : INFINITY;
            col_lim[threadIdx.x] = real ? visible : 0;
            col_lo[threadIdx.x] = p.window > 0 ? max(0, visible - p.window) : 0;
        }
        for (int i = threadIdx.x; i < NC * (D / 4); i += 256) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            const int f = c0 + r;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (f < ncols && f % p.q_len < qn)
                x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + (row0 + f) * D + d);
            *reinterpret_cast<float4 *>(sQ + r * KS + d) = x;
        }
        __syncthreads();
        float2 s[4][CPT];  // even and odd elements' sums
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < CPT; ++c) s[r][c] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int d = 0; d < D; d += 4) {
            float4 k4[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                k4[r] = *reinterpret_cast<const float4 *>(sK + (kg + 32 * r) * KS + d);
#pragma unroll
            for (int c = 0; c < CPT; ++c) {
                const float4 q4 = *reinterpret_cast<const float4 *>(sQ + (cg + 8 * c) * KS + d);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[r][c] = ffma2(make_float2(q4.x, q4.y), make_float2(k4[r].x, k4[r].y), s[r][c]);
                    s[r][c] = ffma2(make_float2(q4.z, q4.w), make_float2(k4[r].z, k4[r].w), s[r][c]);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
            const float lse2 = col_lse[cg + 8 * c];
            const int lim = col_lim[cg + 8 * c], lo = col_lo[cg + 8 * c];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = kb + kg + 32 * r;
                sum[r] += t < lim && t >= lo ? ex2(score_log2(p, s[r][c].x + s[r][c].y) - lse2) : 0.f;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 4);
        const int t = kb + kg + 32 * r;
        if (cg == 0 && t < L && page_ok(p, b, t, lp)) {
            float *w = p.weights + ((int64_t)b * p.Hkv + hkv) * p.row_tokens + t;
            *w = (p.accumulate ? *w : 0.f) + sum[r];
        }
    }
}

// One warp per 8 keys and step; grid (key ranges, Hkv, B).
constexpr int kWarpKeys = 8, kWarpThreads = 256;

template <int D, int NC>
__global__ void __launch_bounds__(kWarpThreads, NC == 8 ? 2 : 3) weights_warp_kernel(const WeightsParams p, const int chunk) {
    constexpr int DPL = D / 32;  // elements of a row per lane: 2 or 4
    const int b = blockIdx.z, hkv = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    const int first = (int)blockIdx.x * chunk, end = min(L, first + chunk);
    if (first >= end) return;
    const int lp = 31 - __clz(p.P);
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    // The columns, packed: column c is row c % qn of head c / qn of the group.
    const int ncols = p.G * qn;
    float q[NC][DPL];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const float *src = static_cast<const float *>(p.q) +
                           (row0 + (c < ncols ? (int64_t)(c / qn) * p.q_len + c % qn : 0)) * D + lane * DPL;
#pragma unroll
        for (int e = 0; e < DPL; ++e) q[c][e] = c < ncols ? src[e] : 0.f;
    }
    // The columns go through the halving kShare at a time (8 at once held too many
    // registers); after it a lane holds column i * kShare + share of one key.
    constexpr int kShare = NC < 4 ? NC : 4, kMine = NC / kShare;
    constexpr int kSpread = 32 / (kWarpKeys * kShare);  // lanes left over: they hold copies
    const int key = lane / kSpread / kShare, share = lane / kSpread % kShare;
    float lse2[kMine];
    int lim[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int c = i * kShare + share;
        const bool real = c < ncols;
        lse2[i] = real ? lse_log2(p.lse[row0 + (int64_t)(c / qn) * p.q_len + c % qn]) : INFINITY;
        lim[i] = real ? L - qn + c % qn + 1 : 0;
    }
    float *w = p.weights + ((int64_t)b * p.Hkv + hkv) * p.row_tokens;
    const int32_t *table = p.page_table + (int64_t)b * p.max_pages;
    // Page ids are read by the lanes that own a key, a step ahead, and handed round.
    auto page_of = [&](int kb) {
        const int t = kb + key;
        const int id = t < end ? table[t >> lp] : -1;
        if (t < end && (id < 0 || id >= p.num_pages) && lane % (kSpread * kShare) == 0)
            record(p.status, ATLAS_DEV_BAD_PAGE);
        return id < p.num_pages ? id : -1;
    };
    const int step = kWarpThreads / 32 * kWarpKeys;
    int kb = first + warp * kWarpKeys;
    int id_next = page_of(kb);
    for (; kb < end; kb += step) {
        const int id = id_next, t = kb + key;
        float x[kWarpKeys][DPL];
#pragma unroll
        for (int k = 0; k < kWarpKeys; ++k) {
            const int page = __shfl_sync(0xffffffffu, id, k * kSpread * kShare);
            const float *src = static_cast<const float *>(p.k_pages) +
                               (((int64_t)max(page, 0) * p.Hkv + hkv) * p.P + ((kb + k) & (p.P - 1))) * D +
                               lane * DPL;
            if (DPL == 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (page >= 0) v = __ldcs(reinterpret_cast<const float4 *>(src));
                x[k][0] = v.x;
                x[k][1] = v.y;
                x[k][2 % DPL] = v.z;
                x[k][3 % DPL] = v.w;
            } else {
                float2 v = make_float2(0.f, 0.f);
                if (page >= 0) v = __ldcs(reinterpret_cast<const float2 *>(src));
                x[k][0] = v.x;
                x[k][1] = v.y;
            }
        }
        const float old = t < end && p.accumulate ? w[t] : 0.f;
        id_next = page_of(kb + step);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            // Partial dot products, value (key, column) at key * kShare + column.
            float s[kWarpKeys * kShare];
#pragma unroll
            for (int k = 0; k < kWarpKeys; ++k)
#pragma unroll
                for (int c = 0; c < kShare; ++c) {
                    const float *qc = q[i * kShare + c];
                    float a = qc[0] * x[k][0];
#pragma unroll
                    for (int e = 1; e < DPL; ++e) a = fmaf(qc[e], x[k][e], a);
                    s[k * kShare + c] = a;
                }
            // Halving: lane bit `o` keeps the upper or the lower half of the values; once
            // one is left, the lanes that hold the same one add theirs up.
            int n = kWarpKeys * kShare;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                if (n > 1) {
                    n /= 2;
                    const bool upper = lane & o;
#pragma unroll
                    for (int v = 0; v < kWarpKeys * kShare / 2; ++v) {
                        if (v >= n) break;
                        const float send = upper ? s[v] : s[v + n];
                        s[v] = (upper ? s[v + n] : s[v]) + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                } else {
                    s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
                }
            }
            const bool sees = t < lim[i] && (p.window == 0 || t >= lim[i] - p.window);
            sum += sees ? ex2(score_log2(p, s[0]) - lse2[i]) : 0.f;
        }
#pragma unroll
        for (int o = kSpread; o < kSpread * kShare; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (t < end && id >= 0 && lane % (kSpread * kShare) == 0) w[t] = old + sum;
    }
}

template <int D, int NC>
cudaError_t launch_warp(const WeightsParams &p, cudaStream_t stream) {
    // Key ranges that give each SM its 8 CTAs twice over at the largest context, of at
    // least one step.
    const int64_t ctx = (int64_t)p.max_pages * p.P, units = (int64_t)p.B * p.Hkv;
    const int64_t step = kWarpThreads / 32 * kWarpKeys;
    const int64_t want = (ctx * units / ((int64_t)device_sm_count() * 16) + step - 1) / step;
    const int64_t chunk = (want < 1 ? 1 : want > 64 ? 64 : want) * step;
    const dim3 grid((unsigned)((ctx + chunk - 1) / chunk), (unsigned)p.Hkv, (unsigned)p.B);
    weights_warp_kernel<D, NC><<<grid, kWarpThreads, 0, stream>>>(p, (int)chunk);
    return cudaGetLastError();
}

template <int D, int NC>
cudaError_t launch_ffma(const WeightsParams &p, cudaStream_t stream) {
    using Lay = FfmaLayout<D, NC>;
    auto kern = weights_ffma_kernel<D, NC>;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !configured[dev]) {
        err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kBytes);
        if (err != cudaSuccess) return err;
        if (dev < 64) configured[dev] = 1;
    }
    const int64_t ctx = (int64_t)p.max_pages * p.P;
    const dim3 grid((unsigned)((ctx + kKeys - 1) / kKeys), (unsigned)p.Hkv, (unsigned)p.B);
    kern<<<grid, 256, Lay::kBytes, stream>>>(p);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_f32(const WeightsParams &p, cudaStream_t stream) {
    const int64_t cols = (int64_t)p.G * p.q_len;
    return cols <= 1    ? launch_warp<D, 1>(p, stream)
           : cols <= 2  ? launch_warp<D, 2>(p, stream)
           : cols <= 4  ? launch_warp<D, 4>(p, stream)
           : cols <= 8  ? launch_warp<D, 8>(p, stream)
                        : launch_ffma<D, 16>(p, stream);
}

atlas_status check(int32_t Hq, int32_t Hkv, int32_t D, int32_t P, const atlas_weights *W) {
    if (!W || W->batch < 1 || W->max_pages_per_seq < 1 || W->num_pages < 1 || W->q_len < 1 ||
        Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || W->row_tokens < 1 || W->window < 0 ||
        !(W->softcap >= 0.f) || W->softcap == INFINITY || W->sm_count < 0 ||
        (W->accumulate != 0 && W->accumulate != 1))
        return ATLAS_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATLAS_ERR_UNSUPPORTED;
    if (P < 8 || P > 128 || (P & (P - 1))) return ATLAS_ERR_UNSUPPORTED;
    if (W->dtype != ATLAS_F32 && W->dtype != ATLAS_BF16) return ATLAS_ERR_UNSUPPORTED;
    const int64_t ctx = (int64_t)W->max_pages_per_seq * P;
    // the limits of the attention calls (32-bit rows and keys), and the grid's
    if (ctx > INT32_MAX / 2 || W->q_len > ctx || (int64_t)W->num_pages * Hkv * P >= INT32_MAX ||
        (int64_t)W->batch * Hq * W->q_len >= INT32_MAX || W->batch > 65535 || Hkv > 65535)
        return ATLAS_ERR_INVALID_ARG;
    return ATLAS_OK;
}

#ifndef F32TC
#define F32TC 16
#endif
// fp32 with at most this many columns runs without the tensor cores and a plan.
constexpr int64_t kF32Columns = F32TC;

WeightsPlan plan_of(int32_t Hq, int32_t Hkv, int32_t D, int32_t P, const atlas_weights *W) {
    const int sms = W->sm_count > 0 ? W->sm_count : device_sm_count();
    const int64_t ctx = (int64_t)W->max_pages_per_seq * P;
    const int G = Hq / Hkv;
    if (W->dtype == ATLAS_BF16) return weights_tc_plan(W->batch, Hkv, G, W->q_len, ctx, sms);
    if ((int64_t)G * W->q_len <= kF32Columns) return WeightsPlan{};
    return weights_tf32x3_plan(W->batch, Hkv, G, W->q_len, D, ctx, sms);
}

}  // namespace
}  // namespace atlas

extern "C" {

size_t atlas_kv_weights_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t page_tokens, const atlas_weights *W) {
    if (atlas::check(n_q_heads, n_kv_heads, head_dim, page_tokens, W) != ATLAS_OK) return SIZE_MAX;
    return atlas::plan_of(n_q_heads, n_kv_heads, head_dim, page_tokens, W).ws_bytes;
}

atlas_status atlas_kv_weights(const void *q, const void *k_pages, const int32_t *page_table,
                              const int32_t *seq_lens, const float *lse, int32_t n_q_heads,
                              int32_t n_kv_heads, int32_t head_dim, int32_t page_tokens,
                              float scale, const atlas_weights *W) {
    using namespace atlas;
    if (!q || !k_pages || !page_table || !seq_lens || !lse || !W || !W->weights)
        return ATLAS_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pages) |
          reinterpret_cast<uintptr_t>(W->workspace)) & 15u) ||
        (reinterpret_cast<uintptr_t>(W->weights) & 3u))
        return ATLAS_ERR_INVALID_ARG;
    if (!(fabsf(scale) < INFINITY)) return ATLAS_ERR_INVALID_ARG;
    const atlas_status st = check(n_q_heads, n_kv_heads, head_dim, page_tokens, W);
    if (st != ATLAS_OK) return st;
    const WeightsPlan plan = plan_of(n_q_heads, n_kv_heads, head_dim, page_tokens, W);
    if (plan.ws_bytes > 0 && (!W->workspace || W->workspace_bytes < plan.ws_bytes))
        return ATLAS_ERR_WORKSPACE;
    WeightsParams p{};
    p.q = q;
    p.k_pages = k_pages;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.q_lens = W->q_lens;
    p.lse = lse;
    p.weights = W->weights;
    p.B = W->batch;
    p.Hq = n_q_heads;
    p.Hkv = n_kv_heads;
    p.G = n_q_heads / n_kv_heads;
    p.P = page_tokens;
    p.q_len = W->q_len;
    p.max_pages = W->max_pages_per_seq;
    p.num_pages = W->num_pages;
    p.row_tokens = W->row_tokens;
    p.accumulate = W->accumulate;
    p.window = W->window < (1 << 30) ? W->window : 1 << 30;  // key + window fits 32 bits
    p.scale_log2 = scale * kLog2e;
    p.softcap_log2 = W->softcap > 0.f ? W->softcap * kLog2e : 0.f;
    p.softcap_inv = W->softcap > 0.f ? scale / W->softcap : 0.f;
    p.status = W->status_word;
    const cudaStream_t stream = static_cast<cudaStream_t>(W->stream);
    (void)cudaGetLastError();
    cudaError_t err;
    const bool bf16 = W->dtype == ATLAS_BF16;
    if (bf16 || plan.parts > 0) {
        p.parts = static_cast<float *>(W->workspace);
        p.n_parts = plan.parts;
        p.tiles_per_part = plan.tiles_per_part;
        CUtensorMap tmQ, tmK;
        if (encode_rows_map(&tmQ, q, (int64_t)p.B * p.Hq * p.q_len, head_dim, 128, !bf16) != ATLAS_OK)
            return ATLAS_ERR_CUDA;
        if (bf16 && encode_rows_map(&tmK, k_pages, (int64_t)p.num_pages * p.Hkv * p.P, head_dim, p.P) !=
                        ATLAS_OK)
            return ATLAS_ERR_CUDA;
        err = bf16 ? launch_weights_tc(p, plan, head_dim, tmQ, tmK, stream)
                   : launch_weights_tf32x3(p, head_dim, tmQ, stream);
    } else {
        err = head_dim == 128 ? launch_f32<128>(p, stream) : launch_f32<64>(p, stream);
    }
    return err == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
