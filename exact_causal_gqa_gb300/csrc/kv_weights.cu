// kv_weights.cu -- the attention weight each cached key received: for key t of
// (sequence, kv head),
//   w[t] (+)= sum over columns c that see t of 2^(s2(t, c) - lse2(c)),
// a column being one (q head of the group, query row) pair, s2 its score with key t and
// lse2 the row's log-sum-exp that the attention call returned, both in log2 units.  No
// softmax state is needed -- lse normalises every row -- and K is read once.
//
// bf16 runs on the tensor cores (kv_weights_tc.cu), and so does fp32 with more than two
// columns (kv_weights_tc_f32.cu); this file has the entry point and the rest.
//
// weights_warp_kernel, one or two columns (decode without or with two shared heads): K is
//   read once, straight into registers, and its bytes are the bound.  A warp takes 8 keys at
//   a time, a lane D / 32 elements of each; the 8 x NC partial dot products are added across
//   the lanes by halving -- each step sends half of a lane's values to the lane that keeps
//   them, one shuffle per score in all -- which leaves every score in one lane, and the
//   columns' weights are added over neighbouring lanes.  8 sequences of 16384 keys, 8 kv
//   heads of 128: 94 us, 5.7 TB/s with one column, 96 us with two (4 keys a warp are slower).
#include "kv_weights.cuh"

namespace atlas {
namespace {

// One warp per 8 keys and step; grid (key ranges, Hkv, B).
constexpr int kWarpKeys = 8, kWarpThreads = 256;

template <int D, int NC>
__global__ void __launch_bounds__(kWarpThreads, 3)
    weights_warp_kernel(const WeightsParams p, const int chunk) {
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
    // After the halving a lane holds one column of one key; kSpread lanes hold copies.
    constexpr int kSpread = 32 / (kWarpKeys * NC);
    const int key = lane / kSpread / NC, mine = lane / kSpread % NC;
    const bool real = mine < ncols;
    const float lse2 =
        real ? lse_log2(p.lse[row0 + (int64_t)(mine / qn) * p.q_len + mine % qn]) : INFINITY;
    const int lim = real ? L - qn + mine % qn + 1 : 0;
    float *w = p.weights + ((int64_t)b * p.Hkv + hkv) * p.row_tokens;
    const int32_t *table = p.page_table + (int64_t)b * p.max_pages;
    // Page ids are read by the lanes that own a key, a step ahead, and handed round.
    auto page_of = [&](int kb) {
        const int t = kb + key;
        const int id = t < end ? table[t >> lp] : -1;
        if (t < end && (id < 0 || id >= p.num_pages) && lane % (kSpread * NC) == 0)
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
            const int page = __shfl_sync(0xffffffffu, id, k * kSpread * NC);
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
        // Partial dot products, value (key, column) at key * NC + column.
        float s[kWarpKeys * NC];
#pragma unroll
        for (int k = 0; k < kWarpKeys; ++k)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                float a = q[c][0] * x[k][0];
#pragma unroll
                for (int e = 1; e < DPL; ++e) a = fmaf(q[c][e], x[k][e], a);
                s[k * NC + c] = a;
            }
        // Halving: lane bit `o` keeps the upper or the lower half of the values; once one is
        // left, the lanes that hold the same one add theirs up.
        int n = kWarpKeys * NC;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            if (n > 1) {
                n /= 2;
                const bool upper = lane & o;
#pragma unroll
                for (int v = 0; v < kWarpKeys * NC / 2; ++v) {
                    if (v >= n) break;
                    const float send = upper ? s[v] : s[v + n];
                    s[v] = (upper ? s[v + n] : s[v]) + __shfl_xor_sync(0xffffffffu, send, o);
                }
            } else {
                s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
            }
        }
        const bool sees = t < lim && (p.window == 0 || t >= lim - p.window);
        float sum = sees ? ex2(score_log2(p, s[0]) - lse2) : 0.f;
#pragma unroll
        for (int o = kSpread; o < kSpread * NC; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (t < end && id >= 0 && lane % (kSpread * NC) == 0) w[t] = old + sum;
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

// fp32 with at most this many columns runs on weights_warp_kernel, without a plan: at 8
// sequences x 8 kv heads x 16384 keys of 128 it takes 94 / 96 / 104 us for 1 / 2 / 4
// columns where the tensor-core stream takes 88, at 1 x 8 x 8192 keys 7.5 / 8.4 / 10.8
// against 8.7, at 2 x 8 x 1000 keys 3.5 / 4.0 / 5.1 against 5.9 (head_dim 64, 8 x 8 x 16384
// keys: 57 / 63 / 82 against 59).
constexpr int64_t kWarpColumns = 2;

WeightsPlan plan_of(int32_t Hq, int32_t Hkv, int32_t D, int32_t P, const atlas_weights *W) {
    const int sms = W->sm_count > 0 ? W->sm_count : device_sm_count();
    const int64_t ctx = (int64_t)W->max_pages_per_seq * P;
    const int G = Hq / Hkv;
    if (W->dtype == ATLAS_BF16) return weights_tc_plan(W->batch, Hkv, G, W->q_len, ctx, sms);
    if ((int64_t)G * W->q_len <= kWarpColumns) return WeightsPlan{};
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
        !aligned4({page_table, seq_lens, lse, W->weights, W->q_lens, W->status_word}))
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
    if (bf16 || plan.stream || plan.parts > 0) {
        p.parts = static_cast<float *>(W->workspace);
        p.n_parts = plan.parts;
        p.tiles_per_part = plan.tiles_per_part;
        // (the stream kernels pack their columns themselves; the fp32 tile kernel reads K so)
        CUtensorMap tmQ{}, tmK{};
        if (!plan.stream &&
            encode_rows_map(&tmQ, q, (int64_t)p.B * p.Hq * p.q_len, head_dim, 128, !bf16) != ATLAS_OK)
            return ATLAS_ERR_CUDA;
        if ((bf16 || plan.stream) &&
            encode_rows_map(&tmK, k_pages, (int64_t)p.num_pages * p.Hkv * p.P, head_dim, p.P, !bf16) !=
                ATLAS_OK)
            return ATLAS_ERR_CUDA;
        err = bf16 ? launch_weights_tc(p, plan, head_dim, tmQ, tmK, stream)
                   : launch_weights_tf32x3(p, plan, head_dim, tmQ, tmK, stream);
    } else {
        const bool one = p.G * p.q_len == 1;
        err = head_dim == 128 ? (one ? launch_warp<128, 1>(p, stream) : launch_warp<128, 2>(p, stream))
                              : (one ? launch_warp<64, 1>(p, stream) : launch_warp<64, 2>(p, stream));
    }
    return err == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
