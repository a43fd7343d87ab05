// kv_weights.cu -- the attention weight each cached key received: for key t of
// (sequence, kv head),
//   w[t] (+)= sum over columns c that see t of 2^(s2(t, c) - lse2(c)),
// a column being one (q head of the group, query row) pair, s2 its score with key t and
// lse2 the row's log-sum-exp that the attention call returned, both in log2 units.  No
// softmax state is needed -- lse normalises every row -- and K is read once.
//
// bf16 runs on the tensor cores (kv_weights_tc.cu); this file has the entry point and
// fp32.  weights_ffma_kernel: a CTA owns 128 keys of one (sequence, kv head), held in shared
// memory, and walks the columns in tiles of NC.  A thread forms 4 keys x NC / 8
// columns of scores as whole dot products, exponentiates them and keeps one sum per key;
// the 8 lanes that share a key add up at the end.
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
__global__ void __launch_bounds__(256) weights_ffma_kernel(const WeightsParams p) {
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
        float s[4][CPT];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < CPT; ++c) s[r][c] = 0.f;
#pragma unroll 4
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
                    s[r][c] = fmaf(q4.x, k4[r].x, s[r][c]);
                    s[r][c] = fmaf(q4.y, k4[r].y, s[r][c]);
                    s[r][c] = fmaf(q4.z, k4[r].z, s[r][c]);
                    s[r][c] = fmaf(q4.w, k4[r].w, s[r][c]);
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
                sum[r] += t < lim && t >= lo ? ex2(score_log2(p, s[r][c]) - lse2) : 0.f;
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

// fp32 has no plan to make: one CTA per 128 keys, no workspace.
WeightsPlan plan_of(int32_t Hq, int32_t Hkv, int32_t P, const atlas_weights *W) {
    if (W->dtype == ATLAS_F32) return WeightsPlan{};
    return weights_tc_plan(W->batch, Hkv, Hq / Hkv, W->q_len, (int64_t)W->max_pages_per_seq * P,
                           W->sm_count > 0 ? W->sm_count : device_sm_count());
}

}  // namespace
}  // namespace atlas

extern "C" {

size_t atlas_kv_weights_workspace_size(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                       int32_t page_tokens, const atlas_weights *W) {
    if (atlas::check(n_q_heads, n_kv_heads, head_dim, page_tokens, W) != ATLAS_OK) return SIZE_MAX;
    return atlas::plan_of(n_q_heads, n_kv_heads, page_tokens, W).ws_bytes;
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
    const WeightsPlan plan = plan_of(n_q_heads, n_kv_heads, page_tokens, W);
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
    if (W->dtype == ATLAS_BF16) {
        p.parts = static_cast<float *>(W->workspace);
        p.n_parts = plan.parts;
        p.tiles_per_part = plan.tiles_per_part;
        CUtensorMap tmQ, tmK;
        if (encode_rows_map(&tmQ, q, (int64_t)p.B * p.Hq * p.q_len, head_dim, 128) != ATLAS_OK ||
            encode_rows_map(&tmK, k_pages, (int64_t)p.num_pages * p.Hkv * p.P, head_dim, p.P) != ATLAS_OK)
            return ATLAS_ERR_CUDA;
        err = launch_weights_tc(p, plan, head_dim, tmQ, tmK, stream);
    } else {
        const bool few = (int64_t)p.G * p.q_len <= 8;
        err = head_dim == 128 ? (few ? launch_ffma<128, 8>(p, stream) : launch_ffma<128, 32>(p, stream))
                              : (few ? launch_ffma<64, 8>(p, stream) : launch_ffma<64, 32>(p, stream));
    }
    return err == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // extern "C"
