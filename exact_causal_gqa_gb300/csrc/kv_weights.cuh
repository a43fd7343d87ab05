// kv_weights.cuh -- what the attention-weight kernels share.
#pragma once

#include "internal.h"
#include "ptx.cuh"

#include "atlas_evict.h"

#include <math.h>

namespace atlas {

struct WeightsParams {
    const void *q, *k_pages;
    const int32_t *page_table, *seq_lens, *q_lens;
    const float *lse;
    float *weights;
    int32_t B, Hq, Hkv, G, P, q_len, max_pages, num_pages, row_tokens;
    int32_t accumulate, window;
    float scale_log2, softcap_log2, softcap_inv;
    float *parts;   // tile kernels: [n_parts][B * Hkv][max_pages * P] partial sums
    int32_t n_parts, tiles_per_part;
    uint32_t *status;
};

__device__ __forceinline__ void record(uint32_t *status, uint32_t bit) {
    if (status) atomicOr(status, bit);
}

__device__ __forceinline__ bool bad_lens(const WeightsParams &p, int L, int qn) {
    return qn < 0 || qn > p.q_len || L < qn || L > p.max_pages * p.P || L > p.row_tokens;
}

// Whether key t (< the sequence's length) lies on a page of the pool.
__device__ __forceinline__ bool page_ok(const WeightsParams &p, int b, int t, int lp) {
    const int id = p.page_table[(int64_t)b * p.max_pages + (t >> lp)];
    return id >= 0 && id < p.num_pages;
}

// Score in log2 units from a raw dot product: scale (and the softcap, if any).  The cap
// takes tanhf, good relative to its value: an absolute error (1e-7 from one exponential)
// would be scaled up by the cap, into a relative error of the weight (measured 1.4e-6 at
// a cap of 30 where tanhf leaves 2e-7).
__device__ __forceinline__ float score_log2(const WeightsParams &p, float raw) {
    return p.softcap_log2 > 0.f ? p.softcap_log2 * tanhf(raw * p.softcap_inv)
                                : raw * p.scale_log2;
}

// Whether rows of which the earliest sees keys below lim_min and the latest keys below
// lim_max see one of [k0, k0 + keys).
__device__ __forceinline__ bool sees(const WeightsParams &p, int lim_min, int lim_max, int k0, int keys) {
    return k0 < lim_max && (p.window == 0 || k0 + keys > lim_min - p.window);
}

// A row's log-sum-exp in log2 units; a row that saw nothing (-inf) becomes +inf, so
// that 2^(s2 - it) is 0.
__device__ __forceinline__ float lse_log2(float lse) {
    return lse == -INFINITY ? INFINITY : lse * kLog2e;
}

// How a call on the tensor cores runs, and the workspace it needs.
struct WeightsPlan {
    int stream;          // 1: few columns, K streamed past the resident queries
    int chunk_tiles;     // stream: 128-key tiles of a CTA
    int parts, tiles_per_part;  // tile kernels: query tiles split between CTAs
    size_t ws_bytes;
};
// bf16 (kv_weights_tc.cu).
WeightsPlan weights_tc_plan(int B, int Hkv, int G, int q_len, int64_t ctx, int sms);
cudaError_t launch_weights_tc(const WeightsParams &p, const WeightsPlan &plan, int D,
                              const CUtensorMap &tmQ, const CUtensorMap &tmK, cudaStream_t stream);
// fp32 with more columns than weights_warp_kernel takes (kv_weights_tc_f32.cu).
WeightsPlan weights_tf32x3_plan(int B, int Hkv, int G, int q_len, int D, int64_t ctx, int sms);
cudaError_t launch_weights_tf32x3(const WeightsParams &p, const WeightsPlan &plan, int D,
                                  const CUtensorMap &tmQ, const CUtensorMap &tmK, cudaStream_t stream);

}  // namespace atlas
