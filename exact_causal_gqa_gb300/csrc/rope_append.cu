// rope_append.cu -- rotary positions with several axes, applied on the way into the
// cache: one pass rotates a step's queries, rotates its new keys and writes keys and
// values to their page slots (atlas_kv_append with the rotation that the pages of the
// CFR-Atlas README leave to the backend fused in).
//
// The mathematics.  Pair p of a row (elements p and p + R/2 of the R rotated ones, or
// 2p and 2p + 1) turns by the angle  z = positions[axis(p)][b][j] * f_p:
//   (x, y) -> (x cos z - y sin z,  y cos z + x sin z),   in fp32, rounded once.
// Far positions make z large (1e6 rad and more), where an fp32 product has lost the
// angle.  Here z is taken in turns, as a 64-bit fraction of one turn: the host rounds
// f_p / 2 pi mod 1 to F_p / 2^64, and the integer product position * F_p mod 2^64 is the
// exact fraction of a turn of that F_p -- the 64-bit wrap is the range reduction, two
// integer multiplies where an fp64 product would cost a slow pipe.  What is left is
// |position| times the rounding of f_p / 2 pi (2^-53 of it): below 2^-24 turns for any
// int32 position and |f_p| <= 1.  The top two bits (rounded) give the quadrant and the
// rest an angle within an eighth of a turn, for sincospif.
//
// What bounds it: memory, (read + write) of every row of q, k and v once.  A thread owns
// one token and one slot of its rows -- V pairs, i.e. two vectors of V elements (16 bytes
// each at V = 8 bf16) -- computes those V sines and cosines once and walks heads with
// them, kUnroll rows in flight.  Consecutive threads take consecutive slots of a row, so
// a warp reads and writes whole rows.  Few tokens (a decode step) leave too few threads
// for that: the heads are then shared between CTAs (grid.y), each redoing the angles.
#include "internal.h"

#include <cuda_bf16.h>
#include <math.h>

namespace atlas {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxPairs = 64;  // head_dim 128 / 2

struct RopeParams {
    const void *q, *k_new, *v_new;
    void *q_out, *k_pages, *v_pages;
    const int32_t *page_table, *seq_lens, *n_new, *positions;
    int64_t qs[3], ks[3], vs[3];  // element strides: batch, head, token
    int32_t B, Hq, Hkv, D, P, n, max_pages, num_pages;
    int32_t pairs;                // rotated pairs of a row; the D - 2 pairs others are copied
    int32_t interleaved;
    int32_t heads_per_cta;
    uint32_t *status;
    uint64_t turn[kMaxPairs];     // f_p / 2 pi mod 1, times 2^64
    uint8_t axis[kMaxPairs];
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// cos and sin of `turn` / 2^64 turns: the nearest quarter turn and a remainder within
// an eighth of a turn either side, whose fp32 form is exact to 2^-24 of itself.
__device__ __forceinline__ void cos_sin_turns(uint64_t turn, float &c, float &s) {
    const uint32_t top = (uint32_t)(turn >> 32);
    const uint32_t quarter = (top + (1u << 29)) >> 30;
    const int32_t rest = (int32_t)(top - (quarter << 30));
    float rs, rc;
    sincospif((float)rest * 0x1p-31f, &rs, &rc);
    const float a = (quarter & 1) ? rs : rc, b = (quarter & 1) ? rc : rs;
    c = (quarter == 1 || quarter == 2) ? -a : a;
    s = (quarter & 2) ? -b : b;
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ RopeParams p) {
    const int lg_slots = 30 - __clz(p.D) - (V == 8 ? 3 : V == 4 ? 2 : V == 2 ? 1 : 0);
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;  // slots: D / (2 V)
    const int64_t token = at >> lg_slots;
    if (token >= (int64_t)p.B * p.n) return;
    const int slot = (int)at & ((1 << lg_slots) - 1);
    const int b = (int32_t)token / p.n, j = (int32_t)token % p.n;  // B * n < 2^31
    const int count = p.n_new ? p.n_new[b] : p.n;
    if (count < 0 || count > p.n) {
        if (j == 0 && slot == 0 && blockIdx.y == 0 && p.status)
            atomicOr(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    if (j >= count) return;
    const int h0 = (int)blockIdx.y * p.heads_per_cta;
    const int heads = p.Hq + 2 * p.Hkv;
    const int h1 = min(heads, h0 + p.heads_per_cta);

    // The two vectors of this slot: pairs V slot .. V slot + V - 1, or (past the rotated
    // part, which V divides too) two vectors of the elements that are only copied.
    const int pair0 = slot * V;
    const bool turns = pair0 < p.pairs;
    int e0, e1;
    if (turns && !p.interleaved) {
        e0 = pair0;
        e1 = pair0 + p.pairs;
    } else {
        e0 = 2 * pair0;
        e1 = e0 + V;
    }
    float c[V], s[V];
    if (turns && h0 < p.Hq + p.Hkv) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int32_t pos = p.positions[((int64_t)p.axis[pair0 + i] * p.B + b) * p.n + j];
            cos_sin_turns((uint64_t)(int64_t)pos * p.turn[pair0 + i], c[i], s[i]);
        }
    }
    // The cache slot of this token; -1: nowhere (reported).
    int64_t cache = -1;
    if (h1 > p.Hq) {
        const int64_t t = (int64_t)p.seq_lens[b] + j;
        uint32_t bad = ATLAS_DEV_BAD_SEQLEN;
        if (t >= 0 && t < (int64_t)p.max_pages * p.P) {
            const int lp = 31 - __clz(p.P);  // page_tokens is a power of two
            const int page = p.page_table[(int64_t)b * p.max_pages + (t >> lp)];
            bad = page < 0 || page >= p.num_pages ? ATLAS_DEV_BAD_PAGE : 0u;
            if (!bad) cache = ((int64_t)page * p.Hkv * p.P + (t & (p.P - 1))) * p.D;
        }
        if (bad && slot == 0 && p.status) atomicOr(p.status, bad);
    }
    using X = Vec<T, V>;
    for (int h = h0; h < h1; h += kUnroll) {
        X x0[kUnroll], x1[kUnroll];
        T *dst[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            dst[u] = nullptr;
            const int hh = h + u;
            if (hh >= h1) continue;
            const T *src;
            if (hh < p.Hq) {
                src = static_cast<const T *>(p.q) + b * p.qs[0] + hh * p.qs[1] + j * p.qs[2];
                dst[u] = static_cast<T *>(p.q_out) + (((int64_t)b * p.Hq + hh) * p.n + j) * p.D;
            } else {
                const bool is_k = hh < p.Hq + p.Hkv;
                const int g = hh - p.Hq - (is_k ? 0 : p.Hkv);
                if (cache < 0) continue;
                src = is_k ? static_cast<const T *>(p.k_new) + b * p.ks[0] + g * p.ks[1] + j * p.ks[2]
                           : static_cast<const T *>(p.v_new) + b * p.vs[0] + g * p.vs[1] + j * p.vs[2];
                dst[u] = static_cast<T *>(is_k ? p.k_pages : p.v_pages) + cache +
                         (int64_t)g * p.P * p.D;
            }
            x0[u] = *reinterpret_cast<const X *>(src + e0);
            x1[u] = *reinterpret_cast<const X *>(src + e1);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (!dst[u]) continue;
            if (turns && h + u < p.Hq + p.Hkv) {
                X y0, y1;
                if (!p.interleaved) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float x = widen(x0[u].e[i]), y = widen(x1[u].e[i]);
                        y0.e[i] = narrow<T>(x * c[i] - y * s[i]);
                        y1.e[i] = narrow<T>(y * c[i] + x * s[i]);
                    }
                } else {
                    // x0 and x1 hold 2 V consecutive elements: pair i at 2i, 2i + 1
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const T &ex = 2 * i < V ? x0[u].e[2 * i % V] : x1[u].e[2 * i % V];
                        const T &ey = 2 * i + 1 < V ? x0[u].e[(2 * i + 1) % V]
                                                    : x1[u].e[(2 * i + 1) % V];
                        const float x = widen(ex), y = widen(ey);
                        (2 * i < V ? y0 : y1).e[2 * i % V] = narrow<T>(x * c[i] - y * s[i]);
                        (2 * i + 1 < V ? y0 : y1).e[(2 * i + 1) % V] = narrow<T>(y * c[i] + x * s[i]);
                    }
                }
                x0[u] = y0;
                x1[u] = y1;
            }
            *reinterpret_cast<X *>(dst[u] + e0) = x0[u];
            *reinterpret_cast<X *>(dst[u] + e1) = x1[u];
        }
    }
}

template <typename T, int V>
cudaError_t launch(RopeParams &p, cudaStream_t stream) {
    const int64_t threads = (int64_t)p.B * p.n * (p.D / (2 * V));
    const int heads = p.Hq + 2 * p.Hkv;
    // As many head groups as it takes to give every SM its 2048 threads.
    const int64_t want = (int64_t)device_sm_count() * 2048;
    int64_t groups = (want + threads - 1) / threads;
    if (groups > heads) groups = heads;
    p.heads_per_cta = (int)((heads + groups - 1) / groups);
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads),
                    (unsigned)((heads + p.heads_per_cta - 1) / p.heads_per_cta));
    rope_append_kernel<T, V><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// A stride triple (batch, head, token) in elements; all zero means dense rows.
bool take_strides(const int64_t given[3], int64_t heads, int64_t n, int64_t D, int64_t per16,
                  int64_t out[3]) {
    if (!given[0] && !given[1] && !given[2]) {
        out[0] = heads * n * D;
        out[1] = n * D;
        out[2] = D;
        return true;
    }
    for (int i = 0; i < 3; ++i) {
        if (given[i] % per16) return false;
        out[i] = given[i];
    }
    return true;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace atlas

extern "C" atlas_status atlas_kv_append_rope(const void *k_new, const void *v_new, void *k_pages,
                                             void *v_pages, const int32_t *page_table,
                                             const int32_t *seq_lens, const int32_t *n_new,
                                             int32_t n_kv_heads, int32_t head_dim,
                                             int32_t page_tokens, const atlas_rope *R) {
    using namespace atlas;
    if (!R || !k_new || !v_new || !k_pages || !v_pages || !page_table || !seq_lens || !R->positions)
        return ATLAS_ERR_INVALID_ARG;
    if (R->batch < 1 || R->max_pages_per_seq < 1 || R->num_pages < 1 || R->max_new < 0 ||
        n_kv_heads < 1 || R->n_q_heads < 0 || (R->n_q_heads > 0 && (!R->q || !R->q_out)))
        return ATLAS_ERR_INVALID_ARG;
    if (head_dim != 64 && head_dim != 128) return ATLAS_ERR_UNSUPPORTED;
    if (page_tokens < 1 || page_tokens > 128 || (page_tokens & (page_tokens - 1)))
        return ATLAS_ERR_UNSUPPORTED;
    if (R->kv_dtype != ATLAS_F32 && R->kv_dtype != ATLAS_BF16) return ATLAS_ERR_UNSUPPORTED;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
        (R->n_q_heads > 0 && (!aligned16(R->q) || !aligned16(R->q_out))))
        return ATLAS_ERR_INVALID_ARG;
    if (R->n_axes < 1 || R->n_axes > ATLAS_ROPE_MAX_AXES || R->rot_dim < 2 || R->rot_dim % 2 ||
        R->rot_dim > head_dim || (R->interleaved != 0 && R->interleaved != 1))
        return ATLAS_ERR_INVALID_ARG;
    // the kernel's index limits: tokens in 32 bits, (token, head) rows of q_out below 2^31
    const int64_t heads = (int64_t)R->n_q_heads + 2 * (int64_t)n_kv_heads;
    if ((int64_t)R->batch * R->max_new * (head_dim / 2) >= (int64_t)INT32_MAX * 256 ||
        (int64_t)R->batch * R->max_new >= INT32_MAX || heads > 65535)
        return ATLAS_ERR_INVALID_ARG;

    RopeParams p{};
    const int pairs = R->rot_dim / 2;
    for (int i = 0; i < pairs; ++i) {
        const int32_t axis = R->pair_axis ? R->pair_axis[i] : 0;
        if (axis < 0 || axis >= R->n_axes) return ATLAS_ERR_INVALID_ARG;
        p.axis[i] = (uint8_t)axis;
        if (!R->inv_freq && !(R->theta > 0.0 && R->theta < HUGE_VAL)) return ATLAS_ERR_INVALID_ARG;
        const double f = R->inv_freq ? R->inv_freq[i] : pow(R->theta, -2.0 * i / R->rot_dim);
        if (!(fabs(f) < HUGE_VAL)) return ATLAS_ERR_INVALID_ARG;
        const double turns = f / 6.283185307179586476925;
        const double part = turns - floor(turns);  // in [0, 1]; 1 only by rounding: no turn
        p.turn[i] = part < 1.0 ? (uint64_t)ldexp(part, 64) : 0;
    }
    const int64_t per16 = R->kv_dtype == ATLAS_BF16 ? 8 : 4;
    const int64_t n = R->max_new, D = head_dim;
    if (!take_strides(R->q_strides, R->n_q_heads, n, D, per16, p.qs) ||
        !take_strides(R->k_strides, n_kv_heads, n, D, per16, p.ks) ||
        !take_strides(R->v_strides, n_kv_heads, n, D, per16, p.vs))
        return ATLAS_ERR_INVALID_ARG;
    if (R->max_new == 0) return ATLAS_OK;
    p.q = R->q;
    p.q_out = R->q_out;
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.page_table = page_table;
    p.seq_lens = seq_lens;
    p.n_new = n_new;
    p.positions = R->positions;
    p.B = R->batch;
    p.Hq = R->n_q_heads;
    p.Hkv = n_kv_heads;
    p.D = head_dim;
    p.P = page_tokens;
    p.n = R->max_new;
    p.max_pages = R->max_pages_per_seq;
    p.num_pages = R->num_pages;
    p.pairs = pairs;
    p.interleaved = R->interleaved;
    p.status = R->status_word;
    // The widest vector (at most 16 bytes) that divides the rotated part's halves.
    const cudaStream_t stream = static_cast<cudaStream_t>(R->stream);
    (void)cudaGetLastError();
    cudaError_t err;
    if (R->kv_dtype == ATLAS_BF16) {
        using T = __nv_bfloat16;
        err = pairs % 8 == 0   ? launch<T, 8>(p, stream)
              : pairs % 4 == 0 ? launch<T, 4>(p, stream)
              : pairs % 2 == 0 ? launch<T, 2>(p, stream)
                               : launch<T, 1>(p, stream);
    } else {
        err = pairs % 4 == 0   ? launch<float, 4>(p, stream)
              : pairs % 2 == 0 ? launch<float, 2>(p, stream)
                               : launch<float, 1>(p, stream);
    }
    return err == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}
