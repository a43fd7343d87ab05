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
// f_p / 2 pi, less its nearest whole number, to F_p / 2^64, and the integer product
// position * F_p mod 2^64 is the exact fraction of a turn of that F_p -- the 64-bit wrap is
// the range reduction, two integer multiplies where an fp64 product would cost a slow pipe.
// What is left is |position| times the rounding of f_p / 2 pi (2^-53 of it, twice): below
// 2^-24 turns for any int32 position and |f_p| <= 1 of either sign (0.7 of that over random
// frequencies).  The top two bits (rounded) give the quadrant and the rest an angle within
// an eighth of a turn, for sincospif.
//
// What bounds it: memory, (read + write) of every row of q, k and v once.  A CTA takes
// kMaxTokens neighbouring tokens: it puts their cosines and sines (shared by all heads)
// and row offsets into shared memory once, then its threads walk the tokens' rows, one
// slot -- V pairs, i.e. two vectors of V elements, 16 bytes each at V = 8 bf16 -- of one
// head at a time.  Consecutive threads take consecutive slots, then heads, so a fused
// projection is read front to back.  With 32 registers a thread, all 2048 threads of an
// SM have their two loads in flight; more slots in flight per thread cost that occupancy
// and were slower, as were angles held in registers.  4 x 8192 tokens of 32 + 8 + 8 heads
// of 128 bf16 (806 MB): 125 us, 6.4 TB/s (95 % of the measured copy); 2 slots a thread
// 149 us, a slot of one token for all heads per thread 197 us; 1, 4, 8, 16, 32 tokens
// per CTA 139, 128, 133, 143, 169 us.  Few tokens (a decode step) leave too few CTAs: the
// heads are then shared between CTAs (grid.y).
#include "internal.h"

#include <cuda_bf16.h>
#include <math.h>

namespace atlas {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 2;
constexpr int kMaxPairs = 64;  // head_dim 128 / 2

struct RopeParams {
    const void *q, *k_new, *v_new;
    void *q_out, *k_pages, *v_pages;
    const int32_t *page_table, *seq_lens, *n_new, *positions;
    int64_t qs[3], ks[3], vs[3];  // element strides: batch, head, token
    int32_t B, Hq, Hkv, D, P, n, max_pages, num_pages;
    int32_t pairs;                // rotated pairs of a row; the D - 2 pairs others are copied
    int32_t interleaved;
    int32_t tokens_per_cta, heads_per_cta;
    uint32_t *status;
    uint64_t turn[kMaxPairs];     // f_p / 2 pi mod 1, times 2^64
    uint8_t axis[kMaxPairs];
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// One access of the whole vector (16 bytes as uint4: a struct copy became narrower ones).
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T *p) {
    Vec<T, V> x;
    if constexpr (sizeof(x) == 16)
        *reinterpret_cast<uint4 *>(&x) = *reinterpret_cast<const uint4 *>(p);
    else
        x = *reinterpret_cast<const Vec<T, V> *>(p);
    return x;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const Vec<T, V> &x) {
    if constexpr (sizeof(x) == 16)
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&x);
    else
        *reinterpret_cast<Vec<T, V> *>(p) = x;
}

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// cos and sin of `turn` / 2^64 turns: the nearest quarter turn and a remainder within an
// eighth of a turn either side.  The low 32 bits are dropped, 2^-32 turns at most, and the
// rest's fp32 form rounds by 2^-24 of it, 2^-27 turns at most: small next to a turn, which
// is what counts for an angle, though the angles of the slowest pairs at the first
// positions (2e-7 turns) keep but ten bits of their own.
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

// Element offsets of a token's rows of head 0; cache < 0: no slot (reported).
struct TokenRows {
    int64_t q, k, v, q_out, cache;
    bool any;  // a real token
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 8) rope_append_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float cs[kMaxTokens][2][kMaxPairs];  // cosines, sines
    __shared__ TokenRows rows[kMaxTokens];
    const int token0 = (int)blockIdx.x * p.tokens_per_cta;
    const int tokens = min(p.tokens_per_cta, p.B * p.n - token0);  // B * n < 2^31
    const int h0 = (int)blockIdx.y * p.heads_per_cta;
    const int h1 = min(p.Hq + 2 * p.Hkv, h0 + p.heads_per_cta);

    for (int i = threadIdx.x; i < tokens * p.pairs && h0 < p.Hq + p.Hkv; i += kThreads) {
        const int k = i / p.pairs, pair = i - k * p.pairs;
        const int32_t pos = p.positions[(int64_t)p.axis[pair] * p.B * p.n + token0 + k];
        cos_sin_turns((uint64_t)(int64_t)pos * p.turn[pair], cs[k][0][pair], cs[k][1][pair]);
    }
    if ((int)threadIdx.x < tokens) {
        const int b = (token0 + (int)threadIdx.x) / p.n, j = (token0 + (int)threadIdx.x) % p.n;
        const int count = p.n_new ? p.n_new[b] : p.n;
        uint32_t bad = 0;
        TokenRows r;
        r.any = count >= 0 && count <= p.n && j < count;
        if (count < 0 || count > p.n) bad = ATLAS_DEV_BAD_SEQLEN;
        r.q = b * p.qs[0] + j * p.qs[2];
        r.k = b * p.ks[0] + j * p.ks[2];
        r.v = b * p.vs[0] + j * p.vs[2];
        r.q_out = ((int64_t)b * p.Hq * p.n + j) * p.D;
        r.cache = -1;
        if (r.any && h1 > p.Hq) {
            const int64_t t = (int64_t)p.seq_lens[b] + j;
            if (t < 0 || t >= (int64_t)p.max_pages * p.P) {
                bad = ATLAS_DEV_BAD_SEQLEN;
            } else {
                const int lp = 31 - __clz(p.P);  // page_tokens is a power of two
                const int page = p.page_table[(int64_t)b * p.max_pages + (t >> lp)];
                if (page < 0 || page >= p.num_pages) bad = ATLAS_DEV_BAD_PAGE;
                else r.cache = ((int64_t)page * p.Hkv * p.P + (t & (p.P - 1))) * p.D;
            }
        }
        if (bad && p.status) atomicOr(p.status, bad);
        rows[threadIdx.x] = r;
    }
    __syncthreads();

    // Item: slot `slot` of head h0 + item / slots of token `k`; D / (2 V) slots a row.
    using X = Vec<T, V>;
    const int lg_slots = 30 - __clz(p.D) - (V == 8 ? 3 : V == 4 ? 2 : V == 2 ? 1 : 0);
    const int per_token = (h1 - h0) << lg_slots;
    for (int k = 0, item = threadIdx.x;; item += kThreads) {
        while (k < tokens && item >= per_token) {
            item -= per_token;
            ++k;
        }
        if (k >= tokens) break;
        const TokenRows &r = rows[k];
        const int h = h0 + (item >> lg_slots), slot = item & ((1 << lg_slots) - 1);
        if (!r.any || (h >= p.Hq && r.cache < 0)) continue;
        const T *src;
        T *dst;
        if (h < p.Hq) {
            src = static_cast<const T *>(p.q) + r.q + h * p.qs[1];
            dst = static_cast<T *>(p.q_out) + r.q_out + (int64_t)h * p.n * p.D;
        } else if (h < p.Hq + p.Hkv) {
            src = static_cast<const T *>(p.k_new) + r.k + (h - p.Hq) * p.ks[1];
            dst = static_cast<T *>(p.k_pages) + r.cache + (int64_t)(h - p.Hq) * p.P * p.D;
        } else {
            src = static_cast<const T *>(p.v_new) + r.v + (h - p.Hq - p.Hkv) * p.vs[1];
            dst = static_cast<T *>(p.v_pages) + r.cache + (int64_t)(h - p.Hq - p.Hkv) * p.P * p.D;
        }
        // The slot's two vectors: of its pairs, or (past the rotated part, which V divides
        // too) of the elements that are only copied.
        const int pair0 = slot * V;
        const bool turned = pair0 < p.pairs;
        const int e0 = turned && !p.interleaved ? pair0 : 2 * pair0;
        const int e1 = turned && !p.interleaved ? pair0 + p.pairs : e0 + V;
        X x0 = load_vec<T, V>(src + e0), x1 = load_vec<T, V>(src + e1);
        if (turned && h < p.Hq + p.Hkv) {
            const float *c = cs[k][0] + pair0, *s = cs[k][1] + pair0;
            X y0, y1;
            if (!p.interleaved) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = widen(x0.e[i]), y = widen(x1.e[i]);
                    y0.e[i] = narrow<T>(x * c[i] - y * s[i]);
                    y1.e[i] = narrow<T>(y * c[i] + x * s[i]);
                }
            } else {
                // x0 and x1 hold 2 V consecutive elements: pair i at 2i, 2i + 1
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float x = widen(2 * i < V ? x0.e[2 * i % V] : x1.e[2 * i % V]);
                    const float y = widen(2 * i + 1 < V ? x0.e[(2 * i + 1) % V] : x1.e[(2 * i + 1) % V]);
                    (2 * i < V ? y0 : y1).e[2 * i % V] = narrow<T>(x * c[i] - y * s[i]);
                    (2 * i + 1 < V ? y0 : y1).e[(2 * i + 1) % V] = narrow<T>(y * c[i] + x * s[i]);
                }
            }
            x0 = y0;
            x1 = y1;
        }
        store_vec<T, V>(dst + e0, x0);
        store_vec<T, V>(dst + e1, x1);
    }
}

template <typename T, int V>
cudaError_t launch(RopeParams &p, cudaStream_t stream) {
    const int64_t tokens = (int64_t)p.B * p.n;
    const int heads = p.Hq + 2 * p.Hkv;
    // kMaxTokens tokens per CTA while that leaves eight CTAs for each SM; with fewer
    // than that of single tokens, the heads in as many groups as it takes.
    const int64_t want = (int64_t)device_sm_count() * 8;
    p.tokens_per_cta = tokens >= want * kMaxTokens ? kMaxTokens : 1;
    const int64_t ctas = (tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
    int64_t groups = (want + ctas - 1) / ctas;
    // (a group has at least one item for each thread)
    const int64_t most = ((int64_t)heads * (p.D / (2 * V)) + kThreads - 1) / kThreads;
    if (groups > most) groups = most;
    p.heads_per_cta = (int)((heads + groups - 1) / groups);
    const dim3 grid((unsigned)ctas, (unsigned)((heads + p.heads_per_cta - 1) / p.heads_per_cta));
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
        (R->n_q_heads > 0 && (!aligned16(R->q) || !aligned16(R->q_out))) ||
        !aligned4({page_table, seq_lens, n_new, R->positions, R->status_word}))
        return ATLAS_ERR_INVALID_ARG;
    if (R->n_axes < 1 || R->n_axes > ATLAS_ROPE_MAX_AXES || R->rot_dim < 2 || R->rot_dim % 2 ||
        R->rot_dim > head_dim || (R->interleaved != 0 && R->interleaved != 1))
        return ATLAS_ERR_INVALID_ARG;
    // the kernel's index limits: tokens and a token's slots in 32 bits
    const int64_t heads = (int64_t)R->n_q_heads + 2 * (int64_t)n_kv_heads;
    if ((int64_t)R->batch * R->max_new >= INT32_MAX - kMaxTokens || heads > 65535)
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
        // The nearest whole turn off, not the one below: that would leave a small negative
        // frequency next to 1, with the last bit of 1 for its own.
        const double turns = f / 6.283185307179586476925;
        const double part = turns - rint(turns);  // exact, at most half a turn either way
        const uint64_t size = (uint64_t)(fabs(part) * 18446744073709551616.0);  // 2^64
        p.turn[i] = part < 0.0 ? 0 - size : size;
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
