// kv_weights_tc_f32.cu -- attention weights per cached key (kv_weights.cuh) for fp32 q and K
// with many columns, on the 5th-generation tensor cores.
//
// Precision.  Each fp32 operand is split as x = hi + lo, hi with the 13 low mantissa bits
// cleared (a tf32 value) and lo the exact rest; a score is taken as
//   K_hi . Q_lo + K_lo . Q_hi + K_hi . Q_hi,
// three tf32 products into one fp32 accumulator, small terms first: about 20 bits of each
// term, where a single tf32 product keeps 10.
//
// Layout as in the bf16 kernel: keys on M, one per TMEM lane, so that a thread sums along
// its own columns.  A CTA keeps 128 / D * 128 keys, hi and lo, in tensor memory (256
// columns) as A operands, and streams 128-row query tiles past them.  A tile arrives raw
// (TMA, two slots); the converter warps split it, hi in place and lo into the one lo
// buffer.  The product that needs lo goes first, so the next tile is split while the other
// two products run.  Two 128-column score buffers: at head_dim 64 one per key tile, at 128
// they alternate between query tiles, each with an epilogue warpgroup of its own.
//
// What bounds it: the three products, 3 x D / 8 x 65 cycles per 128 x 128 scores, next to
// the shared memory that they (B operand), the splitting and the loads read and write.
//
// Warps: 0 producer, 1 MMA issuer (and TMEM), 2 columns, 4-7 converters, 8-15 epilogue
// (which bring the keys in first).  Every mbarrier wait is bounded; a CTA that gives up
// records ATLAS_DEV_TIMEOUT, lets its copies and MMAs finish, frees TMEM and writes NaN.
#include "kv_weights_tc.cuh"

namespace atlas {
namespace {

template <int D>
struct Cfg {
    static constexpr int kKeyTiles = 128 / D;
    static constexpr int kKeys = kKeyTiles * BT;      // of a CTA: 128 or 256
    static constexpr int kTile = BT * D * 4;          // 128 query rows
    static constexpr int kSlabs = D / 32;             // 32-element (128-byte) slabs of a row
    static constexpr int kSlabBytes = BT * 128;
    static constexpr int kColSlots = 4;
    static constexpr int kThreads = 512;
    static constexpr int OFF_RAW = 0;                 // [2] raw tiles, then their hi parts
    static constexpr int OFF_LO = 2 * kTile;
    static constexpr int OFF_LSE = OFF_LO + kTile;
    static constexpr int OFF_LIM = OFF_LSE + kColSlots * BT * 4;
    static constexpr int OFF_INFO = OFF_LIM + kColSlots * BT * 4;
    static constexpr int OFF_SUM = OFF_INFO + kColSlots * 16;  // [128] the second group's sums
    static constexpr int OFF_BAR = OFF_SUM + BT * 4;
    static constexpr int B_K = 0;                     // [2] keys in TMEM (128 arrivals)
    static constexpr int B_QFULL = 2;                 // [2] raw tile landed
    static constexpr int B_SPLIT = 4;                 // [2] tile split (128 arrivals)
    static constexpr int B_QEMPTY = 6;                // [2] products done with the tile
    static constexpr int B_LOFREE = 8;                // products done with its lo part
    static constexpr int B_SFULL = 9, B_SEMPTY = 11;  // [2]
    static constexpr int B_CFULL = 13, B_CEMPTY = B_CFULL + kColSlots;
    static constexpr int B_FINAL = B_CEMPTY + kColSlots;
    static constexpr int kBars = B_FINAL + 1;
    static constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
    static constexpr int kSmem = OFF_TMEM + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
    // TMEM columns of key tile x: hi at 2 D x, lo D further; scores from 256 on.
    static constexpr uint32_t SCORES = 256;
};

__host__ __device__ constexpr uint32_t idesc_tf32_f32(int M, int N) {
    return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem desc] with tf32 operands.
__device__ __forceinline__ void umma_tf32_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float tf32_hi(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u);
}

// One of the three products of a key tile (columns k_tmem) and a query tile.
template <int D>
__device__ __forceinline__ void issue_product(uint32_t d_tmem, uint32_t k_tmem, uint32_t q_smem,
                                              uint32_t idesc, bool first) {
    const uint64_t qd = sdesc_sw128(q_smem, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 8; ++kk)
        umma_tf32_tmem_a(d_tmem, k_tmem + 8 * kk,
                         qd + (((kk >> 2) * Cfg<D>::kSlabBytes + (kk & 3) * 32) >> 4), idesc,
                         !first || kk > 0);
}

// grid: items, the key groups of every (sequence, kv head) in ascending order, the parts of
// one group together.
template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    weights_tf32x3_kernel(const __grid_constant__ CUtensorMap tmQ, const WeightsParams p) {
    using C = Cfg<D>;
    constexpr int KT = C::kKeyTiles;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t sb = smem_u32(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_TMEM + 8);
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
#define BAR(i) (sb + C::OFF_BAR + 8u * (uint32_t)(i))
    const int units = p.B * p.Hkv;
    const int part = (int)(blockIdx.x % (unsigned)p.n_parts);
    const int u = (int)(blockIdx.x / (unsigned)p.n_parts % (unsigned)units);
    const int kb0 = (int)(blockIdx.x / (unsigned)p.n_parts / (unsigned)units) * C::kKeys;
    const int b = u / p.Hkv, hkv = u % p.Hkv;
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && kb0 == 0 && part == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    if (kb0 >= L) return;
    const int lp = 31 - __clz(p.P);
    const int end = min(L, kb0 + C::kKeys);
    const int nq = (p.G * p.q_len + BT - 1) / BT;
    const int q_begin = part * p.tiles_per_part, q_end = min(nq, q_begin + p.tiles_per_part);
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    const int ktiles = (end - kb0 + BT - 1) / BT;

    if (threadIdx.x == 0) {
        for (int k = 0; k < 2; ++k) {
            mbar_init(BAR(C::B_K + k), 128);
            mbar_init(BAR(C::B_QFULL + k), 1);
            mbar_init(BAR(C::B_SPLIT + k), 128);
            mbar_init(BAR(C::B_QEMPTY + k), 1);
            mbar_init(BAR(C::B_SFULL + k), 1);
            mbar_init(BAR(C::B_SEMPTY + k), 128);
        }
        mbar_init(BAR(C::B_LOFREE), 1);
        for (int s = 0; s < C::kColSlots; ++s) {
            mbar_init(BAR(C::B_CFULL + s), 1);
            mbar_init(BAR(C::B_CEMPTY + s), 4 * KT);  // a warpgroup per key tile, or one in turn
        }
        mbar_init(BAR(C::B_FINAL), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    bool failed = false;
    QueryTiles q(p, L, qn, kb0, C::kKeys, q_begin, q_end);
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) prefetch_tmap(&tmQ);
        const uint64_t keep = policy_evict_last();  // other CTAs read the same queries
        int issued = 0;
        while (q.next()) {
            const int s = q.n & 1;
            if (q.n >= 2 && !wait_warp(BAR(C::B_QEMPTY + s), ((q.n >> 1) - 1) & 1, abort_flag)) {
                failed = true;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(BAR(C::B_QFULL + s), C::kTile);
#pragma unroll
                for (int sl = 0; sl < C::kSlabs; ++sl)
                    tma_load_2d_hint(sb + C::OFF_RAW + s * C::kTile + sl * C::kSlabBytes, &tmQ, 32 * sl,
                                     (int)(row0 + q.j * BT), BAR(C::B_QFULL + s), keep);
            }
            issued = q.n + 1;
        }
        if (failed && lane == 0) {
            *abort_flag = 1;
            int no_abort = 0;  // the copies in flight land before the CTA leaves
            for (int k = max(0, issued - 2); k < issued; ++k)
                mbar_wait_bounded(BAR(C::B_QFULL + (k & 1)), (k >> 1) & 1, &no_abort, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc = idesc_tf32_f32(128, 128);
        bool ok = true;
        int used[2] = {0, 0};  // times each score buffer was written
        while (ok && q.next()) {
            const int s = q.n & 1;
            ok = wait_warp(BAR(C::B_SPLIT + s), (q.n >> 1) & 1, abort_flag);
            bool on[KT];
#pragma unroll
            for (int x = 0; x < KT; ++x) {
                const int buf = KT == 2 ? x : s;
                on[x] = ok && x < ktiles && q.seen(kb0 + x * BT, BT);
                if (!on[x]) continue;
                if (used[buf] == 0 || (KT == 1 && q.n < 2)) ok = wait_warp(BAR(C::B_K + x), 0, abort_flag);
                if (ok && used[buf] > 0)
                    ok = wait_warp(BAR(C::B_SEMPTY + buf), (used[buf] - 1) & 1, abort_flag);
                ++used[buf];
            }
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t hi = sb + C::OFF_RAW + s * C::kTile, lo = sb + C::OFF_LO;
#pragma unroll
                for (int x = 0; x < KT; ++x)
                    if (on[x])
                        issue_product<D>(tmem + C::SCORES + (KT == 2 ? x : s) * BT, tmem + 2 * D * x, lo,
                                         idesc, true);
                umma_commit(BAR(C::B_LOFREE));
#pragma unroll
                for (int x = 0; x < KT; ++x)
                    if (on[x]) {
                        const uint32_t d = tmem + C::SCORES + (KT == 2 ? x : s) * BT;
                        issue_product<D>(d, tmem + 2 * D * x + D, hi, idesc, false);
                        issue_product<D>(d, tmem + 2 * D * x, hi, idesc, false);
                        umma_commit(BAR(C::B_SFULL + (KT == 2 ? x : s)));
                    }
                umma_commit(BAR(C::B_QEMPTY + s));
            }
            __syncwarp();
        }
        if (!ok) {
            failed = true;
            *abort_flag = 1;
        }
        // every MMA is done before TMEM is released
        if (elect_one()) umma_commit(BAR(C::B_FINAL));
        int no_abort = 0;
        mbar_wait_bounded(BAR(C::B_FINAL), 0, &no_abort, kWaitLimitNs);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ lse and limits
        // (at head_dim 128 the warpgroups take turns: each meets a stop of its own)
        failed = !bring_columns<C::kColSlots>(p, q, row0, smem, C::OFF_LSE, C::OFF_LIM, C::OFF_INFO,
                                              BAR(C::B_CFULL), BAR(C::B_CEMPTY), 2, abort_flag);
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ converters
        const int i = (int)threadIdx.x - 128;
        while (q.next()) {
            const int s = q.n & 1;
            if (!wait_warp(BAR(C::B_QFULL + s), (q.n >> 1) & 1, abort_flag) ||
                (q.n > 0 && !wait_warp(BAR(C::B_LOFREE), (q.n - 1) & 1, abort_flag))) {
                failed = true;
                if (lane == 0) *abort_flag = 1;
                break;
            }
            float4 *raw = reinterpret_cast<float4 *>(smem + C::OFF_RAW + s * C::kTile);
            float4 *lo = reinterpret_cast<float4 *>(smem + C::OFF_LO);
#pragma unroll 4
            for (int k = i; k < C::kTile / 16; k += 128) {
                const float4 x = raw[k];
                const float4 h = make_float4(tf32_hi(x.x), tf32_hi(x.y), tf32_hi(x.z), tf32_hi(x.w));
                raw[k] = h;
                lo[k] = make_float4(x.x - h.x, x.y - h.y, x.z - h.z, x.w - h.w);
            }
            fence_proxy_async_smem();
            mbar_arrive(BAR(C::B_SPLIT + s));
        }
    } else if (warp >= 8) {
        // ------------------------------------------------------------ epilogue
        const int group = (warp - 8) / 4, q4 = warp % 4;
        const int x = KT == 2 ? group : 0;  // this warpgroup's key tile
        const int r = q4 * 32 + lane, kb = kb0 + x * BT, t = kb + r;
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        const int id = t < end ? p.page_table[(int64_t)b * p.max_pages + (t >> lp)] : -1;
        const bool good = id >= 0 && id < p.num_pages;
        if (t < end && !good && part == 0) record(p.status, ATLAS_DEV_BAD_PAGE);
        // This thread's key, split, into its lane of tensor memory; zeros past the end or on
        // a bad page.  (At head_dim 128 the first warpgroup brings the one tile.)
        if (x < ktiles && (KT == 2 || group == 0)) {
            const float4 *src = reinterpret_cast<const float4 *>(
                static_cast<const float *>(p.k_pages) +
                (good ? (((int64_t)id * p.Hkv + hkv) * p.P + (t & (p.P - 1))) * D : 0));
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t h[32], l[32];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 v = good ? src[c0 / 4 + e] : make_float4(0.f, 0.f, 0.f, 0.f);
                    const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[4 * e + k] = __float_as_uint(tf32_hi(w[k]));
                        l[4 * e + k] = __float_as_uint(w[k] - tf32_hi(w[k]));
                    }
                }
                tmem_st32(tl + 2 * D * x + c0, h);
                tmem_st32(tl + 2 * D * x + D + c0, l);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(BAR(C::B_K + x));
        }
        const uint32_t ts = tl + C::SCORES + group * BT;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        int used = 0;
        for (int n = KT == 2 ? 0 : group;; n += KT == 2 ? 1 : 2) {
            const int s = n % C::kColSlots;
            if (!wait_warp(BAR(C::B_CFULL + s), (n / C::kColSlots) & 1, abort_flag)) {
                failed = true;
                break;
            }
            const TileInfo info = reinterpret_cast<const TileInfo *>(smem + C::OFF_INFO)[s];
            if (info.stop) break;
            if (x < ktiles && sees(p, info.lim_min, info.lim_max, kb, BT)) {
                if (!wait_warp(BAR(C::B_SFULL + group), used & 1, abort_flag)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const bool masked = !info.whole || kb + BT > info.lim_min ||
                                    (p.window > 0 && kb < info.lim_max - p.window);
                const float *nlse = reinterpret_cast<const float *>(smem + C::OFF_LSE) + s * BT;
                const int *lim = reinterpret_cast<const int *>(smem + C::OFF_LIM) + s * BT;
#pragma unroll 1
                for (int c0 = 0; c0 < BT; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(ts + c0, v);
                    tmem_wait_ld32(v);
                    if (c0 == BT - 32) {  // all read: the next product may overwrite them
                        tc_fence_before();
                        mbar_arrive(BAR(C::B_SEMPTY + group));
                    }
                    add_weights<32>(p, v, nlse + c0, lim + c0, t, masked, sum);
                }
                ++used;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_CEMPTY + s));
        }
        if (failed && lane == 0) *abort_flag = 1;
        float total = failed ? __int_as_float(0x7fc00000)
                             : (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (KT == 1) {  // the two warpgroups' shares of the same key
            float *other = reinterpret_cast<float *>(smem + C::OFF_SUM) + r;
            if (group == 1) *other = total;
            group_barrier(1, 256);
            if (group == 0) total += *other;
        }
        if (t < end && good && (KT == 2 || group == 0)) {
            if (p.n_parts > 1) {
                p.parts[((int64_t)part * units + u) * ((int64_t)p.max_pages * p.P) + t] = total;
            } else {
                float *w = p.weights + (int64_t)u * p.row_tokens + t;
                *w = (p.accumulate ? *w : 0.f) + total;
            }
        }
    }
    tc_fence_before();
    const bool any_failed = __syncthreads_or(failed) != 0;
    if (any_failed && threadIdx.x == 0) record(p.status, ATLAS_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
#undef BAR
}

template <int D>
cudaError_t launch_d(const WeightsParams &p, const CUtensorMap &tmQ, cudaStream_t stream) {
    using C = Cfg<D>;
    static int done[64] = {0};
    auto kern = weights_tf32x3_kernel<D>;
    cudaError_t err = configure_smem(reinterpret_cast<const void *>(kern), C::kSmem, done);
    if (err != cudaSuccess) return err;
    const int64_t ctx = (int64_t)p.max_pages * p.P, units = (int64_t)p.B * p.Hkv;
    const int64_t items = (ctx + C::kKeys - 1) / C::kKeys * units * p.n_parts;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    kern<<<(unsigned)items, C::kThreads, C::kSmem, stream>>>(tmQ, p);
    err = cudaGetLastError();
    return err == cudaSuccess && p.n_parts > 1 ? launch_weights_join(p, stream) : err;
}

}  // namespace

cudaError_t launch_weights_tf32x3(const WeightsParams &p, int D, const CUtensorMap &tmQ,
                                  cudaStream_t stream) {
    return D == 128 ? launch_d<128>(p, tmQ, stream) : launch_d<64>(p, tmQ, stream);
}

}  // namespace atlas
