// kv_weights_tc_f32.cu -- attention weights per cached key (kv_weights.cuh) for fp32 q and K
// on the 5th-generation tensor cores.
//
// Precision.  Each fp32 operand is split as x = hi + lo, hi with the 13 low mantissa bits
// cleared (a tf32 value) and lo the exact rest; a score is taken as
//   K_hi . Q_hi + (K_hi . Q_lo + K_lo . Q_hi),
// three tf32 products into fp32 accumulators, the small terms apart from the main one or
// before it: about 20 bits of each term, where a single tf32 product keeps 10.  Weights
// differ from 64-bit ones by 2e-7 to 6e-7 of their value.  An infinite element has no
// such parts (inf - inf): its key's weight is NaN, the other keys' are as ever.
//
// Layout as in the bf16 kernels: keys on M, one per TMEM lane, so that a thread sums along
// its own columns, and the split keys in tensor memory as A operands.
//
// weights_stream_tf32x3_kernel, few columns (decode, observer rows): 64 packed columns stay
//   in shared memory as rows of zeros, hi and lo parts; a CTA streams the keys of
//   its share of the context past them in slabs of 128 keys x 32 elements.  A slab arrives
//   raw by TMA (seven in flight: 112 KB), a converter thread splits its key's 128 bytes into
//   one of four TMEM slots, and two products make of it K_hi . [Q_hi | Q_lo] and
//   K_lo . [0 | Q_hi], main and small terms side by side.  Keeping the two sums apart costs
//   one addition per score in the epilogue and saves a third of the products.
//   Bound by K's bytes up to 16 columns (8 sequences x 8 kv heads x 16384 keys of 128: 88
//   us, 6.1 TB/s; head_dim 64: 58 us, 4.7 TB/s) and by the products at 64 (100 us).  More
//   columns take a launch per 64, which add up in order.
//
// weights_tf32x3_kernel, many columns (a prompt's rows): a CTA keeps 128 / D * 128 keys
//   (256 TMEM columns) and streams 128-row query tiles past them.  A tile arrives raw (TMA,
//   two slots); the converter warps split it, hi in place and lo into the one lo buffer.
//   The product that needs lo goes first, so the next tile is split while the other two run.
//   Two 128-column score buffers: at head_dim 64 one per key tile, at 128 they alternate
//   between query tiles, each with an epilogue warpgroup of its own.  Bound by the three
//   products next to the shared memory that they (B operand), the splitting and the loads
//   read and write: an 8192-row prompt of 32 heads over 8 kv heads of 128 takes 1.21 ms,
//   228 TFLOP/s of scores (9.9 ms with FFMA).
//
// Every mbarrier wait is bounded; a CTA that gives up records ATLAS_DEV_TIMEOUT, lets its
// copies and MMAs finish, frees TMEM and writes NaN.
#include "kv_weights_tc.cuh"

namespace atlas {
namespace {

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

// ---------------------------------------------------------------- few columns
template <int D>
struct StreamCfg {
    static constexpr int N = 64;                      // columns of one pass
    static constexpr int kSlabs = D / 32;
    static constexpr int kSlabBytes = BT * 128;       // 32 elements of 128 keys
    static constexpr int kQSlab = 3 * N * 128;        // 32 elements of zero, hi and lo rows
    static constexpr int S = 7;                       // raw slabs in flight
    static constexpr int kChunks = 4;                 // split slabs in TMEM
    static constexpr int kThreads = 512;
    static constexpr int OFF_Q = S * kSlabBytes;
    static constexpr int OFF_LSE = OFF_Q + kSlabs * kQSlab;
    static constexpr int OFF_LIM = OFF_LSE + N * 4;
    static constexpr int OFF_BAR = OFF_LIM + N * 4;
    static constexpr int B_FULL = 0, B_EMPTY = S;     // raw slab landed / split
    static constexpr int B_READY = 2 * S, B_FREE = B_READY + kChunks;  // split slab in TMEM / used
    static constexpr int B_SFULL = B_FREE + kChunks, B_SEMPTY = B_SFULL + 2;
    static constexpr int B_FINAL = B_SEMPTY + 2, kBars = B_FINAL + 1;
    static constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
    static constexpr int kSmem = OFF_TMEM + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
    // TMEM: split slab k at 64 k (hi, then lo); score buffer i at SCORES + 128 i, nmma
    // columns of main terms, then as many of small ones.
    static constexpr uint32_t SCORES = 64 * kChunks;
};

// grid (chunks of the context, Hkv, B).  The columns col0 .. col0 + 63 of the packed ones.
// Warps: 0 producer, 1 MMA issuer (and TMEM), 4-11 converters, 12-15 epilogue.
template <int D>
__global__ void __launch_bounds__(StreamCfg<D>::kThreads, 1)
    weights_stream_tf32x3_kernel(const __grid_constant__ CUtensorMap tmK, const WeightsParams p,
                                 const int chunk, const int col0) {
    using C = StreamCfg<D>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t sb = smem_u32(smem);
    float *nlse = reinterpret_cast<float *>(smem + C::OFF_LSE);
    int *lim = reinterpret_cast<int *>(smem + C::OFF_LIM);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_TMEM + 8);
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int b = blockIdx.z, hkv = blockIdx.y;
#define BAR(i) (sb + C::OFF_BAR + 8u * (uint32_t)(i))
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    const bool first_pass = col0 == 0, adds = p.accumulate || !first_pass;
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && first_pass) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    const int lp = 31 - __clz(p.P);
    const int first = (int)blockIdx.x * chunk, end = min(L, first + chunk);
    if (first >= end) return;
    float *w = p.weights + ((int64_t)b * p.Hkv + hkv) * p.row_tokens;
    // Keys below every row's window (or all of them, without rows) get nothing.
    const int ncols = min(C::N, p.G * qn - col0);
    const int seen = p.window > 0 ? min(end, max(first, L - qn + 1 - p.window)) : first;
    const int begin = ncols <= 0 ? end : max(first, seen / BT * BT);
    if (first_pass) {
        for (int pg = (first >> lp) + (int)threadIdx.x; pg <= (end - 1) >> lp; pg += C::kThreads) {
            const int id = p.page_table[(int64_t)b * p.max_pages + pg];
            if (id < 0 || id >= p.num_pages) record(p.status, ATLAS_DEV_BAD_PAGE);
        }
    }
    if (!adds)
        for (int t = first + (int)threadIdx.x; t < begin; t += C::kThreads)
            if (page_ok(p, b, t, lp)) w[t] = 0.f;
    if (begin >= end) return;
    const int tiles = (end - begin + BT - 1) / BT;
    const int nmma = (ncols + 15) / 16 * 16;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(BAR(C::B_FULL + s), 1);
            mbar_init(BAR(C::B_EMPTY + s), 4);
        }
        for (int k = 0; k < C::kChunks; ++k) {
            mbar_init(BAR(C::B_READY + k), 128);
            mbar_init(BAR(C::B_FREE + k), 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(BAR(C::B_SFULL + k), 1);
            mbar_init(BAR(C::B_SEMPTY + k), 128);
        }
        mbar_init(BAR(C::B_FINAL), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
    // The columns, packed (column c is row c % qn of head c / qn) and zero-filled to nmma:
    // nmma rows of zeros, then the hi parts, then the lo parts.
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    for (int i = threadIdx.x; i < nmma * (D / 4); i += C::kThreads) {
        const int c = i / (D / 4), ch = i % (D / 4), f = col0 + c;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < ncols)
            v = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                  (row0 + (int64_t)(f / qn) * p.q_len + f % qn) * D + ch * 4);
        const float4 h = make_float4(tf32_hi(v.x), tf32_hi(v.y), tf32_hi(v.z), tf32_hi(v.w));
        uint8_t *slab = smem + C::OFF_Q + (ch / 8) * C::kQSlab;
        *reinterpret_cast<float4 *>(slab + sw128(c, ch % 8)) = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(slab + sw128(nmma + c, ch % 8)) = h;
        *reinterpret_cast<float4 *>(slab + sw128(2 * nmma + c, ch % 8)) =
            make_float4(v.x - h.x, v.y - h.y, v.z - h.z, v.w - h.w);
    }
    for (int c = threadIdx.x; c < C::N; c += C::kThreads) {
        const bool real = c < ncols;
        const int f = col0 + c, i = real ? f % qn : 0;
        nlse[c] = real ? -lse_log2(p.lse[row0 + (int64_t)(f / qn) * p.q_len + i]) : -INFINITY;
        lim[c] = real ? L - qn + i + 1 : 0;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    bool failed = false;
    const int n_slabs = tiles * C::kSlabs;  // slab g: elements 32 (g % kSlabs) on of tile g / kSlabs

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) prefetch_tmap(&tmK);
        const uint64_t policy = policy_evict_first();
        PageIdCache pages{p.page_table + (int64_t)b * p.max_pages, (end - 1) >> lp};
        int issued = 0;
        for (int j = 0; j < tiles && !failed; ++j) {
            const int kb = begin + j * BT;
            const int nbox = (min(BT, end - kb) + p.P - 1) >> lp;  // <= 16
            const int id = pages.get_line(kb >> lp, lane < nbox ? lane : 0);
            const bool good = lane < nbox && id >= 0 && id < p.num_pages;
            const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, good));
            for (int sl = 0; sl < C::kSlabs; ++sl) {
                const int g = j * C::kSlabs + sl, s = g % S;
                if (g >= S && !wait_warp(BAR(C::B_EMPTY + s), (g / S - 1) & 1, abort_flag)) {
                    failed = true;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(BAR(C::B_FULL + s), (boxes << lp) * 128u);
                __syncwarp();
                if (good)
                    tma_load_2d_hint(sb + s * C::kSlabBytes + (lane << lp) * 128, &tmK, 32 * sl,
                                     (id * p.Hkv + hkv) << lp, BAR(C::B_FULL + s), policy);
                __syncwarp();
                issued = g + 1;
            }
        }
        if (failed && lane == 0) {
            *abort_flag = 1;
            int no_abort = 0;  // the copies in flight land before the CTA leaves
            for (int g = max(0, issued - S); g < issued; ++g)
                mbar_wait_bounded(BAR(C::B_FULL + g % S), (g / S) & 1, &no_abort, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        const uint32_t idesc = idesc_tf32_f32(128, 2 * nmma);
        const uint32_t q_hi = (uint32_t)nmma * 128 >> 4;  // the hi rows, in descriptor units
        bool ok = true;
        for (int g = 0; ok && g < n_slabs; ++g) {
            const int j = g / C::kSlabs, sl = g % C::kSlabs, buf = j & 1, k = g % C::kChunks;
            ok = wait_warp(BAR(C::B_READY + k), (g / C::kChunks) & 1, abort_flag);
            if (ok && sl == 0 && j >= 2)
                ok = wait_warp(BAR(C::B_SEMPTY + buf), (j / 2 - 1) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                // K_hi . [Q_hi | Q_lo] and K_lo . [0 | Q_hi] into [main | small] terms: only
                // products of one accumulator and one shape are sure to run in order, which
                // K_lo . Q_hi into the small columns alone would not be
                const uint32_t d = tmem + C::SCORES + buf * 128, a = tmem + 64 * k;
                const uint64_t qd = sdesc_sw128(sb + C::OFF_Q + sl * C::kQSlab, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_tf32_tmem_a(d, a + 8 * kk, qd + q_hi + 2 * kk, idesc, sl > 0 || kk > 0);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_tf32_tmem_a(d, a + 32 + 8 * kk, qd + 2 * kk, idesc, 1u);
                umma_commit(BAR(C::B_FREE + k));
                if (sl == C::kSlabs - 1) umma_commit(BAR(C::B_SFULL + buf));
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
    } else if (warp >= 4 && warp < 12) {
        // ------------------------------------------------------------ converters
        // Two warpgroups take turns at the slabs; a thread splits its key's 32 elements.
        const int q4 = warp % 4, r = q4 * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)(q4 * 32) << 16);
        for (int g = (warp - 4) / 4; g < n_slabs; g += 2) {
            const int s = g % S, k = g % C::kChunks;
            if (!wait_warp(BAR(C::B_FULL + s), (g / S) & 1, abort_flag)) {
                failed = true;
                break;
            }
            uint32_t h[32], l[32];
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
                const float4 v = *reinterpret_cast<const float4 *>(smem + s * C::kSlabBytes + sw128(r, ch));
                const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[4 * ch + e] = __float_as_uint(tf32_hi(x[e]));
                    l[4 * ch + e] = __float_as_uint(x[e] - tf32_hi(x[e]));
                }
            }
            if (g >= C::kChunks && !wait_warp(BAR(C::B_FREE + k), (g / C::kChunks - 1) & 1, abort_flag)) {
                failed = true;
                break;
            }
            tc_fence_after();
            tmem_st32(tl + 64 * k, h);
            tmem_st32(tl + 64 * k + 32, l);
            // Free the raw slab only now, its values in use: right after the loads, some were
            // still on their way when the copy of a later slab landed (a few keys wrong in a
            // million, most on cold data).
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_EMPTY + s));
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(BAR(C::B_READY + k));
        }
        if (failed && lane == 0) *abort_flag = 1;
    } else if (warp >= 12) {
        // ------------------------------------------------------------ epilogue
        const int q4 = warp % 4, r = q4 * 32 + lane;
        const int32_t *table = p.page_table + (int64_t)b * p.max_pages;
        // A tile's page id and old weight are read while the tile before is worked on.
        int id_next = 0;
        float old_next = 0.f;
        auto ahead = [&](int j) {
            const int t = begin + j * BT + r;
            if (t < end) {
                id_next = table[t >> lp];
                old_next = adds ? w[t] : 0.f;
            }
        };
        ahead(0);
        for (int j = 0; j < tiles; ++j) {
            const int buf = j & 1, kb = begin + j * BT, t = kb + r;
            const int id = id_next;
            const float old = old_next;
            ahead(j + 1);
            // a tile that every row sees whole needs no limits (padding columns are zero
            // rows: 0 times a non-finite key is not 0)
            const bool masked = kb + BT > L - qn + 1 || (p.window > 0 && kb < L - p.window) || ncols < nmma;
            if (!wait_warp(BAR(C::B_SFULL + buf), (j >> 1) & 1, abort_flag)) {
                failed = true;
                if (lane == 0) *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint32_t ts = tmem + C::SCORES + buf * 128 + ((uint32_t)(q4 * 32) << 16);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
            for (int c0 = 0; c0 < nmma; c0 += 16) {
                uint32_t v[16], u[16];
                tmem_ld16(ts + c0, v);
                tmem_ld16(ts + nmma + c0, u);
                tmem_wait_ld16(v);
                tmem_wait_ld16(u);
                if (c0 + 16 >= nmma) {  // all read: the next product may overwrite them
                    tc_fence_before();
                    mbar_arrive(BAR(C::B_SEMPTY + buf));
                }
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    v[c] = __float_as_uint(__uint_as_float(v[c]) + __uint_as_float(u[c]));
                add_weights<16>(p, v, nlse + c0, lim + c0, t, masked, sum);
            }
            const float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (t < end && id >= 0 && id < p.num_pages) w[t] = old + total;
        }
    }
    tc_fence_before();
    const bool any_failed = __syncthreads_or(failed) != 0;
    if (any_failed) {
        if (threadIdx.x == 0) record(p.status, ATLAS_DEV_TIMEOUT);
        for (int t = begin + (int)threadIdx.x; t < end; t += C::kThreads)
            if (page_ok(p, b, t, lp)) w[t] = __int_as_float(0x7fc00000);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
#undef BAR
}

template <int D>
cudaError_t launch_stream(const WeightsParams &p, int chunk_tiles, const CUtensorMap &tmK,
                          cudaStream_t stream) {
    using C = StreamCfg<D>;
    static int done[64] = {0};
    auto kern = weights_stream_tf32x3_kernel<D>;
    cudaError_t err = configure_smem(reinterpret_cast<const void *>(kern), C::kSmem, done);
    const int64_t ctx = (int64_t)p.max_pages * p.P, chunk = (int64_t)chunk_tiles * BT;
    const dim3 grid((unsigned)((ctx + chunk - 1) / chunk), (unsigned)p.Hkv, (unsigned)p.B);
    for (int col0 = 0; err == cudaSuccess && col0 < p.G * p.q_len; col0 += C::N) {
        kern<<<grid, C::kThreads, C::kSmem, stream>>>(tmK, p, (int)chunk, col0);
        err = cudaGetLastError();
    }
    return err;
}

// ---------------------------------------------------------------- many columns
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
// one group together.  Warps: 0 producer, 1 MMA issuer (and TMEM), 2 columns, 4-7
// converters, 8-15 epilogue (which bring the keys in first).
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
cudaError_t launch_d(const WeightsParams &p, const WeightsPlan &plan, const CUtensorMap &tmQ,
                     const CUtensorMap &tmK, cudaStream_t stream) {
    if (plan.stream) return launch_stream<D>(p, plan.chunk_tiles, tmK, stream);
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

cudaError_t launch_weights_tf32x3(const WeightsParams &p, const WeightsPlan &plan, int D,
                                  const CUtensorMap &tmQ, const CUtensorMap &tmK, cudaStream_t stream) {
    return D == 128 ? launch_d<128>(p, plan, tmQ, tmK, stream) : launch_d<64>(p, plan, tmQ, tmK, stream);
}

}  // namespace atlas
