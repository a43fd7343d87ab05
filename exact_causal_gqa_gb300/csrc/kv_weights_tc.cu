// kv_weights_tc.cu -- attention weights per cached key (kv_weights.cuh) for bf16 q and K
// on the 5th-generation tensor cores.
//
// The keys go on M: S^T[128 keys x N columns] = K . Q^T lands in tensor memory with one
// key per lane, so the sum over columns that the operator wants runs along the lane's
// TMEM columns: each epilogue thread owns one key, reads its scores, exponentiates
// (2^(s scale log2 e - lse log2 e): one packed FMA and one MUFU exponential per score) and
// adds in a register.  No shuffles, no atomics, no second pass; the order of a key's sum
// depends only on the call's sizes.
//
// weights_stream_kernel, at most 256 columns (decode, observer rows): the columns stay in
//   shared memory, packed so that only real rows take part, and a CTA streams the 128-key
//   tiles of its share of the context past them.  Bound by K's bytes up to 128 columns: 8
//   sequences x 8 kv heads x 32768 keys of 128 (537 MB) take 82 us with up to 32 columns
//   (6.5 TB/s), 91 with 64, 95 with 128; beyond, products, exponentials and loads no longer
//   fit side by side: 115 us with 192, 132 with 256 (leaving out the exponentials 123, the
//   products 126, both 102).
// weights_tile_kernel, more columns (a prompt's rows): a CTA keeps 512 keys (four tiles)
//   and streams 128-row query tiles past them, each loaded once for four products; query
//   tiles no key of the CTA is visible to are not loaded.  Bound by the products (operands
//   from shared memory: 65 clocks per 128 x 128 x 16, as long as one of 64 columns) and the
//   exponentials, each busy 54 % of the time: an 8192-row prompt of 32 heads over 8 kv heads
//   of 128 takes 222 us, 1.24 PFLOP/s of scores.  When (sequence, kv head) x 512-key groups
//   alone would not fill the GPU, the query tiles are split between CTAs; their sums per key
//   go to the workspace and weights_join_kernel adds them in order.
//
// Keys on a bad page, or behind the end, only fill lanes of their own, whose results are
// dropped.  Every mbarrier wait is bounded; a CTA that gives up records
// ATLAS_DEV_TIMEOUT, lets its copies and MMAs finish, frees TMEM and writes NaN.
#include "kv_weights_tc.cuh"

namespace atlas {
namespace {

// One tile of 128 keys from kb (keys below `end`) into shared memory, page by page; the
// whole warp calls it.  Boxes of bad pages are left out (`bar` counts the others' bytes).
template <int D>
__device__ __forceinline__ void load_keys(const WeightsParams &p, const CUtensorMap &tmK,
                                          PageIdCache &pages, int hkv, int kb, int end, int lp,
                                          uint32_t dst, uint32_t bar, uint64_t policy) {
    const int lane = threadIdx.x & 31;
    const int nbox = (min(BT, end - kb) + p.P - 1) >> lp;  // <= 16
    const int id = pages.get_line(kb >> lp, lane < nbox ? lane : 0);
    const bool good = lane < nbox && id >= 0 && id < p.num_pages;
    const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, good));
    if (lane == 0) mbar_arrive_expect_tx(bar, (boxes << lp) * 128u * (D / 64));
    __syncwarp();
    if (good) {
        const int y = (id * p.Hkv + hkv) << lp;
#pragma unroll
        for (int sl = 0; sl < D / 64; ++sl)
            tma_load_2d_hint(dst + sl * kSlab + (lane << lp) * 128, &tmK, 64 * sl, y, bar, policy);
    }
    __syncwarp();
}

// S^T[128 x n] of one key tile and a query tile of n rows (K-major, 128-byte swizzle;
// its 64-element slabs q_slab bytes apart).
template <int D>
__device__ __forceinline__ void issue_scores(uint32_t d_tmem, uint32_t k_smem, uint32_t q_smem,
                                             uint32_t q_slab, uint32_t idesc) {
    const uint64_t kd = sdesc_sw128(k_smem, 16, 1024), qd = sdesc_sw128(q_smem, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        umma_bf16(d_tmem, kd + (((kk >> 2) * kSlab + (kk & 3) * 32) >> 4),
                  qd + (((kk >> 2) * q_slab + (kk & 3) * 32) >> 4), idesc, kk > 0);
}

// ---------------------------------------------------------------- few columns
template <int D, int N>
struct StreamCfg {
    static constexpr int kTile = BT * D * 2;
    static constexpr int kQ = N * D * 2;
    // Up to 32 columns two CTAs share an SM (one's start-up hides behind the other);
    // beyond, the accumulators and queries leave room for one with a deeper ring.
    static constexpr int kCtas = N <= 32 ? 2 : 1;
    static constexpr int kStages = (N <= 32 ? 3 : N <= 128 ? 5 : 4) * (128 / D);
    // Epilogue warpgroups: kGroups that take turns at the tiles, of kHalves that share a
    // tile's columns.  From 64 columns on each has a score buffer and products of its own,
    // so that four of them keep the exponential unit busy while products are under way
    // (64 sequences x heads, 413K keys, 256 columns: 207 us; 237 us with two 256-column
    // buffers); fewer columns need one warpgroup, with two buffers.
    static constexpr int kGroups = N >= 256 ? 2 : N >= 64 ? 4 : 1;
    static constexpr int kHalves = N >= 256 ? 2 : 1;
    static constexpr int kBufs = kGroups == 1 ? 2 : kGroups;  // score buffers of a half
    static constexpr int kPart = N / kHalves;                 // columns of a half
    static constexpr int kThreads = 128 + 128 * kGroups * kHalves;
    static constexpr uint32_t kCols = kBufs * N < 32 ? 32 : kBufs * N;  // TMEM
    static constexpr int OFF_Q = kStages * kTile;
    static constexpr int OFF_LSE = OFF_Q + kQ;
    static constexpr int OFF_LIM = OFF_LSE + N * 4;
    static constexpr int OFF_HALF = OFF_LIM + N * 4;  // [kGroups][128] the second halves' sums
    static constexpr int OFF_BAR = OFF_HALF + (kHalves == 2 ? kGroups * BT * 4 : 0);
    static constexpr int B_FULL = 0, B_EMPTY = kStages, B_SFULL = 2 * kStages,
                         B_SEMPTY = B_SFULL + kBufs * kHalves,
                         B_FINAL = B_SEMPTY + kBufs * kHalves, kBars = B_FINAL + 1;
    static constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
    static constexpr int kSmem = OFF_TMEM + 16 + 1024;
    static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory of an SM");
};

// grid (chunks of the context, Hkv, B)
template <int D, int N>
__global__ void __launch_bounds__(StreamCfg<D, N>::kThreads, StreamCfg<D, N>::kCtas)
    weights_stream_kernel(const __grid_constant__ CUtensorMap tmK, const WeightsParams p,
                          const int chunk) {
    using C = StreamCfg<D, N>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset: the compiler still sees shared memory, not a generic address
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
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && blockIdx.x == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    const int lp = 31 - __clz(p.P);
    const int first = (int)blockIdx.x * chunk, end = min(L, first + chunk);
    if (first >= end) return;
    float *w = p.weights + ((int64_t)b * p.Hkv + hkv) * p.row_tokens;
    // Keys below every row's window (or all of them, without rows) get nothing.
    const int seen = qn == 0 ? end : p.window > 0 ? min(end, max(first, L - qn + 1 - p.window)) : first;
    const int begin = qn == 0 ? end : seen / BT * BT < first ? first : seen / BT * BT;
    for (int pg = (first >> lp) + (int)threadIdx.x; pg <= (end - 1) >> lp; pg += blockDim.x) {
        const int id = p.page_table[(int64_t)b * p.max_pages + pg];
        if (id < 0 || id >= p.num_pages) record(p.status, ATLAS_DEV_BAD_PAGE);
    }
    if (!p.accumulate)
        for (int t = first + (int)threadIdx.x; t < begin; t += blockDim.x)
            if (page_ok(p, b, t, lp)) w[t] = 0.f;
    if (begin >= end) return;
    const int tiles = (end - begin + BT - 1) / BT;
    const int ncols = p.G * qn;                  // packed: column c is row c % qn of head c / qn
    constexpr int kStep = N == 16 ? 16 : 32;     // columns of one TMEM load
    const int nmma = (ncols + kStep - 1) / kStep * kStep;
    const int halves = nmma > C::kPart ? 2 : 1;  // in use (kHalves at most)

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(BAR(C::B_FULL + s), 1);
            mbar_init(BAR(C::B_EMPTY + s), 1);
        }
        for (int s = 0; s < C::kBufs * C::kHalves; ++s) {
            mbar_init(BAR(C::B_SFULL + s), 1);
            mbar_init(BAR(C::B_SEMPTY + s), 128);
        }
        mbar_init(BAR(C::B_FINAL), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), C::kCols);
    // The columns: rows packed and zero-filled to the product's N, their lse and limits.
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    for (int i = threadIdx.x; i < nmma * (D / 8); i += C::kThreads) {
        const int c = i / (D / 8), ch = i % (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c < ncols)
            v = *reinterpret_cast<const uint4 *>(
                static_cast<const __nv_bfloat16 *>(p.q) +
                (row0 + (int64_t)(c / qn) * p.q_len + c % qn) * D + ch * 8);
        st_shared_v4(sb + C::OFF_Q + (ch / 8) * (N * 128) + sw128(c, ch % 8), v.x, v.y, v.z, v.w);
    }
    for (int c = threadIdx.x; c < N; c += C::kThreads) {
        const bool real = c < ncols;
        const int i = real ? c % qn : 0;
        nlse[c] = real ? -lse_log2(p.lse[row0 + (int64_t)(c / qn) * p.q_len + i]) : -INFINITY;
        lim[c] = real ? L - qn + i + 1 : 0;
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(*tmem_slot);
    bool failed = false;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) prefetch_tmap(&tmK);
        const uint64_t policy = policy_evict_first();
        PageIdCache pages{p.page_table + (int64_t)b * p.max_pages, (end - 1) >> lp};
        int issued = 0;
        for (int j = 0; j < tiles; ++j) {
            const int s = j % S;
            if (j >= S && !wait_warp(BAR(C::B_EMPTY + s), ((j / S) - 1) & 1, abort_flag)) {
                failed = true;
                break;
            }
            load_keys<D>(p, tmK, pages, hkv, begin + j * BT, end, lp, sb + s * C::kTile,
                         BAR(C::B_FULL + s), policy);
            issued = j + 1;
        }
        if (failed && lane == 0) {
            *abort_flag = 1;
            int no_abort = 0;  // the copies in flight land before the CTA leaves
            for (int j = max(0, issued - S); j < issued; ++j)
                mbar_wait_bounded(BAR(C::B_FULL + j % S), (j / S) & 1, &no_abort, kWaitLimitNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // (nmma columns in all; the last half used may have fewer than kPart)
        const uint32_t idesc = idesc_bf16_f32(128, min(nmma, C::kPart), false);
        const uint32_t idesc1 = idesc_bf16_f32(128, max(nmma - C::kPart, 16), false);
        bool ok = true;
        for (int j = 0; ok && j < tiles; ++j) {
            const int s = j % S, buf = j % C::kBufs;
            ok = wait_warp(BAR(C::B_FULL + s), (j / S) & 1, abort_flag);
#pragma unroll
            for (int half = 0; half < C::kHalves; ++half) {
                if (!ok || half >= halves) continue;
                const int i = buf * C::kHalves + half;
                if (j >= C::kBufs)
                    ok = wait_warp(BAR(C::B_SEMPTY + i), (j / C::kBufs - 1) & 1, abort_flag);
                if (!ok) continue;
                tc_fence_after();
                if (elect_one()) {
                    issue_scores<D>(tmem + i * C::kPart, sb + s * C::kTile,
                                    sb + C::OFF_Q + half * C::kPart * 128, N * 128,
                                    half ? idesc1 : idesc);
                    umma_commit(BAR(C::B_SFULL + i));
                    if (half == halves - 1) umma_commit(BAR(C::B_EMPTY + s));
                }
                __syncwarp();
            }
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
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        const int group = (warp - 4) / 4 % C::kGroups, half = (warp - 4) / 4 / C::kGroups;
        const int q4 = warp % 4, r = q4 * 32 + lane;
        const int c_begin = half * C::kPart, c_end = min(nmma, c_begin + C::kPart);
        float *other = reinterpret_cast<float *>(smem + C::OFF_HALF) + group * BT + r;
        const int32_t *table = p.page_table + (int64_t)b * p.max_pages;
        // A tile's page id and old weight are read while the tile before is worked on (one
        // after the other and in the loop, they were its longest step).
        const bool reads = half == 0;
        int id = 0, id_next = 0;
        float old = 0.f, old_next = 0.f;
        auto ahead = [&](int j) {
            const int t = begin + j * BT + r;
            if (reads && t < end) {
                id_next = table[t >> lp];
                old_next = p.accumulate ? w[t] : 0.f;
            }
        };
        ahead(group);
        for (int j = half < halves ? group : tiles; j < tiles; j += C::kGroups) {
            const int buf = j % C::kBufs * C::kHalves + half;
            const int kb = begin + j * BT, t = kb + r;
            id = id_next;
            old = old_next;
            ahead(j + C::kGroups);
            // a tile that every row sees whole needs no limits
            const bool masked = kb + BT > L - qn + 1 || (p.window > 0 && kb < L - p.window);
            if (!wait_warp(BAR(C::B_SFULL + buf), (j / C::kBufs) & 1, abort_flag)) {
                failed = true;
                *abort_flag = 1;
            }
            tc_fence_after();
            const uint32_t ts = tmem + buf * C::kPart + ((uint32_t)(q4 * 32) << 16);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // (padding columns are zero rows: 0 times a non-finite key is not 0)
            if (N == 16) {
                uint32_t s[16];
                tmem_ld16(ts, s);
                tmem_wait_ld16(s);
                tc_fence_before();
                mbar_arrive(BAR(C::B_SEMPTY + buf));
                add_weights<16>(p, s, nlse, lim, t, masked || ncols < 16, sum);
            } else {
#pragma unroll 1
                for (int c0 = c_begin; c0 < c_end; c0 += 64) {
                    const bool two = c0 + 32 < c_end;
                    uint32_t s[32], u[32];
                    tmem_ld32(ts + c0 - c_begin, s);
                    if (two) tmem_ld32(ts + c0 - c_begin + 32, u);
                    tmem_wait_ld32(s);
                    if (two) tmem_wait_ld32(u);
                    if (c0 + 64 >= c_end) {
                        // all read: the next product overwrites them meanwhile
                        tc_fence_before();
                        mbar_arrive(BAR(C::B_SEMPTY + buf));
                    }
                    add_weights<32>(p, s, nlse + c0, lim + c0, t, masked || c0 + 32 > ncols, sum);
                    if (two)
                        add_weights<32>(p, u, nlse + c0 + 32, lim + c0 + 32, t,
                                        masked || c0 + 64 > ncols, sum);
                }
            }
            float total = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (C::kHalves == 2 && halves == 2) {
                // the second half's sum through shared memory: written, read, free again
                if (half == 1) *other = total;
                group_barrier(1 + group, 256);
                if (half == 0) total += *other;
                group_barrier(1 + group, 256);
            }
            if (reads && t < end && id >= 0 && id < p.num_pages && !failed) w[t] = old + total;
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
        tmem_dealloc(tmem, C::kCols);
    }
#undef BAR
}

// ---------------------------------------------------------------- many columns
constexpr int kTiles = 4;                // key tiles of a CTA
constexpr int kGroupKeys = kTiles * BT;  // 512

template <int D>
struct TileCfg {
    static constexpr int kTile = BT * D * 2;  // 128 rows of K or Q
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int kThreads = 128 + 128 * kTiles;
    static constexpr int OFF_Q = kTiles * kTile;
    static constexpr int OFF_LSE = OFF_Q + kStages * kTile;    // [kStages][128]
    static constexpr int OFF_LIM = OFF_LSE + kStages * BT * 4;  // [kStages][128]
    static constexpr int OFF_INFO = OFF_LIM + kStages * BT * 4;  // [kStages] TileInfo
    static constexpr int OFF_BAR = OFF_INFO + kStages * 16;
    static constexpr int B_K = 0;
    static constexpr int B_QFULL = B_K + kTiles;
    static constexpr int B_QEMPTY = B_QFULL + kStages;
    static constexpr int B_CFULL = B_QEMPTY + kStages;   // the tile's lse and limits
    static constexpr int B_CEMPTY = B_CFULL + kStages;   // one arrival per epilogue warp
    static constexpr int B_SFULL = B_CEMPTY + kStages;
    static constexpr int B_SEMPTY = B_SFULL + kTiles;
    static constexpr int B_FINAL = B_SEMPTY + kTiles;
    static constexpr int kBars = B_FINAL + 1;
    static constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
    static constexpr int kSmem = OFF_TMEM + 16 + 1024;
    static_assert(kSmem <= 232448, "shared memory budget");
};

// grid: items, the key groups of every (sequence, kv head) in ascending order (under a
// causal mask the first groups have the most rows), the parts of one group together.
template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1)
    weights_tile_kernel(const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmK, const WeightsParams p) {
    using C = TileCfg<D>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset: the compiler still sees shared memory, not a generic address
    uint8_t *smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    const uint32_t sb = smem_u32(smem);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_TMEM);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_TMEM + 8);
    const int warp = uniform((int)threadIdx.x >> 5), lane = threadIdx.x & 31;
#define BAR(i) (sb + C::OFF_BAR + 8u * (uint32_t)(i))
    const int units = p.B * p.Hkv;
    const int part = (int)(blockIdx.x % (unsigned)p.n_parts);
    const int u = (int)(blockIdx.x / (unsigned)p.n_parts % (unsigned)units);
    const int kb0 = (int)(blockIdx.x / (unsigned)p.n_parts / (unsigned)units) * kGroupKeys;
    const int b = u / p.Hkv, hkv = u % p.Hkv;
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bad_lens(p, L, qn)) {
        if (threadIdx.x == 0 && kb0 == 0 && part == 0) record(p.status, ATLAS_DEV_BAD_SEQLEN);
        return;
    }
    if (kb0 >= L) return;
    const int lp = 31 - __clz(p.P);
    const int end = min(L, kb0 + kGroupKeys);
    for (int pg = (kb0 >> lp) + (int)threadIdx.x; pg <= (end - 1) >> lp; pg += blockDim.x) {
        const int id = p.page_table[(int64_t)b * p.max_pages + pg];
        if (id < 0 || id >= p.num_pages) record(p.status, ATLAS_DEV_BAD_PAGE);
    }
    const int nq = (p.G * p.q_len + BT - 1) / BT;
    const int q_begin = part * p.tiles_per_part, q_end = min(nq, q_begin + p.tiles_per_part);
    const int64_t row0 = ((int64_t)b * p.Hq + (int64_t)hkv * p.G) * p.q_len;
    const int ktiles = (end - kb0 + BT - 1) / BT;

    if (threadIdx.x == 0) {
        for (int x = 0; x < kTiles; ++x) {
            mbar_init(BAR(C::B_K + x), 1);
            mbar_init(BAR(C::B_SFULL + x), 1);
            mbar_init(BAR(C::B_SEMPTY + x), 128);
        }
        for (int s = 0; s < S; ++s) {
            mbar_init(BAR(C::B_QFULL + s), 1);
            mbar_init(BAR(C::B_QEMPTY + s), 1);
            mbar_init(BAR(C::B_CFULL + s), 1);
            mbar_init(BAR(C::B_CEMPTY + s), 4 * kTiles);
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
    QueryTiles q(p, L, qn, kb0, kGroupKeys, q_begin, q_end);
    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&tmQ);
            prefetch_tmap(&tmK);
        }
        const uint64_t keep = policy_evict_last();  // other CTAs read the same K and Q
        PageIdCache pages{p.page_table + (int64_t)b * p.max_pages, (end - 1) >> lp};
        int issued = 0;
        for (int x = 0; x < ktiles; ++x)
            load_keys<D>(p, tmK, pages, hkv, kb0 + x * BT, end, lp, sb + x * C::kTile,
                         BAR(C::B_K + x), keep);
        while (q.next()) {
            const int s = q.n % S;
            if (q.n >= S && !wait_warp(BAR(C::B_QEMPTY + s), ((q.n / S) - 1) & 1, abort_flag)) {
                failed = true;
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(BAR(C::B_QFULL + s), C::kTile);
#pragma unroll
                for (int sl = 0; sl < D / 64; ++sl)
                    tma_load_2d_hint(sb + C::OFF_Q + s * C::kTile + sl * kSlab, &tmQ, 64 * sl,
                                     (int)(row0 + q.j * BT), BAR(C::B_QFULL + s), keep);
            }
            issued = q.n + 1;
        }
        if (lane == 0) {
            // Nothing is in flight when the CTA leaves: K tiles that no product waited for
            // (a part without rows for them), and after an abort the queries too.
            int no_abort = 0;
            for (int x = 0; x < ktiles; ++x)
                mbar_wait_bounded(BAR(C::B_K + x), 0, &no_abort, kWaitLimitNs);
            if (failed) {
                *abort_flag = 1;
                for (int k = max(0, issued - S); k < issued; ++k)
                    mbar_wait_bounded(BAR(C::B_QFULL + k % S), (k / S) & 1, &no_abort, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false);
        bool ok = true;
        int used[kTiles] = {0, 0, 0, 0};  // products so far of each key tile
        while (ok && q.next()) {
            const int s = q.n % S;
            ok = wait_warp(BAR(C::B_QFULL + s), (q.n / S) & 1, abort_flag);
            if (!ok) break;
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
                if (!ok || x >= ktiles || !q.seen(kb0 + x * BT, BT)) continue;
                ok = used[x] == 0 ? wait_warp(BAR(C::B_K + x), 0, abort_flag)
                                  : wait_warp(BAR(C::B_SEMPTY + x), (used[x] - 1) & 1, abort_flag);
                if (!ok) continue;
                tc_fence_after();
                if (elect_one()) {
                    issue_scores<D>(tmem + x * BT, sb + x * C::kTile, sb + C::OFF_Q + s * C::kTile,
                                    kSlab, idesc);
                    umma_commit(BAR(C::B_SFULL + x));
                }
                __syncwarp();
                ++used[x];
            }
            if (elect_one()) umma_commit(BAR(C::B_QEMPTY + s));
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
        failed = !bring_columns<S>(p, q, row0, smem, C::OFF_LSE, C::OFF_LIM, C::OFF_INFO,
                                   BAR(C::B_CFULL), BAR(C::B_CEMPTY), 1, abort_flag);
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        const int x = (warp - 4) / 4, q4 = warp % 4;
        const int kb = kb0 + x * BT, t = kb + q4 * 32 + lane;
        const uint32_t ts = tmem + x * BT + ((uint32_t)(q4 * 32) << 16);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        int used = 0;
        for (int n = 0;; ++n) {
            const int s = n % S;
            // (also for a tile this warpgroup skips: it frees the slot like the others)
            if (!wait_warp(BAR(C::B_CFULL + s), (n / S) & 1, abort_flag)) {
                failed = true;
                break;
            }
            const TileInfo info = reinterpret_cast<const TileInfo *>(smem + C::OFF_INFO)[s];
            if (info.stop) break;
            if (x < ktiles && sees(p, info.lim_min, info.lim_max, kb, BT)) {
                if (!wait_warp(BAR(C::B_SFULL + x), used & 1, abort_flag)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                const bool masked = !info.whole || kb + BT > info.lim_min ||
                                    (p.window > 0 && kb < info.lim_max - p.window);
                const float *nlse = reinterpret_cast<const float *>(smem + C::OFF_LSE) + s * BT;
                const int *lim = reinterpret_cast<const int *>(smem + C::OFF_LIM) + s * BT;
#pragma unroll 1
                for (int c0 = 0; c0 < BT; c0 += 64) {
                    uint32_t v[32], u[32];
                    tmem_ld32(ts + c0, v);
                    tmem_ld32(ts + c0 + 32, u);
                    tmem_wait_ld32(v);
                    tmem_wait_ld32(u);
                    if (c0 == BT - 64) {
                        // all read: the next product overwrites them while the last half
                        // is exponentiated from registers
                        tc_fence_before();
                        mbar_arrive(BAR(C::B_SEMPTY + x));
                    }
                    add_weights<32>(p, v, nlse + c0, lim + c0, t, masked, sum);
                    add_weights<32>(p, u, nlse + c0 + 32, lim + c0 + 32, t, masked, sum);
                }
                ++used;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_CEMPTY + s));
        }
        if (failed && lane == 0) *abort_flag = 1;
        if (t < end && page_ok(p, b, t, lp)) {
            const float total = failed ? __int_as_float(0x7fc00000)
                                       : (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
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

// The parts' sums of each key, in order.  grid (keys / 256, Hkv, B)
__global__ void __launch_bounds__(256) weights_join_kernel(const WeightsParams p) {
    const int b = blockIdx.z, u = b * p.Hkv + (int)blockIdx.y;
    const int t = (int)blockIdx.x * 256 + (int)threadIdx.x;
    const int L = p.seq_lens[b];
    const int qn = p.q_lens ? p.q_lens[b] : p.q_len;
    if (bad_lens(p, L, qn) || t >= L || !page_ok(p, b, t, 31 - __clz(p.P))) return;
    const int64_t ctx = (int64_t)p.max_pages * p.P, units = (int64_t)p.B * p.Hkv;
    float sum = 0.f;
    for (int k = 0; k < p.n_parts; ++k) sum += p.parts[(k * units + u) * ctx + t];
    float *w = p.weights + (int64_t)u * p.row_tokens + t;
    *w = (p.accumulate ? *w : 0.f) + sum;
}

template <int D, int N>
cudaError_t launch_stream(const WeightsParams &p, int chunk_tiles, const CUtensorMap &tmK,
                          cudaStream_t stream) {
    using C = StreamCfg<D, N>;
    static int done[64] = {0};
    auto kern = weights_stream_kernel<D, N>;
    const cudaError_t err = configure_smem(reinterpret_cast<const void *>(kern), C::kSmem, done);
    if (err != cudaSuccess) return err;
    const int64_t ctx = (int64_t)p.max_pages * p.P, chunk = (int64_t)chunk_tiles * BT;
    const dim3 grid((unsigned)((ctx + chunk - 1) / chunk), (unsigned)p.Hkv, (unsigned)p.B);
    kern<<<grid, C::kThreads, C::kSmem, stream>>>(tmK, p, (int)chunk);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const WeightsParams &p, const WeightsPlan &plan, const CUtensorMap &tmQ,
                     const CUtensorMap &tmK, cudaStream_t stream) {
    if (plan.stream) {
        const int cols = p.G * p.q_len;
        return cols <= 16    ? launch_stream<D, 16>(p, plan.chunk_tiles, tmK, stream)
               : cols <= 32  ? launch_stream<D, 32>(p, plan.chunk_tiles, tmK, stream)
               : cols <= 64  ? launch_stream<D, 64>(p, plan.chunk_tiles, tmK, stream)
               : cols <= 128 ? launch_stream<D, 128>(p, plan.chunk_tiles, tmK, stream)
                             : launch_stream<D, 256>(p, plan.chunk_tiles, tmK, stream);
    }
    using C = TileCfg<D>;
    static int done[64] = {0};
    auto kern = weights_tile_kernel<D>;
    cudaError_t err = configure_smem(reinterpret_cast<const void *>(kern), C::kSmem, done);
    if (err != cudaSuccess) return err;
    const int64_t ctx = (int64_t)p.max_pages * p.P, units = (int64_t)p.B * p.Hkv;
    const int64_t items = (ctx + kGroupKeys - 1) / kGroupKeys * units * p.n_parts;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    kern<<<(unsigned)items, C::kThreads, C::kSmem, stream>>>(tmQ, tmK, p);
    err = cudaGetLastError();
    return err == cudaSuccess && p.n_parts > 1 ? launch_weights_join(p, stream) : err;
}

}  // namespace

cudaError_t launch_weights_join(const WeightsParams &p, cudaStream_t stream) {
    const int64_t ctx = (int64_t)p.max_pages * p.P;
    weights_join_kernel<<<dim3((unsigned)((ctx + 255) / 256), (unsigned)p.Hkv, (unsigned)p.B), 256, 0,
                          stream>>>(p);
    return cudaGetLastError();
}

// Query tiles of 128 rows split between CTAs of `group_keys` keys: the number of parts with
// the least estimated time, in query tiles.  More items than SMs: their tiles (a key group is
// seen by the rows at and behind it) and start-ups, spread evenly, and a quarter of an item
// for the tail, the long ones going first; else one item.  `startup` is a CTA's in query
// tiles: 6 for bf16 (4: the same times; 8 and 12: 7 % more for one 8192-row prompt of 32 / 8
// heads, 22 % for one of 4096 rows), 3 for fp32 (2 and 4: up to 12 % and 7 % more).  Against
// about three items an SM of at least 8 tiles: one prompt of 512 / 1024 / 4096 / 8192 rows 20 /
// 21 / 78 / 228 -> 11 / 16 / 67 / 222 us, in fp32 30 / 36 / 327 / 1220 -> 19 / 38 / 332 / 1206.
// The join counts as half a start-up: left out, small calls took it for 2 us less on the device
// and 8 more from Python (421 rows x 4 heads x 2 sequences: 10.4 and 22.6 us, now 12.9 and 14.5).
static void split_query_tiles(WeightsPlan &plan, int64_t units, int64_t cols, int q_len, int64_t ctx,
                              int64_t group_keys, int startup, int sms) {
    const int64_t nq = (cols + BT - 1) / BT;
    const int64_t groups = (ctx + group_keys - 1) / group_keys * units;
    const double seen = (double)groups * nq * (1.0 - 0.5 * q_len / ctx);
    double best = INFINITY;
    for (int64_t parts = 1; parts <= nq && parts <= 64; ++parts) {
        const int64_t tiles = (nq + parts - 1) / parts, items = groups * parts;
        const double work = items <= sms ? (double)(tiles + startup)
                                         : (seen + (double)items * startup) / sms +
                                               0.25 * (tiles + startup);
        const double cost = work + (parts > 1 ? 0.5 * startup : 0.0);  // the join
        if (cost < best) {
            best = cost;
            plan.tiles_per_part = (int)tiles;
        }
    }
    plan.parts = (int)((nq + plan.tiles_per_part - 1) / plan.tiles_per_part);
    plan.ws_bytes = plan.parts > 1 ? (size_t)plan.parts * units * ctx * sizeof(float) : 0;
}

// Share of a CTA that streams keys: the 1 to 32 tiles (4096 keys) that take least time, in
// whole waves of `slots` CTAs at the largest context, a CTA's start-up counted as `startup`
// tiles.
static int share_tiles(int64_t units, int64_t ctx, int64_t slots, int startup) {
    const int64_t tiles = (ctx + BT - 1) / BT;
    int share = 1;
    int64_t best = INT64_MAX;
    for (int c = 1; c <= 32; ++c) {
        const int64_t ctas = (tiles + c - 1) / c * units;
        const int64_t cost = (ctas + slots - 1) / slots * (c + startup);
        if (cost < best) {
            best = cost;
            share = c;
        }
    }
    return share;
}

// Pure functions of the call's sizes.
WeightsPlan weights_tc_plan(int B, int Hkv, int G, int q_len, int64_t ctx, int sms) {
    WeightsPlan plan{};
    const int64_t units = (int64_t)B * Hkv, cols = (int64_t)G * q_len;
    if (cols > 256) {
        split_query_tiles(plan, units, cols, q_len, ctx, kGroupKeys, 6, sms);
        return plan;
    }
    // (start-up counted as four tiles: weights at 8 x 8 x 16384 keys of 128 take 40 / 48 / 53
    // / 74 us with 32 / 64 / 128 / 256 columns; with shares that give each SM about eight
    // CTAs 44 / 68 / 81 / 114, and at 4 x 8 x 8192 keys 10 to 23 against 26 to 93)
    plan.stream = 1;
    plan.chunk_tiles = share_tiles(units, ctx, (int64_t)sms * (cols <= 32 ? 2 : 1), 4);
    return plan;
}

// fp32.  Up to 256 columns K is streamed past 64 of them at a time, one launch each: at 8
// sequences x 8 kv heads x 16384 keys of 128, 88 us for up to 16 columns, 100 for 64, 200
// for 128, 397 for 256; the tile kernel takes 535, 535, 510 and 653 us, but 791 for 384
// where the passes would take 600 and lose at smaller sizes (1 x 8 x 8192 keys: 45 us each
// at 256 columns).  More than one pass also needs more key groups than SMs: with fewer the
// tile kernel is done in one wave (2 x 8 x 1000 keys, 128 columns: 9.9 us, 14.1 by passes).
WeightsPlan weights_tf32x3_plan(int B, int Hkv, int G, int q_len, int D, int64_t ctx, int sms) {
    WeightsPlan plan{};
    const int64_t units = (int64_t)B * Hkv, cols = (int64_t)G * q_len, group_keys = 128 / D * BT;
    if (cols <= 64 || (cols <= 256 && (ctx + group_keys - 1) / group_keys * units > sms)) {
        // (start-up counted as two of its tiles)
        plan.stream = 1;
        plan.chunk_tiles = share_tiles(units, ctx, sms, 2);
        return plan;
    }
    split_query_tiles(plan, units, cols, q_len, ctx, group_keys, 3, sms);
    return plan;
}

cudaError_t launch_weights_tc(const WeightsParams &p, const WeightsPlan &plan, int D,
                              const CUtensorMap &tmQ, const CUtensorMap &tmK, cudaStream_t stream) {
    return D == 128 ? launch_d<128>(p, plan, tmQ, tmK, stream) : launch_d<64>(p, plan, tmQ, tmK, stream);
}

}  // namespace atlas
