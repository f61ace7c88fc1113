// Attention weight of cached keys from many query rows a kv head: the same sums as
// weigh_kernel (weigh.cu), on tcgen05.
//
//   w_x = sum over rows r of 2^(c q_r . k_x - l_r),  c = sm_scale log2(e) k_head,  l_r = lse_r log2(e)
//
// The products are laid out as S^T = K Q^T: 128 keys a tile on the tensor memory's
// lanes, up to 128 rows on its columns.  A thread owns a key, runs along the
// columns and keeps the sum in a register over all tiles of rows: no maximum, no
// exchange between threads, and the weights of a key have one owner (same bits in
// every run).  Tensor and exponential bound for many rows (2 D flops and one
// exponential a pair), HBM bound for few (9/16 D bytes a key).
//  * A unit is 256 keys (four pages) of a kv head.  Its K is converted once, to
//    bf16 (code * scale has at most 6 significant bits: exact), straight into
//    tensor memory as the A operand, while the queries stream through shared
//    memory as they are (bf16, TMA, 128-byte swizzle) as the B operand: each tile
//    of rows serves two tiles of keys, so that L2 gives 32 KB for some 1000 cycles.
//  * Warp roles (640 threads): warp 0 loads queries, warp 1 owns TMEM and issues the
//    products, warp 2 copies pages, warp 3 loads log-sums; warps 4..7 and 8..11
//    convert the two key tiles, warps 12..15 and 16..19 sum them up.
//  * TMEM (512 columns): K of two units, S^T of the two key tiles.
//  * Units are dealt to the CTAs in turn.  Where there are few, the row tiles of a
//    unit are dealt to the CTAs of a cluster and their sums added in rank order.
//  * Every wait is bounded; one that runs out raises the CTA's abort flag and the
//    device error word, and each role winds down.
#include <stddef.h>

#include <algorithm>

#include "weigh.cuh"

namespace vsa {

namespace {

constexpr int kThreads = 640;
constexpr int kKeys = 256, kPages = kKeys / kPageTokens;
constexpr int kNlStages = 8, kHeldUnits = 8;
constexpr int kRawUnits = 2;  // units whose pages are on their way or being converted
constexpr uint32_t kSlots = kRawUnits * kPages;
constexpr int kTmemS = 256;

template <int kD>
struct Sm {
    static constexpr int kHalf = 128 * 128;               // 128 rows x 64 channels of bf16, swizzled
    static constexpr int kTile = kHalf * (kD / 64);
    static constexpr int kStages = 5;                     // of queries
    static constexpr int kCodes = kPageTokens * kD / 2, kScales = kPageTokens * kD / 16;
    static constexpr int kRaw = kCodes + kScales;
    static constexpr int kOffRaw = kStages * kTile;       // [unit parity][page]
    static constexpr int kOffMisc = kOffRaw + kRawUnits * kPages * kRaw;
    static constexpr int kKCols = kD / 2;                 // TMEM columns of a key tile
};

struct __align__(16) Misc {
    uint64_t q_full[5], q_empty[5];
    uint64_t raw_full[kRawUnits][kPages], raw_empty[kRawUnits][kPages];
    uint64_t k_full[2][2], k_empty[2];  // [key tile][unit parity], [unit parity]
    uint64_t s_full[2], s_free[2];      // per key tile
    uint64_t nl_full[kNlStages], nl_empty[kNlStages];
    uint64_t drain;
    alignas(16) float nl[kNlStages][128];  // minus the log-sums (log2 units), read in 16 bytes
    int odd[kNlStages];                 // a row of the tile weighs nothing: its logits may be anything
    int held[kHeldUnits][kPages];       // the page is there
    float sums[kKeys];                  // of a cluster's CTA
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(offsetof(Misc, nl) % 16 == 0, "16-byte loads");

template <int kD>
constexpr int smem_bytes() {
    return Sm<kD>::kOffMisc + (int)sizeof(Misc) + 1024;  // slack for 1024-byte alignment
}
static_assert(smem_bytes<128>() <= 232448, "shared memory of the chunk kernel");

struct ChunkParams {
    WeighParams w;
    int per;      // queries of a tile (one, with 128 heads of it, for groups of more than 128)
    int splits;   // tiles of a query for such groups, else 1
    int cluster;  // CTAs that share a unit
};

// A unit of the walk: keys [first, first + 256) of (b, h), its row tiles [t0, tiles)
// in steps of p.cluster.
struct Unit {
    int b, h, first, kv, fresh, t0, tiles;
    __device__ int count(const ChunkParams& p) const { return t0 < tiles ? (tiles - t0 - 1) / p.cluster + 1 : 0; }
};
struct TileRows {
    int query, head, columns;  // first query and head (of the kv head's); rows
};
__device__ __forceinline__ TileRows tile_rows_of(const ChunkParams& p, const Unit& u, int t) {
    if (p.splits == 1) return {t * p.per, 0, min(p.per, u.fresh - t * p.per) * p.w.group};
    const int q = t / p.splits, head = (t - q * p.splits) * 128;
    return {q, head, min(128, p.w.group - head)};
}

__device__ __forceinline__ int blocks_of(int kv) { return kv > 0 ? (kv - 1) / kKeys + 1 : 0; }

// Units of all sequences and heads, those of cluster i of n: i, i + n, ... (a whole warp walks).
struct UnitWalk {
    long long at;  // the next unit, from sequence b0's first on
    int b0;
    long long step;
    int rank;
    __device__ void begin(const ChunkParams& p) {
        at = blockIdx.x / p.cluster;
        step = gridDim.x / p.cluster;
        rank = blockIdx.x % p.cluster;
        b0 = 0;
    }
    __device__ bool next(const ChunkParams& p, Unit& u) {
        const CacheView& c = p.w.c;
        const int lane = threadIdx.x & 31;
        for (;;) {
            const int b = b0 + lane;
            const int kv = b < c.B ? cache_len(c, b, false) : 0;
            const long long mine = (long long)c.kv_heads * blocks_of(kv);
            const long long incl = scan_warp(mine);
            const unsigned past = __ballot_sync(0xffffffffu, at < incl);
            if (!past) {
                at -= __shfl_sync(0xffffffffu, incl, 31);
                b0 += 32;
                if (b0 >= c.B) return false;
                continue;
            }
            const int l = __ffs(past) - 1;
            const long long within = at - __shfl_sync(0xffffffffu, incl - mine, l);
            u.b = b0 + l;
            u.kv = __shfl_sync(0xffffffffu, kv, l);
            const int blocks = blocks_of(u.kv);
            u.h = (int)(within / blocks);
            u.first = (int)(within - (long long)u.h * blocks) * kKeys;
            break;
        }
        u.fresh = p.w.q_lens ? min(max(p.w.q_lens[u.b], 0), p.w.Sq) : p.w.Sq;
        u.tiles = p.splits == 1 ? (u.fresh + p.per - 1) / p.per : u.fresh * p.splits;
        // Tiles whose queries all come before the unit's keys see none of them.
        int t0 = 0;
        if (p.w.causal) {
            const int q0 = min(max(u.first - (u.kv - u.fresh), 0), u.fresh);
            t0 = p.splits == 1 ? q0 / p.per : q0 * p.splits;
        }
        u.t0 = t0 + rank;
        at += step;
        return true;
    }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* desc, uint32_t bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(desc), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// Two fp16 as two bf16 (exact for code * scale).
__device__ __forceinline__ uint32_t f16_to_bf16x2(uint32_t h) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
    return x;
}

template <int kD>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const ChunkParams p) {
    using L = PageLayout<kD>;
    using S = Sm<kD>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Misc& ms = *reinterpret_cast<Misc*>(smem + S::kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &ms.abort_flag;
    const CacheView& c = p.w.c;
    unsigned int* err = c.err;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_q);
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&ms.q_full[s]), 1);
            mbar_init(smem_u32(&ms.q_empty[s]), 1);
        }
        for (int s = 0; s < kRawUnits * kPages; ++s) {
            mbar_init(smem_u32(&ms.raw_full[0][s]), 1);
            mbar_init(smem_u32(&ms.raw_empty[0][s]), 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&ms.k_full[s][0]), 4);
            mbar_init(smem_u32(&ms.k_full[s][1]), 4);
            mbar_init(smem_u32(&ms.k_empty[s]), 1);
            mbar_init(smem_u32(&ms.s_full[s]), 1);
            mbar_init(smem_u32(&ms.s_free[s]), 4);
        }
        for (int s = 0; s < kNlStages; ++s) {
            mbar_init(smem_u32(&ms.nl_full[s]), 1);
            mbar_init(smem_u32(&ms.nl_empty[s]), 8);
        }
        mbar_init(smem_u32(&ms.drain), 1);
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&ms.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    early();
    begin_work();
    const uint32_t tmem = ms.tmem_base;
    UnitWalk walk;
    walk.begin(p);
    Unit u;

    if (warp == 0) {
        // ====================================================== queries by TMA
        const int box_rows = p.splits == 1 ? p.per * p.w.group : 128;
        uint32_t i = 0;  // tiles so far
        bool ok = true;
        while (ok && walk.next(p, u)) {
            for (int t = u.t0; t < u.tiles; t += p.cluster, ++i) {
                const int st = i % S::kStages;
                if (i >= S::kStages) ok = cache_wait<kSleepLong>(smem_u32(&ms.q_empty[st]), (i / S::kStages + 1) & 1, abort_flag, err);
                if (!ok) break;
                if (lane == 0) {
                    const TileRows x = tile_rows_of(p, u, t);
                    const uint32_t bar = smem_u32(&ms.q_full[st]);
                    mbar_arrive_expect_tx(bar, box_rows * kD * 2);
#pragma unroll
                    for (int half = 0; half < kD / 64; ++half)
                        tma_load_4d(sbase + st * S::kTile + half * S::kHalf, &tm_q, bar, half * 64,
                                    u.h * p.w.group + x.head, x.query, u.b);
                }
                __syncwarp();
            }
        }
        // The last load into each stage has landed before the CTA's shared memory is released.
        if (lane == 0)
            for (uint32_t s = 0; s < (uint32_t)S::kStages && s < i; ++s)
                mbar_wait_drain_1(smem_u32(&ms.q_full[s]), ((i - 1 - s) / S::kStages) & 1, err, kCacheWaitNs);
    } else if (warp == 1) {
        // ============================================================ K Q^T
        const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
        const uint32_t lo_q = (uint32_t)smem_desc_sw128(sbase, 16, 1024);
        uint32_t i = 0, n = 0;  // tiles, units with tiles so far
        bool ok = true;
        while (ok && walk.next(p, u)) {
            if (u.count(p) == 0) continue;
            for (int t = u.t0; t < u.tiles && ok; t += p.cluster, ++i) {
                const int st = i % S::kStages;
                const int columns = tile_rows_of(p, u, t).columns;
                const uint32_t idesc = idesc_bf16_f32(128, (columns + 15) & ~15, 0, 0);
                ok = cache_wait<kSleepShort>(smem_u32(&ms.q_full[st]), (i / S::kStages) & 1, abort_flag, err);
                const uint32_t b0 = lo_q + ((uint32_t)(st * S::kTile) >> 4);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (ok && t == u.t0)
                        ok = cache_wait<kSleepShort>(smem_u32(&ms.k_full[s][n & 1]), (n >> 1) & 1, abort_flag, err);
                    if (ok && i > 0) ok = cache_wait<kSleepShort>(smem_u32(&ms.s_free[s]), (i - 1) & 1, abort_flag, err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a0 = tmem + ((n & 1) * 2 + s) * S::kKCols;
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        mma_ts_warp(tmem + kTmemS + s * 128, a0 + kk * 8,
                                    b0 + (((kk >> 2) * S::kHalf + (kk & 3) * 32) >> 4), hi, idesc, kk > 0);
                    mma_commit_warp(smem_u32(&ms.s_full[s]));
                }
                if (!ok) break;
                mma_commit_warp(smem_u32(&ms.q_empty[st]));
            }
            if (!ok) break;
            mma_commit_warp(smem_u32(&ms.k_empty[n & 1]));
            ++n;
        }
        mma_commit_warp(smem_u32(&ms.drain));
        if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain), 0, err, kCacheWaitNs);
    } else if (warp == 2) {
        // ============================================================= pages
        if (blockIdx.x == 0)  // lengths out of range are noted once
            for (int b = lane; b < c.B; b += 32) cache_len(c, b, true);
        uint32_t g = 0;  // pages so far
        bool ok = true;
        while (ok && walk.next(p, u)) {
            if (u.count(p) == 0) continue;
            int id = -1;
            const int page0 = u.first / kPageTokens;
            if (lane < kPages && (page0 + lane) * kPageTokens < u.kv) {
                id = c.table[(size_t)u.b * c.width + page0 + lane];
                if (id < 0 || id >= c.pages) {
                    atomicOr(err, VSA_DEVERR_INDEX);
                    id = -1;
                }
            }
            for (int i = 0; i < kPages; ++i, ++g) {
                const int page = __shfl_sync(0xffffffffu, id, i);
                const int slot = g % kSlots;
                if (g >= kSlots)
                    ok = cache_wait<kSleepLong>(smem_u32(&ms.raw_empty[0][slot]), (g / kSlots + 1) & 1, abort_flag, err);
                if (!ok) break;
                if (lane == 0) {
                    ms.held[(g / kPages) % kHeldUnits][i] = page >= 0;
                    const uint32_t bar = smem_u32(&ms.raw_full[0][slot]);
                    if (page < 0) {
                        mbar_arrive(bar);
                    } else {
                        mbar_arrive_expect_tx(bar, S::kRaw);
                        const uint32_t dst = sbase + S::kOffRaw + slot * S::kRaw;
                        const unsigned char* src = c.pool + ((size_t)page * c.kv_heads + u.h) * L::kBytes;
                        bulk_load(dst, src, S::kCodes, bar);
                        bulk_load(dst + S::kCodes, src + L::kKScale, S::kScales, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0)
            for (uint32_t s = 0; s < kSlots && s < g; ++s)
                mbar_wait_drain_1(smem_u32(&ms.raw_full[0][s]), ((g - 1 - s) / kSlots) & 1, err, kCacheWaitNs);
    } else if (warp == 3) {
        // ========================================================= log-sums
        uint32_t i = 0;
        bool ok = true;
        while (ok && walk.next(p, u)) {
            for (int t = u.t0; t < u.tiles; t += p.cluster, ++i) {
                const TileRows x = tile_rows_of(p, u, t);
                float y[4];
                bool odd = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 32 * k + lane;
                    y[k] = -INFINITY;
                    if (r < x.columns) {
                        const int q = p.splits == 1 ? r / p.w.group : 0;
                        const int head = u.h * p.w.group + x.head + r - q * p.w.group;
                        const float l = p.w.lse[((size_t)u.b * p.w.heads + head) * p.w.Sq + x.query + q];
                        if (fabsf(l) < INFINITY)
                            y[k] = l * -1.4426950408889634f;
                        else
                            odd = true;
                    }
                }
                const int st = i % kNlStages;
                if (i >= kNlStages) ok = cache_wait<kSleepLong>(smem_u32(&ms.nl_empty[st]), (i / kNlStages + 1) & 1, abort_flag, err);
                if (!ok) break;
                odd = __any_sync(0xffffffffu, odd);
#pragma unroll
                for (int k = 0; k < 4; ++k) ms.nl[st][32 * k + lane] = y[k];
                if (lane == 0) ms.odd[st] = odd;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.nl_full[st]));
            }
        }
    } else if (warp < 12) {
        // ============================ convert: warps 4..7 the first 128 keys, 8..11 the others
        const int s = (warp - 4) >> 2, quarter = warp & 3;
        const int key = quarter * 32 + lane;          // of the tile
        const int page = 2 * s + (key >> 6), slot = key & 63;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t n = 0;
        bool ok = true;
        while (ok && walk.next(p, u)) {
            if (u.count(p) == 0) continue;
            const int par = n & 1;
            ok = cache_wait<kSleepShort>(smem_u32(&ms.raw_full[par][page]), (n >> 1) & 1, abort_flag, err);
            if (ok && n >= 2) ok = cache_wait<kSleepShort>(smem_u32(&ms.k_empty[par]), ((n >> 1) + 1) & 1, abort_flag, err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t raw = sbase + S::kOffRaw + (par * kPages + page) * S::kRaw;
            const uint32_t codes = raw + slot * L::kRow, scales = raw + S::kCodes + slot * L::kGroups;
            const uint32_t to = t_lane + (par * 2 + s) * S::kKCols;
            uint32_t sc[kD / 64];
#pragma unroll
            for (int k = 0; k < kD / 64; ++k) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc[k]) : "r"(scales + 4 * k));
#pragma unroll
            for (int piece = 0; piece < kD / 32; ++piece) {
                const uint4 x = lds128(codes + piece * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                const uint32_t two = e4m3_to_f16(sc[piece / 2] >> (16 * (piece & 1)));
                const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
                uint32_t out[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t y[4];
                    e2m1_to_f16(w[k], y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) out[4 * k + j] = f16_to_bf16x2(mul_f16x2(y[j], k < 2 ? s0 : s1));
                }
                tmem_st16(to + piece * 16, out);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.raw_empty[par][page]));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.k_full[s][par]));
            ++n;
        }
    } else {
        // ============================ sums: warps 12..15 the first 128 keys, 16..19 the others
        const int s = (warp - 12) >> 2, quarter = warp & 3;
        const int key = quarter * 32 + lane;
        const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemS + s * 128;
        uint32_t i = 0, n = 0;
        bool ok = true;
        while (ok && walk.next(p, u)) {
            const int x = u.first + s * 128 + key;  // the thread's key
            const float c2 = p.w.scale_log2 * (c.kv_scale ? c.kv_scale[u.h] : 1.f);
            const float2 c2v = make_float2(c2, c2);
            float total = 0.f;
            for (int t = u.t0; t < u.tiles; t += p.cluster, ++i) {
                const TileRows rows = tile_rows_of(p, u, t);
                const int st = i % kNlStages;
                // Columns [low, columns) are rows that see the key.
                int low = 0;
                if (p.w.causal) {
                    const int ahead = x - (u.kv - u.fresh) - rows.query;  // queries of the tile before the key
                    low = ahead <= 0 ? 0 : p.splits > 1 ? 128 : min(ahead, 128) * p.w.group;
                }
                ok = cache_wait<kSleepShort>(smem_u32(&ms.nl_full[st]), (i / kNlStages) & 1, abort_flag, err) &&
                     cache_wait<kSleepShort>(smem_u32(&ms.s_full[s]), i & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                const bool odd = *reinterpret_cast<volatile int*>(&ms.odd[st]);
                float2 a = make_float2(0.f, 0.f), b = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int c0 = 0; c0 < rows.columns; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(t_s + c0, v);
                    const float4* nl = reinterpret_cast<const float4*>(&ms.nl[st][c0]);
                    tmem_wait_ld();
                    if (__any_sync(0xffffffffu, low > c0) || odd || c0 + 32 > rows.columns) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 l = nl[k / 4];
                            const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int col = c0 + k + j;
                                const bool sees = col >= low && col < rows.columns && ls[j] > -INFINITY;
                                const float y = ex2_approx(fmaf(__uint_as_float(v[k + j]), c2, ls[j]));
                                a.x += sees ? y : 0.f;
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 l = nl[k / 4];
                            const float2 e0 = __ffma2_rn(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2v,
                                                         make_float2(l.x, l.y));
                            const float2 e1 = __ffma2_rn(
                                make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), c2v, make_float2(l.z, l.w));
                            a = __fadd2_rn(a, make_float2(ex2_approx(e0.x), ex2_approx(e0.y)));
                            b = __fadd2_rn(b, make_float2(ex2_approx(e1.x), ex2_approx(e1.y)));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&ms.s_free[s]));
                    mbar_arrive(smem_u32(&ms.nl_empty[st]));
                }
                total += (a.x + a.y) + (b.x + b.y);
            }
            if (!ok) break;
            if (u.count(p) > 0) {  // (a page that is not there has no weight)
                if (!*reinterpret_cast<volatile int*>(&ms.held[n % kHeldUnits][2 * s + (key >> 6)])) total = 0.f;
                ++n;
            }
            if (p.cluster > 1) {
                ms.sums[s * 128 + key] = total;
            } else if (x < u.kv) {
                const size_t at = ((size_t)u.b * c.kv_heads + u.h) * ((size_t)c.width * kPageTokens) + x;
                p.w.out[at] = (p.w.weights ? p.w.weights[at] : 0.f) + total;
            }
        }
    }

    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if (p.cluster > 1) {
        // The cluster's one unit: its CTAs' sums in the order of their ranks, a share of the keys each.
        walk.begin(p);
        const bool has = walk.next(p, u);
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        const int each = kKeys / p.cluster, key = walk.rank * each + (int)threadIdx.x;
        if (has && (int)threadIdx.x < each && u.first + key < u.kv && !*abort_flag) {
            float total = 0.f;
            for (int r = 0; r < p.cluster; ++r) {
                uint32_t at;
                float y;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&ms.sums[key])), "r"(r));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(y) : "r"(at) : "memory");
                total += y;
            }
            const size_t at = ((size_t)u.b * c.kv_heads + u.h) * ((size_t)c.width * kPageTokens) + u.first + key;
            p.w.out[at] = (p.w.weights ? p.w.weights[at] : 0.f) + total;
        }
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
    }
    fill_rest(p.w);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                   CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                   CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static std::atomic<EncodeTiledFn> known{nullptr};
    EncodeTiledFn fn = known.load(std::memory_order_relaxed);
    if (fn) return fn;
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return nullptr;
    fn = reinterpret_cast<EncodeTiledFn>(ptr);
    known.store(fn, std::memory_order_relaxed);
    return fn;
}

template <int kD>
cudaError_t launch(const ChunkParams& p, int grid, cudaStream_t stream) {
    const WeighParams& w = p.w;
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    CUtensorMap map;
    // The rows of a tile: `per` queries of the group's heads, or 128 heads of one.
    const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)w.heads, (cuuint64_t)w.Sq, (cuuint64_t)w.c.B};
    const cuuint64_t row = (cuuint64_t)kD * 2;
    const cuuint64_t strides[3] = {row, row * w.heads, row * w.heads * w.Sq};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(w.group, 128), (cuuint32_t)p.per, 1};
    const cuuint32_t each[4] = {1, 1, 1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint4*>(w.q), dims, strides, box, each,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(weigh_chunk_kernel<kD>, smem_bytes<kD>(), done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem_bytes<kD>();
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)p.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, weigh_chunk_kernel<kD>, map, p);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_weigh_chunk(const WeighParams& w, int D, int num_sms, cudaStream_t stream) {
    ChunkParams p;
    p.w = w;
    p.per = std::max(1, 128 / w.group);
    p.splits = w.group > 128 ? (w.group + 127) / 128 : 1;
    // Where all units there may be leave half of the SMs without one, up to 8 CTAs
    // share the row tiles of a unit; each such cluster has one unit.
    const long long most = (long long)w.c.B * w.c.kv_heads * (((long long)w.c.width * kPageTokens + kKeys - 1) / kKeys);
    const long long tiles = p.splits == 1 ? (w.Sq + p.per - 1) / p.per : (long long)w.Sq * p.splits;
    p.cluster = 1;
    while (p.cluster < 8 && 2 * p.cluster * most <= num_sms && 2 * p.cluster <= tiles) p.cluster *= 2;
    const int grid = p.cluster > 1 ? (int)most * p.cluster : (int)std::min<long long>(num_sms, most);
    return D == 64 ? launch<64>(p, grid, stream) : launch<128>(p, grid, stream);
}

}  // namespace vsa
