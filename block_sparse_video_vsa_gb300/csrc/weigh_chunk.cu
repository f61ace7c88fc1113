// Attention weight of cached keys from many query rows a kv head: the same sums as
// weigh_kernel (weigh.cu), on tcgen05.
//
//   w_x = sum over rows r of 2^(c q_r . k_x - l_r),  c = sm_scale log2(e) k_head,  l_r = lse_r log2(e)
//
// The products are laid out as S^T = K Q^T: 128 keys a tile on the tensor memory's
// lanes, up to 128 rows on its columns.  A thread owns a key, runs along the
// columns and keeps the sum in a register over all tiles of rows: no maximum, no
// exchange between threads, and the weights of a key have one owner (same bits in
// every run).  The floor is that of products and exponentials for many rows (2 D flops
// and one exponential a pair), of memory for few (9/16 D bytes a key); the kernel is bound
// by waits of its roles for one another and by instructions (figures below).
//  * A unit is 256 keys (four pages) of a kv head.  Its K is converted once, to
//    bf16 (code * scale has at most 6 significant bits: exact), straight into
//    tensor memory as the A operand, while the queries stream through shared
//    memory as they are (bf16, TMA, 128-byte swizzle) as the B operand: each tile
//    of rows serves two tiles of keys, so that L2 gives 32 KB for some 1000 cycles.
//  * Rows that fit one tile (a window of recent queries) stay in shared memory for
//    all units of their head: the CTAs take runs of neighbouring units then, and
//    pages are all that moves.  Converting K is then much of the work, and 2.6
//    instructions a pair to fp16 instead of 5.6 to bf16 pay for turning the rows into
//    fp16 as well, once a head: a power of two a row, as everywhere (kHalf).  Else
//    units are dealt to the CTAs in turn, which balances causal calls.  Where there are few units, the row tiles of one are
//    dealt to the CTAs of a cluster and their sums added in rank order.
//  * S^T is issued and summed in halves of a tile's columns, with a buffer and a
//    warpgroup for each half and key tile: a half's products run while the others'
//    exponentials do, and four warps a scheduler cover one another's loads.
//  * Warp roles (896 threads): warp 0 loads queries and log-sums, warps 1 (which owns
//    TMEM) and 3 issue the products of a key tile each, warp 2 walks the units,
//    describes them to the others and copies their pages; warps 4..7 and 8..11
//    convert the two key tiles; warps 12..27 sum up.
//  * TMEM (512 columns): K of two units, two halves of S^T of the two key tiles.
//  * Every wait is bounded; one that runs out raises the CTA's abort flag and the
//    device error word, and each role winds down.
// Measured on a GB300, D = 128, one sequence of 32760 tokens, 40 kv heads: 1560 rows
// 437 us = 1.20 PFLOP/s (63% of the measured bf16 rate; tensor pipe 49% busy,
// exponentials 51%, in turns; 0.69 instructions a scheduler and cycle, and of the 10 cycles
// that each of its seven warps takes an instruction 3.6 are waits for tensor memory and barriers);
// 64 rows 51 us = 1.9 TB/s of pages (28% of the copy rate; 0.62 instructions, of 11 cycles 3.2 such
// waits and 1.3 for shared memory; describing, converting and summing a unit of 256 keys takes some
// 1760 instructions a scheduler).
#include <float.h>
#include <stddef.h>

#include <algorithm>

#include "weigh.cuh"

namespace vsa {

namespace {

constexpr int kThreads = 896;
constexpr int kKeys = 256, kPages = kKeys / kPageTokens;
// Log-sums of the last tiles.  A place is written again 8 tiles later, when the products
// of the tile three before that have been issued and completed: those waited for the
// sums of the tiles before, so the place's readers are done.
constexpr int kNlStages = 8;
constexpr int kUnits = 16;                       // described at a time
constexpr int kReaders = kThreads / 32 - 1;      // warps that read the descriptions
// Registers, for rows that stream (which are summed more than converted: 452 us for a
// frame's queries without, 436; a window's 50 and 53): 7 warpgroups launched with 72
// each; the shares add up to 504.
constexpr int kLaunchRegs = 72, kIssueRegs = 56, kConvertRegs = 48, kSumRegs = 88;
static_assert(kIssueRegs + 2 * kConvertRegs + 4 * kSumRegs <= 7 * kLaunchRegs, "register split exceeds the launch");
constexpr uint32_t kRaw = 6;     // units whose pages are on their way or being converted
constexpr int kTmemS = 256;

template <int kD>
struct Sm {
    static constexpr int kHalf = 128 * 128;               // 128 rows x 64 channels of bf16, swizzled
    static constexpr int kTile = kHalf * (kD / 64);
    static constexpr int kStages = 3;                     // of queries
    static constexpr int kCodes = kPageTokens * kD / 2, kScales = kPageTokens * kD / 16;
    static constexpr int kPage = kCodes + kScales;        // K of a page
    static constexpr int kOffRaw = kStages * kTile;       // [unit][page]
    static constexpr int kOffMisc = kOffRaw + (int)kRaw * kPages * kPage;
    static constexpr int kKCols = kD / 2;                 // TMEM columns of a key tile
};

// A unit: keys [first, first + 256) of (b, h), its row tiles [t0, tiles) in steps of
// p.cluster; fresh_rows: other rows than the unit before had.  b < 0: no more units.
struct alignas(16) Unit {
    int b, h, first, kv;
    int fresh, t0, tiles, fresh_rows;
    float c2;  // logit (log2 units) of a product
    int held;  // bit i: page i is there
};

struct __align__(16) Misc {
    uint64_t q_full[3], q_empty[3];
    uint64_t q_here[3];  // kHalf: the queries have landed
    uint64_t raw_full[kRaw][2], raw_empty[kRaw];  // [unit][key tile]
    uint64_t k_full[2][2], k_empty[2][2];  // [key tile][unit parity]
    uint64_t s_full[2][2], s_free[2][2];  // [key tile][buffer]
    uint64_t unit_full[kUnits], unit_empty[kUnits];
    uint64_t part_full[2][2], part_empty[2][2];  // [key tile][unit parity]
    uint64_t drain[2];
    alignas(16) float nl[kNlStages][128];  // minus the log-sums (log2 units), read in 16 bytes
    float cf[kNlStages][128];              // kHalf: logit (log2 units) of a product
    int odd[kNlStages];                    // a row of the tile weighs nothing: its logits may be anything
    float part[2][kKeys];                  // [unit parity]: the odd buffers' share of the sums
    float sums[kKeys];                     // of a cluster's CTA
    Unit unit[kUnits];
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(offsetof(Misc, nl) % 16 == 0 && offsetof(Misc, cf) % 16 == 0, "16-byte loads");

template <int kD>
constexpr int smem_bytes() {
    return Sm<kD>::kOffMisc + (int)sizeof(Misc) + 1024;  // slack for 1024-byte alignment
}
static_assert(smem_bytes<128>() <= 232448, "shared memory of the chunk kernel");

struct ChunkParams {
    WeighParams w;
    int per;       // queries of a tile (one, with 128 heads of it, for groups of more than 128)
    int splits;    // tiles of a query for such groups, else 1
    int cluster;   // CTAs that share a unit
    int resident;  // one tile of rows: CTAs take runs of units and keep it for all of a head
    int half;      // columns of a tile that are issued and summed at once
    int one_half;  // resident rows that fit half a tile: units alternate between the buffers
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

// The units of all sequences and heads in their order; CTA (or cluster) i of n takes
// i, i + n, ..., or the i-th of n equal runs (a whole warp walks).
struct UnitWalk {
    int b, h, block;  // the next unit
    int kv, blocks;   // of its sequence
    int step;
    int rank;
    long long left;  // units of a run
    bool any, moved;
    int known, fresh, tiles;  // the sequence whose queries are known, and they
    int ids, ids_b, ids_from;  // lane i: the page number of page ids_from + i of sequence ids_b
    int scale_h;               // the head whose scale is known
    float c2;

    // The unit `at` places behind sequence b0's first; false: there is none.
    __device__ bool find(const ChunkParams& p, int b0, long long at) {
        const CacheView& c = p.w.c;
        const int lane = threadIdx.x & 31;
        for (; b0 < c.B; b0 += 32) {
            const int n = b0 + lane < c.B ? cache_len(c, b0 + lane, false) : 0;
            const long long mine = (long long)c.kv_heads * blocks_of(n);
            const long long incl = scan_warp(mine);
            const unsigned past = __ballot_sync(0xffffffffu, at < incl);
            if (!past) {
                at -= __shfl_sync(0xffffffffu, incl, 31);
                continue;
            }
            const int l = __ffs(past) - 1;
            at -= __shfl_sync(0xffffffffu, incl - mine, l);
            b = b0 + l;
            kv = __shfl_sync(0xffffffffu, n, l);
            blocks = blocks_of(kv);
            h = (int)(at / blocks);
            block = (int)(at - (long long)h * blocks);
            return true;
        }
        return false;
    }
    __device__ void begin(const ChunkParams& p) {
        const CacheView& c = p.w.c;
        rank = blockIdx.x % p.cluster;
        const int i = blockIdx.x / p.cluster, n = gridDim.x / p.cluster;
        moved = true;
        known = ids_b = scale_h = -1;
        step = n;
        left = 1LL << 62;
        long long from = i;
        if (p.resident) {
            long long total = 0;
            for (int b0 = threadIdx.x & 31; b0 < c.B; b0 += 32)
                total += (long long)c.kv_heads * blocks_of(cache_len(c, b0, false));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
            from = total / n * i + min((long long)i, total % n);
            left = total / n + (i < total % n ? 1 : 0);
            step = 1;
        }
        any = left > 0 && find(p, 0, from);
    }
    // The next unit with tiles, and which lanes' `ids` are its page numbers, from `at` on.
    __device__ bool next(const ChunkParams& p, Unit& u, int& at) {
        const CacheView& c = p.w.c;
        while (any) {
            if (b != known) {
                known = b;
                fresh = p.w.q_lens ? min(max(p.w.q_lens[b], 0), p.w.Sq) : p.w.Sq;
                tiles = p.splits == 1 ? (fresh + p.per - 1) / p.per : fresh * p.splits;
            }
            u.b = b;
            u.h = h;
            u.first = block * kKeys;
            u.kv = kv;
            u.fresh = fresh;
            u.tiles = tiles;
            // Tiles whose queries all come before the unit's keys see none of them.
            int t0 = 0;
            if (p.w.causal && tiles > 1) {
                const int q0 = min(max(u.first - (kv - fresh), 0), fresh);
                t0 = p.splits == 1 ? q0 / p.per : q0 * p.splits;
            }
            u.t0 = t0 + rank;
            u.fresh_rows = moved || !p.resident;
            // On to the next.
            moved = false;
            any = --left > 0;
            block += step;
            if (any && block >= blocks) {
                h += block / blocks;
                block %= blocks;
                moved = true;
                if (h >= c.kv_heads) any = find(p, b + 1, (long long)(h - c.kv_heads) * blocks + block);
            }
            if (u.t0 >= u.tiles) continue;
            // Page numbers are looked up 32 at a time: a run of units needs the next eight
            // units' with one wait for memory.
            const int page = u.first / kPageTokens, lane = threadIdx.x & 31;
            if (u.b != ids_b || page < ids_from || page + kPages > ids_from + 32) {
                ids_b = u.b;
                ids_from = page;
                ids = -1;
                if ((long long)(page + lane) * kPageTokens < u.kv) ids = c.table[(size_t)u.b * c.width + page + lane];
            }
            at = page - ids_from;
            if (u.h != scale_h) {
                scale_h = u.h;
                c2 = p.w.scale_log2 * (c.kv_scale ? c.kv_scale[u.h] : 1.f);
            }
            u.c2 = c2;
            return true;
        }
        return false;
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

// The kD / 16 products of a half: d = a (kD / 2 columns of tensor memory) * b (shared
// memory, 16 channels 32 bytes apart, 64 channels kHalf), and an arrival on `done` (and
// on `also`, where that is not 0) once they and those before have completed.  All lanes call it; one issues, in one branch.
#define VSA_MMA "tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, "
#define VSA_NEXT "add.u32 ta, ta, 8;\n\tadd.u64 db, db, 2;\n\t"
template <int kD>
__device__ __forceinline__ void issue_half(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                           uint32_t done, uint32_t also) {
    if constexpr (kD == 128)
        asm volatile(
            "{\n\t.reg .pred one, p;\n\t.reg .b32 ta;\n\t.reg .b64 db;\n\t"
            "elect.sync _|one, 0xffffffff;\n\t"
            "mov.b64 db, {%2, %3};\n\tmov.b32 ta, %1;\n\tsetp.ne.b32 p, 0, 0;\n\t"
            "@!one bra skip%=;\n\t" VSA_MMA "p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
            VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t"
            "add.u64 db, db, 1016;\n\t"  // (the next 64 channels: 1024 from the first of these)
            VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t"
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t"
            "skip%=:\n\t}" ::"r"(d),
            "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(done), "r"(also)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred one, p;\n\t.reg .b32 ta;\n\t.reg .b64 db;\n\t"
            "elect.sync _|one, 0xffffffff;\n\t"
            "mov.b64 db, {%2, %3};\n\tmov.b32 ta, %1;\n\tsetp.ne.b32 p, 0, 0;\n\t"
            "@!one bra skip%=;\n\t" VSA_MMA "p;\n\tsetp.eq.b32 p, 0, 0;\n\t"
            VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t" VSA_NEXT VSA_MMA "p;\n\t"
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n\t"
            "skip%=:\n\t}" ::"r"(d),
            "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(done), "r"(also)
            : "memory");
    __syncwarp();
}
#undef VSA_MMA
#undef VSA_NEXT
// An arrival once everything issued so far has completed, by the lane that issues.
__device__ __forceinline__ void commit_one(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
        "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
    return x;
}

// One of two threads of a row of a query tile (`tile`: its first half's channels, the
// second kHalf behind): bf16 to fp16, scaled by the power of two it returns; side 0
// the first half of the channels, side 1 the other.  Pieces of 16 bytes are taken where
// they lie (the swizzle keeps a row's together), each row from another one on, so that
// 8 rows do not meet in a bank.
template <int kD>
__device__ __forceinline__ int half_row(uint32_t tile, int row, int side) {
    constexpr int kPieces = kD / 16;  // of this thread
    const uint32_t at = tile + row * 128 + (kD == 128 ? side * Sm<kD>::kHalf : 0);
    const int first = kD == 128 ? 0 : side * kPieces;
    uint32_t mx = 0u;
#pragma unroll 1
    for (int k = 0; k < kPieces; ++k) {
        const uint4 x = lds128(at + (first + (k + row) % kPieces) * 16);
        mx = __vimax3_u16x2(mx, x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
        mx = __vimax3_u16x2(mx, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu);
    }
    uint32_t top = max(mx & 0xFFFFu, mx >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    const int e = q_exponent(__uint_as_float(top << 16));
    const float f = pow2i(e);
#pragma unroll 1
    for (int k = 0; k < kPieces; ++k) {
        const uint32_t to = at + (first + (k + row) % kPieces) * 16;
        const uint4 x = lds128(to);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = pack_f16x2(bf16_lo(w[j]) * f, bf16_hi(w[j]) * f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                     : "memory");
    }
    return e;
}

// 128 keys by N rows, bf16 or fp16.
__device__ __forceinline__ uint32_t idesc(bool half, int N) {
    const uint32_t x = idesc_bf16_f32(128, N, 0, 0);
    return half ? x & ~((1u << 7) | (1u << 10)) : x;
}

// cache_wait for a barrier and a phase of each lane's own, where it is `needed`.
__device__ __forceinline__ bool wait_lanes(uint32_t bar, uint32_t parity, bool needed, volatile int* abort,
                                           unsigned int* err) {
    bool there = !needed;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (!there) there = mbar_try_wait(bar, parity);
        if (__all_sync(0xffffffffu, there)) {
            __syncwarp();  // (what one lane has seen the others may rely on)
            return true;
        }
        __nanosleep(kSleepShort);
        if (i % 64 != 0) continue;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, now - t0 > kCacheWaitNs)) {
            *abort = 1;
            if ((threadIdx.x & 31) == 0) atomicOr(err, VSA_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// The same number for the compiler, too, all over the warp (which holds it in a
// uniform register then, as the products' operands have to be).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }


// kHalf: K and the queries in fp16, each row's scale beside its log-sum (resident rows).
template <int kD, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ ChunkParams p) {
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
            mbar_init(smem_u32(&ms.q_full[s]), kHalf ? 1 + 8 : 2);  // log-sums; the converting warps, or the queries
            mbar_init(smem_u32(&ms.q_here[s]), 1);
            mbar_init(smem_u32(&ms.q_empty[s]), 2);
        }
        for (int s = 0; s < (int)kRaw; ++s) {
            mbar_init(smem_u32(&ms.raw_full[s][0]), 1);
            mbar_init(smem_u32(&ms.raw_full[s][1]), 1);
            mbar_init(smem_u32(&ms.raw_empty[s]), 8);
        }
        for (int s = 0; s < 2; ++s) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&ms.k_full[s][i]), 4);
                mbar_init(smem_u32(&ms.k_empty[s][i]), 1);
                mbar_init(smem_u32(&ms.s_full[s][i]), 1);
                mbar_init(smem_u32(&ms.s_free[s][i]), 4);
                mbar_init(smem_u32(&ms.part_full[s][i]), 4);
                mbar_init(smem_u32(&ms.part_empty[s][i]), 4);
            }
            mbar_init(smem_u32(&ms.drain[s]), 1);
        }
        for (int s = 0; s < kUnits; ++s) {
            mbar_init(smem_u32(&ms.unit_full[s]), 1);
            mbar_init(smem_u32(&ms.unit_empty[s]), kReaders);
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x < kKeys) ms.sums[threadIdx.x] = 0.f;
    // Rows of the query tiles that no load fills are zeros.
    for (int i = threadIdx.x; i < S::kStages * S::kTile / 16; i += kThreads)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
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

    // The n-th unit, once it is described; false: there are no more (or the kernel was called off).
    auto take = [&](uint32_t n, bool& ok, Unit& u) {
        ok = ok && cache_wait<kSleepShort>(smem_u32(&ms.unit_full[n % kUnits]), (n / kUnits) & 1, abort_flag, err);
        if (!ok) return false;
        u = ms.unit[n % kUnits];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ms.unit_empty[n % kUnits]));
        return __any_sync(0xffffffffu, u.b >= 0) != 0;
    };

    if (!kHalf && warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
        // =================================== queries (by TMA) and their log-sums
        // The log-sums are copied to their place asynchronously, and when the next tile
        // of the unit has been asked for turned into what the sums take there.  A
        // column without a row gets the largest number: it becomes -infinity, as a row's
        // log-sum does that is not finite, but is finite itself, so that no tile is marked for it.
        constexpr float kNoRow = FLT_MAX;
        const int box_rows = p.splits == 1 ? p.per * p.w.group : 128;
        int off[4];  // of the lane's columns from the tile's first log-sum on
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 32 * k + lane, q = p.splits == 1 ? r / p.w.group : 0;
            off[k] = min(r - q * p.w.group, p.w.group) * p.w.Sq + q;  // (below 2^25: the rows of a kv head are below 2^24)
        }
        uint32_t i = 0;  // tiles so far
        bool ok = true;
        auto finish = [&](uint32_t tile) {  // whose log-sums have landed
            float* nl = ms.nl[tile % kNlStages];
            bool odd = false;
#pragma unroll
            for (int k = 0; k < 128; k += 32) {
                const float l = nl[k + lane];
                const bool finite = fabsf(l) < INFINITY;
                odd |= !finite;
                nl[k + lane] = finite ? l * -1.4426950408889634f : -INFINITY;
            }
            odd = __any_sync(0xffffffffu, odd);
            if (lane == 0) ms.odd[tile % kNlStages] = odd;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.q_full[tile % S::kStages]));
        };
        Unit u;
        for (uint32_t n = 0; take(n, ok, u); ++n) {
            if (!u.fresh_rows) continue;
            bool pending = false;
#pragma unroll 1
            for (int t = u.t0; t < u.tiles; t += p.cluster, ++i) {
                const uint32_t st = i % S::kStages;
                if (i >= S::kStages)
                    ok = cache_wait<kSleepShort>(smem_u32(&ms.q_empty[st]), (i / S::kStages + 1) & 1, abort_flag, err);
                if (!ok) break;
                const TileRows x = tile_rows_of(p, u, t);
                if (lane == 0) {
                    const uint32_t bar = smem_u32(kHalf ? &ms.q_here[st] : &ms.q_full[st]);
                    mbar_arrive_expect_tx(bar, box_rows * kD * 2);
#pragma unroll
                    for (int half = 0; half < kD / 64; ++half)
                        tma_load_4d(sbase + st * S::kTile + half * S::kHalf, &tm_q, bar, half * 64,
                                    u.h * p.w.group + x.head, x.query, u.b);
                }
                __syncwarp();
                const float* lse = p.w.lse + ((size_t)u.b * p.w.heads + u.h * p.w.group + x.head) * p.w.Sq + x.query;
                float* nl = ms.nl[i % kNlStages];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 32 * k + lane;
                    if (r < x.columns)
                        cp_async4(smem_u32(&nl[r]), lse + off[k]);
                    else
                        nl[r] = kNoRow;
                }
                cp_async_commit();
                if (pending) {
                    cp_async_wait<1>();
                    finish(i - 1);
                }
                pending = true;
            }
            cp_async_wait<0>();
            if (pending) finish(i - 1);  // (the last one asked for, also where a wait ran out)
        }
        // The last load into each stage has landed before the CTA's shared memory is released.
        if (lane == 0)
            for (uint32_t s = 0; s < (uint32_t)S::kStages && s < i; ++s)
                mbar_wait_drain_1(smem_u32(kHalf ? &ms.q_here[s] : &ms.q_full[s]), ((i - 1 - s) / S::kStages) & 1, err,
                                  kCacheWaitNs);
    } else if (warp == 1 || warp == 3) {
        // ================================ K Q^T: warp 1 of the first key tile, warp 3 of the other
        const int s = warp >> 1;
        const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
        const uint32_t lo_q = uniform((uint32_t)smem_desc_sw128(sbase, 16, 1024));
        const uint32_t t_k = uniform(tmem) + s * S::kKCols, t_s = uniform(tmem) + kTmemS + s * 128;
        uint32_t i = 0, used[2] = {0, 0};  // tiles so far, products so far in each buffer
        bool ok = true;
        Unit u;
        for (uint32_t n = 0; take(n, ok, u); ++n) {
            // (A resident tile is the one that was loaded last: it is let go when the next is taken up.)
            if (p.resident && u.fresh_rows && i++ > 0) commit_one(smem_u32(&ms.q_empty[(i - 2) % S::kStages]));
            const uint32_t a0 = t_k + (n & 1) * 2 * S::kKCols, k_empty = smem_u32(&ms.k_empty[s][n & 1]);
#pragma unroll 1
            for (int t = u.t0; t < u.tiles; t += p.cluster) {
                const uint32_t tile = p.resident ? i - 1 : i++;
                const uint32_t st = tile % S::kStages;
                const int columns = p.splits == 1 ? min(p.per, u.fresh - t * p.per) * p.w.group : tile_rows_of(p, u, t).columns;
                // The halves in both buffers, or (one_half) the tile in the buffer of the unit's parity.
                const int e0 = p.one_half ? (int)(n & 1) : 0, halves = !p.one_half && columns > p.half ? 2 : 1;
                const uint32_t q_empty = p.resident ? 0u : smem_u32(&ms.q_empty[st]);
                const bool last = t + p.cluster >= u.tiles;
                // Lane by lane, what the first half waits for: the buffer, the unit's K, the tile's rows.
                {
                    const uint32_t use = e0 ? used[1] : used[0];
                    uint32_t bar = smem_u32(&ms.s_free[s][e0]), parity = (use + 1) & 1;
                    bool needed = use > 0;
                    if (lane & 1) {
                        bar = smem_u32(&ms.k_full[s][n & 1]);
                        parity = (n >> 1) & 1;
                        needed = t == u.t0;
                    } else if (lane & 2) {
                        bar = smem_u32(&ms.q_full[st]);
                        parity = (tile / S::kStages) & 1;
                        needed = u.fresh_rows;
                    }
                    ok = wait_lanes(bar, parity, needed, abort_flag, err);
                }
                if (!ok) break;
                tc_fence_after();
                const uint32_t b0 = lo_q + ((st * S::kTile) >> 4);
                issue_half<kD>(t_s + e0 * 64, a0, b0, hi, idesc(kHalf, (min(columns, p.half) + 31) & ~31),
                               smem_u32(&ms.s_full[s][e0]), halves == 1 ? q_empty : 0u);
                if (e0)
                    ++used[1];
                else
                    ++used[0];
                if (halves == 2) {
                    if (used[1] > 0)
                        ok = cache_wait<kSleepShort>(smem_u32(&ms.s_free[s][1]), (used[1] + 1) & 1, abort_flag, err);
                    if (!ok) break;
                    ++used[1];
                    tc_fence_after();
                    issue_half<kD>(t_s + 64, a0, b0 + (p.half * 128 >> 4), hi,
                                   idesc(kHalf, (columns - p.half + 31) & ~31), smem_u32(&ms.s_full[s][1]), q_empty);
                }
                if (last) commit_one(k_empty);
            }
            if (!ok) break;
        }
        commit_one(smem_u32(&ms.drain[s]));
        if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain[s]), 0, err, kCacheWaitNs);
    } else if (warp == 2) {
        // ===================================================== units and pages
        if (blockIdx.x == 0)  // lengths out of range are noted once
            for (int b = lane; b < c.B; b += 32) cache_len(c, b, true);
        UnitWalk walk;
        walk.begin(p);
        uint32_t n = 0;  // units so far
        bool ok = true;
        Unit u;
        int at = 0;
        bool more = walk.next(p, u, at);
        for (; ok && more; ++n) {
            int id = __shfl_sync(0xffffffffu, walk.ids, at + lane % kPages);
            const bool there = lane < kPages && (long long)(u.first + lane * kPageTokens) < u.kv;
            if (there && (id < 0 || id >= c.pages)) {
                atomicOr(err, VSA_DEVERR_INDEX);
                id = -1;
            }
            u.held = (int)__ballot_sync(0xffffffffu, there && id >= 0);
            const int h = u.h, held = u.held, ids = id;
            const uint32_t raw = n % kRaw;
            if (n >= kUnits)
                ok = cache_wait<kSleepShort>(smem_u32(&ms.unit_empty[n % kUnits]), (n / kUnits + 1) & 1, abort_flag, err);
            if (!ok) break;
            if (lane == 0) {
                ms.unit[n % kUnits] = u;
                mbar_arrive(smem_u32(&ms.unit_full[n % kUnits]));
            }
            more = walk.next(p, u, at);  // (its page numbers are asked for before this unit's pages)
            if (n >= kRaw)
                ok = cache_wait<kSleepShort>(smem_u32(&ms.raw_empty[raw]), (n / kRaw + 1) & 1, abort_flag, err);
            if (!ok) break;
            // Lanes 0 and 1 announce the bytes of a key tile's two pages; lane 2 i copies
            // page i's codes, lane 2 i + 1 its scales.
            if (lane < 2) mbar_arrive_expect_tx(smem_u32(&ms.raw_full[raw][lane]), S::kPage * __popc((held >> (2 * lane)) & 3));
            __syncwarp();
            const int page = __shfl_sync(0xffffffffu, ids, (lane >> 1) % kPages);
            if (lane < 2 * kPages && ((held >> (lane >> 1)) & 1)) {
                const uint32_t dst = sbase + S::kOffRaw + (raw * kPages + (lane >> 1)) * S::kPage;
                const unsigned char* src = c.pool + ((size_t)page * c.kv_heads + h) * L::kBytes;
                const uint32_t bar = smem_u32(&ms.raw_full[raw][lane >> 2]);
                if (lane & 1)
                    bulk_load(dst + S::kCodes, src + L::kKScale, S::kScales, bar);
                else
                    bulk_load(dst, src, S::kCodes, bar);
            }
            __syncwarp();
        }
        const uint32_t asked = n;  // (a unit that a wait cut short has none asked for)
        if (ok && n >= kUnits)
            ok = cache_wait<kSleepShort>(smem_u32(&ms.unit_empty[n % kUnits]), (n / kUnits + 1) & 1, abort_flag, err);
        if (lane == 0 && ok) {
            ms.unit[n % kUnits].b = -1;
            mbar_arrive(smem_u32(&ms.unit_full[n % kUnits]));
        }
        if (lane < 2)
            for (uint32_t s = 0; s < kRaw && s < asked; ++s)
                mbar_wait_drain_1(smem_u32(&ms.raw_full[s][lane]), ((asked - 1 - s) / kRaw) & 1, err, kCacheWaitNs);
    } else if (warp < 12) {
        // ============================ convert: warps 4..7 the first 128 keys, 8..11 the others
        if (!kHalf) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        const int s = (warp - 4) >> 2, quarter = warp & 3;
        const int key = quarter * 32 + lane;  // of the tile
        const int page = 2 * s + (key >> 6), place = key & 63;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t slot = 0, turn = 0;
        uint32_t i = 0;  // kHalf: row tiles so far
        bool ok = true;
        Unit u;
        for (uint32_t n = 0; take(n, ok, u); ++n) {
            if (kHalf && u.fresh_rows) {
                // The head's rows to fp16 in their places: two threads a row.
                const int th = threadIdx.x - 128, row = th >> 1, side = th & 1;
                const uint32_t st = i % S::kStages;
                ok = cache_wait<kSleepShort>(smem_u32(&ms.q_here[st]), (i / S::kStages) & 1, abort_flag, err);
                if (!ok) break;
                const int e = half_row<kD>(sbase + st * S::kTile, row, side);
                if (side == 0)
                    ms.cf[i % kNlStages][row] = logit_scale(p.w.scale_log2, c.kv_scale ? c.kv_scale[u.h] : 1.f, e);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.q_full[st]));
                ++i;
            }
            const int par = n & 1;
            ok = cache_wait<kSleepShort>(smem_u32(&ms.raw_full[slot][s]), turn & 1, abort_flag, err);
            if (ok && n >= 2) ok = cache_wait<kSleepShort>(smem_u32(&ms.k_empty[s][par]), ((n >> 1) + 1) & 1, abort_flag, err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t raw = sbase + S::kOffRaw + (slot * kPages + page) * S::kPage;
            const uint32_t codes = raw + place * L::kRow, scales = raw + S::kCodes + place * L::kGroups;
            const uint32_t to = t_lane + (par * 2 + s) * S::kKCols;
            // (A short loop: code that runs once a unit costs more to fetch than to run.)
#pragma unroll 1
            for (int piece = 0; piece < kD / 32; ++piece) {
                const uint4 x = lds128(codes + piece * 16);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint16_t sc;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(sc) : "r"(scales + piece * 2));
                const uint32_t two = e4m3_to_f16(sc);
                const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
                uint32_t out[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t y[4];
                    e2m1_to_f16(w[k], y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t z = mul_f16x2(y[j], k < 2 ? s0 : s1);
                        out[4 * k + j] = kHalf ? z : f16_to_bf16x2(z);
                    }
                }
                tmem_st16(to + piece * 16, out);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.raw_empty[slot]));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.k_full[s][par]));
            if (++slot == kRaw) {
                slot = 0;
                ++turn;
            }
        }
    } else if (warp < 28) {
        // ============================ sums: a warpgroup for each key tile s and buffer e
        if (!kHalf) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        const int s = (warp - 12) >> 3, e = ((warp - 12) >> 2) & 1, quarter = warp & 3;
        const int key = quarter * 32 + lane;
        const uint32_t t_s = tmem + ((uint32_t)(quarter * 32) << 16) + kTmemS + s * 128 + e * 64;
        uint32_t i = 0, used = 0;  // tiles, halves of this group so far
        bool ok = true;
        Unit u;
        for (uint32_t n = 0; take(n, ok, u); ++n) {
            const int x = u.first + s * 128 + key;  // the thread's key
            const bool there = (u.held >> (2 * s + (key >> 6))) & 1;
            const size_t at = ((size_t)u.b * c.kv_heads + u.h) * ((size_t)c.width * kPageTokens) + x;
            float before = 0.f;
            if ((e == 0 || p.one_half) && p.cluster == 1 && p.w.weights && x < u.kv) before = p.w.weights[at];
            if (p.one_half && (int)(n & 1) != e) {
                if (p.resident && u.fresh_rows) ++i;
                continue;
            }
            float total = 0.f;
            if (p.resident && u.fresh_rows) ++i;
            const int c0 = p.one_half ? 0 : e * p.half;
            // Columns from `low` on are rows that see the key; of the tile at hand.  (A call's steps
            // together are below 2^24 rows and a tile, whole tiles of a group of up to 128 heads; wider
            // groups set `low` for each tile, or never.)
            const int step = p.splits == 1 ? p.per * p.w.group * p.cluster : 0;
            int low = -0x40000000;
            if (p.w.causal && p.splits == 1) low = (max(x - (u.kv - u.fresh), 0) - u.t0 * p.per) * p.w.group;
#pragma unroll 1
            for (int t = u.t0; t < u.tiles; t += p.cluster, low -= step) {
                const uint32_t place = (p.resident ? i - 1 : i++) % kNlStages;
                int columns;
                if (p.splits == 1) {
                    columns = min(p.per, u.fresh - t * p.per) * p.w.group;
                } else {
                    const TileRows rows = tile_rows_of(p, u, t);
                    columns = rows.columns;
                    if (p.w.causal) low = x - (u.kv - u.fresh) > rows.query ? 128 : 0;
                }
                const int end = min(c0 + p.half, columns);
                if (c0 >= end) continue;
                ok = cache_wait<kSleepShort>(smem_u32(&ms.s_full[s][e]), used++ & 1, abort_flag, err);
                if (!ok) break;
                tc_fence_after();
                const bool odd = *reinterpret_cast<volatile int*>(&ms.odd[place]);
                // (Columns past the last row are products with zeros, and weigh 2^-infinity, where
                // the tile ends with all of the tensor's queries; else they may be products with
                // anything: with queries behind the sequence's, or, in the last tile of a group of
                // more than 128 heads, with the next kv head's.)
                const bool plain = !odd && (end == c0 + p.half || (p.splits == 1 && u.fresh == p.w.Sq)) &&
                                   !__any_sync(0xffffffffu, low > c0);
                float2 a = make_float2(0.f, 0.f), b = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int c1 = c0; c1 < end; c1 += 32) {
                    uint32_t v[32];
                    tmem_ld32(t_s + c1 - c0, v);
                    const float4* nl = reinterpret_cast<const float4*>(&ms.nl[place][c1]);
                    const float4* cf = reinterpret_cast<const float4*>(&ms.cf[place][c1]);
                    tmem_wait_ld();
                    if (c1 + 32 >= end) {
                        // All of S is in registers: its columns may take the next tile's.
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&ms.s_free[s][e]));
                    }
                    if (plain) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 l = nl[k / 4], f = kHalf ? cf[k / 4] : make_float4(u.c2, u.c2, u.c2, u.c2);
                            const float2 e0 = __ffma2_rn(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                                         make_float2(f.x, f.y), make_float2(l.x, l.y));
                            const float2 e1 = __ffma2_rn(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])),
                                                         make_float2(f.z, f.w), make_float2(l.z, l.w));
                            a = __fadd2_rn(a, make_float2(ex2_approx(e0.x), ex2_approx(e0.y)));
                            b = __fadd2_rn(b, make_float2(ex2_approx(e1.x), ex2_approx(e1.y)));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 l = nl[k / 4];
                            const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int col = c1 + k + q;
                                const bool sees = col >= low && col < columns && ls[q] > -INFINITY;
                                const float y = ex2_approx(fmaf(__uint_as_float(v[k + q]), kHalf ? ms.cf[place][c1 + k + q] : u.c2, ls[q]));
                                a.x += sees ? y : 0.f;
                            }
                        }
                    }
                }
                total += (a.x + a.y) + (b.x + b.y);
            }
            if (!ok) break;
            // The two halves' shares.
            if (!p.one_half) {
                float* part = &ms.part[n & 1][s * 128 + key];
                const uint32_t part_full = smem_u32(&ms.part_full[s][n & 1]), part_empty = smem_u32(&ms.part_empty[s][n & 1]);
                if (e == 1) {
                    if (n >= 2) ok = cache_wait<kSleepShort>(part_empty, ((n >> 1) + 1) & 1, abort_flag, err);
                    if (!ok) break;
                    *part = total;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(part_full);
                    continue;
                }
                ok = cache_wait<kSleepShort>(part_full, (n >> 1) & 1, abort_flag, err);
                if (!ok) break;
                total += *part;
                __syncwarp();
                if (lane == 0) mbar_arrive(part_empty);
            }
            if (!there) total = 0.f;  // (a page that is not there has no weight)
            if (p.cluster > 1)
                ms.sums[s * 128 + key] = total;
            else if (x < u.kv)
                p.w.out[at] = before + total;
        }
    }

    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    if (p.cluster > 1) {
        // The cluster's one unit: its CTAs' sums in the order of their ranks, a share of the keys each.
        UnitWalk walk;
        walk.begin(p);
        walk.rank = 0;
        Unit u;
        int at_page;
        const bool has = walk.next(p, u, at_page);
        const int rank = blockIdx.x % p.cluster;
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
        const int each = kKeys / p.cluster, key = rank * each + (int)threadIdx.x;
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
    fill_rest(p.w, true);
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

template <int kD, bool kHalf>
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
    static std::atomic<int> known{0};
    // The register split draws on the launch's registers; with fewer, setmaxnreg
    // would wait forever, so such a build is refused.
    int regs = 0;
    cudaError_t e = launch_registers(weigh_chunk_kernel<kD, kHalf>, known, &regs);
    if (e != cudaSuccess) return e;
    if (!kHalf && regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    e = allow_smem(weigh_chunk_kernel<kD, kHalf>, smem_bytes<kD>(), done);
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
    e = cudaLaunchKernelEx(&cfg, weigh_chunk_kernel<kD, kHalf>, map, p);
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
    p.resident = tiles == 1;
    p.half = 64;
    p.one_half = p.resident && w.Sq * w.group <= p.half;
    const int grid = p.cluster > 1 ? (int)most * p.cluster : (int)std::min<long long>(num_sms, most);
    if (p.resident) return D == 64 ? launch<64, true>(p, grid, stream) : launch<128, true>(p, grid, stream);
    return D == 64 ? launch<64, false>(p, grid, stream) : launch<128, false>(p, grid, stream);
}

}  // namespace vsa
