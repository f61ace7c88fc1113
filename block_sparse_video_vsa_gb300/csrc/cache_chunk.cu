// Attention over the 4-bit paged cache, many query rows a kv head (chunks of
// tokens): the same function as token_kernel (cache_attn.cu), on tcgen05.
//
// Tensor bound for long chunks (4 * D flops for each row and key), so the
// structure is the fine stage's: 128 query rows a unit, one TMEM lane each,
// 128 keys (two pages) a step, Q and P as A operands in TMEM, two softmax
// groups that take the steps in turn with a reference, sum and output of their
// own, joined at the unit's end.  What differs is where K and V come from: two
// producer warps copy pages (halves: codes and scales of K or of V) into rings,
// and two warpgroups, one for K and one for V, convert each step's two pages
// into fp16 tiles (exact, see cache.cuh) in the 128-byte swizzled layout the
// tensor core reads.  So a page crosses HBM and L2 in 9 bits a pair of K and V
// elements instead of 32.
//  * Warp roles (640 threads): warps 0 and 2 copy pages; warp 1 owns TMEM and
//    issues Q K^T, warp 3 P V; warps 4..7 convert K, warps 8..11 V; warps
//    12..15 and 16..19 are the softmax groups (group 0 the CTA's even steps).
//  * TMEM (512 columns): S [0,128); P (fp16 pairs) [128,192); Q [192,256);
//    O_0 [256,384); O_1 [384,512).
//  * A query row is scaled by a power of two on its way to fp16 (its bf16
//    values keep all their bits down to 2^-31 of its largest, see q_exponent)
//    and the inverse joins its softmax scale.
//  * Every wait is bounded; one that runs out raises the CTA's abort flag and
//    the device error word, and each role winds down.
//  * Measured (GB300): 1560 queries x 40 heads of 128 over 32760 keys, 960 us =
//    1.09 PFLOP/s (57% of the measured bf16 burst).  A step takes some 2010
//    cycles of an SM, of which the tensor pipe is busy 51%; the converting and
//    softmax warps and the waiting roles issue 5540 instructions for it, 0.69 a
//    scheduler and cycle.  1% of them are spills (144 bytes stored and 248 loaded
//    by ptxas at D = 128, 112 and 216 at D = 64; 45 loads and 9 stores a step).
//    With one converting warpgroup it took 1200 us, with
//    256 rows a unit, a tile a softmax group (a conversion then serves twice the
//    rows, but TMEM has no room for Q, so Q K^T reads both operands from shared
//    memory, nor for a second S to work ahead in) 1160 to 1215: at D = 128, where
//    all was measured; at D = 64 two tiles would leave room for Q.  How long the
//    waits sleep (20 to 250 ns) changes nothing.
#include "cache.cuh"

namespace vsa {

namespace {

constexpr int kChunkThreads = 640;
constexpr int kKStages = 2;
constexpr int kMetaSteps = 16;
constexpr int kRawHalves = 4;  // slots of a ring of half pages
constexpr int kRowPitch = 256 + 16;  // bytes of a row on its way in (queries) or out: rows start in other banks
// Registers: 5 warpgroups launched with 96 each; the shares add up to 480.
constexpr int kLaunchRegs = 96, kIssueRegs = 48, kConvertRegs = 56, kSoftRegs = 160;
static_assert(kIssueRegs + 2 * kConvertRegs + 2 * kSoftRegs <= 5 * kLaunchRegs, "register split exceeds the launch");

constexpr int kTmemS = 0, kTmemP = 128, kTmemQ = 192, kTmemO0 = 256, kTmemO1 = 384;

template <int kD>
struct ChunkSmem {
    static constexpr int kHalf = 128 * 128;          // 128 keys x 64 channels of fp16, swizzled
    static constexpr int kTile = kHalf * (kD / 64);  // K or V of a step
    static constexpr int kCodes = kPageTokens * kD / 2, kScales = kPageTokens * kD / 16;
    static constexpr int kRawBytes = kCodes + kScales;
    static constexpr int kVStages = kD == 64 ? 3 : 2;  // (as many as fit)
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kKStages * kTile;
    static constexpr int kOffRaw = kOffV + kVStages * kTile;  // [K, V][slot]
    static constexpr int kOffRows = kOffRaw + 2 * kRawHalves * kRawBytes;
    static constexpr int kOffMisc = kOffRows + 128 * kRowPitch;
};

// A softmax warp's walk, its present unit and the two after that: kept in
// shared memory, the steps need the registers.
struct SoftWalk {
    Walk walk;
    Segment unit[3];
};

struct __align__(16) ChunkMisc {
    uint64_t raw_full[2][kRawHalves], raw_empty[2][kRawHalves];  // of K, of V
    uint64_t k_full[kKStages], k_empty[kKStages];
    uint64_t v_full[3], v_empty[3];
    uint64_t s_full[2];  // per softmax group: S of its next step is ready
    uint64_t s_free;     // S has been loaded into registers
    uint64_t p_full;     // P of the step (and any rescaling of O) is in TMEM
    uint64_t pv_grp[2];  // per group: P V of its step has completed
    uint64_t unit_done;  // every P V of the unit has completed
    uint64_t rows_full;  // the next unit's queries are in the row buffer
    uint64_t q_full, q_empty;
    uint64_t o_free;     // O_0 and O_1 have been read by the unit's epilogue
    uint64_t drain[2];
    int2 key0[kMetaSteps];   // first key of a step's pages (kNoKey: none)
    int raw_keys[2][kRawHalves];  // keys of a half page's slots that the sequence has (0: passed over)
    float xm[2][2][128];     // [unit parity][group][row]: reference, sum at the unit's end
    float xl[2][2][128];
    float scale[2][128];     // [unit parity][row]: logit -> log2 units
    SoftWalk soft[8];
    PlanScratch plan;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kNoKey = 0x7FFFFFFF;  // beyond every row's limit

template <int kD>
constexpr int chunk_smem() {
    return ChunkSmem<kD>::kOffMisc + (int)sizeof(ChunkMisc) + 1024;  // slack for 1024-byte alignment
}
static_assert(chunk_smem<128>() <= 232448, "shared memory of the chunk kernel");

// As idesc_bf16_f32, fp16 inputs.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16_f32(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

__device__ __forceinline__ float max3f(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Maximum of x[0..63], as four running chains.
__device__ __forceinline__ float chunk_max64(const float* x) {
    float a[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int c = 4; c < 60; c += 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = max3f(a[j], x[c + j], x[c + 4 + j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = fmaxf(a[j], x[60 + j]);
    return fmaxf(max3f(a[0], a[1], a[2]), a[3]);
}

// exp2(x * c2 - mb) of 64 logits as 32 fp16 pairs; adds the fp32 values to l.
__device__ __forceinline__ void chunk_exp64(const float* x, float c2, float mb, uint32_t* pk, float& l) {
    const float2 c2v = make_float2(c2, c2), nmb = make_float2(-mb, -mb);
    float2 s01 = make_float2(0.f, 0.f), s23 = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 64; c += 4) {
        const float2 a01 = __ffma2_rn(make_float2(x[c], x[c + 1]), c2v, nmb);
        const float2 a23 = __ffma2_rn(make_float2(x[c + 2], x[c + 3]), c2v, nmb);
        const float p0 = ex2_approx(a01.x), p1 = ex2_approx(a01.y);
        const float p2 = ex2_approx(a23.x), p3 = ex2_approx(a23.y);
        s01 = __fadd2_rn(s01, make_float2(p0, p1));
        s23 = __fadd2_rn(s23, make_float2(p2, p3));
        pk[c >> 1] = pack_f16x2(p0, p1);
        pk[(c >> 1) + 1] = pack_f16x2(p2, p3);
    }
    l += (s01.x + s01.y) + (s23.x + s23.y);
}

__device__ __forceinline__ int steps_of(const Segment& s) { return (s.last - s.first + 1) >> 1; }

__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 x;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
    return x;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Row r of unit s in q or out, in 16-byte pieces; real: there is such a row.
struct RowAt {
    int head, qi;
    bool real;
    size_t at;
};
template <int kD>
__device__ __forceinline__ RowAt row_at(const AttnParams& p, const Segment& s, int r) {
    RowAt x;
    const int row = s.t * 128 + r;
    x.real = row < p.Sq * p.group;
    x.qi = x.real ? row / p.group : 0;
    x.head = s.h * p.group + (x.real ? row - x.qi * p.group : 0);
    x.at = (((size_t)s.b * p.Sq + x.qi) * p.heads + x.head) * (kD / 8);
    return x;
}

// This thread's asynchronous 16-byte copies arrive on `bar` once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Rows [r0, r0 + 64) of a unit that has nothing to attend (a whole warp calls it).
template <int kD>
__device__ __forceinline__ void no_keys(const AttnParams& p, const Segment& s, int r0) {
    constexpr int kLanes = kD / 8;  // of a row
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int r = r0; r < r0 + 64; r += 32) {
        const RowAt x = row_at<kD>(p, s, r + lane);
        if (x.real && p.lse) p.lse[((size_t)s.b * p.heads + x.head) * p.Sq + x.qi] = -INFINITY;
        const unsigned reals = __ballot_sync(0xffffffffu, x.real);
#pragma unroll 1
        for (int k = lane / kLanes; k < 32; k += 32 / kLanes) {
            const size_t at = __shfl_sync(0xffffffffu, x.at, k) + lane % kLanes;
            if ((reals >> k) & 1u) p.out[at] = make_uint4(0, 0, 0, 0);
        }
    }
}

// Softmax thread of a row: puts its query (at `src` in shared memory, the second
// half of its channels 128 bytes after the first) into the
// TMEM Q columns of its lane as fp16, scaled by a power of two, and returns the
// power.  The largest magnitude is found as integers: the bit patterns of bf16
// magnitudes are in their order.  (Short loops: code that runs once a unit costs
// more to fetch than to run.)
template <int kD>
__device__ __forceinline__ int stage_query(uint32_t src, uint32_t t_q) {
    uint32_t mx = 0u;
#pragma unroll 1
    for (int c = 0; c < kD * 2; c += 64) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = lds128(src + c * (128 / kD) + 16 * i);
            mx = __vimax3_u16x2(mx, x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
            mx = __vimax3_u16x2(mx, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu);
        }
    }
    const int e = q_exponent(__uint_as_float(max(mx & 0xFFFFu, mx >> 16) << 16));
    const float f = pow2i(e);
#pragma unroll 1
    for (int c = 0; c < kD * 2; c += 64) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 x = lds128(src + c * (128 / kD) + 16 * i);
            w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 x = __fmul2_rn(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), make_float2(f, f));
            w[i] = pack_f16x2(x.x, x.y);
        }
        tmem_st16(t_q + c / 4, w);
    }
    tmem_wait_st();
    return e;
}

// Half of one key's codes of K or V and their scales (`codes`, `scales`: the
// key's, in shared memory) to row `row` of a fp16 tile: channels [h kD / 2,
// (h + 1) kD / 2).  Two threads a key, neighbouring lanes, each starting at
// another 16-byte piece (kD = 128) so that neither the loads nor the swizzled
// stores of 8 lanes meet in a bank.
template <int kD>
__device__ __forceinline__ void convert_half_row(uint32_t codes, uint32_t scales, int row, int h, bool zero,
                                                 uint32_t tile) {
    constexpr int kPieces = kD / 64;  // of 32 channels
    const int flip = kPieces == 2 ? ((row >> 1) ^ h) & 1 : 0;
    uint4 w[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = lds128(codes + h * (kD / 4) + (i ^ flip) * 16);
    uint32_t sc = 0u;  // scale bytes, two a piece
    if (!zero) {
        if constexpr (kD == 128)
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(sc) : "r"(scales + h * 4));
        else
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc) : "r"(scales + h * 2));
    }
    // Unit u of 16 bytes (8 channels) of a 64-channel half goes to u ^ (row & 7).
    const uint32_t base = tile + row * 128 + (kD == 128 ? h * ChunkSmem<kD>::kHalf : 0);
    const uint32_t low = (row & 3) << 4, top = (row & 4) << 4;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int c = kD == 128 ? i ^ flip : h;  // piece of the 64 channels
        const uint32_t two = e4m3_to_f16(kD == 128 ? sc >> (16 * c) : sc);
        const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        const uint32_t at = base + ((c << 6) ^ top);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
            e2m1_to_f16(ws[k], y);
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = mul_f16x2(y[j], k < 2 ? s0 : s1);
            sts128(at + ((k << 4) ^ low), y[0], y[1], y[2], y[3]);
        }
    }
}

// A place in a ring of kN slots: the slot and how many times the ring has been gone round.
template <int kN>
struct Ring {
    int slot = 0;
    uint32_t turn = 0;
    __device__ __forceinline__ void step() {
        if (++slot == kN) {
            slot = 0;
            ++turn;
        }
    }
    __device__ __forceinline__ uint32_t full() const { return turn & 1; }         // parity of the slot's next filling
    __device__ __forceinline__ uint32_t empty() const { return (turn + 1) & 1; }  // and of its last emptying (turn > 0)
};

template <int kD>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(AttnParams p) {
    using L = PageLayout<kD>;
    using Sm = ChunkSmem<kD>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    ChunkMisc& ms = *reinterpret_cast<ChunkMisc*>(smem + Sm::kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &ms.abort_flag;
    unsigned int* err = p.c.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2 * kRawHalves; ++s) {
            mbar_init(smem_u32(&ms.raw_full[0][s]), 1);
            mbar_init(smem_u32(&ms.raw_empty[0][s]), 4);
        }
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(smem_u32(&ms.k_full[s]), 4);
            mbar_init(smem_u32(&ms.k_empty[s]), 1);
        }
        for (int s = 0; s < Sm::kVStages; ++s) {
            mbar_init(smem_u32(&ms.v_full[s]), 4);
            mbar_init(smem_u32(&ms.v_empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&ms.s_full[s]), 1);
            mbar_init(smem_u32(&ms.pv_grp[s]), 1);
            mbar_init(smem_u32(&ms.drain[s]), 1);
        }
        mbar_init(smem_u32(&ms.s_free), 4);
        mbar_init(smem_u32(&ms.p_full), 4);
        mbar_init(smem_u32(&ms.unit_done), 1);
        mbar_init(smem_u32(&ms.rows_full), 256);
        mbar_init(smem_u32(&ms.q_full), 4);
        mbar_init(smem_u32(&ms.q_empty), 1);
        mbar_init(smem_u32(&ms.o_free), 8);
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    // The tiles start as zeros: the tensor core multiplies rows that no page
    // filled (an odd last page, pages passed over) by probabilities of zero.
    {
        int4* z = reinterpret_cast<int4*>(smem);
        for (int e = threadIdx.x; e < Sm::kOffRaw / 16; e += kChunkThreads) z[e] = make_int4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    early();
    Walk walk;
    if (!walk.begin(p, ms.plan)) return;  // the whole CTA: TMEM is not allocated yet
    if (warp == 1) {
        tmem_alloc(smem_u32(&ms.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_base;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0 || warp == 2) {
            // ================================ page producers: warp 0 K, warp 2 V
            const int side = warp >> 1;
            Ring<kRawHalves> raw;
            uint32_t g = 0;  // steps so far
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                if (sg.first == sg.last) {  // a unit without pages: zeros, half of the rows by each producer
                    no_keys<kD>(p, sg, side * 64);
                    continue;
                }
                const unsigned char* pool = p.c.pool + (size_t)sg.h * L::kBytes + (side ? L::kV : 0);
                for (int base = sg.first; base < sg.last && ok; base += 32) {
                    int logical = 0, id = -1;
                    if (base + lane < sg.last) look_up(p, sg, base + lane, logical, id);
                    const int n = min(32, sg.last - base);
                    for (int i = 0; i < n; ++i, raw.step()) {
                        const int page = __shfl_sync(0xffffffffu, id, i);
                        const int first = __shfl_sync(0xffffffffu, logical, i) * kPageTokens;
                        const int slot = raw.slot;
                        if (raw.turn > 0) {
                            ok = cache_wait<kSleepLong>(smem_u32(&ms.raw_empty[side][slot]), raw.empty(), abort_flag, err);
                            if (!ok) break;
                        }
                        if (lane == 0) {
                            if (side == 0) {  // (steps start at even pages of the segment: 32 is even)
                                int* key0 = &ms.key0[g % kMetaSteps].x;
                                key0[i & 1] = page < 0 ? kNoKey : first;
                                if (!(i & 1)) key0[1] = kNoKey;
                            }
                            ms.raw_keys[side][slot] = page < 0 ? 0 : sg.len.kv - first;
                            const uint32_t bar = smem_u32(&ms.raw_full[side][slot]);
                            if (page < 0) {
                                mbar_arrive(bar);
                            } else {
                                mbar_arrive_expect_tx(bar, Sm::kRawBytes);
                                const uint32_t dst = sbase + Sm::kOffRaw + (side * kRawHalves + slot) * Sm::kRawBytes;
                                const unsigned char* src = pool + (size_t)page * p.c.kv_heads * L::kBytes;
                                bulk_load(dst, src, Sm::kCodes, bar);
                                bulk_load(dst + Sm::kCodes, src + (side ? L::kVScale - L::kV : L::kKScale), Sm::kScales,
                                          bar);
                            }
                        }
                        if ((i & 1) || base + i + 1 == sg.last) ++g;
                        __syncwarp();
                    }
                }
            }
            // The last copy into each slot: of this turn up to raw.slot, of the last one from there on.
            if (lane == 0) {
                for (int s = 0; s < kRawHalves; ++s) {
                    const uint32_t turns = raw.turn + (s < raw.slot ? 1 : 0);
                    if (turns > 0)
                        mbar_wait_drain_1(smem_u32(&ms.raw_full[side][s]), (turns - 1) & 1, err, kCacheWaitNs);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ========================================================= Q K^T
            const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
            const uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
            const uint32_t lo_k = (uint32_t)smem_desc_sw128(sbase + Sm::kOffK, 16, 1024);
            Ring<kKStages> ring;
            uint32_t g = 0, ul = 0;  // so far: steps, units with steps
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                const int nst = steps_of(sg);
                if (nst == 0) continue;
                ok = cache_wait<kSleepShort>(smem_u32(&ms.q_full), ul++ & 1, abort_flag, err);
                for (int t = 0; t < nst && ok; ++t, ++g, ring.step()) {
                    if (g >= 1)
                        ok = cache_wait<kSleepShort>(smem_u32(&ms.s_free), (g - 1) & 1, abort_flag, err);
                    const int slot = ring.slot;
                    if (ok)
                        ok = cache_wait<kSleepShort>(smem_u32(&ms.k_full[slot]), ring.full(), abort_flag, err);
                    if (!ok) break;
                    const uint32_t b0 = lo_k + ((uint32_t)(slot * Sm::kTile) >> 4);
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk)
                        mma_ts_warp(tmem + kTmemS, tmem + kTmemQ + kk * 8,
                                    b0 + (((kk >> 2) * Sm::kHalf + (kk & 3) * 32) >> 4), hi, idesc, kk > 0);
                    mma_commit_warp(smem_u32(&ms.s_full[g & 1]));
                    mma_commit_warp(smem_u32(&ms.k_empty[slot]));
                }
                if (!ok) break;
                mma_commit_warp(smem_u32(&ms.q_empty));
            }
            mma_commit_warp(smem_u32(&ms.drain[0]));
            if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain[0]), 0, err, kCacheWaitNs);
            __syncwarp();
        } else if (warp == 3) {
            // =========================================================== P V
            const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
            const uint32_t idesc = idesc_f16_f32(128, kD, 0, 1);
            const uint32_t lo_v = (uint32_t)smem_desc_sw128(sbase + Sm::kOffV, Sm::kHalf, 1024);
            Ring<Sm::kVStages> ring;
            uint32_t g = 0, ul = 0;  // so far: steps, units with steps
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                const int nst = steps_of(sg);
                if (nst == 0) continue;
                // O_0 and O_1 start over once the last epilogue has read them.
                if (ul >= 1) ok = cache_wait<kSleepShort>(smem_u32(&ms.o_free), (ul - 1) & 1, abort_flag, err);
                for (int t = 0; t < nst && ok; ++t, ++g, ring.step()) {
                    const int slot = ring.slot;
                    ok = cache_wait<kSleepShort>(smem_u32(&ms.p_full), g & 1, abort_flag, err) &&
                         cache_wait<kSleepShort>(smem_u32(&ms.v_full[slot]), ring.full(), abort_flag, err);
                    if (!ok) break;
                    const uint32_t b0 = lo_v + ((uint32_t)(slot * Sm::kTile) >> 4);
                    const uint32_t d = tmem + ((g & 1) ? kTmemO1 : kTmemO0);
                    const uint32_t acc = t >= 2 ? 1u : 0u;  // a group's first step of the unit overwrites its O
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts_warp(d, tmem + kTmemP + kk * 8, b0 + ((kk * 2048) >> 4), hi, idesc,
                                    acc | (kk > 0 ? 1u : 0u));
                    if (sg.first + 2 * t + 1 < sg.last) {
#pragma unroll
                        for (int kk = 4; kk < 8; ++kk)
                            mma_ts_warp(d, tmem + kTmemP + kk * 8, b0 + ((kk * 2048) >> 4), hi, idesc, 1u);
                    }
                    mma_commit_warp(smem_u32(&ms.pv_grp[g & 1]));
                    mma_commit_warp(smem_u32(&ms.v_empty[slot]));
                }
                if (!ok) break;
                ++ul;
                mma_commit_warp(smem_u32(&ms.unit_done));
            }
            mma_commit_warp(smem_u32(&ms.drain[1]));
            if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain[1]), 0, err, kCacheWaitNs);
            __syncwarp();
        }
    } else if (warp < 12) {
        // ============================================ convert: warps 4..7 K, 8..11 V
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        const int side = (warp - 4) >> 2;
        const int th = threadIdx.x & 127, key = th >> 1, h = th & 1;  // two threads a key of a page
        const uint32_t raw_at = sbase + Sm::kOffRaw + side * kRawHalves * Sm::kRawBytes;
        const uint32_t tiles = sbase + (side ? Sm::kOffV : Sm::kOffK);
        const uint32_t full = smem_u32(side ? ms.v_full : ms.k_full), empty = smem_u32(side ? ms.v_empty : ms.k_empty);
        const int stages = side ? Sm::kVStages : kKStages;
        Ring<kRawHalves> raw;
        int st = 0;
        uint32_t turn = 0;  // of the tile's ring
        bool ok = true;
        for (Segment sg; ok && walk.next(p, sg);) {
            for (int i = sg.first; i < sg.last && ok; i += 2) {
                const int held = min(2, sg.last - i);
                if (turn > 0) ok = cache_wait<kSleepLong>(empty + 8 * st, (turn + 1) & 1, abort_flag, err);
                for (int which = 0; which < held && ok; ++which, raw.step()) {
                    ok = cache_wait<kSleepLong>(smem_u32(&ms.raw_full[side][raw.slot]), raw.full(), abort_flag, err);
                    if (!ok) break;
                    const uint32_t at = raw_at + raw.slot * Sm::kRawBytes;
                    // Slots past the sequence's end hold anything, and a page passed
                    // over nothing: their V is zero (their K is masked).
                    const bool zero = key >= *reinterpret_cast<volatile int*>(&ms.raw_keys[side][raw.slot]);
                    convert_half_row<kD>(at + key * (kD / 2), at + Sm::kCodes + key * (kD / 16),
                                         which * kPageTokens + key, h, zero, tiles + st * Sm::kTile);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&ms.raw_empty[side][raw.slot]));
                }
                if (!ok) break;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full + 8 * st);
                if (++st == stages) {
                    st = 0;
                    ++turn;
                }
            }
        }
    } else {
        // ============================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int G = (warp - 12) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t o_mine = t_lane + (G ? kTmemO1 : kTmemO0);
        constexpr int dh = kD / 2;  // output columns of this thread: [G * dh, G * dh + dh)
        const float ninf = -INFINITY;
        bool ok = true;
        uint32_t g0 = 0, ul = 0;  // steps before the unit, units with steps
        SoftWalk& sw = ms.soft[warp - 12];
        auto advance = [&](int to) -> bool {  // the walk's next unit with steps into sw.unit[to]
            Walk w = sw.walk;
            Segment s;
            bool has;
            do has = w.next(p, s);
            while (has && s.first == s.last);
            __syncwarp();
            if (lane == 0) {
                sw.walk = w;
                sw.unit[to] = s;
            }
            __syncwarp();
            return has;
        };
        if (lane == 0) sw.walk = walk;
        __syncwarp();
        const uint32_t row_s = sbase + Sm::kOffRows + r * kRowPitch;  // the row's place in the row buffer
        auto queries = [&](const Segment& s, uint32_t u) {  // of unit s, the u-th
            if (ok) ok = cache_wait<kSleepShort>(smem_u32(&ms.rows_full), u & 1, abort_flag, err);
            if (ok) {
                tc_fence_after();
                const int e = stage_query<kD>(row_s, t_lane + kTmemQ);
                ms.scale[u & 1][r] = logit_scale(p.scale_log2, p.c.kv_scale ? p.c.kv_scale[s.h] : 1.f, e);
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.q_full));
        };
        // This warp's share of the queries of unit s on their way to the row
        // buffer: half G of the channels of its quarter's rows.
        const uint32_t mine = row_s + G * 128;
        auto ask_queries = [&](const Segment& s) {
            constexpr int kLanes = kD / 16, kRows = 32 / kLanes;  // lanes of a half row, rows a turn
            const RowAt x = row_at<kD>(p, s, r);
            const unsigned reals = __ballot_sync(0xffffffffu, x.real);
            const int sub = lane % kLanes;
#pragma unroll 1
            for (int k = lane / kLanes; k < 32; k += kRows) {
                const size_t at = __shfl_sync(0xffffffffu, x.at, k) + G * kLanes + sub;
                if ((reals >> k) & 1u) cp_async16(mine + (k - lane) * kRowPitch + sub * 16, p.q + at);
            }
            cp_async_arrive(smem_u32(&ms.rows_full));
        };
        auto place = [](uint32_t u) { return (int)(u % 3u); };
        bool more = advance(0), next = more && advance(1);
        if (more) {
            ask_queries(sw.unit[0]);
            if (G == 0) queries(sw.unit[0], 0);
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
            if (next) ask_queries(sw.unit[1]);
        }
#pragma unroll 1
        for (; more; ++ul) {
            const Segment& sg = sw.unit[place(ul)];
            const int nst = steps_of(sg);
            int lim = sg.len.kv;  // first key the row does not see
            if (p.causal && sg.t * 128 + r < sg.len.q * p.group)
                lim = max(0, min(lim, sg.len.kv - sg.len.q + (sg.t * 128 + r) / p.group + 1));
            float c2 = 0.f, m = ninf, l = 0.f;
            bool first = true;
#pragma unroll 1
            for (int t = (int)((g0 + G) & 1); t < nst; t += 2) {
                const uint32_t gs = g0 + t;
                if (ok) ok = cache_wait<kSleepShort>(smem_u32(&ms.s_full[G]), (gs >> 1) & 1, abort_flag, err);
                tc_fence_after();
                c2 = ms.scale[ul & 1][r];
                const int2 k0 = ms.key0[gs % kMetaSteps];
                // Keys of the two pages that this row sees (none where no page is).
                const int va = lim - k0.x, vb = lim - k0.y;
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32)
                    tmem_ld32(t_lane + kTmemS + c, *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
                tmem_wait_ld();
                // S is in registers: its columns may take the next step's.
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.s_free));
                if (__any_sync(0xffffffffu, va < kPageTokens || vb < kPageTokens)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        x[c] = c < va ? x[c] : ninf;
                        x[64 + c] = c < vb ? x[64 + c] : ninf;
                    }
                }
                const float mx = fmaxf(chunk_max64(x), chunk_max64(x + 64)) * c2;
                // The reference m follows the maximum lazily: O and l are rescaled on a jump only.
                float alpha = 1.f;
                if (mx > m + (kCacheHeadroom + kCacheRescale)) {
                    const float next = mx - kCacheHeadroom;
                    alpha = m == ninf ? 0.f : ex2_approx(m - next);
                    m = next;
                    l *= alpha;
                }
                const float mb = m == ninf ? 0.f : m;
                uint32_t pk[64];
                chunk_exp64(x, c2, mb, pk, l);
                chunk_exp64(x + 64, c2, mb, pk + 32, l);
                // P V of the step before (the other group's) has read P.
                if (gs > 0 && ok)
                    ok = cache_wait<kSleepShort>(smem_u32(&ms.pv_grp[G ^ 1]), ((gs - 1) >> 1) & 1, abort_flag, err);
                tc_fence_after();
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 64; c += 16)
                        tmem_st16(t_lane + kTmemP + c, *reinterpret_cast<uint32_t(*)[16]>(&pk[c]));
                }
                if (ok && !first && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // The last P V into this group's O has completed.
                    ok = cache_wait<kSleepShort>(smem_u32(&ms.pv_grp[G]), ((gs - 2) >> 1) & 1, abort_flag, err);
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < kD; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld32(o_mine + c0, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
                        tmem_st32(o_mine + c0, o);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.p_full));
                first = false;
            }
            // The group that takes the next unit's first step stages its queries.
            if (next && ((g0 + nst) & 1) == (uint32_t)G) {
                // The unit's Q K^T have completed: Q may be overwritten.
                if (ok) ok = cache_wait<kSleepShort>(smem_u32(&ms.q_empty), ul & 1, abort_flag, err);
                queries(sw.unit[place(ul + 1)], ul + 1);
            }
            const bool after = next && advance(place(ul + 2));
            // ------------------------------------------------ unit epilogue
            //   m = max(m_0, m_1), a_k = 2^(m_k - m), l = a_0 l_0 + a_1 l_1, O = a_0 O_0 + a_1 O_1
            ms.xm[ul & 1][G][r] = m;
            ms.xl[ul & 1][G][r] = l;
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
            // The group of the unit's even steps comes first, whatever it is:
            // the sums do not depend on what the CTA did before the unit.
            const int ge = (int)(g0 & 1u);
            const float m_e = ms.xm[ul & 1][ge][r], l_e = ms.xl[ul & 1][ge][r];
            const float m_o = ms.xm[ul & 1][ge ^ 1][r], l_o = ms.xl[ul & 1][ge ^ 1][r];
            const float mt = fmaxf(m_e, m_o);
            float a_e = m_e == ninf ? 0.f : ex2_approx(m_e - mt);
            float a_o = m_o == ninf ? 0.f : ex2_approx(m_o - mt);
            const float lt = __fmaf_rn(a_e, l_e, __fmul_rn(a_o, l_o));
            const uint32_t o_e = ge ? kTmemO1 : kTmemO0, o_o = ge ? kTmemO0 : kTmemO1;
            const RowAt x = row_at<kD>(p, sg, r);
            const bool live = sg.t * 128 + r < sg.len.q * p.group && lt != 0.f;
            const size_t part = (2 * (size_t)blockIdx.x + (sg.first > 0 ? 0 : 1)) * 128 + r;
            if (sg.whole) {
                const float inv =
                    live ? (p.c.kv_scale ? p.c.kv_scale[p.c.kv_heads + sg.h] : 1.f) / lt : 0.f;
                a_e *= inv;
                a_o *= inv;
            }
            if (ok) ok = cache_wait<kSleepShort>(smem_u32(&ms.unit_done), ul & 1, abort_flag, err);
            tc_fence_after();
            const bool real = ok && x.real;  // (a wait that ran out leaves no whole O to store)
            // Each thread's columns go to its place in the row buffer (the bar.sync
            // above: the next queries have been taken from there), and from there
            // to memory by the lanes together, 64 or 128 bytes of a row: lanes
            // that store rows of their own take some 3 cycles a lane and piece.
            const unsigned reals = __ballot_sync(0xffffffffu, real);
            const bool whole = sg.whole;
            const size_t to = whole ? x.at + G * (dh / 8) : (part * kD + G * dh) / 4;  // in 16 bytes
            uint4* const base = whole ? p.out : reinterpret_cast<uint4*>(p.part_o);
            const int lanes = whole ? 4 : 8, sub = lane & (lanes - 1);  // of a row
#pragma unroll 1
            for (int c0 = 0; c0 < dh; c0 += 32) {
                uint32_t o[32];
                float2 f[16];
#pragma unroll
                for (int q = 0; q < 16; ++q) f[q] = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int side = 0; side < min(nst, 2); ++side) {  // (a group without a step holds no O of the unit)
                    tmem_ld32(t_lane + (side ? o_o : o_e) + G * dh + c0, o);
                    tmem_wait_ld();
                    const float2 a = side ? make_float2(a_o, a_o) : make_float2(a_e, a_e);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        f[q] = __ffma2_rn(make_float2(__uint_as_float(o[2 * q]), __uint_as_float(o[2 * q + 1])), a, f[q]);
                }
                if (whole) {
#pragma unroll
                    for (int q = 0; q < 16; ++q) o[q] = live ? pack_bf16x2(f[q].x, f[q].y) : 0u;
#pragma unroll
                    for (int q = 0; q < 16; q += 4) sts128(mine + q * 4, o[q], o[q + 1], o[q + 2], o[q + 3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 16; q += 2)
                        sts128(mine + q * 8, __float_as_uint(f[q].x), __float_as_uint(f[q].y),
                               __float_as_uint(f[q + 1].x), __float_as_uint(f[q + 1].y));
                }
                __syncwarp();
#pragma unroll 1
                for (int k = lane / lanes; k < 32; k += 32 / lanes) {  // row k of the warp
                    const size_t at = __shfl_sync(0xffffffffu, to, k) + sub;
                    const uint4 y = lds128(mine + (k - lane) * kRowPitch + sub * 16);
                    if ((reals >> k) & 1u) base[at + c0 / (whole ? 8 : 4)] = y;
                }
                __syncwarp();
            }
            // O_0 and O_1 have been read: the next unit may start them over.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.o_free));
            if (real && ok && G == 0) {
                if (!sg.whole)
                    p.part_ml[part] = make_float2(mt, lt);
                else if (p.lse)
                    p.lse[((size_t)sg.b * p.heads + x.head) * p.Sq + x.qi] =
                        live ? (mt + __log2f(lt)) * 0.69314718055994531f : ninf;
            }
            if (after) ask_queries(sw.unit[place(ul + 2)]);
            g0 += nst;
            more = next;
            next = after;
        }
        cp_async_wait<0>();
    }

    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

template <int kD>
static cudaError_t launch_chunk_d(const AttnParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> known{0};
    // The register split draws on the launch's registers; with fewer, setmaxnreg
    // would wait forever, so such a build is refused.
    int regs = 0;
    cudaError_t e = launch_registers(chunk_kernel<kD>, known, &regs);
    if (e != cudaSuccess) return e;
    if (regs != kLaunchRegs) return cudaErrorInvalidKernelImage;
    e = allow_smem(chunk_kernel<kD>, chunk_smem<kD>(), done);
    if (e != cudaSuccess) return e;
    // Not launched early itself: over 32760 keys, 64 rows of 40 heads take 95.4 us
    // so and 102.2 launched early (a ragged batch of prompts 289.6 and 281.1).
    chunk_kernel<kD><<<p.grid, kChunkThreads, chunk_smem<kD>(), stream>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_chunk(const AttnParams& p, int D, cudaStream_t stream) {
    return D == 64 ? launch_chunk_d<64>(p, stream) : launch_chunk_d<128>(p, stream);
}

}  // namespace vsa
