// Attention over the 4-bit paged cache, many query rows a kv head (chunks of
// tokens): the same function as token_kernel (cache_attn.cu), on tcgen05.
//
// Tensor bound for long chunks (4 * D flops for each row and key).  A unit is
// kQ tiles of 128 query rows, one TMEM lane each; a step is 128 keys (two
// pages).  What stands between the cache and the tensor core is the conversion
// of codes to fp16 operands, about 1.5 instructions an element and as many
// bytes of shared-memory writes as the tensor core reads, so it is shared by
// as many rows as TMEM has room for:
//  * kQ = 2 (more than 128 rows): each softmax group has a tile of its own and
//    takes every step; K and V are converted once for 256 rows.
//  * kQ = 1: both groups have the same rows and take the steps in turn, each
//    with a maximum, sum and output of its own, joined at the unit's end.
// A producer warp copies pages (halves: K and V with their scales) into a
// ring; a warpgroup converts them (exact, see cache.cuh) to K and V tiles in
// the 128-byte swizzled layout the tensor core reads.  A page crosses HBM and
// L2 in 9 bits a pair of K and V elements instead of 32.
//  * Warp roles (512 threads): warp 0 looks pages up and copies them; warp 1
//    owns TMEM and issues Q K^T, warp 3 P V; warps 4..7 convert; warps 8..11
//    and 12..15 are the softmax groups.
//  * TMEM (512 columns): S_0 [0,128), S_1 [128,256), O_0 [256,384), O_1
//    [384,512).  P (fp16 pairs) takes the first 64 columns of its S once the
//    softmax has loaded that; Q is in shared memory.
//  * A query row is scaled by a power of two on its way to fp16 (its bf16
//    values keep all their bits) and the inverse joins its softmax scale.
//  * Every wait is bounded; one that runs out raises the CTA's abort flag and
//    the device error word, and each role winds down.
#include "cache.cuh"

namespace vsa {

namespace {

constexpr int kChunkThreads = 512;
constexpr int kMetaSteps = 16;
// Registers: 4 warpgroups launched with 128 each; the shares add up to 512.
constexpr int kIssueRegs = 64, kConvertRegs = 80, kSoftRegs = 184;
static_assert(kIssueRegs + kConvertRegs + 2 * kSoftRegs <= 512, "register split exceeds the launch");

constexpr int kTmemS = 0, kTmemO = 256, kTmemGroup = 128;  // of group G: + G * kTmemGroup

template <int kD, int kQ>
struct ChunkSmem {
    static constexpr int kKStages = 2;
    static constexpr int kVStages = kD == 128 && kQ == 2 ? 2 : 3;
    static constexpr int kRaw = kD == 128 ? 6 : 12;  // half pages
    static constexpr int kHalf = 128 * 128;          // 128 rows x 64 channels of fp16, swizzled
    static constexpr int kTile = kHalf * (kD / 64);  // Q of a tile, K or V of a step
    static constexpr int kCodes = kPageTokens * kD / 2, kScales = kPageTokens * kD / 16;
    static constexpr int kRawBytes = kCodes + kScales;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kQ * kTile;
    static constexpr int kOffV = kOffK + kKStages * kTile;
    static constexpr int kOffRaw = kOffV + kVStages * kTile;
    static constexpr int kOffMisc = kOffRaw + kRaw * kRawBytes;
};

// A softmax warp's walk and its present and next unit: kept in shared memory,
// the steps need the registers.
struct SoftWalk {
    Walk walk;
    Segment unit[2];
};

struct __align__(16) ChunkMisc {
    uint64_t raw_full[12], raw_empty[12];
    uint64_t k_full[2], k_empty[2];
    uint64_t v_full[3], v_empty[3];
    // Per softmax group: S of its next step is ready; P of it (and any
    // rescaling of O) is in TMEM; P V has completed (S may be overwritten).
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t q_full[2], q_empty[2];  // per tile
    uint64_t drain[2];
    int2 key0[kMetaSteps];  // first key of a step's pages (kNoKey: none)
    float xm[2][128], xl[2][128];  // kQ = 1: the groups' maxima and sums at the unit's end
    float scale[2][128];           // kQ = 1: [unit parity][row]: logit -> log2 units
    SoftWalk soft[8];
    PlanScratch plan;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kNoKey = 0x7FFFFFFF;  // beyond every row's limit

template <int kD, int kQ>
constexpr int chunk_smem() {
    return ChunkSmem<kD, kQ>::kOffMisc + (int)sizeof(ChunkMisc) + 1024;  // slack for 1024-byte alignment
}
static_assert(chunk_smem<128, 1>() <= 232448 && chunk_smem<128, 2>() <= 232448, "shared memory of the chunk kernel");

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

// Softmax thread of row r of a tile: puts query row `row` of unit s into the
// tile's Q as fp16, scaled by a power of two, and returns the row's factor from
// logits to log2 units.
template <int kD, int kQ>
__device__ __forceinline__ float stage_query(const AttnParams& p, const Segment& s, int row, int r, uint32_t tile) {
    const bool real = row < p.Sq * p.group;
    const int qi = real ? row / p.group : 0;
    const int head = s.h * p.group + (real ? row - qi * p.group : 0);
    const uint4* src = p.q + (((size_t)s.b * p.Sq + qi) * p.heads + head) * (kD / 8);
    uint32_t w[kD / 2];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kD / 8; ++i) {
        const uint4 x = real ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int i = 0; i < kD / 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    const int e = q_exponent(amax);
    const float f = pow2i(e);
#pragma unroll
    for (int i = 0; i < kD / 8; ++i) {
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = pack_f16x2(bf16_lo(w[4 * i + j]) * f, bf16_hi(w[4 * i + j]) * f);
        sts128(tile + (i >> 3) * ChunkSmem<kD, kQ>::kHalf + r * 128 + (((i & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
    }
    fence_proxy_async_smem();
    return p.scale_log2 * (p.c.kv_scale ? __ldg(p.c.kv_scale + s.h) : 1.f) * pow2i(-e);
}

// Half of one key's codes of K or V and their scales (`codes`, `scales`: the
// key's, in shared memory) to row `row` of a fp16 tile: channels [h kD / 2,
// (h + 1) kD / 2).  Two threads a key, neighbouring lanes, each starting at
// another 16-byte piece (kD = 128) so that neither the loads nor the swizzled
// stores of 8 lanes meet in a bank.
template <int kD, int kQ>
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
    const uint32_t base = tile + row * 128 + (kD == 128 ? h * ChunkSmem<kD, kQ>::kHalf : 0);
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

// Groups with rows of a unit.
template <int kQ>
__device__ __forceinline__ int groups_of(const AttnParams& p, const Segment& s) {
    return kQ == 2 && s.t * 256 + 128 < p.Sq * p.group ? 2 : 1;
}

template <int kD, int kQ>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(AttnParams p) {
    using L = PageLayout<kD>;
    using Sm = ChunkSmem<kD, kQ>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    ChunkMisc& ms = *reinterpret_cast<ChunkMisc*>(smem + Sm::kOffMisc);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &ms.abort_flag;
    unsigned int* err = p.c.err;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Sm::kRaw; ++s) {
            mbar_init(smem_u32(&ms.raw_full[s]), 1);
            mbar_init(smem_u32(&ms.raw_empty[s]), 4);
        }
        for (int s = 0; s < Sm::kKStages; ++s) {
            mbar_init(smem_u32(&ms.k_full[s]), 4);
            mbar_init(smem_u32(&ms.k_empty[s]), 1);
        }
        for (int s = 0; s < Sm::kVStages; ++s) {
            mbar_init(smem_u32(&ms.v_full[s]), 4);
            mbar_init(smem_u32(&ms.v_empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&ms.s_full[s]), 1);
            mbar_init(smem_u32(&ms.p_full[s]), 4);
            mbar_init(smem_u32(&ms.pv_done[s]), 1);
            mbar_init(smem_u32(&ms.q_full[s]), 4);
            mbar_init(smem_u32(&ms.q_empty[s]), 1);
            mbar_init(smem_u32(&ms.drain[s]), 1);
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    // The tiles start as zeros: the tensor core multiplies rows that no page
    // filled (an odd last page, pages passed over) by probabilities of zero.
    {
        int4* z = reinterpret_cast<int4*>(smem + Sm::kOffK);
        for (int e = threadIdx.x; e < (Sm::kOffRaw - Sm::kOffK) / 16; e += kChunkThreads) z[e] = make_int4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
        if (warp == 0) {
            // ================================================= page producer
            // Half pages in the order of their conversion: K of the step's
            // pages, then V of them.
            uint32_t j = 0, g = 0;  // half pages and steps so far
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                const unsigned char* pool = p.c.pool + (size_t)sg.h * L::kBytes;
                for (int base = sg.first; base < sg.last && ok; base += 32) {
                    int logical = 0, id = -1;
                    if (base + lane < sg.last) look_up(p, sg, base + lane, logical, id);
                    const int n = min(32, sg.last - base);  // (32 is even: steps do not straddle)
                    for (int i = 0; i < n && ok; i += 2, ++g) {
                        const int held = min(2, n - i);
                        const int page0 = __shfl_sync(0xffffffffu, id, i);
                        const int page1 = held == 2 ? __shfl_sync(0xffffffffu, id, i + 1) : -1;
                        const int num0 = __shfl_sync(0xffffffffu, logical, i);
                        const int num1 = held == 2 ? __shfl_sync(0xffffffffu, logical, i + 1) : 0;
                        if (lane == 0)
                            ms.key0[g % kMetaSteps] = make_int2(page0 < 0 ? kNoKey : num0 * kPageTokens,
                                                                page1 < 0 ? kNoKey : num1 * kPageTokens);
                        for (int k = 0; k < 2 * held; ++k, ++j) {
                            const int side = k >= held;
                            const int page = (k - side * held) ? page1 : page0;
                            const int slot = j % Sm::kRaw;
                            if (j >= (uint32_t)Sm::kRaw) {
                                ok = mbar_wait_bounded(smem_u32(&ms.raw_empty[slot]), (j / Sm::kRaw + 1) & 1,
                                                       abort_flag, err, kCacheWaitNs);
                                if (!ok) break;
                            }
                            if (lane == 0) {
                                const uint32_t bar = smem_u32(&ms.raw_full[slot]);
                                if (page < 0) {
                                    mbar_arrive(bar);
                                } else {
                                    mbar_arrive_expect_tx(bar, Sm::kRawBytes);
                                    const uint32_t dst = sbase + Sm::kOffRaw + slot * Sm::kRawBytes;
                                    const unsigned char* src = pool + (size_t)page * p.c.kv_heads * L::kBytes;
                                    bulk_load(dst, src + side * L::kV, Sm::kCodes, bar);
                                    bulk_load(dst + Sm::kCodes, src + (side ? L::kVScale : L::kKScale), Sm::kScales,
                                              bar);
                                }
                            }
                            __syncwarp();
                        }
                    }
                }
            }
            if (lane == 0) {
                for (int s = 0; s < Sm::kRaw && (uint32_t)s < j; ++s) {
                    const uint32_t last = j - 1 - ((j - 1 - s) % Sm::kRaw);
                    mbar_wait_drain_1(smem_u32(&ms.raw_full[s]), (last / Sm::kRaw) & 1, err, kCacheWaitNs);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ========================================================= Q K^T
            const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
            const uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
            const uint32_t lo_q = (uint32_t)smem_desc_sw128(sbase + Sm::kOffQ, 16, 1024);
            const uint32_t lo_k = (uint32_t)smem_desc_sw128(sbase + Sm::kOffK, 16, 1024);
            uint32_t g = 0, n_s[2] = {0, 0}, n_q[2] = {0, 0};  // steps; S written, units staged, per group
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                const int nst = steps_of(sg), groups = groups_of<kQ>(p, sg);
                for (int t = 0; t < nst && ok; ++t, ++g) {
                    const int slot = g % Sm::kKStages;
                    ok = mbar_wait_bounded(smem_u32(&ms.k_full[slot]), (g / Sm::kKStages) & 1, abort_flag, err,
                                           kCacheWaitNs);
                    const uint32_t b0 = lo_k + ((uint32_t)(slot * Sm::kTile) >> 4);
#pragma unroll
                    for (int G = 0; G < 2; ++G) {
                        if (kQ == 1 ? (g & 1) != (uint32_t)G : G >= groups) continue;
                        const int tile = kQ == 1 ? 0 : G;
                        if (t == 0 && ok)
                            ok = mbar_wait_bounded(smem_u32(&ms.q_full[tile]), n_q[tile] & 1, abort_flag, err,
                                                   kCacheWaitNs);
                        if (n_s[G] > 0 && ok)  // P V of the group's last step has read P, which lies in S
                            ok = mbar_wait_bounded(smem_u32(&ms.pv_done[G]), (n_s[G] - 1) & 1, abort_flag, err,
                                                   kCacheWaitNs);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a0 = lo_q + ((uint32_t)(tile * Sm::kTile) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk) {
                            const uint32_t step = ((kk >> 2) * Sm::kHalf + (kk & 3) * 32) >> 4;
                            mma_ss_warp(tmem + kTmemS + G * kTmemGroup, a0 + step, hi, b0 + step, hi, idesc, kk > 0);
                        }
                        mma_commit_warp(smem_u32(&ms.s_full[G]));
                        ++n_s[G];
                    }
                    if (!ok) break;
                    mma_commit_warp(smem_u32(&ms.k_empty[slot]));
                }
                if (!ok) break;
#pragma unroll
                for (int tile = 0; tile < kQ; ++tile) {
                    if (tile >= groups) continue;
                    // (A unit without steps has its queries staged all the same.)
                    if (nst == 0 && ok)
                        ok = mbar_wait_bounded(smem_u32(&ms.q_full[tile]), n_q[tile] & 1, abort_flag, err,
                                               kCacheWaitNs);
                    mma_commit_warp(smem_u32(&ms.q_empty[tile]));
                    ++n_q[tile];
                }
            }
            mma_commit_warp(smem_u32(&ms.drain[0]));
            if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain[0]), 0, err, kCacheWaitNs);
            __syncwarp();
        } else if (warp == 3) {
            // =========================================================== P V
            const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);
            const uint32_t idesc = idesc_f16_f32(128, kD, 0, 1);
            const uint32_t lo_v = (uint32_t)smem_desc_sw128(sbase + Sm::kOffV, Sm::kHalf, 1024);
            uint32_t g = 0, n_p[2] = {0, 0};
            bool ok = true;
            for (Segment sg; ok && walk.next(p, sg);) {
                const int nst = steps_of(sg), groups = groups_of<kQ>(p, sg);
                for (int t = 0; t < nst && ok; ++t, ++g) {
                    const int slot = g % Sm::kVStages;
                    ok = mbar_wait_bounded(smem_u32(&ms.v_full[slot]), (g / Sm::kVStages) & 1, abort_flag, err,
                                           kCacheWaitNs);
                    const uint32_t b0 = lo_v + ((uint32_t)(slot * Sm::kTile) >> 4);
#pragma unroll
                    for (int G = 0; G < 2; ++G) {
                        if (kQ == 1 ? (g & 1) != (uint32_t)G : G >= groups) continue;
                        if (ok)
                            ok = mbar_wait_bounded(smem_u32(&ms.p_full[G]), n_p[G] & 1, abort_flag, err, kCacheWaitNs);
                        if (!ok) break;
                        // The unit's first step of the group starts its O over.
                        const uint32_t acc = t >= (kQ == 1 ? 2 : 1) ? 1u : 0u;
                        const uint32_t d = tmem + kTmemO + G * kTmemGroup, a = tmem + kTmemS + G * kTmemGroup;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts_warp(d, a + kk * 8, b0 + ((kk * 2048) >> 4), hi, idesc, acc | (kk > 0 ? 1u : 0u));
                        if (sg.first + 2 * t + 1 < sg.last) {
#pragma unroll
                            for (int kk = 4; kk < 8; ++kk)
                                mma_ts_warp(d, a + kk * 8, b0 + ((kk * 2048) >> 4), hi, idesc, 1u);
                        }
                        mma_commit_warp(smem_u32(&ms.pv_done[G]));
                        ++n_p[G];
                    }
                    if (!ok) break;
                    mma_commit_warp(smem_u32(&ms.v_empty[slot]));
                }
            }
            mma_commit_warp(smem_u32(&ms.drain[1]));
            if (lane == 0) mbar_wait_drain_1(smem_u32(&ms.drain[1]), 0, err, kCacheWaitNs);
            __syncwarp();
        }
    } else if (warp < 8) {
        // ============================================================ convert
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        const int th = threadIdx.x - 128, key = th >> 1, h = th & 1;  // two threads a key of a page
        uint32_t j = 0, g = 0;
        bool ok = true;
        for (Segment sg; ok && walk.next(p, sg);) {
            for (int i = sg.first; i < sg.last && ok; i += 2, ++g) {
                const int held = min(2, sg.last - i);
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {
                    const int stages = side ? Sm::kVStages : Sm::kKStages, st = g % stages;
                    const uint32_t full = smem_u32(side ? &ms.v_full[st] : &ms.k_full[st]);
                    const uint32_t empty = smem_u32(side ? &ms.v_empty[st] : &ms.k_empty[st]);
                    const uint32_t tile = sbase + (side ? Sm::kOffV : Sm::kOffK) + st * Sm::kTile;
                    if (g >= (uint32_t)stages)
                        ok = mbar_wait_bounded(empty, (g / stages + 1) & 1, abort_flag, err, kCacheWaitNs);
#pragma unroll 1
                    for (int which = 0; which < held && ok; ++which, ++j) {
                        const int slot = j % Sm::kRaw;
                        ok = mbar_wait_bounded(smem_u32(&ms.raw_full[slot]), (j / Sm::kRaw) & 1, abort_flag, err,
                                               kCacheWaitNs);
                        if (!ok) break;
                        const int2 k0 = ms.key0[g % kMetaSteps];
                        const int key0 = which ? k0.y : k0.x;
                        // Slots past the sequence's end hold anything, and a page
                        // passed over nothing: their V is zero (K is masked).
                        const bool zero = side && (key0 == kNoKey || key0 + key >= sg.len.kv);
                        const uint32_t raw = sbase + Sm::kOffRaw + slot * Sm::kRawBytes;
                        convert_half_row<kD, kQ>(raw + key * (kD / 2), raw + Sm::kCodes + key * (kD / 16),
                                                 which * kPageTokens + key, h, zero, tile);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&ms.raw_empty[slot]));
                    }
                    if (!ok) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full);
                }
            }
        }
    } else {
        // ============================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int G = (warp - 8) >> 2;
        const int quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_mine = t_lane + kTmemS + G * kTmemGroup, o_mine = t_lane + kTmemO + G * kTmemGroup;
        const int tile = kQ == 2 ? G : 0;
        const uint32_t q_tile = sbase + Sm::kOffQ + tile * Sm::kTile;
        const float ninf = -INFINITY;
        bool ok = true;
        uint32_t g0 = 0, n = 0, units = 0;  // steps before the unit; steps and units of this group
        SoftWalk& sw = ms.soft[warp - 8];
        auto advance = [&](int to) -> bool {  // the walk's next unit into sw.unit[to]
            Walk w = sw.walk;
            Segment s;
            const bool has = w.next(p, s);
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
        bool more = advance(0);
        float next_c2 = 0.f;
        auto stage = [&](int of) {  // the queries of sw.unit[of]
            const Segment& s = sw.unit[of];
            if (tile >= groups_of<kQ>(p, s)) return;
            next_c2 = stage_query<kD, kQ>(p, s, s.t * (kQ * 128) + tile * 128 + r, r, q_tile);
            if (kQ == 1) ms.scale[of][r] = next_c2;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ms.q_full[tile]));
        };
        if (more && (kQ == 2 || G == 0)) stage(0);
#pragma unroll 1
        for (uint32_t ul = 0; more; ++ul) {
            const bool next = advance((ul + 1) & 1);
            const Segment& sg = sw.unit[ul & 1];
            const int nst = steps_of(sg);
            const bool mine = tile < groups_of<kQ>(p, sg);
            const int row = sg.t * (kQ * 128) + tile * 128 + r;
            const int live_rows = sg.len.q * p.group;
            int lim = sg.len.kv;  // first key the row does not see
            if (p.causal && row < live_rows) lim = max(0, min(lim, sg.len.kv - sg.len.q + row / p.group + 1));
            float c2 = next_c2, m = ninf, l = 0.f;
            bool first = true;
#pragma unroll 1
            for (int t = kQ == 1 ? (int)((g0 + G) & 1) : 0; t < nst && mine; t += kQ == 1 ? 2 : 1, ++n) {
                if (ok) ok = mbar_wait_bounded(smem_u32(&ms.s_full[G]), n & 1, abort_flag, err, kCacheWaitNs);
                tc_fence_after();
                if (kQ == 1) c2 = ms.scale[ul & 1][r];
                const int2 k0 = ms.key0[(g0 + t) % kMetaSteps];
                // Keys of the two pages that this row sees (none where no page is).
                const int va = lim - k0.x, vb = lim - k0.y;
                float x[128];
#pragma unroll
                for (int c = 0; c < 128; c += 32) tmem_ld32(s_mine + c, *reinterpret_cast<uint32_t(*)[32]>(&x[c]));
                tmem_wait_ld();
                if (__any_sync(0xffffffffu, va < kPageTokens || vb < kPageTokens)) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) {
                        x[c] = c < va ? x[c] : ninf;
                        x[64 + c] = c < vb ? x[64 + c] : ninf;
                    }
                }
                const float mx = fmaxf(chunk_max64(x), chunk_max64(x + 64)) * c2;
                // Lazy maximum: O and l are rescaled on a jump only.
                float alpha = 1.f;
                if (mx > m + kCacheRescale) {
                    alpha = m == ninf ? 0.f : ex2_approx(m - mx);
                    m = mx;
                    l *= alpha;
                }
                const float mb = m == ninf ? 0.f : m;
                if (!first && ok && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // (The group's last P V has completed: this S was written after it.)
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
                uint32_t pk[64];
                chunk_exp64(x, c2, mb, pk, l);
                chunk_exp64(x + 64, c2, mb, pk + 32, l);
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 64; c += 16)
                        tmem_st16(s_mine + c, *reinterpret_cast<uint32_t(*)[16]>(&pk[c]));
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ms.p_full[G]));
                first = false;
            }
            // The next unit's queries, once this one's Q K^T have completed.
            if (mine && (kQ == 2 || ((g0 + nst) & 1) == (uint32_t)G)) {
                if (ok && next)
                    ok = mbar_wait_bounded(smem_u32(&ms.q_empty[tile]), units & 1, abort_flag, err, kCacheWaitNs);
            }
            if (mine) ++units;
            if (next && ok && (kQ == 2 || ((g0 + nst) & 1) == (uint32_t)G)) stage((ul + 1) & 1);
            // ------------------------------------------------ unit epilogue
            float a_e = 1.f, a_o = 0.f, mt = m, lt = l;
            const uint32_t ge = kQ == 1 ? (g0 & 1u) : G;  // the group of the unit's even steps comes first
            bool has_e = nst > 0, has_o = false;          // a group without a step holds no O of the unit
            if (kQ == 1) {
                //   m = max(m_0, m_1), a_k = 2^(m_k - m), l = a_0 l_0 + a_1 l_1, O = a_0 O_0 + a_1 O_1
                ms.xm[G][r] = m;
                ms.xl[G][r] = l;
                // This group's O is complete before the other reads its half of it.
                if (n > 0 && ok)
                    ok = mbar_wait_bounded(smem_u32(&ms.pv_done[G]), (n - 1) & 1, abort_flag, err, kCacheWaitNs);
                tc_fence_before();
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                tc_fence_after();
                const float m_e = ms.xm[ge][r], l_e = ms.xl[ge][r], m_o = ms.xm[ge ^ 1][r], l_o = ms.xl[ge ^ 1][r];
                mt = fmaxf(m_e, m_o);
                a_e = m_e == ninf ? 0.f : ex2_approx(m_e - mt);
                a_o = m_o == ninf ? 0.f : ex2_approx(m_o - mt);
                lt = __fmaf_rn(a_e, l_e, __fmul_rn(a_o, l_o));
                has_o = nst > 1;
            } else if (n > 0 && mine && ok) {
                ok = mbar_wait_bounded(smem_u32(&ms.pv_done[G]), (n - 1) & 1, abort_flag, err, kCacheWaitNs);
                tc_fence_after();
            }
            const bool real = ok && mine && row < p.Sq * p.group;
            const int qi = real ? row / p.group : 0;
            const int head = sg.h * p.group + (real ? row - qi * p.group : 0);
            const bool live = row < live_rows && lt != 0.f, whole = sg.whole;
            const size_t part = (2 * (size_t)blockIdx.x + (sg.first > 0 ? 0 : 1)) * (kQ * 128) + tile * 128 + r;
            if (whole) {
                const float inv =
                    live ? (p.c.kv_scale ? __ldg(p.c.kv_scale + p.c.kv_heads + sg.h) : 1.f) / lt : 0.f;
                a_e *= inv;
                a_o *= inv;
            }
            // kQ = 1: the groups write half of the columns each.
            const int col0 = kQ == 1 ? G * (kD / 2) : 0, cols = kQ == 1 ? kD / 2 : kD;
            uint4* dst = p.out + (((size_t)sg.b * p.Sq + qi) * p.heads + head) * (kD / 8) + col0 / 8;
            float4* dst_part = reinterpret_cast<float4*>(p.part_o + part * kD + col0);
#pragma unroll 1
            for (int c0 = 0; c0 < (mine ? cols : 0); c0 += 32) {
                uint32_t oa[32], ob[32];
                tmem_ld32(t_lane + kTmemO + ge * kTmemGroup + col0 + c0, oa);
                if (kQ == 1) tmem_ld32(t_lane + kTmemO + (ge ^ 1) * kTmemGroup + col0 + c0, ob);
                tmem_wait_ld();
                float f[32];
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    const float e = has_e ? __uint_as_float(oa[q]) : 0.f;
                    f[q] = kQ == 1 ? __fmaf_rn(a_e, e, __fmul_rn(a_o, has_o ? __uint_as_float(ob[q]) : 0.f)) : a_e * e;
                }
                if (!real || !ok) continue;
                if (whole) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            w[q] = live ? pack_bf16x2(f[8 * v + 2 * q], f[8 * v + 2 * q + 1]) : 0u;
                        __stcs(dst + c0 / 8 + v, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst_part[c0 / 4 + v] = make_float4(f[4 * v], f[4 * v + 1], f[4 * v + 2], f[4 * v + 3]);
                }
            }
            if (kQ == 1) {
                // Both groups have read O_0 and O_1 (and the exchanged statistics):
                // the next unit's steps, which either announces after this, may start.
                tc_fence_before();
                asm volatile("bar.sync %0, 64;" ::"r"(1 + quarter) : "memory");
                tc_fence_after();
            }
            if (real && ok && (kQ == 2 || G == 0)) {
                if (!whole)
                    p.part_ml[part] = make_float2(mt, lt);
                else if (p.lse)
                    p.lse[((size_t)sg.b * p.heads + head) * p.Sq + qi] =
                        live ? (mt + __log2f(lt)) * 0.69314718055994531f : ninf;
            }
            g0 += nst;
            more = next;
        }
    }

    // ------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

}  // namespace

template <int kD, int kQ>
static cudaError_t launch_chunk_as(const AttnParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    // The register split draws on the launch's 128 registers a thread; with
    // fewer, setmaxnreg would wait forever, so such a build is refused.
    static const int regs = [] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, chunk_kernel<kD, kQ>) == cudaSuccess ? fa.numRegs : 0;
    }();
    if (regs != 128) return cudaErrorInvalidKernelImage;
    const cudaError_t e = allow_smem(chunk_kernel<kD, kQ>, chunk_smem<kD, kQ>(), done);
    if (e != cudaSuccess) return e;
    chunk_kernel<kD, kQ><<<p.grid, kChunkThreads, chunk_smem<kD, kQ>(), stream>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_chunk(const AttnParams& p, int D, cudaStream_t stream) {
    if (p.tile == 256) return D == 64 ? launch_chunk_as<64, 2>(p, stream) : launch_chunk_as<128, 2>(p, stream);
    return D == 64 ? launch_chunk_as<64, 1>(p, stream) : launch_chunk_as<128, 1>(p, stream);
}

}  // namespace vsa
