// Attention weight that cached keys have got, summed over query rows: for each kv
// head and cached token x
//   w_x += sum over the rows r that see x of exp(sm_scale q_r . k_x - lse_r)
// with the rows' log-sum-exp from the attention call.  Only K is read: 9/16 D bytes
// a key and head, 2 D flops and an exponential for each row.
//
// Few rows a kv head (up to 24, or 32 of 64 channels): K Q^T by mma.sync m16n8k16
// (fp16 in, fp32 out) with tokens on the 16-row side, as in token_kernel
// (cache_attn.cu); a weight is the sum over a token's row of the accumulator, so nothing is joined
// across warps and each weight has one owner: same bits in every run.
//  * All warps take equal stretches of the line of half pages (32 tokens) of all
//    sequences and heads; codes, scales and weights so far come to shared memory by
//    asynchronous copies, three half pages ahead, each warp's for itself (61 sequences
//    of up to 12000 tokens, 128 / 64 channels: 56.6 / 43.8 us; two half pages in
//    registers in turns 60.7 / 54.8, four in shared memory 57.6 / 44.2; single calls are
//    up to 0.2 us slower so).
//  * A key's 64 (or 32) code bytes are four lanes' loads; the order of channels
//    within K Q^T is free, so a lane's 32 (16) channels need no shuffle.
// Measured on a GB300, 4 rows a kv head, D = 128: 61 sequences of up to 12000 tokens,
// 8 kv heads, 56.9 us = 4.4 TB/s read (65% of the measured copy rate): some 340
// instructions a half page and warp, and four warps a scheduler, which issue 0.57 a cycle.
// A warp waits 6.8 cycles an instruction: 1.4 for the one before, 1.1 for memory,
// 1.3 for the pipes and dispatch, 1.1 for its turn.  20 rows on 8 sequences of 8000, 19.8 us:
// three warps a scheduler, 0.39 a cycle; 2.0 for the instruction before, 1.7 for memory, 1.1
// for the pipes and dispatch.  One sequence of
// 32760: 9 us, the latency of lengths, page numbers, rows and half pages one after the
// other (its bytes take 3).
#include <float.h>

#include "weigh.cuh"

namespace vsa {

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kUnit = 32;  // tokens

// Half pages of sequence b.
__device__ __forceinline__ int units_of(int kv) { return (kv + kUnit - 1) / kUnit; }

// Where a place on the line is: sequence, half page within all of its heads'.
struct LinePlace {
    int b;
    long long within;
};
// The line's length, and where `part` of `parts` begins and ends on it (a whole warp calls it).
__device__ __forceinline__ long long line_length(const CacheView& c) {
    const int lane = threadIdx.x & 31;
    long long sum = 0;
    for (int b = lane; b < c.B; b += 32) sum += (long long)c.kv_heads * units_of(cache_len(c, b, false));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
__device__ __forceinline__ LinePlace place_on_line(const CacheView& c, long long at) {
    const int lane = threadIdx.x & 31;
    for (int b0 = 0;; b0 += 32) {
        const long long mine =
            b0 + lane < c.B ? (long long)c.kv_heads * units_of(cache_len(c, b0 + lane, false)) : 0;
        const long long incl = scan_warp(mine);
        const unsigned past = __ballot_sync(0xffffffffu, at < incl);
        if (past || b0 + 32 >= c.B) {
            const int l = past ? __ffs(past) - 1 : 31;
            return {b0 + l, at - __shfl_sync(0xffffffffu, incl - mine, l)};
        }
        at -= __shfl_sync(0xffffffffu, incl, 31);
    }
}

// One lane's share of 32 tokens' K: rows 16 m + 8 half + lane / 4, a quarter of their channels.
template <int kD>
struct KUnit {
    uint32_t codes[2][2][kD / 32];
    uint32_t scales[2][2];
    float before;  // the weight of token 16 (t / 2) + 8 (t % 2) + g so far
};

// A half page's K and its tokens' weights so far, on their way to a warp.
template <int kD>
struct alignas(16) Piece {
    static constexpr int kCodes = kUnit * PageLayout<kD>::kRow, kScales = kUnit * PageLayout<kD>::kGroups;
    unsigned char codes[kCodes];
    unsigned char scales[kScales];
    float before[32];  // of the lane's token
};
constexpr int kStages = 3;  // pieces of a warp

template <int kD, int kNT, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1) weigh_kernel(WeighParams p) {
    extern __shared__ __align__(16) unsigned char weigh_smem[];
    using L = PageLayout<kD>;
    constexpr int kWords = kD / 32;
    early();
    begin_work();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const CacheView& c = p.c;
    Piece<kD>* const pieces = reinterpret_cast<Piece<kD>*>(weigh_smem) + warp * kStages;
    if (blockIdx.x == 0 && warp == 0)  // lengths out of range are noted once
        for (int b = lane; b < c.B; b += 32) cache_len(c, b, true);
    const long long total = line_length(c);
    const long long parts = (long long)gridDim.x * kWarps, part = (long long)warp * gridDim.x + blockIdx.x;
    long long left = total / parts + (part < total % parts ? 1 : 0);
    const size_t row_places = (size_t)c.width * kPageTokens;
    if (left > 0) {
        LinePlace at = place_on_line(c, total / parts * part + min(part, total % parts));
        int kv = cache_len(c, at.b, false);
        int h = (int)(at.within / units_of(kv)), u = (int)(at.within - (long long)h * units_of(kv));
        while (left > 0) {
            while (u >= units_of(kv)) {  // the next head, the next sequence
                u = 0;
                if (++h == c.kv_heads) {
                    h = 0;
                    kv = cache_len(c, ++at.b, false);
                    if (units_of(kv) == 0) h = c.kv_heads - 1;  // (none: on to the next)
                }
            }
            const int b = at.b, n = (int)min(left, (long long)(units_of(kv) - u)), end = u + n;
            const int fresh = p.q_lens ? min(max(p.q_lens[b], 0), p.Sq) : p.Sq;
            const int rows = fresh * p.group;
            const float k_head = c.kv_scale ? c.kv_scale[h] : 1.f;
            const float* in = p.weights ? p.weights + ((size_t)b * c.kv_heads + h) * row_places : nullptr;
            float* out = p.out + ((size_t)b * c.kv_heads + h) * row_places;
            // Places in the pool of the 32 pages from page0 on.
            int page0 = u >> 1, id = -1;
            auto look_up = [&]() {
                id = -1;
                if (page0 + lane < (end + 1) >> 1) {
                    id = c.table[(size_t)b * c.width + page0 + lane];
                    if (id < 0 || id >= c.pages) {
                        atomicOr(c.err, VSA_DEVERR_INDEX);
                        id = -1;
                    }
                }
            };
            look_up();
            uint32_t there = 0;  // a bit for each stage: the page is one
            auto ask = [&](int unit, int stage) {
                if (unit < end) {
                    if ((unit >> 1) - page0 == 32) {
                        page0 += 32;
                        look_up();
                    }
                    const int page = __shfl_sync(0xffffffffu, id, (unit >> 1) - page0);
                    there = page >= 0 ? there | 1u << stage : there & ~(1u << stage);
                    Piece<kD>& piece = pieces[stage];
                    if (page >= 0) {
                        using P = Piece<kD>;
                        const unsigned char* base = c.pool + ((size_t)page * c.kv_heads + h) * L::kBytes;
#pragma unroll
                        for (int i = 0; i < P::kCodes / 512; ++i)
                            cp_async16(smem_u32(piece.codes + i * 512 + lane * 16),
                                       base + (unit & 1) * P::kCodes + i * 512 + lane * 16);
                        if (lane < P::kScales / 16)
                            cp_async16(smem_u32(piece.scales + lane * 16),
                                       base + L::kKScale + (unit & 1) * P::kScales + lane * 16);
                    }
                    if (in) cp_async4(smem_u32(&piece.before[lane]), in + unit * kUnit + 16 * (t >> 1) + 8 * (t & 1) + g);
                }
                cp_async_commit();
            };
            auto take = [&](int stage, KUnit<kD>& k) {
                const Piece<kD>& piece = pieces[stage];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int tok = 16 * m + 8 * half + g;
                        const unsigned char* src = piece.codes + tok * L::kRow + t * (kWords * 4);
                        const unsigned char* sc = piece.scales + tok * L::kGroups + t * (kWords / 2);
                        if constexpr (kWords == 4) {
                            const uint4 x = *reinterpret_cast<const uint4*>(src);
                            k.codes[m][half][0] = x.x; k.codes[m][half][1] = x.y;
                            k.codes[m][half][2] = x.z; k.codes[m][half][3] = x.w;
                            k.scales[m][half] = *reinterpret_cast<const uint16_t*>(sc);
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2*>(src);
                            k.codes[m][half][0] = x.x; k.codes[m][half][1] = x.y;
                            k.scales[m][half] = (uint32_t)*sc * 0x101u;
                        }
                    }
                k.before = in ? piece.before[lane] : 0.f;
            };
            // The first keys are on their way before the rows are looked at.
#pragma unroll
            for (int i = 0; i < kStages; ++i) ask(u + i, i);
            // The rows as the matrix instruction's columns.
            uint32_t qf[kNT][2 * kWords][2];
            float scale[kNT][2], off[kNT][2];  // logit = s scale - off (log2 units) of rows nt * 8 + 2 t + i
            int lim[kNT][2], min_lim = kv;     // first key that the row does not see
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                const int r = nt * 8 + g, qi = r / p.group;
                const bool live = r < rows;
                const int head = h * p.group + r - qi * p.group;
                float lse = INFINITY;
                if (live) lse = p.lse[((size_t)b * p.heads + head) * p.Sq + qi];
                const bool used = fabsf(lse) < INFINITY;  // (a row without a finite sum weighs nothing)
                const uint4* src = p.q + (((size_t)b * p.Sq + qi) * p.heads + head) * (kD / 8) + t * kWords;
                uint32_t w[4 * kWords];
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const uint4 x = used ? src[i] : make_uint4(0, 0, 0, 0);
                    w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < 4 * kWords; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                const int e = q_exponent(amax);
                const float f = pow2i(e);
#pragma unroll
                for (int i = 0; i < 2 * kWords; ++i) {
                    qf[nt][i][0] = pack_f16x2(bf16_lo(w[2 * i]) * f, bf16_hi(w[2 * i]) * f);
                    qf[nt][i][1] = pack_f16x2(bf16_lo(w[2 * i + 1]) * f, bf16_hi(w[2 * i + 1]) * f);
                }
                // (Finite below: a key that the row does not see has a logit of -infinity.)
                const float mine = used ? fmaxf(lse * 1.4426950408889634f, -FLT_MAX) : INFINITY;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    scale[nt][i] = logit_scale(p.scale_log2, k_head, __shfl_sync(0xffffffffu, e, (2 * t + i) * 4));
                    off[nt][i] = __shfl_sync(0xffffffffu, mine, (2 * t + i) * 4);
                    const int row = nt * 8 + 2 * t + i;
                    lim[nt][i] = kv;
                    if (p.causal && row < rows) lim[nt][i] = kv - fresh + row / p.group + 1;
                    min_lim = min(min_lim, lim[nt][i]);
                }
            }
            min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 1));
            min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 2));
            auto work = [&](const KUnit<kD>& k, bool held) {
                float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
                if (held && rows > 0) {
                    float s[2][kNT][4];
                    uint32_t ks[2][2][kWords / 2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t two = e4m3_to_f16(k.scales[m][half]);
                            ks[m][half][0] = kWords == 4 ? __byte_perm(two, 0, 0x1010) : two;
                            if constexpr (kWords == 4) ks[m][half][1] = __byte_perm(two, 0, 0x3232);
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt) s[m][nt][2 * half] = s[m][nt][2 * half + 1] = 0.f;
                        }
#pragma unroll
                    for (int w = 0; w < kWords; ++w)
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                e2m1_to_f16(k.codes[m][half][w], a[half]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) a[half][i] = mul_f16x2(a[half][i], ks[m][half][w / 2]);
                            }
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int nt = 0; nt < kNT; ++nt)
                                    mma_f16(s[m][nt], a[0][2 * i], a[1][2 * i], a[0][2 * i + 1], a[1][2 * i + 1],
                                            qf[nt][2 * w + i][0], qf[nt][2 * w + i][1]);
                        }
                    const int key0 = u * kUnit;
                    if (key0 + kUnit > min_lim) {  // keys past a row's limit
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (key0 + 16 * m + 8 * (i >> 1) + g >= lim[nt][i & 1]) s[m][nt][i] = -INFINITY;
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                sum[m][i >> 1] += ex2_approx(fmaf(s[m][nt][i], scale[nt][i & 1], -off[nt][i & 1]));
                }
                // Sums over the four lanes of a token; lane t keeps that of (m, half) = (t / 2, t % 2).
                const bool hi = t & 2, odd = t & 1;
                float a0 = hi ? sum[1][0] : sum[0][0], a1 = hi ? sum[1][1] : sum[0][1];
                a0 += __shfl_xor_sync(0xffffffffu, hi ? sum[0][0] : sum[1][0], 2);
                a1 += __shfl_xor_sync(0xffffffffu, hi ? sum[0][1] : sum[1][1], 2);
                float y = odd ? a1 : a0;
                y += __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
                const int x = u * kUnit + 16 * (t >> 1) + 8 * (t & 1) + g;
                if (x < kv) out[x] = k.before + y;
            };
            int stage = 0;
#pragma unroll 1
            for (; u < end; ++u) {
                cp_async_wait<kStages - 1>();
                __syncwarp();
                KUnit<kD> k;
                take(stage, k);
                const bool held = there >> stage & 1u;
                __syncwarp();  // all have what they need of the stage
                ask(u + kStages, stage);
                work(k, held);
                stage = (stage + 1) % kStages;
            }
            left -= n;
        }
    }
    fill_rest(p, false);
}

template <int kD, int kNT, int kWarps>
cudaError_t launch_few(const WeighParams& p, int num_sms, cudaStream_t stream) {
    constexpr int smem = kWarps * kStages * (int)sizeof(Piece<kD>);
    static_assert(smem <= 232448, "shared memory of the weighing kernel");
    auto kernel = weigh_kernel<kD, kNT, kWarps>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
    return launch_early(kernel, dim3((unsigned)num_sms), kWarps * 32, smem, stream, p);
}

}  // namespace

cudaError_t launch_cache_weigh(const CacheView& c, int D, const void* q, const float* lse, int Sq, int heads,
                               const int32_t* q_lens, int causal, float sm_scale, const float* weights, float* out,
                               int num_sms, cudaStream_t stream) {
    WeighParams p;
    p.c = c;
    p.q = static_cast<const uint4*>(q);
    p.lse = lse;
    p.q_lens = q_lens;
    p.weights = weights;
    p.out = out;
    p.Sq = Sq;
    p.heads = heads;
    p.group = heads / c.kv_heads;
    p.causal = causal;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    const int rows = Sq * p.group;
    // weigh_kernel with as many row tiles of 8 as there are, or the chunk kernel.  Times
    // in us of weigh_kernel | the chunk kernel, 8 kv heads (more rows than these: the
    // registers for the queries leave too few warps):
    //   rows of a kv head           20           32
    //   D = 128,  1 x 32760     14.0 | 16.6  18.1 | 16.5
    //             8 x 8000      20.0 | 24.9  28.2 | 24.8
    //   D = 64,   1 x 32760     11.0 | 14.4  12.9 | 14.6
    //             8 x 8000      15.0 | 22.1  17.4 | 22.2
    // Warps of a block, one tile of 8 rows (61 sequences of up to 12000, D = 128): 57.6 us with
    // 16, 57.0 with 20, which makes single calls slower (9.1 and 9.8).
    if (rows > (D == 64 ? 32 : 24)) return launch_weigh_chunk(p, D, num_sms, stream);
    if (D == 64)
        return rows <= 8    ? launch_few<64, 1, 16>(p, num_sms, stream)
               : rows <= 16 ? launch_few<64, 2, 16>(p, num_sms, stream)
               : rows <= 24 ? launch_few<64, 3, 12>(p, num_sms, stream)
                            : launch_few<64, 4, 12>(p, num_sms, stream);
    return rows <= 8    ? launch_few<128, 1, 16>(p, num_sms, stream)
           : rows <= 16 ? launch_few<128, 2, 12>(p, num_sms, stream)
                        : launch_few<128, 3, 12>(p, num_sms, stream);
}

}  // namespace vsa
