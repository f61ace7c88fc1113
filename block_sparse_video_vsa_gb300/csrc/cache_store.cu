// Writing and reading the 4-bit paged cache.
//
// append_kernel: the keys and values of a step go to their pages, the keys
// (and the step's queries, to an output of their own) rotated on the way:
//   (x, y) -> (x c - y s, y c + x s) for the channel pairs (2i, 2i + 1) or
//   (i, i + R / 2), with c, s the fp32 table row of the token's position.
// Products and sums are rounded one by one (no fused multiply-add), so the
// fp32 result, and with it every code, is the one the formula gives step by
// step.  Then, for 16 channels with y = x / head scale:
//   scale = e4m3(max|y| / 6),  code = e2m1(y / scale)   (nearest, ties to even)
// where both divisions are multiplications by the fp32 reciprocal.
// HBM bound: (heads + 2 kv_heads) * D * 2 bytes in, heads * D * 2 + kv_heads
// * D * 9 / 8 out a token.  A thread takes 32 channels of one token (two
// scale groups, the two halves of a rotated pair among them) and holds their
// cosines and sines in registers over all heads it walks; a warp takes
// neighbouring tokens of one head, whose codes are contiguous in the page.
// Measured: a frame of 1560 tokens x 40 heads of 128, 19.2 us (3.8 TB/s of the
// bytes it needs, 56% of the measured copy rate), 24 ragged chunks of up to 1003
// tokens (24 and 8 heads of 64) 33.9 us (4.4 TB/s, 65%).  16 warps an SM issue 0.47
// instructions a scheduler and cycle and wait for loads otherwise; neither a
// second row on its way nor 16 channels a thread (32 warps an SM, 20.1 and
// 40.3 us beside 18.6 and 34.4 on the same day) made it better.
//
// read_kernel: pages back to bf16 rows, [B, S, kv_heads, D], zero past each
// sequence's length.  HBM bound (9/16 byte in, 2 bytes out an element): one
// block a page and head, 16-byte stores.  Measured: 32760 tokens x 40 heads of
// 128, 139 us, 6.2 TB/s (91% of the measured copy rate).
#include "cache.cuh"

namespace vsa {

namespace {

struct AppendParams {
    CacheView c;
    const unsigned char* q;
    const unsigned char* k;
    const unsigned char* v;
    unsigned char* q_out;
    const int32_t* new_lens;   // [B], or null: S
    const int32_t* positions;  // [B][S], or null: the token's place in its sequence
    const float* rope;         // [rope_rows][R]: R / 2 cosines, R / 2 sines
    int S, heads, rope_rows, R;
    int wide;  // q, k, v and q_out are aligned to 32 bytes
};

// 16 bf16 channels: a 32-byte sector, in one access where the tensor is aligned
// to it (`wide`; two half sectors a lane cost L2 twice the accesses).
struct Sector {
    uint32_t w[8];
};
__device__ __forceinline__ Sector load_sector(const unsigned char* at, bool wide) {
    Sector s;
    if (wide) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]), "=r"(s.w[5]),
                       "=r"(s.w[6]), "=r"(s.w[7])
                     : "l"(at)
                     : "memory");
    } else {
        const uint4 a = reinterpret_cast<const uint4*>(at)[0], b = reinterpret_cast<const uint4*>(at)[1];
        s.w[0] = a.x; s.w[1] = a.y; s.w[2] = a.z; s.w[3] = a.w;
        s.w[4] = b.x; s.w[5] = b.y; s.w[6] = b.z; s.w[7] = b.w;
    }
    return s;
}
__device__ __forceinline__ void store_sector(unsigned char* at, const Sector& s, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(s.w[0]), "r"(s.w[1]),
                     "r"(s.w[2]), "r"(s.w[3]), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(at)[0] = make_uint4(s.w[0], s.w[1], s.w[2], s.w[3]);
        reinterpret_cast<uint4*>(at)[1] = make_uint4(s.w[4], s.w[5], s.w[6], s.w[7]);
    }
}

// Codes (two words) and scale byte of 16 channels.  The cache holds finite
// numbers only: NaN is stored as 0, and what is beyond 448 * 6 saturates.
__device__ __forceinline__ uint32_t quantise16(const float* x, float inv_head, uint32_t (&code)[2]) {
    float y[16];
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        y[i] = __fmul_rn(x[i], inv_head);
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(fabsf(y[i])));
    }
    if (a != a) {  // (one look a group instead of one an element)
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            y[i] = y[i] == y[i] ? y[i] : 0.f;
            a = fmaxf(a, fabsf(y[i]));
        }
    }
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(__fmul_rn(a, 1.f / 6.f)));
    const float s = __half2float(__ushort_as_half((unsigned short)(e4m3_to_f16(s8) & 0xFFFFu)));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // No NaN here: a zero scale has no infinity in its group (that scale is 448).
            const float lo = __fmul_rn(y[8 * w + 2 * j], r), hi = __fmul_rn(y[8 * w + 2 * j + 1], r);
            uint32_t b;
            asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}"
                : "=r"(b)
                : "f"(hi), "f"(lo));
            word |= b << (8 * j);
        }
        code[w] = word;
    }
    return s8 & 0xFFu;
}

constexpr int kAppendThreads = 128;

// kTok tokens a block: 8 neighbouring tokens, or 1 for steps of few tokens
// (then the block's threads spread over heads instead).
template <int kD, int kTok, bool kPairs>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendParams p) {
    using L = PageLayout<kD>;
    constexpr int kSlices = kD / 32;                              // threads of a head row
    constexpr int kHeadLanes = kAppendThreads / (kSlices * kTok);  // heads in flight
    early();
    begin_work();
    const int slice = threadIdx.x % kSlices;
    const int b = blockIdx.z;
    const int tok = blockIdx.x * kTok + (threadIdx.x / kSlices) % kTok;
    if (tok >= p.S) return;
    const size_t token = (size_t)b * p.S + tok;
    const int hq = p.q_out ? p.heads : 0;
    const int all = hq + 2 * p.c.kv_heads;
    // The two groups of 16 channels: [g0, g0 + 16) and [g1, g1 + 16), rotated or
    // not.  Neighbouring lanes take neighbouring groups as far as the pairs
    // allow: an access then covers lines rather than every other sector of them.
    const int R0 = kPairs || slice * 32 < p.R ? 0 : p.R;  // halves: the channels that stay as they are begin at R
    const int g0 = R0 + (slice - R0 / 32) * 16;
    const int g1 = g0 + (kPairs ? kD : R0 == 0 && p.R > 0 ? p.R : kD - p.R) / 2;
    const bool turn0 = g0 < p.R, turn1 = kPairs ? g1 < p.R : turn0;
    const int step = gridDim.y * kHeadLanes;
    // Head h of all: a query head, a key head or a value head; its row of the token.
    auto row_of = [&](int h) -> const unsigned char* {
        const int kh = h < hq ? h : h < hq + p.c.kv_heads ? h - hq : h - hq - p.c.kv_heads;
        return h < hq ? p.q + (token * p.heads + kh) * (kD * 2)
                      : (h < hq + p.c.kv_heads ? p.k : p.v) + (token * p.c.kv_heads + kh) * (kD * 2);
    };
    int h = blockIdx.y * kHeadLanes + threadIdx.x / (kSlices * kTok);
    // The first row is on its way while the lengths, the page and the angles are looked up.
    Sector a, c;
    if (h < all) {
        a = load_sector(row_of(h) + g0 * 2, p.wide);
        c = load_sector(row_of(h) + g1 * 2, p.wide);
    }
    const int n = cache_len(p.c, b, threadIdx.x == 0);
    const int fresh = min(p.new_lens ? max(p.new_lens[b], 0) : p.S, min(p.S, n));
    const bool live = tok < fresh;
    const int at = n - fresh + tok;  // place in the sequence
    // Where the token goes.
    unsigned char* page = nullptr;
    if (live) {
        const int id = p.c.table[(size_t)b * p.c.width + at / kPageTokens];
        if (id >= 0 && id < p.c.pages)
            page = p.c.pool + (size_t)id * p.c.kv_heads * L::kBytes;
        else if (slice == 0)
            atomicOr(p.c.err, VSA_DEVERR_INDEX);
    }
    const int in_page = at % kPageTokens;
    float cs[16], sn[16];
    if (turn0 && live) {
        const int pos = p.positions ? p.positions[(size_t)b * p.S + tok] : at;
        if (pos >= 0 && pos < p.rope_rows) {
            // Angle i is that of channels (g0 + 2i, + 1) and, from 8 on, (g1 + 2i - 16, + 1), or of (g0 + i, g1 + i).
            const float4* row = reinterpret_cast<const float4*>(p.rope + (size_t)pos * p.R + (kPairs ? g0 / 2 : g0));
            const int skip = kPairs ? (turn1 ? (g1 - g0) / 8 - 2 : -2) : 0;  // of 16 bytes, to the second group's
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4* at4 = row + i + (i < 2 ? 0 : skip);
                const float4 u = at4[0], w = at4[p.R / 8];
                cs[4 * i] = u.x; cs[4 * i + 1] = u.y; cs[4 * i + 2] = u.z; cs[4 * i + 3] = u.w;
                sn[4 * i] = w.x; sn[4 * i + 1] = w.y; sn[4 * i + 2] = w.z; sn[4 * i + 3] = w.w;
            }
        } else {  // no such row: a zero rotation
            if (slice == 0) atomicOr(p.c.err, VSA_DEVERR_INDEX);
#pragma unroll
            for (int i = 0; i < 16; ++i) cs[i] = sn[i] = 0.f;
        }
    }
    if (!live) {  // a padding row: nothing to keep, its queries are zero
        Sector zero;
#pragma unroll
        for (int i = 0; i < 8; ++i) zero.w[i] = 0u;
        for (; h < hq; h += step) {
            unsigned char* dst = p.q_out + (token * p.heads + h) * (kD * 2);
            store_sector(dst + g0 * 2, zero, p.wide);
            store_sector(dst + g1 * 2, zero, p.wide);
        }
        return;
    }
    for (; h < all; h += step) {
        float x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[2 * i] = bf16_lo(a.w[i]);
            x[2 * i + 1] = bf16_hi(a.w[i]);
            x[16 + 2 * i] = bf16_lo(c.w[i]);
            x[16 + 2 * i + 1] = bf16_hi(c.w[i]);
        }
        if (h + step < all) {  // the next head's row is on its way while this one is worked on
            a = load_sector(row_of(h + step) + g0 * 2, p.wide);
            c = load_sector(row_of(h + step) + g1 * 2, p.wide);
        }
        const bool is_q = h < hq, is_k = !is_q && h < hq + p.c.kv_heads;
        const int kh = is_q ? h : is_k ? h - hq : h - hq - p.c.kv_heads;
        if (turn0 && (is_q || is_k)) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (kPairs && i >= 8 && !turn1) break;
                // Pair i: (2i, 2i + 1) of the 32 channels, or (i, 16 + i) of the two groups.
                float& u = x[kPairs ? 2 * i : i];
                float& w = x[kPairs ? 2 * i + 1 : 16 + i];
                const float y = u, z = w;
                u = __fsub_rn(__fmul_rn(y, cs[i]), __fmul_rn(z, sn[i]));
                w = __fadd_rn(__fmul_rn(z, cs[i]), __fmul_rn(y, sn[i]));
            }
        }
        if (is_q) {
            Sector y, z;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                z.w[i] = pack_bf16x2(x[16 + 2 * i], x[16 + 2 * i + 1]);
            }
            unsigned char* dst = p.q_out + (token * p.heads + kh) * (kD * 2);
            store_sector(dst + g0 * 2, y, p.wide);
            store_sector(dst + g1 * 2, z, p.wide);
        } else if (page) {
            const float hs = p.c.kv_scale ? p.c.kv_scale[(is_k ? 0 : p.c.kv_heads) + kh] : 1.f;
            const float inv = __frcp_rn(hs);
            uint32_t c0[2], c1[2];
            const uint32_t s0 = quantise16(x, inv, c0), s1 = quantise16(x + 16, inv, c1);
            unsigned char* head = page + (size_t)kh * L::kBytes;
            unsigned char* codes = head + (is_k ? 0 : L::kV) + in_page * L::kRow;
            unsigned char* scales = head + (is_k ? L::kKScale : L::kVScale) + in_page * L::kGroups;
            if (g1 == g0 + 16) {
                *reinterpret_cast<uint4*>(codes + g0 / 2) = make_uint4(c0[0], c0[1], c1[0], c1[1]);
                *reinterpret_cast<uint16_t*>(scales + g0 / 16) = (uint16_t)(s0 | (s1 << 8));
            } else {
                *reinterpret_cast<uint2*>(codes + g0 / 2) = make_uint2(c0[0], c0[1]);
                *reinterpret_cast<uint2*>(codes + g1 / 2) = make_uint2(c1[0], c1[1]);
                scales[g0 / 16] = (unsigned char)s0;
                scales[g1 / 16] = (unsigned char)s1;
            }
        }
    }
}

struct ReadParams {
    CacheView c;
    uint4* k;
    uint4* v;
    int S;
};

constexpr int kReadThreads = 256;

template <int kD>
__global__ void __launch_bounds__(kReadThreads) read_kernel(ReadParams p) {
    using L = PageLayout<kD>;
    constexpr int kLanes = kD / 8;                  // threads of a token row (8 channels each)
    constexpr int kStep = kReadThreads / kLanes;    // tokens a pass
    early();
    begin_work();
    const int h = blockIdx.y, b = blockIdx.z;
    const int first = blockIdx.x * kPageTokens;
    const int lane = threadIdx.x % kLanes;
    const int n = cache_len(p.c, b, threadIdx.x == 0);
    const unsigned char* page = nullptr;
    if (first < n) {
        const int id = p.c.table[(size_t)b * p.c.width + blockIdx.x];
        if (id >= 0 && id < p.c.pages)
            page = p.c.pool + ((size_t)id * p.c.kv_heads + h) * L::kBytes;
        else if (threadIdx.x == 0)
            atomicOr(p.c.err, VSA_DEVERR_INDEX);
    }
    // Both sides' loads come before the first store, which may be to anywhere.
    constexpr int kTurns = kPageTokens / kStep;
    float hs[2];
    uint32_t code[2][kTurns], scale[2][kTurns];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        hs[side] = p.c.kv_scale ? p.c.kv_scale[side * p.c.kv_heads + h] : 1.f;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int t = threadIdx.x / kLanes + i * kStep;
            const bool held = page && first + t < n;
            code[side][i] = held ? reinterpret_cast<const uint32_t*>(page + side * L::kV + t * L::kRow)[lane] : 0u;
            scale[side][i] = held ? (uint32_t)page[(side ? L::kVScale : L::kKScale) + t * L::kGroups + lane / 2] : 0u;
        }
    }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int t = first + threadIdx.x / kLanes + i * kStep;
            if (t >= p.S) continue;
            uint32_t e[4], w[4];
            e2m1_to_f16(code[side][i], e);
            const uint32_t s = e4m3_to_f16(scale[side][i] * 0x101u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t y = mul_f16x2(e[j], s);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y));
                w[j] = pack_bf16x2(f.x * hs[side], f.y * hs[side]);
            }
            uint4* dst = (side ? p.v : p.k) + (((size_t)b * p.S + t) * p.c.kv_heads + h) * kLanes + lane;
            __stcs(dst, make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(const CacheView& c, int D, const void* q, const void* k, const void* v, int S,
                                int heads, const int32_t* new_lens, const float* rope, int rope_rows, int rope_dim,
                                int interleaved, const int32_t* positions, void* q_out, int num_sms,
                                cudaStream_t stream) {
    AppendParams p;
    p.c = c;
    p.q = static_cast<const unsigned char*>(q);
    p.k = static_cast<const unsigned char*>(k);
    p.v = static_cast<const unsigned char*>(v);
    p.q_out = static_cast<unsigned char*>(q_out);
    p.wide = ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
               reinterpret_cast<uintptr_t>(q_out)) & 31u) == 0;
    p.new_lens = new_lens;
    p.positions = positions;
    p.rope = rope;
    p.S = S;
    p.heads = heads;
    p.rope_rows = rope_rows;
    p.R = rope_dim;
    const int all = (q_out ? heads : 0) + 2 * c.kv_heads;
    const int tok = S >= 8 ? 8 : 1;
    const int lanes = kAppendThreads / (D / 32 * tok);
    const int bx = (S + tok - 1) / tok;
    // Heads are spread over blocks as long as all blocks are resident at once (four
    // an SM): a frame's 585 blocks take 18.6 us, 1560 in 2.6 turns 22.5.
    const int most = (all + lanes - 1) / lanes;
    const long long blocks = (long long)bx * c.B;
    int by = (int)(4LL * num_sms / blocks);
    by = by < 1 ? 1 : by > most ? most : by;
    const dim3 grid((unsigned)bx, (unsigned)by, (unsigned)c.B);
    auto of_d64 = interleaved ? (tok == 8 ? append_kernel<64, 8, true> : append_kernel<64, 1, true>)
                              : (tok == 8 ? append_kernel<64, 8, false> : append_kernel<64, 1, false>);
    auto of_d128 = interleaved ? (tok == 8 ? append_kernel<128, 8, true> : append_kernel<128, 1, true>)
                               : (tok == 8 ? append_kernel<128, 8, false> : append_kernel<128, 1, false>);
    return launch_early(D == 64 ? of_d64 : of_d128, grid, kAppendThreads, 0, stream, p);
}

cudaError_t launch_cache_read(const CacheView& c, int D, int S, void* k, void* v, cudaStream_t stream) {
    ReadParams p;
    p.c = c;
    p.k = static_cast<uint4*>(k);
    p.v = static_cast<uint4*>(v);
    p.S = S;
    const dim3 grid((unsigned)((S + kPageTokens - 1) / kPageTokens), (unsigned)c.kv_heads, (unsigned)c.B);
    return launch_early(D == 64 ? read_kernel<64> : read_kernel<128>, grid, kReadThreads, 0, stream, p);
}

}  // namespace vsa
