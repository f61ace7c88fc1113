// Attention over the 4-bit paged cache, few query rows a kv head: the rows of
// a step's tokens times the heads that share the kv head.
//
//   s_x = sm_scale q . k_x,   out = sum_x softmax(s)_x v_x,   lse = log sum_x exp s_x
//
// over the sequence's cached tokens x (up to the query's own place when
// causal; those of the selected pages when a selection is given).
//
// HBM bound: 9/16 byte an element against 4 flops for each query row, so the
// kernel is built to keep bulk copies in flight and to spend few instructions
// on an element.
//  * A producer warp looks pages up and copies them whole (72 * D contiguous
//    bytes) into a ring; consumer warp w takes every kWarps-th page of the
//    CTA's part of the line (see cache.cuh) with a softmax state of its own,
//    and the warps' states are joined once a unit through shared memory.
//  * S^T = K Q^T and O^T = V^T P^T (m16n8k16, fp16 in, fp32 out): the matrix
//    instructions' 16-row side holds tokens, then channels, so 8 query rows
//    fill them.  tcgen05 is no help here: its smallest tile has 64 rows and
//    its operands would have to be written to shared memory first.
//  * Codes go from shared memory to fragments without a shuffle: the order of
//    channels within K Q^T is free, so a lane takes 32 neighbouring channels
//    of a token; for V^T P^T a lane takes the 16 channels of one scale group
//    of four tokens and the conversion's byte holds two tokens' codes of a
//    channel.  Conversion and scale are two instructions for two elements
//    (a conversion and a product), exact in fp16.
//  * P is rounded to fp16 (2^-11 relative; the sum keeps the fp32 values);
//    maximum, sum and output are fp32.  The maximum is followed lazily: the
//    output is rescaled when it grows by more than 2^8.
#include "cache.cuh"

namespace vsa {

namespace {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// (a & m) | (b & ~m)
__device__ __forceinline__ uint32_t bit_select(uint32_t m, uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(m), "r"(a), "r"(b));
    return d;
}

// Shared memory of the kernel: kSlots pages, then the warps' states.
template <int kD, int kNT, int kWarps, int kSlots>
struct TokenSmem {
    static constexpr int kRows = 8 * kNT;
    static constexpr int kRowPad = kD + 4;  // floats: neighbouring rows start in other banks
    unsigned char page[kSlots][PageLayout<kD>::kBytes];
    float o[kWarps][kRows][kRowPad];
    float2 ml[kWarps][kRows];
    uint64_t full[kSlots];
    uint64_t empty[kSlots];
    int logical[kSlots];  // page number within the sequence, or -1: nothing to read
    PlanScratch plan;
    int abort_flag;
    int stop;  // abort_flag as one thread read it between the joining barriers
};

// One unit's rows as the consumer warps hold them.
template <int kNT>
struct RowState {
    float m[kNT][2], l[kNT][2];   // rows nt * 8 + 2 t + e: maximum (log2 units), this lane's share of the sum
    float scale[kNT][2];          // logit -> log2 units
    int lim[kNT][2];              // first key the row does not see
};

template <int kD, int kNT, int kWarps, int kSlots>
__global__ void __launch_bounds__((kWarps + 1) * 32, 1) token_kernel(AttnParams p) {
    using L = PageLayout<kD>;
    using Smem = TokenSmem<kD, kNT, kWarps, kSlots>;
    constexpr int kTiles = kPageTokens / 16;  // token tiles of a page
    constexpr int kWords = kD / 32;           // code words a lane holds of a K row
    constexpr int kChan = kD / 8;             // V channels of a lane
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_u32(&sm.full[s]), 1);
            mbar_init(smem_u32(&sm.empty[s]), 1);
        }
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    // The joining kernel may be set up meanwhile (its blocks wait for this grid's end).
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Walk walk;
    if (!walk.begin(p, sm.plan)) return;
    volatile int* abort_flag = &sm.abort_flag;

    if (warp == kWarps) {
        // =========================================================== producer
        uint32_t j = 0;
        bool ok = true;
        for (Segment sg; ok && walk.next(p, sg);) {
            const unsigned char* pool = p.c.pool + (size_t)sg.h * L::kBytes;
            for (int base = sg.first; base < sg.last && ok; base += 32) {
                // Lane i looks up page base + i.
                int logical = 0, id = -1;
                if (base + lane < sg.last) look_up(p, sg, base + lane, logical, id);
                const int n = min(32, sg.last - base);
                for (int i = 0; i < n; ++i, ++j) {
                    const int slot = j % kSlots;
                    const int page = __shfl_sync(0xffffffffu, id, i), num = __shfl_sync(0xffffffffu, logical, i);
                    if (j >= (uint32_t)kSlots) {
                        ok = mbar_wait_bounded(smem_u32(&sm.empty[slot]), (j / kSlots + 1) & 1, abort_flag, p.c.err,
                                               kCacheWaitNs);
                        if (!ok) break;
                    }
                    if (lane == 0) {
                        sm.logical[slot] = page < 0 ? -1 : num;
                        const uint32_t bar = smem_u32(&sm.full[slot]);
                        if (page < 0) {
                            mbar_arrive(bar);
                        } else {
                            mbar_arrive_expect_tx(bar, L::kBytes);
                            bulk_load(smem_u32(sm.page[slot]), pool + (size_t)page * p.c.kv_heads * L::kBytes,
                                      L::kBytes, bar);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        // The copies in flight land before the CTA's shared memory is released.
        if (lane == 0) {
            for (int s = 0; s < kSlots && (uint32_t)s < j; ++s) {
                const uint32_t lastj = j - 1 - ((j - 1 - s) % kSlots);
                mbar_wait_drain_1(smem_u32(&sm.full[s]), (lastj / kSlots) & 1, p.c.err, kCacheWaitNs);
            }
        }
        return;
    }

    // ============================================================= consumers
    // Row r of a page tile sits at token f(r) = r ^ ((r >> 1) & 1) of its 8: of
    // the four tokens that a V load's lanes t = 0..3 read, two are even and two
    // odd (64-byte rows: 2-way bank conflicts instead of 4-way).
    const int k_row = g ^ ((g >> 1) & 1);
    const int v_row0 = (2 * t) ^ (t & 1), v_row1 = (2 * t + 1) ^ (t & 1);
    const int R = p.Sq * p.group;
    uint32_t j = 0;      // pages of the part before the segment
    bool ok = true;
    for (Segment at; walk.next(p, at);) {
        // ------------------------------------------------ the unit's queries
        uint32_t qf[kNT][2 * kWords][2];
        RowState<kNT> rs;
        const int row0 = at.t * p.tile;
        const int live_rows = min(at.len.q * p.group, row0 + 8 * kNT);
        int min_lim = at.len.kv;
        const float c_head = p.scale_log2 * (p.c.kv_scale ? __ldg(p.c.kv_scale + at.h) : 1.f);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int row = row0 + nt * 8 + g;
            uint32_t w[4 * kWords];
            const bool real = row < R;
            const int qi = real ? row / p.group : 0;
            const int head = at.h * p.group + (real ? row - qi * p.group : 0);
            const uint4* src = p.q + (((size_t)at.b * p.Sq + qi) * p.heads + head) * (kD / 8) + t * kWords;
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint4 x = real ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
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
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int er = __shfl_sync(0xffffffffu, e, (2 * t + c) * 4);
                const int r = row0 + nt * 8 + 2 * t + c;
                rs.scale[nt][c] = c_head * pow2i(-er);
                rs.m[nt][c] = -INFINITY;
                rs.l[nt][c] = 0.f;
                int lim = at.len.kv;
                if (p.causal && r < live_rows) lim = min(lim, at.len.kv - at.len.q + r / p.group + 1);
                rs.lim[nt][c] = lim;
                min_lim = min(min_lim, lim);
            }
        }
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 1));
        min_lim = min(min_lim, __shfl_xor_sync(0xffffffffu, min_lim, 2));
        float o[kChan / 2][kNT][4];
#pragma unroll
        for (int i = 0; i < kChan / 2; ++i)
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][nt][c] = 0.f;

        // ------------------------------------------------------------- pages
        const uint32_t j1 = j + (uint32_t)(at.last - at.first);
        for (uint32_t jj = j + (warp + kWarps - j % kWarps) % kWarps; jj < j1; jj += kWarps) {
            const int slot = jj % kSlots;
            ok = mbar_wait_bounded(smem_u32(&sm.full[slot]), (jj / kSlots) & 1, abort_flag, p.c.err, kCacheWaitNs);
            if (!ok) break;
            const int logical = sm.logical[slot];
            if (logical < 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
                continue;
            }
            const unsigned char* page = sm.page[slot];
            const int key0 = logical * kPageTokens;
            // S^T
            float s[kTiles][kNT][4];
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
                for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[m][nt][c] = 0.f;
                uint32_t kw[2][kWords], ks[2][kWords / 2];
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int tok = 16 * m + 8 * half + k_row;
                    const unsigned char* src = page + tok * L::kRow + t * (kWords * 4);
                    const unsigned char* sc = page + L::kKScale + tok * L::kGroups + t * (kWords / 2);
                    if constexpr (kWords == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src);
                        kw[half][0] = x.x; kw[half][1] = x.y; kw[half][2] = x.z; kw[half][3] = x.w;
                        const uint32_t two = e4m3_to_f16(*reinterpret_cast<const uint16_t*>(sc));
                        ks[half][0] = __byte_perm(two, 0, 0x1010);
                        ks[half][1] = __byte_perm(two, 0, 0x3232);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        kw[half][0] = x.x; kw[half][1] = x.y;
                        ks[half][0] = e4m3_to_f16((uint32_t)*sc * 0x101u);
                    }
                }
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        e2m1_to_f16(kw[half][w], a[half]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) a[half][i] = mul_f16x2(a[half][i], ks[half][w / 2]);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(s[m][nt], a[0][2 * i], a[1][2 * i], a[0][2 * i + 1], a[1][2 * i + 1],
                                    qf[nt][2 * w + i][0], qf[nt][2 * w + i][1]);
                }
            }
            // Keys past a row's limit (and scores of what lies there) do not count.
            const bool masked = key0 + kPageTokens > min_lim;
            if (masked) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int key = key0 + 16 * m + 8 * (c >> 1) + k_row;
                            if (key >= rs.lim[nt][c & 1]) s[m][nt][c] = -INFINITY;
                        }
            }
            // Online softmax; P^T as fp16 fragments.
            uint32_t pf[kTiles][kNT][2];
            float alpha[kNT][2];
            bool rescale = false;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
                    for (int m = 1; m < kTiles; ++m) mx = fmaxf(mx, fmaxf(s[m][nt][c], s[m][nt][c + 2]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    mx *= rs.scale[nt][c];
                    alpha[nt][c] = 1.f;
                    if (mx > rs.m[nt][c] + kCacheRescale || (rs.m[nt][c] == -INFINITY && mx > -INFINITY)) {
                        alpha[nt][c] = rs.m[nt][c] == -INFINITY ? 0.f : ex2_approx(rs.m[nt][c] - mx);
                        rs.m[nt][c] = mx;
                        rs.l[nt][c] *= alpha[nt][c];
                        rescale = true;
                    }
                    const float mb = rs.m[nt][c] == -INFINITY ? 0.f : rs.m[nt][c];
                    float sum = 0.f;
#pragma unroll
                    for (int m = 0; m < kTiles; ++m)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float& x = s[m][nt][c + 2 * half];
                            x = ex2_approx(fmaf(x, rs.scale[nt][c], -mb));
                            sum += x;
                        }
                    rs.l[nt][c] += sum;
                }
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    pf[m][nt][0] = transpose8x8(pack_f16x2(s[m][nt][0], s[m][nt][1]));
                    pf[m][nt][1] = transpose8x8(pack_f16x2(s[m][nt][2], s[m][nt][3]));
                }
            }
            if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
                for (int i = 0; i < kChan / 2; ++i)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) o[i][nt][c] *= alpha[nt][c & 1];
            }
            // O^T += V^T P^T
            const bool ragged = key0 + kPageTokens > at.len.kv;  // slots past the length hold anything
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                int tok[4] = {16 * m + v_row0, 16 * m + v_row1, 16 * m + 8 + v_row0, 16 * m + 8 + v_row1};
                uint32_t vw[4][kChan / 8], sc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned char* src = page + L::kV + tok[i] * L::kRow + g * (kChan / 2);
                    if constexpr (kChan == 16) {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        vw[i][0] = x.x; vw[i][1] = x.y;
                    } else {
                        vw[i][0] = *reinterpret_cast<const uint32_t*>(src);
                    }
                    sc[i] = page[L::kVScale + tok[i] * L::kGroups + g * kChan / 16];
                    if (ragged && key0 + tok[i] >= at.len.kv) sc[i] = 0u;
                }
                const uint32_t s01 = e4m3_to_f16(sc[0] | (sc[1] << 8)), s23 = e4m3_to_f16(sc[2] | (sc[3] << 8));
#pragma unroll
                for (int w = 0; w < kChan / 8; ++w) {
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    e2m1_to_f16(bit_select(0x0F0F0F0Fu, vw[0][w], vw[1][w] << 4), a0);  // even channels
                    e2m1_to_f16(bit_select(0x0F0F0F0Fu, vw[0][w] >> 4, vw[1][w]), a1);  // odd channels
                    e2m1_to_f16(bit_select(0x0F0F0F0Fu, vw[2][w], vw[3][w] << 4), a2);
                    e2m1_to_f16(bit_select(0x0F0F0F0Fu, vw[2][w] >> 4, vw[3][w]), a3);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x0 = mul_f16x2(a0[i], s01), x1 = mul_f16x2(a1[i], s01);
                        const uint32_t x2 = mul_f16x2(a2[i], s23), x3 = mul_f16x2(a3[i], s23);
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt)
                            mma_f16(o[4 * w + i][nt], x0, x1, x2, x3, pf[m][nt][0], pf[m][nt][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
        }
        j = j1;

        // ------------------------------------- join the warps, write the rows
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = rs.l[nt][c];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int r = nt * 8 + 2 * t + c;
                if (g == 0) sm.ml[warp][r] = make_float2(rs.m[nt][c], l);
                float4* dst = reinterpret_cast<float4*>(&sm.o[warp][r][g * kChan]);
#pragma unroll
                for (int i = 0; i < kChan / 4; ++i)
                    dst[i] = make_float4(o[2 * i][nt][c], o[2 * i][nt][c + 2], o[2 * i + 1][nt][c],
                                         o[2 * i + 1][nt][c + 2]);
            }
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        constexpr int kRows = Smem::kRows, kQuads = kD / 4;
        const float v_head = p.c.kv_scale ? __ldg(p.c.kv_scale + p.c.kv_heads + at.h) : 1.f;
        for (int e = threadIdx.x; e < kRows * kQuads; e += kWarps * 32) {
            const int r = e / kQuads, c4 = e % kQuads;
            if (row0 + r >= R) continue;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.ml[w][r].x);
            float l = 0.f;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 ml = sm.ml[w][r];
                const float a = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][r][4 * c4]);
                l = fmaf(a, ml.y, l);
                sum.x = fmaf(a, x.x, sum.x);
                sum.y = fmaf(a, x.y, sum.y);
                sum.z = fmaf(a, x.z, sum.z);
                sum.w = fmaf(a, x.w, sum.w);
            }
            if (at.whole) {
                const int qi = (row0 + r) / p.group, head = at.h * p.group + (row0 + r) - qi * p.group;
                const bool live = row0 + r < live_rows && l != 0.f;
                const float inv = live ? v_head / l : 0.f;
                uint2* dst = reinterpret_cast<uint2*>(p.out + (((size_t)at.b * p.Sq + qi) * p.heads + head) * (kD / 8));
                dst[c4] = live ? make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv))
                               : make_uint2(0u, 0u);
                if (c4 == 0 && p.lse)
                    p.lse[((size_t)at.b * p.heads + head) * p.Sq + qi] =
                        live ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
            } else {
                const size_t slot = 2 * (size_t)blockIdx.x + (at.first > 0 ? 0 : 1);
                reinterpret_cast<float4*>(p.part_o)[(slot * p.tile + r) * kQuads + c4] = sum;
                if (c4 == 0) p.part_ml[slot * p.tile + r] = make_float2(m, l);
            }
        }
        // Every warp goes on or leaves with the others: they read one thread's view of the flag.
        if (threadIdx.x == 0) sm.stop = *abort_flag;
        asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
        if (*reinterpret_cast<volatile int*>(&sm.stop)) break;
    }
}

// Joins the parts of the units that were cut.  Block y looks at the cut before
// CTA y + 1's part; the unit's first cut does the work, one warp a row:
//   m = max m_i, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i
constexpr int kJoinWarps = 4;

template <int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(AttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c0 = blockIdx.y;  // the CTA that begins the unit, if this is its first cut
    const int4 u = p.places[c0 + 1];
    if (u.x < 0 || u.w == 0) return;
    const int4 prev = p.places[c0];
    if (prev.w > 0 && prev.x == u.x && prev.y == u.y && prev.z == u.z) return;
    const int lane = threadIdx.x & 31;
    int c1 = c0 + 1;  // the unit's last CTA
    for (bool in = true; in;) {
        const int c = c1 + 1 + lane;
        int4 x = make_int4(-1, 0, 0, 0);
        if (c < p.grid) x = p.places[c];
        const unsigned same = __ballot_sync(0xffffffffu, x.x == u.x && x.y == u.y && x.z == u.z && x.w > 0);
        const int n = __ffs(~same) - 1;  // -1: all 32
        c1 += n < 0 ? 32 : n;
        in = n < 0;
    }
    const SeqLens len = seq_lens(p, u.x);
    const int R = p.Sq * p.group, live_rows = len.q * p.group;
    const float v_head = p.c.kv_scale ? __ldg(p.c.kv_scale + p.c.kv_heads + u.y) : 1.f;
    const int r = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    const int row = u.z * p.tile + r;
    if (row >= R) return;
    // Slot 1 of the unit's first CTA, slot 0 of the others.
    float m = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) m = fmaxf(m, p.part_ml[(2 * (size_t)c + (c == c0)) * p.tile + r].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    constexpr int kPer = kD / 32;
    float l = 0.f, sum[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
        const size_t at = (2 * (size_t)c + (c == c0)) * p.tile + r;
        const float2 ml = p.part_ml[at];
        const float a = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
        l = fmaf(a, ml.y, l);
        float o[kPer];
        if constexpr (kPer == 4)
            *reinterpret_cast<float4*>(o) = *reinterpret_cast<const float4*>(p.part_o + at * kD + lane * kPer);
        else
            *reinterpret_cast<float2*>(o) = *reinterpret_cast<const float2*>(p.part_o + at * kD + lane * kPer);
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[i] = fmaf(a, o[i], sum[i]);
    }
    const int qi = row / p.group, head = u.y * p.group + row - qi * p.group;
    const bool live = row < live_rows && l != 0.f;
    const float inv = live ? v_head / l : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (((size_t)u.x * p.Sq + qi) * p.heads + head) * (kD / 8)) +
                    lane * (kPer / 2);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) dst[i / 2] = live ? pack_bf16x2(sum[i] * inv, sum[i + 1] * inv) : 0u;
    if (lane == 0 && p.lse)
        p.lse[((size_t)u.x * p.heads + head) * p.Sq + qi] =
            live ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <int kD, int kNT, int kWarps, int kSlots>
cudaError_t launch_token(const AttnParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(TokenSmem<kD, kNT, kWarps, kSlots>);
    static_assert(smem <= 232448, "shared memory of the token kernel");
    // A slot is always read by the same warp, so no warp can look for a slot's
    // next phase before the present one has completed.
    static_assert(kSlots % kWarps == 0, "slots are dealt to warps");
    auto kernel = token_kernel<kD, kNT, kWarps, kSlots>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<p.grid, (kWarps + 1) * 32, smem, stream>>>(p);
    note_launches(1);
    return cudaGetLastError();
}

// Rows of a unit: up to 16 rows a kv head go to token_kernel, more to chunk_kernel.
int tile_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 128; }

}  // namespace

size_t cache_attn_workspace_bytes(int D, int Sq, int group) {
    const int tile = tile_rows(Sq * group);
    return (size_t)kMaxGrid * 16 + (size_t)2 * kMaxGrid * tile * ((size_t)D * 4 + 8);
}

cudaError_t launch_cache_attn(const CacheView& c, int D, const void* q, int Sq, int heads, const int32_t* q_lens,
                              int causal, const int32_t* page_sel, int nsel, float sm_scale, void* workspace,
                              void* out, float* lse, int num_sms, cudaStream_t stream) {
    AttnParams p;
    p.c = c;
    p.q_lens = q_lens;
    p.page_sel = page_sel;
    p.q = static_cast<const uint4*>(q);
    p.out = static_cast<uint4*>(out);
    p.lse = lse;
    p.Sq = Sq;
    p.heads = heads;
    p.group = heads / c.kv_heads;
    p.nsel = nsel;
    p.causal = causal;
    const int rows = Sq * p.group;
    p.tile = tile_rows(rows);
    p.tiles = (rows + p.tile - 1) / p.tile;
    p.grid = num_sms < kMaxGrid ? num_sms : kMaxGrid;
    p.places = static_cast<int4*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.places + kMaxGrid);
    p.part_o = reinterpret_cast<float*>(p.part_ml + (size_t)2 * kMaxGrid * p.tile);
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    // Short walks are not worth joining: a unit of up to kWholePages pages stays in one CTA.
    constexpr int kWholePages = 8;
    const int most = page_sel ? nsel : c.width;
    p.whole = most <= kWholePages;
    cudaError_t e;
    if (p.tile == 128)
        e = launch_chunk(p, D, stream);
    else if (D == 64)
        e = p.tile == 8 ? launch_token<64, 1, 11, 22>(p, stream) : launch_token<64, 2, 7, 21>(p, stream);
    else
        e = p.tile == 8 ? launch_token<128, 1, 7, 21>(p, stream) : launch_token<128, 2, 7, 14>(p, stream);
    if (e != cudaSuccess || p.whole) return e;
    // Launched early (it waits for the attention kernel's end by itself).
    if (p.grid < 2) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.tile + kJoinWarps - 1) / kJoinWarps), (unsigned)(p.grid - 1));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = D == 64 ? cudaLaunchKernelEx(&cfg, combine_kernel<64>, p) : cudaLaunchKernelEx(&cfg, combine_kernel<128>, p);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace vsa
