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
//  * The warps take equal stretches of the CTA's part of the line (see
//    cache.cuh), in pieces of 32 tokens (half pages).  Each looks its pages up,
//    keeps bulk copies of its next pages (72 * D contiguous bytes) in flight and
//    has a softmax state of its own.  At a unit's end each leaves its state, and
//    the warp that comes last joins them and writes the rows, while the others
//    are at the next unit: no barrier among the warps.
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
//  * P is rounded to fp16 (2^-11 relative, down to 2^-32 of the row's largest;
//    the sum keeps the fp32 values); reference, sum and output are fp32.  The
//    reference (7 below the maximum, see kCacheHeadroom) follows lazily: the
//    output is rescaled when the maximum grows by more than 2^8.
//  * Measured (GB300): 61 ragged sequences of up to 12000 tokens, 32 heads on 8
//    of 128: 101 us, 4.45 TB/s (65% of the measured copy rate).  What bounds it
//    is issue: 1200 instructions a page at 0.55 a scheduler and cycle, 12 warps
//    an SM (163 registers).  A producer warp with 7 consumers behind a barrier
//    a unit took 127 us.  One token on one clip of 32760 tokens takes 22 us.
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

// A page is walked in two pieces of 32 tokens.
constexpr int kPieceTokens = 32;

// The CTA's part of the line is cut again, into equal stretches for its warps
// (in half pages): a warp meets few units, and a unit's warps are neighbours.
template <int kWarps>
struct Tasks {
    int width;                // of a warp's stretch
    long long base;           // where the next segment begins
    int first_warp, count;    // of the segment: its warps
    __device__ void begin_part(const AttnParams& p, const Walk& walk) {
        long long n = walk.left;
        if (p.whole) {  // the last unit may reach over the part's end
            Walk w = walk;
            n = 0;
            for (Segment s; w.next(p, s);) n += s.length;
        }
        width = (int)max(1LL, (2 * n + kWarps - 1) / kWarps);
        base = 0;
    }
    // This warp's pieces [first, end) of the segment; false: it has no part in it.
    __device__ bool take(const Segment& s, int warp, int& first, int& end) {
        const int n = 2 * (s.last - s.first);
        first_warp = (int)(base / width);
        count = (int)((base + max(n, 1) - 1) / width) - first_warp + 1;
        const long long lo = (long long)warp * width - base;  // the stretch, from the segment's first piece on
        base += 2LL * s.length;
        first = 2 * s.first + (int)max(0LL, min((long long)n, lo));
        end = 2 * s.first + (int)max(0LL, min((long long)n, lo + width));
        return warp >= first_warp && warp < first_warp + count;
    }
};

// A warp's state at a unit's end: O [kRows][kRowPad], then (reference in log2
// units, sum) [kRows].
template <int kD, int kNT>
struct TokenState {
    static constexpr int kRows = 8 * kNT;
    static constexpr int kRowPad = kD + 4;  // floats: neighbouring rows start in other banks
    float o[kRows][kRowPad];
    float2 ml[kRows];
};

// Shared memory of the kernel: kOwn page slots for each warp.
template <int kD, int kNT, int kWarps, int kOwn>
struct TokenSmem {
    unsigned char page[kWarps][kOwn][PageLayout<kD>::kBytes];
    uint64_t full[kWarps][kOwn];
    int number[kWarps][kOwn];  // page number within the sequence, or -1: nothing to read
    // Of the states that a warp leaves: the unit (from 1) and where it is (in
    // the warp's first slot when the warp has no more pages to come, else in
    // the workspace: the slots are better used for pages).  [0]: of the unit
    // that an earlier warp begins, the first of the warp's stretch; [1]: of a
    // unit that it begins itself.  Those that end in its stretch it joins at
    // once, so neither is ever needed again before it has been read.
    unsigned int left[kWarps][2];
    TokenState<kD, kNT>* state[kWarps][2];
    unsigned int claimed[kWarps];  // by a unit's first warp: the unit, once a warp joins it
    // Each warp's walks of the part (of the pages it asks for, and of those it
    // works on) and the 32 pages it has looked up last.
    Walk ask_walk[kWarps], walk[kWarps];
    Tasks<kWarps> ask_tasks[kWarps], tasks[kWarps];
    Segment ask_unit[kWarps], unit[kWarps];
    int2 pages[kWarps][32];  // place in the pool (-1: passed over), page number
    PlanScratch plan;
    int abort_flag;
    static_assert(sizeof(TokenState<kD, kNT>) <= kOwn * PageLayout<kD>::kBytes, "a state fits a warp's slots");
};

template <int kD, int kNT, int kWarps, int kOwn>
__global__ void __launch_bounds__(kWarps * 32, 1) token_kernel(AttnParams p) {
    using L = PageLayout<kD>;
    using Smem = TokenSmem<kD, kNT, kWarps, kOwn>;
    using State = TokenState<kD, kNT>;
    constexpr int kTiles = kPieceTokens / 16;  // token tiles of a piece
    constexpr int kWords = kD / 32;            // code words a lane holds of a K row
    constexpr int kChan = kD / 8;              // V channels of a lane
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;

    if (threadIdx.x < kWarps * kOwn) {
        mbar_init(smem_u32(&sm.full[0][threadIdx.x]), 1);
        if (threadIdx.x < kWarps) sm.left[threadIdx.x][0] = sm.left[threadIdx.x][1] = sm.claimed[threadIdx.x] = 0;
        if (threadIdx.x == 0) sm.abort_flag = 0;
        fence_barrier_init();
    }
    early();
    begin_work();
    {
        Walk w;
        if (!w.begin(p, sm.plan)) return;
        Tasks<kWarps> tk;
        tk.begin_part(p, w);
        if (lane == 0) {
            sm.walk[warp] = w;
            sm.tasks[warp] = tk;
        }
        __syncthreads();  // the barriers and flags above are every warp's
    }
    volatile int* abort_flag = &sm.abort_flag;

    // Asks for the warp's next page, into its next slot (which it has done
    // with): the pages of its tasks in order, kOwn ahead of its work.
    uint32_t asked = 0;
    int ask = 0, ask_end = 0, page0 = 0;  // the task's pages; first of those looked up
    bool ask_more = true;
    // The next unit of which this warp has pieces [first, end); counts the units on the way.
    auto next_task = [&](Walk& walk, Tasks<kWarps>& tasks, Segment& unit, int& first, int& end, unsigned& units) {
        Walk w = walk;
        Tasks<kWarps> tk = tasks;
        Segment s;
        bool has;
        do {
            has = w.next(p, s);
            ++units;
        } while (has && !tk.take(s, warp, first, end));
        __syncwarp();
        if (lane == 0) {
            walk = w;
            tasks = tk;
            unit = s;
        }
        __syncwarp();
        return has;
    };
    auto look_up_32 = [&](int first) {  // of the unit asked for
        const Segment& u = sm.ask_unit[warp];
        int2 x = make_int2(-1, 0);
        if (first + lane < u.last) look_up(p, u, first + lane, x.y, x.x);
        __syncwarp();
        sm.pages[warp][lane] = x;
        page0 = first;
        __syncwarp();
    };
    auto ask_next = [&]() {
        while (ask == ask_end && ask_more) {
            unsigned units = 0;
            int first = 0, end = 0;
            ask_more = next_task(sm.ask_walk[warp], sm.ask_tasks[warp], sm.ask_unit[warp], first, end, units);
            if (!ask_more) return;
            ask = first >> 1;
            ask_end = (end + 1) >> 1;
            if (ask < ask_end) look_up_32(ask);
        }
        if (!ask_more) return;
        if (ask - page0 == 32) look_up_32(ask);
        const int2 page = sm.pages[warp][ask - page0];
        const int slot = asked % kOwn;
        if (lane == 0) {
            const uint32_t bar = smem_u32(&sm.full[warp][slot]);
            sm.number[warp][slot] = page.x < 0 ? -1 : page.y;
            if (page.x < 0) {
                mbar_arrive(bar);
            } else {
                mbar_arrive_expect_tx(bar, L::kBytes);
                bulk_load(smem_u32(sm.page[warp][slot]),
                          p.c.pool + ((size_t)page.x * p.c.kv_heads + sm.ask_unit[warp].h) * L::kBytes, L::kBytes, bar);
            }
        }
        ++asked;
        ++ask;
    };
    // Row r of a token tile sits at token f(r) = r ^ ((r >> 1) & 1) of its 8: of
    // the four tokens that a V load's lanes t = 0..3 read, two are even and two
    // odd (64-byte rows: 2-way bank conflicts instead of 4-way).
    const int k_row = g ^ ((g >> 1) & 1);
    const int v_row0 = (2 * t) ^ (t & 1), v_row1 = (2 * t + 1) ^ (t & 1);
    const int R = p.Sq * p.group;
    uint32_t j = 0;            // this warp's pages so far
    unsigned int unit = 0;     // units so far
    int piece_begin = 0, piece_end = 0;
    const Segment& at = sm.unit[warp];
    bool ok = next_task(sm.walk[warp], sm.tasks[warp], sm.unit[warp], piece_begin, piece_end, unit);
    if (ok) {  // the first unit is also the first to ask for
        if (lane == 0) {
            sm.ask_walk[warp] = sm.walk[warp];
            sm.ask_tasks[warp] = sm.tasks[warp];
            sm.ask_unit[warp] = at;
        }
        __syncwarp();
        ask = piece_begin >> 1;
        ask_end = (piece_end + 1) >> 1;
        if (ask < ask_end) look_up_32(ask);
#pragma unroll 1
        for (int i = 0; i < kOwn; ++i) ask_next();
    }
    for (; ok; ok = ok && next_task(sm.walk[warp], sm.tasks[warp], sm.unit[warp], piece_begin, piece_end, unit)) {
        const int present = sm.tasks[warp].count, first_warp = sm.tasks[warp].first_warp;  // the unit's warps
        const bool none = at.first == at.last;  // no pages: this warp writes the rows alone
        // ------------------------------------------------ the unit's queries
        uint32_t qf[kNT][2 * kWords][2];
        float rs_m[kNT][2], rs_l[kNT][2];  // rows nt * 8 + 2 t + c: reference (log2 units), this lane's share of the sum
        float rs_scale[kNT][2];            // logit -> log2 units
        int rs_lim[kNT][2];                // first key the row does not see
        const int row0 = at.t * p.tile;
        const int live_rows = min(at.len.q * p.group, row0 + 8 * kNT);
        int min_lim = at.len.kv;
        const float k_head = p.c.kv_scale ? p.c.kv_scale[at.h] : 1.f;
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
                const uint4 x = real ? src[i] : make_uint4(0, 0, 0, 0);
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
                rs_scale[nt][c] = logit_scale(p.scale_log2, k_head, er);
                rs_m[nt][c] = -INFINITY;
                rs_l[nt][c] = 0.f;
                int lim = at.len.kv;
                if (p.causal && r < live_rows) lim = min(lim, at.len.kv - at.len.q + r / p.group + 1);
                rs_lim[nt][c] = lim;
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

        // ------------------------------------------------------------ pieces
#pragma unroll 1
        for (int pc = piece_begin; pc < piece_end; ++pc) {
            const int slot = j % kOwn;
            const int half = pc & 1;
            if (!half || pc == piece_begin) {
                ok = cache_wait<kSleepShort>(smem_u32(&sm.full[warp][slot]), (j / kOwn) & 1, abort_flag, p.c.err);
                if (!ok) break;
            }
            const bool page_end = half || pc + 1 == piece_end;  // done with the page after this piece
            const int number = sm.number[warp][slot];
            const int key0 = number * kPageTokens + half * kPieceTokens;
            if (number < 0 || key0 >= at.len.kv) {
                if (page_end) {
                    ++j;
                    __syncwarp();
                    ask_next();
                }
                continue;
            }
            const unsigned char* page = sm.page[warp][slot];
            const int tok0 = half * kPieceTokens;
            // S^T: the two token tiles side by side (their sums do not wait for one another)
            float s[kTiles][kNT][4];
            uint32_t kw[kTiles][2][kWords], ks[kTiles][2][kWords / 2];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int tok = tok0 + 16 * m + 8 * half + k_row;
                    const unsigned char* src = page + tok * L::kRow + t * (kWords * 4);
                    const unsigned char* sc = page + L::kKScale + tok * L::kGroups + t * (kWords / 2);
                    if constexpr (kWords == 4) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src);
                        kw[m][half][0] = x.x; kw[m][half][1] = x.y; kw[m][half][2] = x.z; kw[m][half][3] = x.w;
                        const uint32_t two = e4m3_to_f16(*reinterpret_cast<const uint16_t*>(sc));
                        ks[m][half][0] = __byte_perm(two, 0, 0x1010);
                        ks[m][half][1] = __byte_perm(two, 0, 0x3232);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        kw[m][half][0] = x.x; kw[m][half][1] = x.y;
                        ks[m][half][0] = e4m3_to_f16((uint32_t)*sc * 0x101u);
                    }
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) s[m][nt][2 * half] = s[m][nt][2 * half + 1] = 0.f;
                }
#pragma unroll
            for (int w = 0; w < kWords; ++w)
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        e2m1_to_f16(kw[m][half][w], a[half]);
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
            // Keys past a row's limit (and scores of what lies there) do not count.
            const bool masked = key0 + kPieceTokens > min_lim;
            if (masked) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int key = key0 + 16 * m + 8 * (c >> 1) + k_row;
                            if (key >= rs_lim[nt][c & 1]) s[m][nt][c] = -INFINITY;
                        }
            }
            // Online softmax; P^T as fp16 fragments.
            uint32_t pf[kTiles][kNT][2];
            float alpha[kNT][2];
            bool rescale = false;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                float mx[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    mx[c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
                    for (int m = 1; m < kTiles; ++m) mx[c] = fmaxf(mx[c], fmaxf(s[m][nt][c], s[m][nt][c + 2]));
                }
#pragma unroll
                for (int x = 4; x < 32; x *= 2)
#pragma unroll
                    for (int c = 0; c < 2; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], x));
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    // (No branch: the exponential of a step that needs none costs less than one.)
                    const float top = mx[c] * rs_scale[nt][c];
                    const bool jump = top > rs_m[nt][c] + (kCacheHeadroom + kCacheRescale);
                    const float next = jump ? top - kCacheHeadroom : rs_m[nt][c];
                    alpha[nt][c] = jump ? ex2_approx(rs_m[nt][c] - next) : 1.f;  // (0 from a reference of -infinity)
                    rs_m[nt][c] = next;
                    rs_l[nt][c] *= alpha[nt][c];
                    rescale |= jump;
                    const float mb = rs_m[nt][c] == -INFINITY ? 0.f : rs_m[nt][c];
                    float sum = 0.f;
#pragma unroll
                    for (int m = 0; m < kTiles; ++m)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float& x = s[m][nt][c + 2 * half];
                            x = ex2_approx(fmaf(x, rs_scale[nt][c], -mb));
                            sum += x;
                        }
                    rs_l[nt][c] += sum;
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
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
                const int tok[4] = {16 * m + v_row0, 16 * m + v_row1, 16 * m + 8 + v_row0, 16 * m + 8 + v_row1};
                uint32_t vw[4][kChan / 8], sc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned char* src = page + L::kV + (tok0 + tok[i]) * L::kRow + g * (kChan / 2);
                    if constexpr (kChan == 16) {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        vw[i][0] = x.x; vw[i][1] = x.y;
                    } else {
                        vw[i][0] = *reinterpret_cast<const uint32_t*>(src);
                    }
                    sc[i] = page[L::kVScale + (tok0 + tok[i]) * L::kGroups + g * kChan / 16];
                }
                if (masked) {  // slots past the length hold anything
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (key0 + tok[i] >= at.len.kv) sc[i] = 0u;
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
            if (page_end) {
                ++j;
                __syncwarp();
                ask_next();
            }
        }
        if (!ok) break;

        // ----------------------------------------------- leave the state
        const int R_tile = min(State::kRows, R - row0);
        if (!none) {
            const int begun = first_warp == warp;
            State* st = j == asked
                            ? reinterpret_cast<State*>(sm.page[warp][0])
                            : static_cast<State*>(p.scratch) + ((size_t)blockIdx.x * kWarps + warp) * 2 + begun;
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float l = rs_l[nt][c];
                    l += __shfl_xor_sync(0xffffffffu, l, 4);
                    l += __shfl_xor_sync(0xffffffffu, l, 8);
                    l += __shfl_xor_sync(0xffffffffu, l, 16);
                    const int r = nt * 8 + 2 * t + c;
                    if (g == 0) st->ml[r] = make_float2(rs_m[nt][c], l);
                    float4* dst = reinterpret_cast<float4*>(&st->o[r][g * kChan]);
#pragma unroll
                    for (int i = 0; i < kChan / 4; ++i)
                        dst[i] = make_float4(o[2 * i][nt][c], o[2 * i][nt][c + 2], o[2 * i + 1][nt][c],
                                             o[2 * i + 1][nt][c + 2]);
                }
            __threadfence_block();
            __syncwarp();
            if (lane == 0) {
                sm.state[warp][begun] = st;
                __threadfence_block();
                *reinterpret_cast<volatile unsigned int*>(&sm.left[warp][begun]) = unit;
            }
            __threadfence_block();
            __syncwarp();
            // All states are there for the last warp at least; one joins them.
            bool there = true;
            if (lane < present)
                there = *reinterpret_cast<volatile unsigned int*>(&sm.left[first_warp + lane][lane == 0]) == unit;
            if (!__all_sync(0xffffffffu, there)) continue;
            unsigned int taken = 0;
            if (lane == 0) taken = atomicMax(&sm.claimed[first_warp], unit);  // units count up
            if (__shfl_sync(0xffffffffu, taken, 0) >= unit) continue;
            __threadfence_block();
        }
        // ------------------------- the last warp: join the states, write the rows
        // (in the order of their pieces: the sums do not depend on which came last).
        constexpr int kPer = kD / 32;  // channels of a lane
        const float v_head = p.c.kv_scale ? p.c.kv_scale[p.c.kv_heads + at.h] : 1.f;
        const int n = none ? 0 : present;
        // (Short loops: code that runs once a unit costs more to fetch than to run.)
        constexpr int kRows = State::kRows, kLanes = 32 / kRows;  // lanes of a row
        constexpr int kTurns = (kWarps + kLanes - 1) / kLanes;
        const int r = lane / kLanes, q = lane % kLanes;  // states q, q + kLanes, ... of row r
        float a[kTurns], row_l[kTurns], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            const int i = k * kLanes + q;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (i < n) ml = sm.state[first_warp + i][i == 0]->ml[r];
            a[k] = ml.x;
            row_l[k] = ml.y;
            m = fmaxf(m, ml.x);
        }
#pragma unroll
        for (int x = 1; x < kLanes; x *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            a[k] = a[k] == -INFINITY ? 0.f : ex2_approx(a[k] - m);
            l = fmaf(a[k], row_l[k], l);
        }
#pragma unroll
        for (int x = 1; x < kLanes; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
        // Where row r goes, and its factor.
        const int qi = (row0 + r) / p.group, head = at.h * p.group + (row0 + r) - qi * p.group;
        const bool live = row0 + r < live_rows && l != 0.f, whole = at.whole;
        long long dst = ((long long)at.b * p.Sq + qi) * p.heads + head;
        float factor = live ? v_head / l : 0.f;
        if (!whole) {
            dst = (2 * (long long)blockIdx.x + (at.first > 0 ? 0 : 1)) * p.tile + r;
            factor = 1.f;
        }
        if (q == 0 && r < R_tile) {
            if (!whole)
                p.part_ml[dst] = make_float2(m, l);
            else if (p.lse)
                p.lse[((size_t)at.b * p.heads + head) * p.Sq + qi] =
                    live ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
        float sum[kRows][kPer];
#pragma unroll
        for (int x = 0; x < kRows; ++x)
#pragma unroll
            for (int c = 0; c < kPer; ++c) sum[x][c] = 0.f;
#pragma unroll
        for (int k = 0; k < kTurns; ++k)
#pragma unroll 1
            for (int i = k * kLanes; i < min(n, (k + 1) * kLanes); ++i) {
                const State* si = sm.state[first_warp + i][i == 0];
                float y[kRows][kPer];
#pragma unroll
                for (int x = 0; x < kRows; ++x) {
                    if constexpr (kPer == 4)
                        *reinterpret_cast<float4*>(y[x]) = *reinterpret_cast<const float4*>(&si->o[x][lane * kPer]);
                    else
                        *reinterpret_cast<float2*>(y[x]) = *reinterpret_cast<const float2*>(&si->o[x][lane * kPer]);
                }
#pragma unroll
                for (int x = 0; x < kRows; ++x) {
                    const float ai = __shfl_sync(0xffffffffu, a[k], x * kLanes + i - k * kLanes);
#pragma unroll
                    for (int c = 0; c < kPer; ++c) sum[x][c] = fmaf(ai, y[x][c], sum[x][c]);
                }
            }
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
            if (x >= R_tile) break;
            const float f = __shfl_sync(0xffffffffu, factor, x * kLanes);
            const bool any = __shfl_sync(0xffffffffu, (int)live, x * kLanes) != 0;
            const long long to = __shfl_sync(0xffffffffu, dst, x * kLanes);
            if (whole) {
                uint32_t w[kPer / 2];
#pragma unroll
                for (int c = 0; c < kPer; c += 2) w[c / 2] = any ? pack_bf16x2(sum[x][c] * f, sum[x][c + 1] * f) : 0u;
                uint32_t* out = reinterpret_cast<uint32_t*>(p.out + to * (kD / 8)) + lane * (kPer / 2);
                if constexpr (kPer == 4)
                    *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
                else
                    *out = w[0];
            } else {
                float* out = p.part_o + to * kD + lane * kPer;
                if constexpr (kPer == 4)
                    *reinterpret_cast<float4*>(out) = make_float4(sum[x][0], sum[x][1], sum[x][2], sum[x][3]);
                else
                    *reinterpret_cast<float2*>(out) = make_float2(sum[x][0], sum[x][1]);
            }
        }
    }
    // Copies still in flight (a walk that an abort cut short) land before the
    // CTA's shared memory is released.
    if (lane == 0)
        for (; j < asked; ++j)
            mbar_wait_drain_1(smem_u32(&sm.full[warp][j % kOwn]), (j / kOwn) & 1, p.c.err, kCacheWaitNs);
}

// Joins the parts of the units that were cut.  Block (x, y) looks at the cut
// before CTA y + 1's part; if it is the unit's first, it joins the rows x,
// x + gridDim.x, ...:
//   m = max m_i, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i
// The warps take the parts in turn and ask for eight at a time: a unit cut
// into many parts is a matter of latency.
constexpr int kJoinWarps = 4;

template <int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) combine_kernel(AttnParams p) {
    __shared__ float s_o[kJoinWarps][kD];
    __shared__ float2 s_ml[kJoinWarps];
    early();
    begin_work();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.y;  // the CTA that begins the unit, if this is its first cut
    // Lane i: where CTA c0 + i's part begins (b < 0: not inside a unit).
    int4 x = make_int4(-1, 0, 0, 0);
    if (c0 + lane < p.grid) x = p.places[c0 + lane];
    const int4 u = make_int4(__shfl_sync(0xffffffffu, x.x, 1), __shfl_sync(0xffffffffu, x.y, 1),
                             __shfl_sync(0xffffffffu, x.z, 1), 0);
    unsigned same = __ballot_sync(0xffffffffu, x.x == u.x && x.y == u.y && x.z == u.z);
    if (u.x < 0 || (same & 1u)) return;
    int c1 = c0 + __ffs(~(same >> 1)) - 1;  // the unit's last CTA
    for (int c = c0 + 32; same >> 31 && c < p.grid; c += 32) {  // (more than 31 parts)
        x = make_int4(-1, 0, 0, 0);
        if (c + lane < p.grid) x = p.places[c + lane];
        const unsigned more = __ballot_sync(0xffffffffu, x.x == u.x && x.y == u.y && x.z == u.z);
        c1 = c - 1 + (more == 0xffffffffu ? 32 : __ffs(~more) - 1);
        if (more != 0xffffffffu) break;
    }
#pragma unroll 1
    for (int r = blockIdx.x; r < p.tile; r += gridDim.x) {
        const int row = u.z * p.tile + r;
        if (row >= p.Sq * p.group) return;
        // Slot 1 of the unit's first CTA, slot 0 of the others.
        constexpr int kPer = kD / 32, kAhead = 8;
        float m = -INFINITY, l = 0.f, sum[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[i] = 0.f;
#pragma unroll 1
        for (int c = c0 + warp; c <= c1; c += kJoinWarps * kAhead) {
            float2 ml[kAhead];
            float o[kAhead][kPer];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int ck = c + k * kJoinWarps;
                const size_t at = (2 * (size_t)ck + (ck == c0)) * p.tile + r;
                ml[k] = make_float2(-INFINITY, 0.f);
                if (ck > c1) continue;
                ml[k] = p.part_ml[at];
                const float* src = p.part_o + at * kD + lane * kPer;
                if constexpr (kPer == 4)
                    *reinterpret_cast<float4*>(o[k]) = *reinterpret_cast<const float4*>(src);
                else
                    *reinterpret_cast<float2*>(o[k]) = *reinterpret_cast<const float2*>(src);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) top = fmaxf(top, ml[k].x);
            // (Parts without a key leave the reference at -infinity, and so does a row of NaN,
            // whose sum is NaN: only an empty part is passed over.)
            const float keep = m == top ? 1.f : ex2_approx(m - top);
            m = top;
            l *= keep;
#pragma unroll
            for (int i = 0; i < kPer; ++i) sum[i] *= keep;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (ml[k].x == -INFINITY && ml[k].y == 0.f) continue;
                const float a = ml[k].x == -INFINITY ? 0.f : ex2_approx(ml[k].x - m);
                l = fmaf(a, ml[k].y, l);
#pragma unroll
                for (int i = 0; i < kPer; ++i) sum[i] = fmaf(a, o[k][i], sum[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_o[warp][lane * kPer + i] = sum[i];
        if (lane == 0) s_ml[warp] = make_float2(m, l);
        __syncthreads();
        if (threadIdx.x < kD / 2) {
            m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_ml[w].x);
            l = 0.f;
            float2 y = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kJoinWarps; ++w) {
                const float2 ml = s_ml[w];
                const float a = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m);
                const float2 z = *reinterpret_cast<const float2*>(&s_o[w][2 * threadIdx.x]);
                l = fmaf(a, ml.y, l);
                y.x = fmaf(a, z.x, y.x);
                y.y = fmaf(a, z.y, y.y);
            }
            const int qi = row / p.group, head = u.y * p.group + row - qi * p.group;
            const bool live = row < seq_lens(p, u.x).q * p.group && l != 0.f;
            const float inv = live ? (p.c.kv_scale ? p.c.kv_scale[p.c.kv_heads + u.y] : 1.f) / l : 0.f;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (((size_t)u.x * p.Sq + qi) * p.heads + head) * (kD / 8));
            dst[threadIdx.x] = live ? pack_bf16x2(y.x * inv, y.y * inv) : 0u;
            if (threadIdx.x == 0 && p.lse)
                p.lse[((size_t)u.x * p.heads + head) * p.Sq + qi] =
                    live ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
        __syncthreads();
    }
}

constexpr int kTokenWarps = 12;  // at most: states in the workspace

template <int kD, int kNT, int kWarps, int kOwn>
cudaError_t launch_token(const AttnParams& p, cudaStream_t stream) {
    constexpr int smem = (int)sizeof(TokenSmem<kD, kNT, kWarps, kOwn>);
    static_assert(smem <= 232448, "shared memory of the token kernel");
    static_assert(kOwn >= 2 && kOwn <= 32, "a piece to come beside the present one");
    auto kernel = token_kernel<kD, kNT, kWarps, kOwn>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
    static_assert(kWarps <= kTokenWarps && kWarps <= 16, "states in the workspace");
    return launch_early(kernel, dim3((unsigned)p.grid), kWarps * 32, smem, stream, p);
}

// How the line is cut, in pages, with what was measured:
//  * unit_cost, what starting and ending a unit takes.  A ragged batch of
//    prompts takes 358 us with 6, 329 with 20, 315 with 30, 334 with 45:
//    chunk_kernel drains its pipeline at a unit's end.  token_kernel's warps go
//    on: 103.9 us with 1, 102.2 with 2, 102.5 with 4.
//  * min_part.  One token on 2000 to 4000 cached ones: 11.8 us with parts of
//    2 pages, 13.4 with 6, 14.5 with 12; chunks gain nothing below 8.
//  * Walks of up to `whole` pages are not cut at all (and need no joining
//    kernel).  Times in us, cut and whole, keys of 8 kv heads of 128:
//      pages                    8            16           32           48
//      8 rows                   10.2  9.5    10.5 11.9    11.0 15.8    11.3 20.3
//      8 rows, 8 sequences      11.7 10.1    12.5 12.6    15.6 16.5    17.4 20.9
//      64 rows                  18.6 13.4    19.3 17.1    22.0 25.3    22.4 33.3
//      64 rows, 8 sequences     22.5 14.7    28.0 19.3    33.7 26.6    37.2 35.3
//      500 rows, 8 sequences    42.1 28.9    55.3 38.3    77.6 54.6    91.1 70.6
//    Whole wins up to 8 pages (token_kernel) and 16 (chunk_kernel) in all cases
//    measured, D = 64 and 40 kv heads too; beyond, it depends on how many units
//    there are.
constexpr int kTokenUnitCost = 2, kChunkUnitCost = 28, kIdleCost = 2;
constexpr int kTokenMinPart = 2, kChunkMinPart = 8;
constexpr int kTokenWhole = 8, kChunkWhole = 16;

// Rows of a unit: up to 16 rows a kv head go to token_kernel, more to chunk_kernel.
// Times in us for 8 kv heads, token_kernel in tiles of 8 | of 16 | chunk_kernel:
//   rows of a kv head                  8                  9..16        17..24       32..48
//   D = 128, 4 sequences of 300        9.4 | 10.9 | 12.2  11.5 | 12.2  13.7 | 12.3  13.7 | 12.6
//            1 of 32760               20.5 | 25.0 | 28.5  26.3 | 28.8  37.7 | 30.7  48.7 | 33.1
//            16 of 8000               41.2 | 56.1 | 85.7  59.3 | 87.6  98.8 | 89.5   139 | 92.9
//   D = 64,  4 of 300                  8.4 |  9.7 |  9.9  10.3 | 10.0  12.6 | 10.0  12.6 | 10.0
//            1 of 32760               15.2 | 18.4 | 24.4  19.4 | 25.0  27.7 | 26.4  33.9 | 29.4
//            16 of 8000               33.0 | 39.4 | 67.8  41.5 | 69.3  64.6 | 71.0  89.6 | 74.4
// (the larger number of rows of each column; D = 64 with 17 to 32 rows on long
// caches could go either way).
int tile_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 128; }

}  // namespace

size_t cache_attn_workspace_bytes(int D, int Sq, int group) {
    const int tile = tile_rows(Sq * group);
    const size_t row = (size_t)D * 4 + 8;
    return (size_t)kMaxGrid * 16 + (size_t)2 * kMaxGrid * tile * row +
           (tile >= 128 ? 0 : (size_t)kMaxGrid * kTokenWarps * 2 * tile * (row + 16));
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
    p.scratch = p.part_o + (size_t)2 * kMaxGrid * p.tile * D;
    p.scale_log2 = sm_scale * 1.4426950408889634f;
    p.unit_cost = p.tile >= 128 ? kChunkUnitCost : kTokenUnitCost;
    p.idle_cost = kIdleCost;
    p.min_part = p.tile >= 128 ? kChunkMinPart : kTokenMinPart;
    const int most = page_sel ? nsel : c.width;
    p.brief = c.B <= 32 && p.tiles == 1 &&
              (long long)c.B * c.kv_heads * ((long long)most + p.unit_cost) < (1LL << 31);
    p.whole = most <= (p.tile >= 128 ? kChunkWhole : kTokenWhole);
    cudaError_t e;
    if (p.tile >= 128)
        e = launch_chunk(p, D, stream);
    else if (D == 64)
        e = p.tile == 8 ? launch_token<64, 1, 12, 4>(p, stream) : launch_token<64, 2, 12, 4>(p, stream);
    else
        e = p.tile == 8 ? launch_token<128, 1, 12, 2>(p, stream) : launch_token<128, 2, 8, 3>(p, stream);
    if (e != cudaSuccess || p.whole) return e;
    if (p.grid < 2) return cudaSuccess;
    const dim3 grid((unsigned)std::min(p.tiles == 1 ? rows : p.tile, 16), (unsigned)(p.grid - 1));
    return launch_early(D == 64 ? combine_kernel<64> : combine_kernel<128>, grid, kJoinWarps * 32, 0, stream, p);
}

}  // namespace vsa
