// Shared pieces of the 4-bit paged cache: the page layout, conversions
// between its codes and fp16, and the split of attention work over a grid.
//
// A page holds 64 tokens of one kv head in 72 * D contiguous bytes:
//   K codes [64][D / 2] | V codes [64][D / 2] | K scales [64][D / 16] | V scales [64][D / 16]
// A code is e2m1 (sign, two exponent bits, one mantissa bit), low nibble =
// even channel; a scale is e4m3 and covers 16 channels.  code * scale has at
// most 2 + 4 significant bits and lies in [2^-10, 2688], so the product is
// exact in fp16 (and in bf16): the kernels multiply in fp16 without rounding.
// The fp32 head scale stays outside (it joins sm_scale and the epilogue).
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include <atomic>

#include "vsa_common.cuh"

namespace vsa {

constexpr int kPageTokens = 64;

// What every cache kernel knows of the cache (device pointers).
struct CacheView {
    unsigned char* pool;
    const int32_t* table;    // [B][width]
    const int32_t* kv_lens;  // [B]
    const float* kv_scale;   // [2][kv_heads], or null: 1
    unsigned int* err;
    int pages, kv_heads, B, width;
};

// Lets `kernel` use `smem` bytes; `done` (one for each kernel) remembers the
// devices, which saves small calls a driver call.
template <class K>
inline cudaError_t allow_smem(K kernel, int smem, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Registers a thread of `kernel` is launched with; `known` (one for each kernel)
// keeps the answer once there is one (0: none yet), and no failure.
template <class K>
inline cudaError_t launch_registers(K kernel, std::atomic<int>& known, int* regs) {
    *regs = known.load(std::memory_order_relaxed);
    if (*regs != 0) return cudaSuccess;
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    *regs = fa.numRegs;
    known.store(fa.numRegs, std::memory_order_relaxed);
    return cudaSuccess;
}

#if defined(__CUDACC__)

// The kernels of the cache calls, chunk_kernel apart, are launched while the
// kernel before them on the stream still runs (where that one allows it by
// early(), as they all do):
// blocks are set up as soon as an SM has room, and wait in begin_work() until
// the kernel before has ended and its writes can be seen.  Nothing is read
// from or written to global memory before that, and nothing is read as
// read-only data (the non-coherent loads): a kernel's life begins before its
// predecessor's last write, so what anything before it on the stream may have
// written is loaded as ordinary memory, which the wait orders.  A step is a
// chain of kernels of 3 to 20 us; one token on 300 takes 8.2 us a call so, 9.2
// without, a frame's append and a read 29.0 and 32.6.
template <class... P>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, P... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}
__device__ __forceinline__ void early() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void begin_work() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int kD>
struct PageLayout {
    static constexpr int kRow = kD / 2;     // code bytes of a token
    static constexpr int kGroups = kD / 16;  // scale bytes of a token
    static constexpr int kV = kPageTokens * kRow;
    static constexpr int kKScale = 2 * kPageTokens * kRow;
    static constexpr int kVScale = kKScale + kPageTokens * kGroups;
    static constexpr int kBytes = kVScale + kPageTokens * kGroups;
};
static_assert(PageLayout<128>::kBytes == 72 * 128 && PageLayout<64>::kBytes == 72 * 64, "page size");

// Tokens of sequence b in the cache; a length the page table cannot hold is
// cut to what it holds (and noted in the error word by the caller's choice).
__device__ __forceinline__ int cache_len(const CacheView& c, int b, bool note) {
    const int n = c.kv_lens[b];
    const long long cap = (long long)c.width * kPageTokens;
    if (n < 0 || n > cap) {
        if (note) atomicOr(c.err, VSA_DEVERR_INDEX);
        return n < 0 ? 0 : (int)cap;
    }
    return n;
}

// Four bytes of code pairs -> four fp16 pairs (byte j's low nibble in the low half).
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes (bits 0..15) -> fp16 pair.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(two));
    return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Power-of-two factor that brings a query row of largest magnitude `amax`
// into [2^14, 2^15), so that its bf16 values (8 significant bits) convert to
// fp16 (11, steps of 2^-24 at least) without rounding down to 2^-31 of the row's
// largest; what is smaller is off by 2^-25 at most, 2^-39 of the largest (rows
// below 2^-106 are scaled by 2^120 only: off by 2^-145).  1 for a row of zeros
// or with an infinity.  The inverse goes into the row's softmax scale.
__device__ __forceinline__ int q_exponent(float amax) {
    if (!(amax > 0.f) || amax > 3.4e38f) return 0;
    const int e = (int)((__float_as_uint(amax) >> 23) & 0xFFu) - 127;  // below the normals: -127
    return min(14 - e, 120);
}
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 126

// What a row's logits are multiplied with (log2 units): a normal number whatever
// its factors are, for keys that a row does not see have a logit of -infinity,
// and -infinity * 0 is NaN.  (A logit is below 2^34 before: one that small a
// factor brings below 2^-92, where it is 0 to the exponential as it should be.)
__device__ __forceinline__ float logit_scale(float scale_log2, float k_head, int e) {
    const float f = scale_log2 * k_head * pow2i(-e);
    return f < 1.17549435e-38f ? 1.17549435e-38f : f;  // (NaN stays NaN)
}

constexpr uint64_t kCacheWaitNs = 2000000000ull;  // limit of the kernels' waits: 2 s

// Bounded wait of a whole warp for a phase of a barrier: false if *abort was
// raised, or if limit_ns have passed since the 64th look (then it raises *abort
// and sets the timeout bit).  Between looks the warp sleeps kSleep ns: waiting
// roles share their scheduler with working ones.
template <int kSleep>
__device__ __forceinline__ bool cache_wait(uint32_t bar, uint32_t parity, volatile int* abort, unsigned int* err,
                                           uint64_t limit_ns = kCacheWaitNs) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (kSleep > 0) __nanosleep(kSleep);
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (i % 64 != 0) continue;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *abort != 0)) return false;
        if (__any_sync(0xffffffffu, now - t0 > limit_ns)) {
            *abort = 1;
            if ((threadIdx.x & 31) == 0) atomicOr(err, VSA_DEVERR_TIMEOUT);
            return false;
        }
    }
}
constexpr int kSleepShort = 20, kSleepLong = 100;

// Untiled bulk copy into shared memory (16-byte aligned, a multiple of 16 bytes), completing on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// ------------------------------------------------- split of attention work
// A unit is (sequence b, kv head, tile of `tile` query rows); row r is head
// kv_head * group + r % group of query r / group.  Units are laid end to end
// in the order (b, kv head, tile), each as long as the pages it walks plus
// unit_cost (what starting and ending a unit costs, in pages; idle_cost for a
// unit that walks none and is written as zeros), and the line
// is cut into equal parts, one for each CTA: batches of ragged lengths and
// single long sequences fill the grid alike.  A unit that lies in one part
// is written by its CTA; the parts of a cut unit go to the workspace (two
// slots a CTA: slot 0 for a unit begun by an earlier CTA, slot 1 for one it
// begins itself and does not finish) and are joined by combine_kernel, a block
// for each cut: there are fewer cuts than CTAs, whatever the batch.
struct AttnParams {
    CacheView c;
    const int32_t* q_lens;    // [B], or null: Sq
    const int32_t* page_sel;  // [B][kv_heads][nsel], or null
    const uint4* q;           // bf16 [B][Sq][heads][D]
    uint4* out;
    float* lse;               // [B][heads][Sq], or null
    float* part_o;            // [2 * grid][tile][D]
    float2* part_ml;          // [2 * grid][tile]: reference (log2 units), sum
    void* scratch;            // token_kernel: [grid][warps][2] states
    int4* places;             // [grid]: where each CTA's part begins (b, h, t, page); b = -1: between units
    int Sq, heads, group, nsel, causal;
    int tile, tiles;          // rows of a unit; units of a (b, kv head)
    int grid;                 // CTAs of the attention kernel
    int unit_cost, idle_cost;  // of a unit beside its pages, of one without pages
    int min_part;             // pages of a part at least
    int brief;                // up to 32 sequences, one tile each, a line shorter than 2^31
    int whole;                // units are not cut: a unit belongs to the CTA that holds its first page
    float scale_log2;         // sm_scale * log2(e)
};

struct SeqLens {
    int kv, q;
};

__device__ __forceinline__ SeqLens seq_lens(const AttnParams& p, int b, bool note = false) {
    SeqLens s;
    const int q = p.q_lens ? p.q_lens[b] : p.Sq;  // (asked for first: both loads are on their way at once)
    s.kv = cache_len(p.c, b, note);
    s.q = min(max(q, 0), p.Sq);
    return s;
}

// Pages that tile t of a sequence walks (0: nothing to attend).
__device__ __forceinline__ int tile_pages(const AttnParams& p, const SeqLens& s, int t) {
    if (p.tiles == 1) return s.q == 0 ? 0 : p.page_sel ? p.nsel : (s.kv + kPageTokens - 1) / kPageTokens;
    const int rows = s.q * p.group;
    const int first = t * p.tile;
    if (first >= rows) return 0;
    if (p.page_sel) return p.nsel;
    int lim = s.kv;
    if (p.causal) lim = min(lim, s.kv - s.q + (min(rows, first + p.tile) - 1) / p.group + 1);
    return lim > 0 ? (lim + kPageTokens - 1) / kPageTokens : 0;
}
__device__ __forceinline__ int tile_cost(const AttnParams& p, const SeqLens& s, int t) {
    const int n = tile_pages(p, s, t);
    return n > 0 ? n + p.unit_cost : p.idle_cost;
}
// sum of floor((k t + c) / g) for t < n (c >= 0, g > 0), in k terms without steps:
// floor(k z) is the sum of floor(z + j / k) over j < k (Hermite's identity), so
// with z = (t + c / k) / g every term is the sum of floor((t + c_j) / g) over j,
// c_j = floor((c + j g) / k), and x / g sums in closed form over whole runs of g.
// (Loops that stay loops: unrolled, the same sums make a ragged batch of prompts
// take 312 us instead of 291, for code that a CTA runs once or twice.)
static __host__ __device__ __noinline__ long long steps_sum(int n, int k, long long c, int g) {
    unsigned long long sum = 0;  // (terms may pass 2^64 for the longest caches, their differences do not)
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        const long long c_j = (c + j * g) / k;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {  // the terms below n + c_j, then less those below c_j
            const long long x = e ? c_j : n + c_j;
            const long long runs = x < (1LL << 31) ? (long long)((unsigned)x / (unsigned)g) : x / g;
            const unsigned long long below =
                (unsigned long long)g * (runs * (runs - 1) / 2) + (unsigned long long)(runs * (x - runs * g));
            sum += e ? 0ull - below : below;
        }
    }
    return (long long)sum;
}
// Cost of one kv head of a sequence: the sum of its tiles.
__device__ __forceinline__ long long head_cost(const AttnParams& p, const SeqLens& s) {
    if (p.tiles == 1) return tile_cost(p, s, 0);
    const int live = min(p.tiles, (s.q * p.group + p.tile - 1) / p.tile);
    const auto sum = [&](int with, long long pages) {  // tiles with pages, pages of all
        return pages + (long long)with * p.unit_cost + (long long)(p.tiles - with) * p.idle_cost;
    };
    if (!p.causal || p.page_sel || live <= 1) {
        const int n = tile_pages(p, s, 0);
        return sum(n > 0 ? live : 0, (long long)live * n);
    }
    // Tile t but the last sees keys up to its last row's place,
    //   pages = ceil((kv - q + 1 + floor(((t + 1) tile - 1) / group)) / 64)
    //         = floor((tile t + tile - 1 + group (kv - q + 64)) / (64 group)),
    // from the first tile with a key on (a sequence may be shorter than its queries).
    // A tile of several is 128 rows, a whole number of 64 (see tile_rows).
    const long long lead = (long long)p.group * (s.kv - s.q + kPageTokens) + p.tile - 1, per = 64LL * p.group;
    long long none = 0;
    if (lead < per) none = min((long long)live - 1, (per - lead + p.tile - 1) / p.tile);
    const int end = tile_pages(p, s, live - 1);
    const long long pages =
        end + steps_sum(live - 1 - (int)none, p.tile / kPageTokens, (lead + none * p.tile) / kPageTokens, p.group);
    return sum(live - (int)none - (end == 0), pages);
}

// A place on the line: page `page` of unit (b, h, t) (from the unit's number of pages on: its end).
struct Place {
    int b, h, t, page;
};

// Where part `c` of `n` of a line of `total` begins (parts of equal length, the first total % n one longer).
__device__ __forceinline__ long long part_begin(long long total, int c, int n) {
    long long q, r;
    if (total < (1LL << 31)) {
        q = (int)total / n;
        r = (int)total - (int)q * n;
    } else {
        q = total / n;
        r = total - q * n;
    }
    return q * c + min((long long)c, r);
}

struct PlanScratch {
    long long warp_sum[32];
    long long within;  // where the part begins: sequence, position in it
    int b;
};

// Tile and page at position `at` of a kv head of sequence s (a whole warp calls it).
__device__ __forceinline__ void tile_at(const AttnParams& p, const SeqLens& s, long long at, Place& x) {
    x.t = 0;
    x.page = (int)at;
    if (p.tiles == 1) return;
    const int lane = threadIdx.x & 31;
    for (int t0 = 0; t0 < p.tiles; t0 += 32) {
        const int n = t0 + lane < p.tiles ? tile_cost(p, s, t0 + lane) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at < incl);
        if (past) {
            const int l = __ffs(past) - 1;
            x.t = t0 + l;
            x.page = (int)at - __shfl_sync(0xffffffffu, incl - n, l);
            return;
        }
        at -= __shfl_sync(0xffffffffu, incl, 31);
    }
}

__device__ __forceinline__ long long scan_warp(long long x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    return x;
}

// Parts of the line: one for each CTA, of min_part pages at least.
__device__ __forceinline__ int used_parts(const AttnParams& p, long long total) {
    const long long n = total < (1LL << 31) ? ((int)total + p.min_part - 1) / p.min_part : p.grid;
    return n < p.grid ? (int)n : p.grid;
}

// A CTA's walk along its part of the line, unit by unit.
struct Segment {
    int b, h, t;
    SeqLens len;
    int first, last;  // pages
    int length;       // on the line
    bool whole;       // the unit from end to end: its rows are written at once
};
struct Walk {
    Place at;
    SeqLens len;
    long long left;  // of the part

    // The start where calls are small: every warp by itself, lane b sequence b, 32 bits.
    __device__ bool begin_brief(const AttnParams& p) {
        const int lane = threadIdx.x & 31;
        SeqLens s = {0, 0};
        if (lane < p.c.B) s = seq_lens(p, lane, threadIdx.x < 32 && blockIdx.x == 0);
        const int hc = tile_cost(p, s, 0);
        const int mine = lane < p.c.B ? p.c.kv_heads * hc : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned total = (unsigned)__shfl_sync(0xffffffffu, incl, 31);
        const unsigned parts = (unsigned)used_parts(p, total), c = blockIdx.x;
        if (c >= parts) {
            if (threadIdx.x == 0) p.places[c] = make_int4(-1, 0, 0, 0);
            return false;
        }
        const unsigned q = total / parts, r = total - q * parts;
        const int from = (int)(q * c + min(c, r));
        left = q + (c < r ? 1 : 0);
        const int l = __ffs(__ballot_sync(0xffffffffu, from < incl)) - 1;
        at.b = l;
        len.kv = __shfl_sync(0xffffffffu, s.kv, l);
        len.q = __shfl_sync(0xffffffffu, s.q, l);
        const int within = from - __shfl_sync(0xffffffffu, incl - mine, l);
        const int cost = __shfl_sync(0xffffffffu, hc, l);
        at.h = (int)((unsigned)within / (unsigned)cost);
        at.t = 0;
        at.page = within - at.h * cost;
        return true;
    }
    // All threads of the block call it; false: nothing for this CTA.
    __device__ bool begin(const AttnParams& p, PlanScratch& sc) {
        if (!(p.brief ? begin_brief(p) : begin_any(p, sc))) return false;
        // A unit's end is its owner's, and so is the rest of a unit that is not cut.
        const bool cut = at.page > 0 && at.page < tile_pages(p, len, at.t) && !p.whole;
        if (threadIdx.x == 0)
            p.places[blockIdx.x] = cut ? make_int4(at.b, at.h, at.t, at.page) : make_int4(-1, 0, 0, 0);
        if (at.page > 0 && !cut) {
            const int rest = tile_cost(p, len, at.t) - at.page;
            left -= rest;
            at.page += rest;
        }
        return true;
    }
    __device__ bool begin_any(const AttnParams& p, PlanScratch& sc) {
        const int lane = threadIdx.x & 31;
        // Sequences [b0, b1) are this thread's: up to 32 of them are dealt to
        // the lanes of every warp, more to the threads of the block.
        const bool few = p.c.B <= 32;
        const int who = few ? lane : (int)threadIdx.x, n = few ? 32 : (int)blockDim.x;
        const int per = few ? 1 : (p.c.B + n - 1) / n;
        const int b0 = min(who * per, p.c.B), b1 = min(b0 + per, p.c.B);
        long long mine = 0;
        for (int b = b0; b < b1; ++b) mine += p.c.kv_heads * head_cost(p, seq_lens(p, b));
        long long incl = scan_warp(mine);
        long long total = __shfl_sync(0xffffffffu, incl, 31);
        if (!few) {
            if (lane == 0) sc.warp_sum[threadIdx.x >> 5] = total;
            __syncthreads();
            total = 0;
            long long base = 0;
            for (int w = 0; w < (int)blockDim.x / 32; ++w) {
                if (w < (int)threadIdx.x >> 5) base += sc.warp_sum[w];
                total += sc.warp_sum[w];
            }
            incl += base;
        }
        const int parts = used_parts(p, total);
        if ((int)blockIdx.x >= parts) {
            if (threadIdx.x == 0) p.places[blockIdx.x] = make_int4(-1, 0, 0, 0);
            return false;
        }
        const long long from = part_begin(total, blockIdx.x, parts);
        left = part_begin(total, blockIdx.x + 1, parts) - from;
        // The thread whose sequences hold `from` finds the sequence.
        long long within = from - (incl - mine);
        int b = -1;
        if (within >= 0 && within < mine) {
            for (b = b0;; ++b) {
                const long long cost = p.c.kv_heads * head_cost(p, seq_lens(p, b));
                if (within < cost) break;
                within -= cost;
            }
        }
        if (few) {
            const int l = __ffs(__ballot_sync(0xffffffffu, b >= 0)) - 1;
            b = __shfl_sync(0xffffffffu, b, l);
            within = __shfl_sync(0xffffffffu, within, l);
        } else {
            if (b >= 0) {
                sc.b = b;
                sc.within = within;
            }
            __syncthreads();
            b = sc.b;
            within = sc.within;
        }
        at.b = b;
        len = seq_lens(p, b, threadIdx.x == 0);
        const long long hc = head_cost(p, len);
        at.h = within < (1LL << 31) ? (int)within / (int)min(hc, 0x7FFFFFFFLL) : (int)(within / hc);
        tile_at(p, len, within - at.h * hc, at);
        return true;
    }
    __device__ bool next(const AttnParams& p, Segment& s) {
        if (left <= 0) return false;
        int cost = tile_cost(p, len, at.t);
        if (at.page >= cost) {  // the next unit
            at.page = 0;
            if (++at.t == p.tiles) {
                at.t = 0;
                if (++at.h == p.c.kv_heads) {
                    at.h = 0;
                    if (++at.b == p.c.B) return false;
                    len = seq_lens(p, at.b, threadIdx.x == 0);
                }
            }
            cost = tile_cost(p, len, at.t);
        }
        const int take = p.whole || cost - at.page < left ? cost - at.page : (int)left;
        const int n = tile_pages(p, len, at.t);
        s.b = at.b;
        s.h = at.h;
        s.t = at.t;
        s.len = len;
        s.first = min(at.page, n);
        s.last = min(at.page + take, n);
        s.length = take;
        s.whole = at.page == 0 && take >= n;
        left -= take;
        at.page += take;
        return true;
    }
};

// Looks up page `i` of a segment's walk: its page number within the sequence,
// and its place in the pool (-1: passed over).
__device__ __forceinline__ void look_up(const AttnParams& p, const Segment& s, int i, int& logical, int& id) {
    logical = p.page_sel ? p.page_sel[((size_t)s.b * p.c.kv_heads + s.h) * p.nsel + i] : i;
    id = -1;
    if (logical < 0 || logical >= (s.len.kv + kPageTokens - 1) / kPageTokens) return;
    id = p.c.table[(size_t)s.b * p.c.width + logical];
    if (id < 0 || id >= p.c.pages) {
        atomicOr(p.c.err, VSA_DEVERR_INDEX);
        id = -1;
    }
}

constexpr int kMaxGrid = 160;                     // CTAs of an attention launch: one for each SM (152 on GB300)
// The reference that a row's weights are taken against, 2^(logit - reference),
// starts kCacheHeadroom (log2 units) below the row's maximum, and moves when the
// maximum has grown by more than kCacheRescale.  Weights then reach 2^15, inside
// fp16, and what fp16 cannot hold at the other end (below 2^-25) is under 2^-32
// of the row's largest; against the maximum itself it would be 2^-25, and many
// such weights on a long cache would be missing from the output, not from the sum.
constexpr float kCacheHeadroom = 7.0f, kCacheRescale = 8.0f;

// cache_chunk.cu
cudaError_t launch_chunk(const AttnParams& p, int D, cudaStream_t stream);

#endif  // __CUDACC__

}  // namespace vsa
