// Eviction from the 4-bit paged cache: of a sequence's n tokens each kv head keeps
// the first few, the most recent, and of those between the ones with the largest
// weights (those that cache_weigh sums, or any others).
//
// choose_kernel writes the places kept, ascending: the k-th largest weight T of
// the middle is found digit by digit from the top (11, 11 and 10 bits of the
// weights' bit patterns, put in their order), every place above T is kept and
// of those at T the lowest.  A block takes a (sequence, kv head), or a cluster of up
// to 8, each a stretch of its places: keys go to shared memory once, histograms are
// summed over the cluster by distributed shared memory (all blocks form the same
// sums, one barrier a digit).  Counting is in integers: the same places in every run.
// 40 rows of 32760 take 19 us for 5 MB from a cold cache (GB300): load, counting (0.58
// instructions a scheduler and cycle), barriers and the ordered list follow one another.
//
// move_kernel and move_within_kernel bring the kept tokens' codes, scales and
// weights to the places 0, 1, ...: 9/8 D + 4 bytes a token and head each way,
// by sectors of 32 bytes, of which a token's scales use 8, and larger fetches: a move
// of every fourth token reads twice the bytes it keeps (8190 of 32760 tokens, 40 heads
// of 128: 96 MB read, 24 us from a cold cache, 4.4 TB/s; 65% of the copy rate).  To other pages a
// block takes a page of 64 places.  Within the sequence's own pages a cluster takes
// a (sequence, kv head) and goes along the places in order: kept[j] >= j and
// ascends, so once all its blocks have read the places of a turn, no place that the
// turn writes is read again.  evict_kernel is choice and move in one, for short rows
// that keep up to 256 tokens.
#include <algorithm>

#include "move.cuh"

namespace vsa {

namespace {

constexpr int kMaxCluster = 8;
constexpr int kDigits = 3;
constexpr int kBins = 2048;
constexpr int kCopies = 4;            // of a histogram: neighbouring lanes add to different ones
constexpr int kHeldKeys = 40 * 1024;  // keys of a block's stretch that go to shared memory

struct EvictParams {
    CacheView c;
    const int32_t* to_table;  // [B][to_width], or null: the tokens stay in their pages
    const float* weights;     // [B][kv_heads][64 * width]
    float* moved;             // [B][kv_heads][64 * to_width] (in place: weights)
    int32_t* kept;            // [B][kv_heads][budget]
    int32_t* lens;            // [B]
    int budget, first, recent, to_width;
    int keys;                 // of shared memory, a block
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The words at `p`, a shared address of this block, in block `rank` of the cluster.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    return at;
}
__device__ __forceinline__ uint32_t load_from_rank(const void* p, uint32_t rank) {
    uint32_t x;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at_rank(p, rank)) : "memory");
    return x;
}
__device__ __forceinline__ uint2 load2_from_rank(const void* p, uint32_t rank) {
    uint2 x;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at_rank(p, rank)) : "memory");
    return x;
}
__device__ __forceinline__ unsigned scan_warp32(unsigned x) {  // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    return x;
}

// Bit patterns in the order of the numbers: NaN below all, -0 with 0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct ChooseSmem {
    unsigned int hist[kCopies][kBins];
    alignas(16) unsigned int total[kDigits][kBins];  // of this block, for the others of the cluster
    unsigned int warp_sum[32];
    unsigned int counts[2][32];  // above T, at T: of a warp's stretch
    unsigned int totals[2];                // of the block
    unsigned int found, before, there, unused[3];
};

extern __shared__ __align__(16) unsigned char choose_smem[];

template <int kChooseThreads, bool kClusters>
__device__ __forceinline__ void choose(const EvictParams& p) {
    constexpr int kChooseWarps = kChooseThreads / 32;
    ChooseSmem& sm = *reinterpret_cast<ChooseSmem*>(choose_smem);
    uint32_t* keys = reinterpret_cast<uint32_t*>(choose_smem + sizeof(ChooseSmem));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blocks = kClusters ? (int)cluster_size() : 1, rank = kClusters ? (int)cluster_rank() : 0;
    const int row = blockIdx.x / blocks;  // of B * kv_heads
    const int b = row / p.c.kv_heads, h = row - b * p.c.kv_heads;
    const int n = cache_len(p.c, b, h == 0 && rank == 0 && threadIdx.x == 0);
    int32_t* kept = p.kept + (size_t)row * p.budget;
    const int me = rank * kChooseThreads + threadIdx.x, all = blocks * kChooseThreads;
    if (h == 0 && me == 0) p.lens[b] = min(n, p.budget);
    if (n <= p.budget) {  // nothing to choose
        for (int j = me; j < p.budget; j += all) kept[j] = j < n ? j : -1;
        return;
    }
    for (int j = me; j < p.first; j += all) kept[j] = j;
    for (int j = me; j < p.recent; j += all) kept[p.budget - p.recent + j] = n - p.recent + j;
    const int want = p.budget - p.first - p.recent;
    if (want == 0) return;
    // This block's stretch of the middle, in whole warps' worth.
    const int middle = n - p.recent - p.first;
    const long long per = (long long)((middle - 1) / blocks / 128 + 1) * 128;
    const int begin = (int)min((long long)middle, rank * per), size = (int)min((long long)middle, begin + per) - begin;
    const float* w = p.weights + (size_t)row * p.c.width * kPageTokens + p.first + begin;
    const bool held = size <= p.keys;
    // Keys i .. i + 3 (i a multiple of 4; those from `size` on are anything).
    auto keys_at = [&](int i) {
        if (held) return *reinterpret_cast<const uint4*>(&keys[i]);
        uint4 k;
        k.x = order_key(w[i]);
        k.y = i + 1 < size ? order_key(w[i + 1]) : 0u;
        k.z = i + 2 < size ? order_key(w[i + 2]) : 0u;
        k.w = i + 3 < size ? order_key(w[i + 3]) : 0u;
        return k;
    };
    if (held) {
        constexpr int kAhead = 16;
        for (int i0 = threadIdx.x; i0 < size; i0 += kAhead * kChooseThreads) {
            float x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) x[k] = i0 + k * kChooseThreads < size ? w[i0 + k * kChooseThreads] : 0.f;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i0 + k * kChooseThreads < size) keys[i0 + k * kChooseThreads] = order_key(x[k]);
        }
    }
    // The digits of T; `left` of the places with T's digits so far are still to be found.
    uint32_t top = 0u, mask = 0u;
    unsigned left = (unsigned)want;
    if (threadIdx.x == 0) sm.found = sm.before = sm.there = 0u;
#pragma unroll 1
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = d == 2 ? 1024 : 2048;
        for (int i = threadIdx.x; i < kCopies * kBins / 4; i += kChooseThreads)
            reinterpret_cast<uint4*>(sm.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        unsigned* hist = sm.hist[lane % kCopies];
        for (int i = 4 * threadIdx.x; i < size; i += 4 * kChooseThreads) {
            const uint4 k4 = keys_at(i);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < size && (k[j] & mask) == top) atomicAdd(&hist[(k[j] >> shift) & (bins - 1)], 1u);
        }
        __syncthreads();
        // Thread t: the kPer bins from x on, x = bins - kPer (t + 1): from the top down.
        constexpr int kPer = kBins / kChooseThreads;
        const int x = bins - kPer * ((int)threadIdx.x + 1);
        unsigned bin[kPer], sum = 0u;
#pragma unroll
        for (int j = 0; j < kPer; j += 2) {
            uint2 y = make_uint2(0u, 0u);
            if (x >= 0) {
#pragma unroll
                for (int k = 0; k < kCopies; ++k) {
                    const uint2 z = *reinterpret_cast<const uint2*>(&sm.hist[k][x + j]);
                    y.x += z.x;
                    y.y += z.y;
                }
                if (blocks > 1) *reinterpret_cast<uint2*>(&sm.total[d][x + j]) = y;
            }
            bin[j] = y.x;
            bin[j + 1] = y.y;
        }
        if (blocks > 1) {  // sums over the cluster
            cluster_arrive();
            cluster_wait();
            if (x >= 0) {
#pragma unroll
                for (int j = 0; j < kPer; j += 2) {
                    uint2 y = make_uint2(0u, 0u);
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        if (r >= blocks) break;
                        const uint2 z = load2_from_rank(&sm.total[d][x + j], (uint32_t)r);
                        y.x += z.x;
                        y.y += z.y;
                    }
                    bin[j] = y.x;
                    bin[j + 1] = y.y;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += bin[j];
        const unsigned incl = scan_warp32(sum);
        if (lane == 31) sm.warp_sum[warp] = incl;
        __syncthreads();
        const unsigned of_warp = lane < kChooseWarps ? sm.warp_sum[lane] : 0u;
        const unsigned base = scan_warp32(of_warp) - of_warp;
        unsigned before = __shfl_sync(0xffffffffu, base, warp) + incl - sum;
        if (before < left && before + sum >= left) {
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j) {
                if (before < left && before + bin[j] >= left) {
                    sm.found = (unsigned)(x + j);
                    sm.before = before;
                    sm.there = bin[j];
                }
                before += bin[j];
            }
        }
        __syncthreads();
        top |= sm.found << shift;
        mask |= (unsigned)(bins - 1) << shift;
        left -= sm.before;
        if (sm.there == left) break;  // all of them are kept: their other digits do not matter
        __syncthreads();              // (the next digit writes what was read here)
    }
    // `left` of the places at T are kept, the lowest.  (All of them as a rule: then every
    // key from T on is one, and only those are counted.)  Where each warp's kept places go:
    const bool ties = sm.there != left;  // (T is known to its last bit then)
    const int part = ((size - 1) / kChooseWarps / 128 + 1) * 128;  // of a warp (size > 0 or nothing to do)
    const int from = min(size, warp * part), to = min(size, from + part);
    unsigned above = 0u, same = 0u;
    for (int i = from + 4 * lane; i < to; i += 128) {
        const uint4 k4 = keys_at(i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        if (!ties) {
#pragma unroll
            for (int j = 0; j < 4; ++j) above += i + j < to && k[j] >= top;
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            above += i + j < to && k[j] > top;
            same += i + j < to && k[j] == top;
        }
    }
    above = __reduce_add_sync(0xffffffffu, above);
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0) {
        sm.counts[0][warp] = above;
        sm.counts[1][warp] = same;
    }
    __syncthreads();
    const unsigned above_of = lane < kChooseWarps ? sm.counts[0][lane] : 0u, same_of = lane < kChooseWarps ? sm.counts[1][lane] : 0u;
    const unsigned above_to = scan_warp32(above_of), same_to = scan_warp32(same_of);
    above = __shfl_sync(0xffffffffu, above_to - above_of, warp);
    same = __shfl_sync(0xffffffffu, same_to - same_of, warp);
    if (blocks > 1) {
        if (threadIdx.x == 31) {
            sm.totals[0] = above_to;
            sm.totals[1] = same_to;
        }
        cluster_arrive();
        cluster_wait();
        for (int r = 0; r < rank; ++r) {
            above += load_from_rank(&sm.totals[0], (uint32_t)r);
            same += load_from_rank(&sm.totals[1], (uint32_t)r);
        }
        cluster_arrive();  // no block leaves while another reads from it
    }
    if (!ties) {
        unsigned j = above;  // (in the row's list whoever writes the weights meanwhile)
        for (int i0 = from; i0 < to; i0 += 128) {
            const int i = i0 + 4 * lane;
            bool keep[4] = {false, false, false, false};
            if (i < to) {
                const uint4 k = keys_at(i);
                keep[0] = k.x >= top;
                keep[1] = i + 1 < to && k.y >= top;
                keep[2] = i + 2 < to && k.z >= top;
                keep[3] = i + 3 < to && k.w >= top;
            }
            const unsigned mine = keep[0] + keep[1] + keep[2] + keep[3], incl = scan_warp32(mine);
            unsigned to_j = j + incl - mine;
            int32_t* list = kept + p.first + to_j;
            const int place = p.first + begin + i;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (keep[e] && to_j < (unsigned)want) *list = place + e;
                list += keep[e];
                to_j += keep[e];
            }
            j += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (blocks > 1) cluster_wait();
        return;
    }
    for (int i0 = from; i0 < to; i0 += 128) {
        const int i = i0 + 4 * lane;
        bool over[4] = {false, false, false, false}, at_t[4] = {false, false, false, false};
        if (i < to) {
            const uint4 k4 = keys_at(i);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                over[e] = i + e < to && k[e] > top;
                at_t[e] = i + e < to && k[e] == top;
            }
        }
        unsigned mine = 0u;  // above T in the low half, at T in the high one
#pragma unroll
        for (int e = 0; e < 4; ++e) mine += (over[e] ? 1u : 0u) + (at_t[e] ? 0x10000u : 0u);
        const unsigned incl = scan_warp32(mine);
        unsigned t = same + ((incl - mine) >> 16);  // at T before this lane's
        unsigned j = above + ((incl - mine) & 0xFFFFu) + min(t, left);
        int32_t* list = kept + p.first + j;
        const int place = p.first + begin + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool keep = over[e] || (at_t[e] && t < left);
            if (keep && j < (unsigned)want) *list = place + e;
            list += keep;
            j += keep;
            t += at_t[e];
        }
        const unsigned all_of_them = __shfl_sync(0xffffffffu, incl, 31);
        above += all_of_them & 0xFFFFu;
        same += all_of_them >> 16;
    }
    if (blocks > 1) cluster_wait();
}

template <int kChooseThreads>
__global__ void __launch_bounds__(kChooseThreads, 1) choose_kernel(EvictParams p) {
    early();
    begin_work();
    choose<kChooseThreads, true>(p);
}

// To other pages: block (x, h, b) fills places 64 x .. 64 x + 63.  (All the blocks an SM holds, 32
// registers a thread: what has to be waited for, one after the other, is most of a block's life.  40
// heads of 8190 from 32760 tokens with a read 77.0 us at 40 registers, 75.8 so.)
template <int kD>
__global__ void __launch_bounds__(kMoveThreads, 16) move_kernel(EvictParams p) {
    __shared__ int source[kPageTokens];
    early();
    begin_work();
    const int h = blockIdx.y, b = blockIdx.z, first = blockIdx.x * kPageTokens;
    const size_t row = (size_t)b * p.c.kv_heads + h;
    const int held = cache_len(p.c, b, false), n = min(held, p.budget), size = min(kPageTokens, n - first);
    if (threadIdx.x < kPageTokens) {
        const int t = threadIdx.x;
        int s = t < size ? p.kept[row * p.budget + first + t] : -1;
        if (s >= held) s = -1;
        source[t] = s;
        p.moved[row * p.to_width * kPageTokens + first + t] =
            s >= 0 ? p.weights[row * p.c.width * kPageTokens + s] : 0.f;
    }
    if (size <= 0) return;
    __syncthreads();
    MovedToken<kD> x[MovedToken<kD>::kTurns];
    take_tokens<kD>(p.c, p.c.table, p.c.width, b, h, source, size, threadIdx.x, x);
    put_tokens<kD>(p.c, p.to_table, p.to_width, b, h, first, size, threadIdx.x, x);
}

// Within the sequence's pages: a cluster goes along the row, 64 places a block and turn.
template <int kD>
__global__ void __launch_bounds__(kMoveThreads) move_within_kernel(EvictParams p) {
    __shared__ int source[2][kPageTokens];
    early();
    begin_work();
    const int blocks = (int)cluster_size(), rank = (int)cluster_rank();
    const size_t row = blockIdx.x / blocks;
    const int b = (int)(row / p.c.kv_heads), h = (int)(row - (size_t)b * p.c.kv_heads);
    const int n = cache_len(p.c, b, false);
    if (n <= p.budget) return;  // (the whole cluster)
    const int32_t* kept = p.kept + row * p.budget;
    float* w = p.moved + row * p.c.width * kPageTokens;
    MovedToken<kD> x[MovedToken<kD>::kTurns];
    float weight = 0.f;
    const int step = blocks * kPageTokens;
    int turn = 0;
    for (int first = rank * kPageTokens; first - rank * kPageTokens < p.budget; first += step, turn ^= 1) {
        const int size = min(kPageTokens, p.budget - first);
        if ((int)threadIdx.x < size) {
            int s = kept[first + threadIdx.x];
            if (s >= n) s = -1;
            source[turn][threadIdx.x] = s;
            weight = s >= 0 ? w[s] : 0.f;
        }
        __syncthreads();
        if (size > 0) take_tokens<kD>(p.c, p.c.table, p.c.width, b, h, source[turn], size, threadIdx.x, x);
        cluster_arrive();
        cluster_wait();
        if (size > 0) put_tokens<kD>(p.c, p.c.table, p.c.width, b, h, first, size, threadIdx.x, x);
        if ((int)threadIdx.x < size) w[first + threadIdx.x] = weight;
    }
    for (unsigned i = p.budget + rank * kMoveThreads + threadIdx.x; i < (unsigned)n; i += blocks * kMoveThreads) w[i] = 0.f;
}

// Choice and move in one, for few tokens to keep: a block a row, 64 places for each 128 threads.
constexpr int kFewThreads = 512, kFewBudget = kFewThreads / kMoveThreads * kPageTokens;
template <int kD>
__global__ void __launch_bounds__(kFewThreads, 1) evict_kernel(EvictParams p) {
    __shared__ int source[kFewThreads / kMoveThreads][kPageTokens];
    early();
    begin_work();
    choose<kFewThreads, false>(p);
    __syncthreads();  // (the list is the block's own)
    const size_t row = blockIdx.x;
    const int b = (int)(row / p.c.kv_heads), h = (int)(row - (size_t)b * p.c.kv_heads);
    const int n = cache_len(p.c, b, false);
    const bool within = p.to_table == nullptr;
    if (within && n <= p.budget) return;
    const int32_t* table = within ? p.c.table : p.to_table;
    const int width = within ? p.c.width : p.to_width;
    const int32_t* kept = p.kept + row * p.budget;
    const float* w = p.weights + row * p.c.width * kPageTokens;
    float* moved = p.moved + row * width * kPageTokens;
    const int group = threadIdx.x / kMoveThreads, thread = threadIdx.x % kMoveThreads, first = group * kPageTokens;
    const int m = min(n, p.budget), size = min(kPageTokens, m - first);
    float weight = 0.f;
    if (thread < size) {
        int s = kept[first + thread];
        if (s >= n) s = -1;
        source[group][thread] = s;
        weight = s >= 0 ? w[s] : 0.f;
    }
    __syncthreads();
    MovedToken<kD> x[MovedToken<kD>::kTurns];
    if (size > 0) take_tokens<kD>(p.c, p.c.table, p.c.width, b, h, source[group], size, thread, x);
    __syncthreads();  // all have read before any writes
    if (size > 0) put_tokens<kD>(p.c, table, width, b, h, first, size, thread, x);
    if (thread < size) moved[first + thread] = weight;
    const unsigned end = within ? (unsigned)n : (unsigned)width * kPageTokens;
    for (unsigned i = m + threadIdx.x; i < end; i += kFewThreads) moved[i] = 0.f;
}

// As launch_early, in clusters of `cluster` blocks along x.
template <class... P>
cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int cluster, int threads, int smem, cudaStream_t stream,
                            P... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    note_launches(1);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_evict(const CacheView& c, int D, const float* weights, int budget, int first, int recent,
                               const int32_t* to_table, int to_width, int32_t* kept, int32_t* lens, float* moved,
                               int num_sms, cudaStream_t stream) {
    EvictParams p;
    p.c = c;
    p.to_table = to_table;
    p.weights = weights;
    p.moved = moved;
    p.kept = kept;
    p.lens = lens;
    p.budget = budget;
    p.first = first;
    p.recent = recent;
    p.to_width = to_width;
    // Blocks of a row: as many as its keys need shared memory of, and more while the
    // rows leave SMs idle and a block has keys enough to pay for the barriers.  The choice
    // and a move of 1000 tokens, in us, with 1 / 2 / 4 / 8 blocks a row:
    //    8 heads, 12000 keys    11.1 / 12.4 / 14.5 / 17.9
    //    8 heads, 32760         17.6 / 16.2 / 14.0 / 20.6
    //   40 heads, 32760         19.4 / 16.3 / 24.7 / 54.1 (blocks share SMs from four on)
    //    8 heads, 115200           - /    - / 20.7 / 18.9
    const long long places = (long long)c.width * kPageTokens;
    const long long rows = (long long)c.B * c.kv_heads;
    int cluster = 1;
    while (cluster < kMaxCluster &&
           (places > (long long)kHeldKeys * cluster || (2 * rows * cluster <= num_sms && places > 12288LL * cluster)))
        cluster *= 2;
    const long long stretch = ((places + cluster - 1) / cluster + 127) / 128 * 128 + 128;
    p.keys = (int)std::min<long long>(stretch, kHeldKeys);
    // 512 threads where a thread has few keys: 300 keys of 2 heads 7.0 us as above (1024
    // threads: 7.4), 2000 of 8 heads 7.7 (8.5), 4000 8.6 (8.8), 32760 20.6 (18.7); 12000 in 192
    // rows 32.7 (29.5).
    constexpr int kFixed = (int)sizeof(ChooseSmem), kSmall = 4352;
    static_assert(kFixed % 16 == 0 && kFixed + kHeldKeys * 4 <= 232448, "shared memory of the choosing kernel");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(choose_kernel<1024>, kFixed + kHeldKeys * 4, done);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> done_small{0};
    e = allow_smem(choose_kernel<512>, kFixed + kSmall * 4, done_small);
    if (e != cudaSuccess) return e;
    // Choice and move in one kernel where a block moves all that its row keeps at once.  In us, two
    // kernels | one, D = 128, 4000 keys, to other pages and within their own (two turns of a
    // block's threads for 512 tokens are as slow as they look):
    //   budget 256,  1 sequence of 8 heads  9.6 |  8.9   8.5 |  7.4
    //               61                     27.0 | 24.6  22.2 | 18.3
    //   budget 512,  1                      9.6 | 10.8   8.5 |  9.1
    //               61                     38.7 | 50.2  29.6 | 32.9
    if (cluster == 1 && p.keys <= kSmall && budget <= kFewBudget) {
        static std::atomic<uint64_t> done_few[2];
        const auto kernel = D == 64 ? evict_kernel<64> : evict_kernel<128>;
        e = allow_smem(kernel, kFixed + kSmall * 4, done_few[D == 64]);
        if (e != cudaSuccess) return e;
        return launch_early(kernel, dim3((unsigned)rows), kFewThreads, kFixed + p.keys * 4, stream, p);
    }
    e = launch_clusters(p.keys <= kSmall ? choose_kernel<512> : choose_kernel<1024>, dim3((unsigned)(rows * cluster)), cluster,
                        p.keys <= kSmall ? 512 : 1024, kFixed + p.keys * 4, stream, p);
    if (e != cudaSuccess) return e;
    if (to_table) {
        const dim3 grid((unsigned)to_width, (unsigned)c.kv_heads, (unsigned)c.B);
        return launch_early(D == 64 ? move_kernel<64> : move_kernel<128>, grid, kMoveThreads, 0, stream, p);
    }
    const int turns = (budget + kPageTokens - 1) / kPageTokens;
    cluster = 1;
    while (cluster < kMaxCluster && cluster < turns) cluster *= 2;
    return launch_clusters(D == 64 ? move_within_kernel<64> : move_within_kernel<128>, dim3((unsigned)(rows * cluster)), cluster,
                           kMoveThreads, 0, stream, p);
}

}  // namespace vsa
