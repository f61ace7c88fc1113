// A draft's tree of tokens: its masks and positions, and the accepted path.
//
// tree_kernel: node i of a sequence's m drafted tokens has a parent p_i < i (or
// hangs on the cached tokens).  Its mask is the set of its ancestors and itself,
//   mask_i = {i} u mask_{p_i},  position_i = start + |mask_i| - 1,
// as bits in 64-bit words, which is what the attention reads.  A thread forms one
// word of one node by walking up from the node (parents in shared memory; a
// path of some ten nodes, 1024 at most), so no thread waits for another's.
// Latency bound: a block a few hundred words, 4 S bytes in, 8 S ceil(S / 64) + 4 S
// out: 2 us for a tree of 12, 3 for 61 of up to 48 (GB300).
//
// accept_kernel: of the step's tokens at places base .. base + m - 1 those on the
// accepted path move to base, base + 1, ...; the codes and scales of K and V of
// all kv heads, 9/8 D bytes each way.  A block takes a kv head of a sequence, 64
// tokens at a time: all are read before any is written, and a path ascends
// (path_i >= i), so nothing is read that was written before.  Latency bound: lengths,
// path, page numbers, tokens, one after the other; 2.7 us for one path, 7.2 for 61 paths
// in 8 heads of 128 channels from a cold cache.
#include "move.cuh"

namespace vsa {

namespace {

struct TreeParams {
    const int32_t* parents;   // [B][S]
    const int32_t* kv_lens;   // [B], or null: positions are depths
    const int32_t* new_lens;  // [B], or null: S
    const int32_t* starts;    // [B], or null: kv_lens - new_lens
    uint64_t* mask;           // [B][S][words]
    int32_t* positions;       // [B][S], or null
    unsigned int* err;
    int S, words;
};

constexpr int kTreeThreads = 128;

__global__ void __launch_bounds__(kTreeThreads) tree_kernel(TreeParams p) {
    __shared__ int parent[kMaxTree];
    early();
    begin_work();
    const int b = blockIdx.y;
    const int fresh = p.new_lens ? min(max(p.new_lens[b], 0), p.S) : p.S;
    bool bad = false;
    for (int i = threadIdx.x; i < fresh; i += kTreeThreads) {
        const int x = p.parents[(size_t)b * p.S + i];
        const bool ok = x >= -1 && x < i;
        bad |= !ok;
        parent[i] = ok ? x : -1;
    }
    if (bad && blockIdx.x == 0) atomicOr(p.err, VSA_DEVERR_INDEX);
    __syncthreads();
    const int at = blockIdx.x * kTreeThreads + threadIdx.x;
    if (at >= p.S * p.words) return;
    const int node = at / p.words, word = at - node * p.words;
    uint64_t bits = 0;
    int depth = -1;
    if (node < fresh)
        for (int i = node; i >= 0; i = parent[i]) {  // (parents come before: it ends)
            if (i >> 6 == word) bits |= 1ull << (i & 63);
            ++depth;
        }
    p.mask[((size_t)b * p.S + node) * p.words + word] = bits;
    if (p.positions && word == 0) {
        int start = 0;
        if (p.starts)
            start = p.starts[b];
        else if (p.kv_lens)
            start = p.kv_lens[b] - fresh;
        p.positions[(size_t)b * p.S + node] = node < fresh ? start + depth : 0;
    }
}

struct AcceptParams {
    CacheView c;
    const int32_t* new_lens;   // [B]
    const int32_t* path;       // [B][n]
    const int32_t* path_lens;  // [B]
    int32_t* lens;             // [B]
    int n;
};

template <int kD>
__global__ void __launch_bounds__(kMoveThreads) accept_kernel(AcceptParams p) {
    __shared__ int source[kPageTokens];
    early();
    begin_work();
    const int h = blockIdx.x, b = blockIdx.y;
    const int held = cache_len(p.c, b, h == 0 && threadIdx.x == 0);
    const int fresh = min(max(p.new_lens[b], 0), held);
    const int base = held - fresh;
    const int count = min(min(max(p.path_lens[b], 0), p.n), fresh);
    if (h == 0 && threadIdx.x == 0) {
        if (p.path_lens[b] != count) atomicOr(p.c.err, VSA_DEVERR_INDEX);
        p.lens[b] = base + count;
    }
    for (int first = 0; first < count; first += kPageTokens) {
        const int size = min(kPageTokens, count - first);
        if (threadIdx.x < size) {
            const int i = first + threadIdx.x;
            const int32_t* path = p.path + (size_t)b * p.n;
            const int x = path[i], before = i > 0 ? path[i - 1] : -1;
            const bool ok = x >= i && x < fresh && x > before;
            if (!ok) atomicOr(p.c.err, VSA_DEVERR_INDEX);
            source[threadIdx.x] = ok ? base + x : -1;
        }
        __syncthreads();
        MovedToken<kD> moved[MovedToken<kD>::kTurns];
        take_tokens<kD>(p.c, p.c.table, p.c.width, b, h, source, size, threadIdx.x, moved);
        __syncthreads();  // (and `source` is free again)
        put_tokens<kD>(p.c, p.c.table, p.c.width, b, h, base + first, size, threadIdx.x, moved);
    }
}

}  // namespace

int tree_max_nodes() { return kMaxTree; }

cudaError_t launch_cache_tree(const int32_t* parents, int B, int S, const int32_t* kv_lens, const int32_t* new_lens,
                              const int32_t* starts, uint64_t* mask, int32_t* positions, unsigned int* err,
                              cudaStream_t stream) {
    TreeParams p;
    p.parents = parents;
    p.kv_lens = kv_lens;
    p.new_lens = new_lens;
    p.starts = starts;
    p.mask = mask;
    p.positions = positions;
    p.err = err;
    p.S = S;
    p.words = (S + 63) / 64;
    const dim3 grid((unsigned)((S * p.words + kTreeThreads - 1) / kTreeThreads), (unsigned)B);
    return launch_early(tree_kernel, grid, kTreeThreads, 0, stream, p);
}

cudaError_t launch_cache_accept(const CacheView& c, int D, const int32_t* new_lens, const int32_t* path,
                                const int32_t* path_lens, int n, int32_t* lens, cudaStream_t stream) {
    AcceptParams p;
    p.c = c;
    p.new_lens = new_lens;
    p.path = path;
    p.path_lens = path_lens;
    p.lens = lens;
    p.n = n;
    const dim3 grid((unsigned)c.kv_heads, (unsigned)c.B);
    return launch_early(D == 64 ? accept_kernel<64> : accept_kernel<128>, grid, kMoveThreads, 0, stream, p);
}

}  // namespace vsa
