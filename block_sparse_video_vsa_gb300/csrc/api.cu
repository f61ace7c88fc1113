// C ABI of the VSA library: argument validation on the host, then dispatch
// to the kernels of tile.cu, coarse.cu, pair.cu, fine.cu, coarse_attn.cu,
// block_select.cu, cache_store.cu, cache_attn.cu (which passes on to cache_chunk.cu),
// tree.cu, weigh.cu (which passes on to weigh_chunk.cu) and evict.cu
// (coarse_noalloc.cu holds the allocation-free coarse entry point).  See
// include/vsa.h for the contract of each entry point.
#include <float.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "cache.cuh"

namespace vsa {

// Library-wide device error word (one per device that loads the library).
__device__ unsigned int g_device_error;

namespace {
constexpr int kMaxDevices = 64;
std::atomic<uint64_t> g_launches{0};
std::mutex g_ctx_mu;
DevCtx g_ctx[kMaxDevices];
bool g_ctx_ok[kMaxDevices];
}  // namespace

void note_launches(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

// Element counts that index int32 loops in the kernels must stay below 2^31.
bool sizes_fit(int64_t B, int64_t rows, int64_t heads, int64_t D) {
    const int64_t lim = (int64_t)1 << 31;
    return heads * D < lim / 64 && B * rows < lim && B * heads * rows / 64 < lim;
}

cudaError_t get_dev_ctx(DevCtx* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_ctx_mu);
    if (!g_ctx_ok[dev]) {
        DevCtx c;
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_device_error);
        if (e != cudaSuccess) return e;
        c.err = static_cast<unsigned int*>(p);
        e = cudaDeviceGetAttribute(&c.num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        e = cudaDeviceGetAttribute(&c.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
        if (e != cudaSuccess) return e;
        g_ctx[dev] = c;
        g_ctx_ok[dev] = true;
    }
    *out = g_ctx[dev];
    return cudaSuccess;
}

}  // namespace vsa

using namespace vsa;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

vsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? VSA_OK : VSA_ERR_CUDA; }

bool grid_ok(const vsa_grid* g) {
    return g && g->B > 0 && g->T > 0 && g->H > 0 && g->W > 0 && g->heads > 0 && g->D > 0;
}

int64_t cubes_of(const vsa_grid* g) {
    return (int64_t)((g->T + 3) / 4) * ((g->H + 3) / 4) * ((g->W + 3) / 4);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// What every vsa_cache_* call asks of the cache and of its rows a sequence.
vsa_status cache_args(const vsa_cache* c, int32_t S) {
    if (!c || !c->pool || !c->table || !c->kv_lens) return VSA_ERR_INVALID_ARG;
    if (c->pages <= 0 || c->kv_heads <= 0 || c->B <= 0 || c->width <= 0 || S <= 0)
        return VSA_ERR_INVALID_ARG;
    const int64_t lim = (int64_t)1 << 31;
    if (c->D != 64 && c->D != 128) return VSA_ERR_UNSUPPORTED;
    if (c->B > 65535 || c->kv_heads > 65535 || (int64_t)c->pages * c->kv_heads >= lim ||
        (int64_t)c->width * kPageTokens >= lim || (int64_t)c->B * S >= lim || S > (64 << 24))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(c->pool) || !aligned4(c->table) || !aligned4(c->kv_lens) || !aligned4(c->kv_scale))
        return VSA_ERR_ALIGNMENT;
    return VSA_OK;
}

vsa_status cache_view(const vsa_cache* c, CacheView* v, DevCtx* ctx) {
    if (get_dev_ctx(ctx) != cudaSuccess) return VSA_ERR_CUDA;
    v->pool = static_cast<unsigned char*>(c->pool);
    v->table = c->table;
    v->kv_lens = c->kv_lens;
    v->kv_scale = c->kv_scale;
    v->err = ctx->err;
    v->pages = c->pages;
    v->kv_heads = c->kv_heads;
    v->B = c->B;
    v->width = c->width;
    return VSA_OK;
}

}  // namespace

extern "C" {

const char* vsa_status_string(vsa_status s) {
    switch (s) {
        case VSA_OK: return "VSA_OK";
        case VSA_ERR_INVALID_ARG: return "VSA_ERR_INVALID_ARG";
        case VSA_ERR_UNSUPPORTED: return "VSA_ERR_UNSUPPORTED";
        case VSA_ERR_ALIGNMENT: return "VSA_ERR_ALIGNMENT";
        case VSA_ERR_INDEX_RANGE: return "VSA_ERR_INDEX_RANGE";
        case VSA_ERR_TIMEOUT: return "VSA_ERR_TIMEOUT";
        case VSA_ERR_CUDA: return "VSA_ERR_CUDA";
    }
    return "VSA_ERR_UNKNOWN";
}

int64_t vsa_num_cubes(const vsa_grid* g) {
    if (!grid_ok(g)) return -1;
    return cubes_of(g);
}

vsa_status vsa_tile(const vsa_grid* g, const void* x, void* xt, int32_t* vbs, vsa_stream_t stream) {
    if (!grid_ok(g) || !x || !xt) return VSA_ERR_INVALID_ARG;
    if ((g->heads * (int64_t)g->D) % 8 != 0) return VSA_ERR_UNSUPPORTED;
    const int64_t N = cubes_of(g);
    if (!sizes_fit(g->B, N * 64, g->heads, g->D) || (int64_t)g->T * g->H * g->W >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(xt) || (vbs && (reinterpret_cast<uintptr_t>(vbs) & 3u)))
        return VSA_ERR_ALIGNMENT;
    return from_cuda(launch_tile(*g, (int)N, x, xt, vbs, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_untile(const vsa_grid* g, const void* yt, void* y, vsa_stream_t stream) {
    if (!grid_ok(g) || !yt || !y) return VSA_ERR_INVALID_ARG;
    if ((g->heads * (int64_t)g->D) % 8 != 0) return VSA_ERR_UNSUPPORTED;
    const int64_t N = cubes_of(g);
    if (!sizes_fit(g->B, N * 64, g->heads, g->D) || (int64_t)g->T * g->H * g->W >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(yt) || !aligned16(y)) return VSA_ERR_ALIGNMENT;
    return from_cuda(launch_untile(*g, (int)N, yt, y, static_cast<cudaStream_t>(stream)));
}

size_t vsa_coarse_workspace_bytes(int32_t B, int32_t heads, int32_t ncubes, int32_t D) {
    if (B <= 0 || heads <= 0 || ncubes <= 0 || D <= 0) return 0;
    return coarse_workspace_bytes(B, heads, ncubes, D, coarse_split_default(ncubes, D));
}

vsa_status vsa_coarse_select(const void* qt, const void* kt, const int32_t* vbs, int32_t B, int32_t ncubes,
                             int32_t heads, int32_t D, int32_t topk, float sm_scale, void* workspace,
                             int32_t* topk_idx, vsa_stream_t stream) {
    if (!qt || !kt || !vbs || !workspace || !topk_idx) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || ncubes <= 0 || heads <= 0 || topk <= 0 || topk > ncubes) return VSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale)) return VSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
    if (ncubes > 4096 || !sizes_fit(B, (int64_t)ncubes * 64, heads, D)) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(qt) || !aligned16(kt) || !aligned16(workspace) || !aligned16(vbs) ||
        (reinterpret_cast<uintptr_t>(topk_idx) & 3u))
        return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    cudaError_t e = get_dev_ctx(&ctx);
    if (e != cudaSuccess) return VSA_ERR_CUDA;
    const bool split = coarse_split_default(ncubes, D);
    const size_t smem = coarse_smem_bytes(ncubes, D, split);
    if (smem > (size_t)ctx.max_smem_optin) return VSA_ERR_UNSUPPORTED;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)D);
    return from_cuda(launch_coarse(qt, kt, vbs, B, ncubes, heads, D, topk, sm_scale, workspace, topk_idx, split, false,
                                   static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_tile_pool(const vsa_grid* g, const void* q, const void* k, void* qt, void* kt, int32_t* vbs,
                         void* workspace, vsa_stream_t stream) {
    if (!grid_ok(g) || !q || !k || !workspace) return VSA_ERR_INVALID_ARG;
    if (g->D != 64 && g->D != 128) return VSA_ERR_UNSUPPORTED;
    const int64_t N = cubes_of(g);
    if (N > 4096 || !sizes_fit(g->B, N * 64, g->heads, g->D) || (int64_t)g->T * g->H * g->W >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if ((int64_t)g->B * N > 2147483647 || g->heads > 65535) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || (qt && !aligned16(qt)) || (kt && !aligned16(kt)) || !aligned16(workspace) ||
        (vbs && (reinterpret_cast<uintptr_t>(vbs) & 3u)))
        return VSA_ERR_ALIGNMENT;
    return from_cuda(launch_tile_pool(*g, (int)N, q, k, qt, kt, vbs, workspace, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_coarse_select_pooled(const int32_t* vbs, int32_t B, int32_t ncubes, int32_t heads, int32_t D,
                                    int32_t topk, float sm_scale, void* workspace, int32_t* topk_idx,
                                    vsa_stream_t stream) {
    if (!vbs || !workspace || !topk_idx) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || ncubes <= 0 || heads <= 0 || topk <= 0 || topk > ncubes) return VSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale)) return VSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
    if (ncubes > 4096 || !sizes_fit(B, (int64_t)ncubes * 64, heads, D)) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(workspace) || !aligned16(vbs) || (reinterpret_cast<uintptr_t>(topk_idx) & 3u))
        return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    cudaError_t e = get_dev_ctx(&ctx);
    if (e != cudaSuccess) return VSA_ERR_CUDA;
    const bool split = coarse_split_default(ncubes, D);
    if (coarse_smem_bytes(ncubes, D, split) > (size_t)ctx.max_smem_optin) return VSA_ERR_UNSUPPORTED;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)D);
    return from_cuda(launch_coarse(nullptr, nullptr, vbs, B, ncubes, heads, D, topk, sm_scale, workspace, topk_idx,
                                   split, true, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// Every fine-stage entry point: validation, then one launch of the fine kernel.
vsa_status fine_entry(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx, const int32_t* counts,
                      const int32_t* vbs, const uint32_t* pairs, int32_t B, int32_t ncubes, int32_t heads, int32_t D,
                      int32_t topk, float sm_scale, const float* coarse_out, const void* gate_c, const void* gate_f,
                      void* out, float* lse, float* max_prob, vsa_stream_t stream, const vsa_grid* raster = nullptr) {
    if (!qt || !kt || !vt || !topk_idx || !vbs || !out) return VSA_ERR_INVALID_ARG;
    const bool gated = coarse_out || gate_c || gate_f;
    if (gated && (!coarse_out || !gate_c || !gate_f)) return VSA_ERR_INVALID_ARG;
    if (raster) {
        // q and out in raster order of this grid; k, v, topk_idx on its cubes.
        if (!grid_ok(raster) || gated) return VSA_ERR_INVALID_ARG;
        if (raster->B != B || raster->heads != heads || raster->D != D || cubes_of(raster) != ncubes)
            return VSA_ERR_INVALID_ARG;
        if ((int64_t)B * raster->T * raster->H * raster->W >= ((int64_t)1 << 31)) return VSA_ERR_UNSUPPORTED;
    }
    if (B <= 0 || ncubes <= 0 || heads <= 0 || topk <= 0 || topk > ncubes) return VSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale)) return VSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
    if (!sizes_fit(B, (int64_t)ncubes * 64, heads, D) || (int64_t)B * ncubes * 64 >= ((int64_t)1 << 31) ||
        (int64_t)B * heads * ncubes >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if (heads > 65535) return VSA_ERR_UNSUPPORTED;  // TMA box coordinate range
    if (topk > fine_max_topk() || ncubes > fine_max_cubes()) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(qt) || !aligned16(kt) || !aligned16(vt) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(topk_idx) & 3u) || (reinterpret_cast<uintptr_t>(vbs) & 3u) ||
        (reinterpret_cast<uintptr_t>(pairs) & 3u) || (reinterpret_cast<uintptr_t>(counts) & 3u) ||
        (lse && (reinterpret_cast<uintptr_t>(lse) & 3u)) ||
        (max_prob && (reinterpret_cast<uintptr_t>(max_prob) & 3u)) ||
        (gated && (!aligned16(coarse_out) || !aligned16(gate_c) || !aligned16(gate_f))))
        return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    cudaError_t e = get_dev_ctx(&ctx);
    if (e != cudaSuccess) return VSA_ERR_CUDA;
    if (fine_smem_bytes() > ctx.max_smem_optin) return VSA_ERR_UNSUPPORTED;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)D);
    return from_cuda(launch_fine(qt, kt, vt, topk_idx, counts, vbs, pairs, B, ncubes, heads, D, topk, sm_scale,
                                 coarse_out, gate_c, gate_f, out, lse, max_prob, raster, ctx.err, ctx.num_sms,
                                 static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

vsa_status vsa_sparse_attn_fwd_gated(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx,
                                     const int32_t* counts, const int32_t* vbs, const uint32_t* pairs, int32_t B,
                                     int32_t ncubes, int32_t heads, int32_t D, int32_t topk, float sm_scale,
                                     const float* coarse_out, const void* gate_c, const void* gate_f, void* out,
                                     float* lse, vsa_stream_t stream) {
    return fine_entry(qt, kt, vt, topk_idx, counts, vbs, pairs, B, ncubes, heads, D, topk, sm_scale, coarse_out,
                      gate_c, gate_f, out, lse, nullptr, stream);
}

vsa_status vsa_sparse_attn_fwd_peak(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx,
                                    const int32_t* counts, const int32_t* vbs, const uint32_t* pairs, int32_t B,
                                    int32_t ncubes, int32_t heads, int32_t D, int32_t topk, float sm_scale, void* out,
                                    float* lse, float* max_prob, vsa_stream_t stream) {
    if (!max_prob) return VSA_ERR_INVALID_ARG;
    return fine_entry(qt, kt, vt, topk_idx, counts, vbs, pairs, B, ncubes, heads, D, topk, sm_scale, nullptr, nullptr,
                      nullptr, out, lse, max_prob, stream);
}


vsa_status vsa_sparse_attn_fwd_raster(const vsa_grid* g, const void* q, const void* kt, const void* vt,
                                      const int32_t* topk_idx, const int32_t* counts, const int32_t* vbs,
                                      const uint32_t* pairs, int32_t topk, float sm_scale, void* out, float* lse,
                                      vsa_stream_t stream) {
    if (!grid_ok(g)) return VSA_ERR_INVALID_ARG;
    const int64_t N = cubes_of(g);
    if (N > 2147483647) return VSA_ERR_UNSUPPORTED;
    return fine_entry(q, kt, vt, topk_idx, counts, vbs, pairs, g->B, (int32_t)N, g->heads, g->D, topk, sm_scale,
                      nullptr, nullptr, nullptr, out, lse, nullptr, stream, g);
}

vsa_status vsa_sparse_attn_fwd_ex(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx,
                                  const int32_t* counts, const int32_t* vbs, const uint32_t* pairs, int32_t B,
                                  int32_t ncubes, int32_t heads, int32_t D, int32_t topk, float sm_scale,
                                  void* out, float* lse, vsa_stream_t stream) {
    return vsa_sparse_attn_fwd_gated(qt, kt, vt, topk_idx, counts, vbs, pairs, B, ncubes, heads, D, topk, sm_scale,
                                     nullptr, nullptr, nullptr, out, lse, stream);
}

size_t vsa_coarse_attn_workspace_bytes(int32_t B, int32_t heads, int32_t ncubes, int32_t D) {
    if (B <= 0 || heads <= 0 || ncubes <= 0 || (D != 64 && D != 128)) return 0;
    return coarse_attn_workspace_bytes(B, heads, ncubes, D);
}

vsa_status vsa_coarse_attn(const void* qt, const void* kt, const void* vt, const int32_t* vbs, int32_t B,
                           int32_t ncubes, int32_t heads, int32_t D, float sm_scale, void* workspace,
                           float* coarse_out, vsa_stream_t stream) {
    if (!qt || !kt || !vt || !vbs || !workspace || !coarse_out) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || ncubes <= 0 || heads <= 0) return VSA_ERR_INVALID_ARG;
    if (!(sm_scale == sm_scale)) return VSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
    if (!sizes_fit(B, (int64_t)ncubes * 64, heads, D) || B > 65535 || heads > 65535 ||
        (int64_t)B * ncubes >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(qt) || !aligned16(kt) || !aligned16(vt) || !aligned16(workspace) || !aligned16(coarse_out) ||
        (reinterpret_cast<uintptr_t>(vbs) & 3u))
        return VSA_ERR_ALIGNMENT;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)D);
    return from_cuda(launch_coarse_attn(qt, kt, vt, vbs, B, ncubes, heads, D, sm_scale, workspace, coarse_out,
                                        static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_sparse_attn_fwd_paired(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx,
                                      const int32_t* vbs, const uint32_t* pairs, int32_t B, int32_t ncubes,
                                      int32_t heads, int32_t D, int32_t topk, float sm_scale, void* out, float* lse,
                                      vsa_stream_t stream) {
    return vsa_sparse_attn_fwd_ex(qt, kt, vt, topk_idx, nullptr, vbs, pairs, B, ncubes, heads, D, topk, sm_scale,
                                  out, lse, stream);
}

vsa_status vsa_sparse_attn_fwd(const void* qt, const void* kt, const void* vt, const int32_t* topk_idx,
                               const int32_t* vbs, int32_t B, int32_t ncubes, int32_t heads, int32_t D,
                               int32_t topk, float sm_scale, void* out, float* lse, vsa_stream_t stream) {
    return vsa_sparse_attn_fwd_ex(qt, kt, vt, topk_idx, nullptr, vbs, nullptr, B, ncubes, heads, D, topk,
                                  sm_scale, out, lse, stream);
}

size_t vsa_block_select_workspace_bytes(int32_t B, int32_t S, int32_t heads, int32_t D) {
    if (B <= 0 || heads <= 0 || S <= 0 || S % 128 || (D != 64 && D != 128)) return 0;
    return block_select_workspace_bytes(B, heads, S / 128, D);
}

vsa_status vsa_block_select(const void* q, const void* k, int32_t B, int32_t S, int32_t heads, int32_t D, float tau,
                            float sm_scale, void* workspace, int32_t* cube_idx, int32_t* cube_counts,
                            vsa_stream_t stream) {
    if (!q || !k || !workspace || !cube_idx || !cube_counts) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || S <= 0 || heads <= 0 || S % 128) return VSA_ERR_INVALID_ARG;
    if (!(tau > 0.f && tau <= 1.f) || !(sm_scale == sm_scale)) return VSA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return VSA_ERR_UNSUPPORTED;
    if (S / 128 > block_select_max_blocks() || B > 65535 || heads > 65535 ||
        !sizes_fit(B, S, heads, D))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(cube_idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(cube_counts) & 3u))
        return VSA_ERR_ALIGNMENT;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)D);
    return from_cuda(launch_block_select(q, k, B, S, heads, D, tau, sm_scale, workspace, cube_idx, cube_counts,
                                         static_cast<cudaStream_t>(stream)));
}

size_t vsa_cache_pool_bytes(int32_t pages, int32_t kv_heads, int32_t D) {
    if (pages <= 0 || kv_heads <= 0 || (D != 64 && D != 128)) return 0;
    return (size_t)pages * kv_heads * 72 * D;
}

vsa_status vsa_cache_append(const vsa_cache* c, const void* q, const void* k, const void* v, int32_t S,
                            int32_t heads, const int32_t* new_lens, const float* rope, int32_t rope_rows,
                            int32_t rope_dim, int32_t interleaved, const int32_t* positions, void* q_out,
                            vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, S);
    if (st != VSA_OK) return st;
    if (!k || !v || (q == nullptr) != (q_out == nullptr) || (q && heads <= 0)) return VSA_ERR_INVALID_ARG;
    if (rope_dim < 0 || (rope_dim > 0) != (rope != nullptr) || (rope && rope_rows <= 0)) return VSA_ERR_INVALID_ARG;
    if (rope_dim % 32 || rope_dim > c->D || (q && heads > 65535)) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(rope) ||
        !aligned4(new_lens) || !aligned4(positions))
        return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    return from_cuda(launch_cache_append(cv, c->D, q, k, v, S, q ? heads : 0, new_lens, rope, rope_rows, rope_dim,
                                         interleaved, positions, q_out, ctx.num_sms,
                                         static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_cache_read(const vsa_cache* c, int32_t S, void* k, void* v, vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, S);
    if (st != VSA_OK) return st;
    if (!k || !v) return VSA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    return from_cuda(launch_cache_read(cv, c->D, S, k, v, static_cast<cudaStream_t>(stream)));
}

size_t vsa_cache_attn_workspace_bytes(int32_t kv_heads, int32_t D, int32_t Sq, int32_t heads) {
    if (kv_heads <= 0 || heads <= 0 || heads % kv_heads || Sq <= 0 || (D != 64 && D != 128) ||
        (int64_t)Sq * (heads / kv_heads) >= (1 << 24))
        return 0;
    return cache_attn_workspace_bytes(D, Sq, heads / kv_heads);
}

}  // extern "C"

namespace {

// vsa_cache_attn, and with a tree vsa_cache_attn_tree.
vsa_status cache_attn(const vsa_cache* c, const void* q, int32_t Sq, int32_t heads, const int32_t* q_lens,
                      int32_t causal, const uint64_t* tree, const int32_t* page_sel, int32_t nsel, float sm_scale,
                      void* workspace, void* out, float* lse, vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, Sq);
    if (st != VSA_OK) return st;
    if (!q || !workspace || !out || heads <= 0 || heads % c->kv_heads) return VSA_ERR_INVALID_ARG;
    if (nsel < 0 || (nsel > 0) != (page_sel != nullptr) || !(fabsf(sm_scale) <= FLT_MAX)) return VSA_ERR_INVALID_ARG;
    if (heads > 65535 || (int64_t)Sq * (heads / c->kv_heads) >= (1 << 24) || nsel >= (1 << 25)) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(workspace) || !aligned16(out) || !aligned4(q_lens) || !aligned4(page_sel) ||
        !aligned4(lse))
        return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)c->D);
    return from_cuda(launch_cache_attn(cv, c->D, q, Sq, heads, q_lens, causal, tree, page_sel, nsel, sm_scale,
                                       workspace, out, lse, ctx.num_sms, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

vsa_status vsa_cache_attn(const vsa_cache* c, const void* q, int32_t Sq, int32_t heads, const int32_t* q_lens,
                          int32_t causal, const int32_t* page_sel, int32_t nsel, float sm_scale, void* workspace,
                          void* out, float* lse, vsa_stream_t stream) {
    return cache_attn(c, q, Sq, heads, q_lens, causal, nullptr, page_sel, nsel, sm_scale, workspace, out, lse, stream);
}

vsa_status vsa_cache_attn_tree(const vsa_cache* c, const void* q, int32_t Sq, int32_t heads, const int32_t* q_lens,
                               const uint64_t* tree, const int32_t* page_sel, int32_t nsel, float sm_scale,
                               void* workspace, void* out, float* lse, vsa_stream_t stream) {
    const vsa_status st = cache_args(c, Sq);
    if (st != VSA_OK) return st;
    if (!tree) return VSA_ERR_INVALID_ARG;
    if (Sq > tree_max_nodes()) return VSA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(tree) & 7u) return VSA_ERR_ALIGNMENT;
    return cache_attn(c, q, Sq, heads, q_lens, 0, tree, page_sel, nsel, sm_scale, workspace, out, lse, stream);
}

vsa_status vsa_cache_tree(const int32_t* parents, int32_t B, int32_t S, const int32_t* kv_lens,
                          const int32_t* new_lens, const int32_t* starts, uint64_t* mask, int32_t* positions,
                          vsa_stream_t stream) {
    if (!parents || !mask || B <= 0 || S <= 0) return VSA_ERR_INVALID_ARG;
    if (B > 65535 || S > tree_max_nodes()) return VSA_ERR_UNSUPPORTED;
    if (!aligned4(parents) || !aligned4(kv_lens) || !aligned4(new_lens) || !aligned4(starts) || !aligned4(positions) ||
        (reinterpret_cast<uintptr_t>(mask) & 7u))
        return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    if (get_dev_ctx(&ctx) != cudaSuccess) return VSA_ERR_CUDA;
    return from_cuda(launch_cache_tree(parents, B, S, kv_lens, new_lens, starts, mask, positions, ctx.err,
                                       static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_cache_accept(const vsa_cache* c, const int32_t* new_lens, const int32_t* path, const int32_t* path_lens,
                            int32_t n, int32_t* lens, vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, n);
    if (st != VSA_OK) return st;
    if (!new_lens || !path || !path_lens || !lens || lens == c->kv_lens || lens == new_lens || lens == path_lens)
        return VSA_ERR_INVALID_ARG;
    if (n > tree_max_nodes()) return VSA_ERR_UNSUPPORTED;
    if (!aligned4(new_lens) || !aligned4(path) || !aligned4(path_lens) || !aligned4(lens)) return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    return from_cuda(launch_cache_accept(cv, c->D, new_lens, path, path_lens, n, lens,
                                         static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_cache_weigh(const vsa_cache* c, const void* q, const float* lse, int32_t Sq, int32_t heads,
                           const int32_t* q_lens, int32_t causal, float sm_scale, const float* weights, float* out,
                           vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, Sq);
    if (st != VSA_OK) return st;
    if (!q || !lse || !out || heads <= 0 || heads % c->kv_heads || !(fabsf(sm_scale) <= FLT_MAX))
        return VSA_ERR_INVALID_ARG;
    if (heads > 65535 || (int64_t)Sq * (heads / c->kv_heads) >= (1 << 24)) return VSA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(weights) || !aligned16(out) || !aligned4(lse) || !aligned4(q_lens))
        return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    if (sm_scale <= 0.f) sm_scale = 1.0f / sqrtf((float)c->D);
    return from_cuda(launch_cache_weigh(cv, c->D, q, lse, Sq, heads, q_lens, causal, sm_scale, weights, out,
                                        ctx.num_sms, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_cache_evict(const vsa_cache* c, float* weights, int32_t budget, int32_t first, int32_t recent,
                           const int32_t* to_table, int32_t to_width, int32_t* kept, int32_t* lens, float* moved,
                           vsa_stream_t stream) {
    CacheView cv;
    DevCtx ctx;
    vsa_status st = cache_args(c, 1);
    if (st != VSA_OK) return st;
    if (!weights || !kept || !lens || lens == c->kv_lens) return VSA_ERR_INVALID_ARG;
    if (budget <= 0 || first < 0 || recent < 0 || (int64_t)first + recent > budget) return VSA_ERR_INVALID_ARG;
    if (to_table ? to_width <= 0 || !moved || moved == weights : to_width != 0 || moved) return VSA_ERR_INVALID_ARG;
    const int64_t most = std::min<int64_t>(budget, (int64_t)c->width * kPageTokens);
    if (to_table && (int64_t)to_width * kPageTokens < most) return VSA_ERR_INVALID_ARG;
    if (budget > (1 << 30) || (int64_t)c->B * c->kv_heads >= (1 << 27) || (int64_t)to_width * kPageTokens >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned4(weights) || !aligned4(moved) || !aligned4(kept) || !aligned4(lens) || !aligned4(to_table))
        return VSA_ERR_ALIGNMENT;
    st = cache_view(c, &cv, &ctx);
    if (st != VSA_OK) return st;
    return from_cuda(launch_cache_evict(cv, c->D, weights, budget, first, recent, to_table, to_width, kept, lens,
                                        to_table ? moved : weights, ctx.num_sms, static_cast<cudaStream_t>(stream)));
}

size_t vsa_pair_workspace_bytes(int32_t B, int32_t heads, int32_t ncubes, int32_t topk) {
    if (B <= 0 || heads <= 0 || ncubes <= 0 || topk <= 0) return 0;
    return pair_workspace_bytes(B, heads, ncubes, topk);
}

vsa_status vsa_pair_cubes(const int32_t* topk_idx, int32_t B, int32_t ncubes, int32_t heads, int32_t topk,
                          void* workspace, uint32_t* pairs, vsa_stream_t stream) {
    if (!topk_idx || !workspace || !pairs) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || ncubes <= 0 || heads <= 0 || topk <= 0 || topk > ncubes) return VSA_ERR_INVALID_ARG;
    if (ncubes > pair_max_cubes() || topk > pair_max_topk() || (int64_t)B * heads > 65535 ||
        (int64_t)B * heads * ncubes >= ((int64_t)1 << 31) ||
        (int64_t)B * heads * ncubes * topk >= ((int64_t)1 << 40))
        return VSA_ERR_UNSUPPORTED;
    if (!aligned16(workspace) || (reinterpret_cast<uintptr_t>(topk_idx) & 3u) ||
        (reinterpret_cast<uintptr_t>(pairs) & 3u))
        return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    if (get_dev_ctx(&ctx) != cudaSuccess) return VSA_ERR_CUDA;
    return from_cuda(launch_pair(topk_idx, B, ncubes, heads, topk, workspace, pairs, ctx.num_sms,
                                 ctx.max_smem_optin, static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_validate_indices_ex(const int32_t* topk_idx, const int32_t* counts, const int32_t* vbs, int32_t B,
                                   int32_t heads, int32_t ncubes, int32_t topk, int32_t* dev_flag,
                                   vsa_stream_t stream) {
    if (!topk_idx || !vbs || !dev_flag) return VSA_ERR_INVALID_ARG;
    if (B <= 0 || heads <= 0 || ncubes <= 0 || topk <= 0) return VSA_ERR_INVALID_ARG;
    if (ncubes > validate_max_cubes() || (int64_t)B * heads * ncubes >= ((int64_t)1 << 31))
        return VSA_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(topk_idx) & 3u) || (reinterpret_cast<uintptr_t>(vbs) & 3u) ||
        (reinterpret_cast<uintptr_t>(counts) & 3u) || (reinterpret_cast<uintptr_t>(dev_flag) & 3u))
        return VSA_ERR_ALIGNMENT;
    return from_cuda(launch_validate(topk_idx, counts, vbs, B * heads * ncubes, ncubes, topk, dev_flag,
                                     static_cast<cudaStream_t>(stream)));
}

vsa_status vsa_validate_indices(const int32_t* topk_idx, const int32_t* vbs, int32_t B, int32_t heads,
                                int32_t ncubes, int32_t topk, int32_t* dev_flag, vsa_stream_t stream) {
    return vsa_validate_indices_ex(topk_idx, nullptr, vbs, B, heads, ncubes, topk, dev_flag, stream);
}

vsa_status vsa_device_error(uint32_t* out, int32_t reset) {
    if (!out) return VSA_ERR_INVALID_ARG;
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof v) != cudaSuccess) return VSA_ERR_CUDA;
    *out = v;
    if (reset) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_device_error, &z, sizeof z) != cudaSuccess) return VSA_ERR_CUDA;
    }
    return VSA_OK;
}

vsa_status vsa_debug_wait_timeout(int64_t limit_ns, int32_t* dev_result, vsa_stream_t stream) {
    if (!dev_result || limit_ns < 1000 || limit_ns > 10000000000ll) return VSA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(dev_result) & 3u) return VSA_ERR_ALIGNMENT;
    DevCtx ctx;
    if (get_dev_ctx(&ctx) != cudaSuccess) return VSA_ERR_CUDA;
    return from_cuda(launch_debug_wait((long long)limit_ns, dev_result, ctx.err, static_cast<cudaStream_t>(stream)));
}

uint64_t vsa_kernel_launches(void) { return g_launches.load(std::memory_order_relaxed); }

vsa_status vsa_table_from_csr(const int64_t* lut_ptr, const int32_t* kv_idx, int64_t nnz, int64_t rows,
                              int32_t width, int32_t ncubes, int32_t* table, int32_t* counts) {
    if (!lut_ptr || !table || !counts || rows <= 0 || width <= 0 || nnz < 0 || ncubes <= 0)
        return VSA_ERR_INVALID_ARG;
    if (lut_ptr[0] != 0) return VSA_ERR_INVALID_ARG;
    for (int64_t r = 0; r < rows; ++r) {
        const int64_t n = lut_ptr[r + 1] - lut_ptr[r];
        if (n < 0 || n > width) return VSA_ERR_INVALID_ARG;
    }
    if (lut_ptr[rows] > nnz) return VSA_ERR_INVALID_ARG;  // the offsets run past kv_idx
    if (lut_ptr[rows] > 0 && !kv_idx) return VSA_ERR_INVALID_ARG;
    for (int64_t e = 0; e < lut_ptr[rows]; ++e)
        if (kv_idx[e] < 0 || kv_idx[e] >= ncubes) return VSA_ERR_INDEX_RANGE;
    for (int64_t r = 0; r < rows; ++r) {
        const int64_t b = lut_ptr[r];
        const int32_t n = (int32_t)(lut_ptr[r + 1] - b);
        int32_t* row = table + r * (int64_t)width;
        for (int32_t e = 0; e < n; ++e) row[e] = kv_idx[b + e];
        for (int32_t e = n; e < width; ++e) row[e] = -1;
        counts[r] = n;
    }
    return VSA_OK;
}

}  // extern "C"
