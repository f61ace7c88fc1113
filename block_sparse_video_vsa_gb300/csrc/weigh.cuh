// What the two kernels of cache_weigh share.
#pragma once

#include "cache.cuh"

namespace vsa {

struct WeighParams {
    CacheView c;
    const uint4* q;         // bf16 [B][Sq][heads][D]
    const float* lse;       // [B][heads][Sq]
    const int32_t* q_lens;  // [B], or null: Sq
    const float* weights;   // [B][kv_heads][64 * width], or null: zeros
    float* out;             // likewise; may be `weights`
    int Sq, heads, group, causal;
    float scale_log2;       // sm_scale * log2(e)
};

#if defined(__CUDACC__)

// 4-byte asynchronous global -> shared copy, tracked by commit groups.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Places from a sequence's length on: what `weights` has there, or zero
// (nothing is to be done in place).  The blocks share the rows.
__device__ __forceinline__ void fill_rest(const WeighParams& p, bool idle) {
    if (p.out == p.weights) return;
    const long long rows = (long long)p.c.B * p.c.kv_heads;
    const long long share = max(1LL, (long long)gridDim.x / rows), step = gridDim.x / share;  // blocks of a row; rows at once
    const long long places = (long long)p.c.width * kPageTokens;
    for (long long row = blockIdx.x / share; row < rows; row += step) {
        const int b = (int)(row / p.c.kv_heads);
        // (All of a sequence without queries, which nobody else writes, where `idle` says so.)
        const int kv = idle && p.q_lens && p.q_lens[b] <= 0 ? 0 : cache_len(p.c, b, false);
        const float* in = p.weights ? p.weights + row * places : nullptr;
        float* out = p.out + row * places;
        const long long whole = ((long long)kv + 3) / 4 * 4;  // from here on in 16 bytes
        const long long i0 = (blockIdx.x % share) * blockDim.x + threadIdx.x;
        if (kv + i0 < whole) out[kv + i0] = in ? in[kv + i0] : 0.f;
        for (long long i = whole / 4 + i0; i < places / 4; i += share * blockDim.x)
            reinterpret_cast<float4*>(out)[i] = in ? reinterpret_cast<const float4*>(in)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

// weigh_chunk.cu
cudaError_t launch_weigh_chunk(const WeighParams& p, int D, int num_sms, cudaStream_t stream);

#endif  // __CUDACC__

}  // namespace vsa
