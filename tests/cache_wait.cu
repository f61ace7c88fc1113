// The cache kernels' bounded wait by itself, for tests/test_gpu_cache_wait.py.
// Two warps; the first waits for a barrier that the second completes (mode 2),
// that nobody arrives at while the second raises the abort flag (mode 1), or
// that nobody arrives at at all (mode 0).
#include "cache.cuh"

__global__ void wait_kernel(int mode, unsigned long long limit_ns, unsigned int* err, int* result) {
    __shared__ __align__(8) uint64_t bar;
    __shared__ int abort_flag;
    const uint32_t b = vsa::smem_u32(&bar);
    if (threadIdx.x == 0) {
        vsa::mbar_init(b, 1);
        abort_flag = 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const bool ok = vsa::cache_wait<vsa::kSleepShort>(b, 0, &abort_flag, err, limit_ns);
        if (threadIdx.x == 0) {
            result[0] = ok;
            result[1] = *(volatile int*)&abort_flag;
        }
    } else if (threadIdx.x == 32) {
        __nanosleep(1000);
        if (mode == 1) *(volatile int*)&abort_flag = 1;
        if (mode == 2) vsa::mbar_arrive(b);
    }
}

// result: {the wait's answer, the abort flag after it, the error word}; returns a CUDA status.
extern "C" int wait_case(int mode, unsigned long long limit_ns, int* result) {
    int* d = nullptr;
    cudaError_t e = cudaMalloc(&d, 3 * sizeof(int));
    if (e != cudaSuccess) return (int)e;
    e = cudaMemset(d, 0, 3 * sizeof(int));
    if (e == cudaSuccess) {
        wait_kernel<<<1, 64>>>(mode, limit_ns, reinterpret_cast<unsigned int*>(d + 2), d);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaMemcpy(result, d, 3 * sizeof(int), cudaMemcpyDeviceToHost);
    cudaFree(d);
    return (int)e;
}
