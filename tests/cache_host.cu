// Host parts of the cache's shared header, for tests/test_cache_header.py: built
// without a GPU, with the runtime's attribute query answered by the test.
#include <cuda_runtime.h>

static int g_error = 0, g_regs = 0, g_asked = 0;
template <class K>
static cudaError_t fake_attributes(cudaFuncAttributes* fa, K) {
    ++g_asked;
    fa->numRegs = g_regs;
    return (cudaError_t)g_error;
}
#define cudaFuncGetAttributes fake_attributes
#include "cache.cuh"

// answers: n pairs {error, registers} of the query; got: n pairs {status, registers} of the call; returns queries made.
extern "C" int registers_case(const int* answers, int n, int* got) {
    static std::atomic<int> known;
    known = 0;
    g_asked = 0;
    for (int i = 0; i < n; ++i) {
        g_error = answers[2 * i];
        g_regs = answers[2 * i + 1];
        got[2 * i + 1] = -1;
        got[2 * i] = (int)vsa::launch_registers(&registers_case, known, &got[2 * i + 1]);
    }
    return g_asked;
}

// Sums for n rows of {n, k, c, g}.
extern "C" void steps_sum_case(const long long* args, int rows, long long* got) {
    for (int i = 0; i < rows; ++i)
        got[i] = vsa::steps_sum((int)args[4 * i], (int)args[4 * i + 1], args[4 * i + 2], (int)args[4 * i + 3]);
}
