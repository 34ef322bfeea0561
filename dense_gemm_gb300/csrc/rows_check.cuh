// The checked build's status of the kernels along rows (sm_103a), which are in a translation
// unit of their own and do not see the products' status words. In the product build there is
// nothing here: G16_CHECK is the constant true.
#pragma once
#include <cuda_runtime.h>

#define G16_CHECK_FAILED rows_check_failed
#include "ops_rows.h"
#include "ptx.cuh"

#ifdef GEMM_DEBUG
namespace g16 {

namespace {
__device__ unsigned int g_rows_check_line;  // source line of the first failed check, 0: none
}

__device__ __noinline__ bool rows_check_failed(int line) {
    atomicCAS(&g_rows_check_line, 0u, unsigned(line));
    return false;
}

__global__ void rows_check_selftest_kernel() {
    if (threadIdx.x == 0) (void)G16_CHECK(false);
}

cudaError_t rows_check_selftest(cudaStream_t stream) {
    rows_check_selftest_kernel<<<1, 32, 0, stream>>>();
    return cudaGetLastError();
}

cudaError_t take_rows_check_line(unsigned int *line) {
    const unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(line, g_rows_check_line, sizeof(zero));
    if (e == cudaSuccess && *line != 0) e = cudaMemcpyToSymbol(g_rows_check_line, &zero, sizeof(zero));
    return e;
}

}  // namespace g16
#endif
