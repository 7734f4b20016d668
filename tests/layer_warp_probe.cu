// Test support: a warp waits, half of its lanes on a barrier that has
// completed and half on one that nothing completes; result[i] is lane i's
// answer.
#include <stdint.h>

#include "mhc_umma.cuh"

__global__ void layer_warp_probe_kernel(unsigned int* result) {
    __shared__ __align__(8) uint64_t bars[2];
    if (threadIdx.x == 0) {
        mhc::mbar_init(bars, 1);
        mhc::mbar_init(bars + 1, 1);
        mhc::mbar_init_fence();
        mhc::mbar_arrive(bars);
    }
    __syncthreads();
    result[threadIdx.x] = mhc::umma::wait_warp(mhc::smem_addr(bars + threadIdx.x % 2), 0) ? 1u : 0u;
}

extern "C" __attribute__((visibility("default"))) int run_warp_probe(void* result) {
    layer_warp_probe_kernel<<<1, 32>>>(static_cast<unsigned int*>(result));
    if (cudaGetLastError() != cudaSuccess) return 1;
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : 2;
}
