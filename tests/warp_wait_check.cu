// Device check of tfk::mbar_warp_wait_or_abort: a warp whose lanes begin to wait at
// different times, while another warp completes the phase and raises the abort flag
// close together, in either order, or raises the flag alone.  The waiting warp then
// goes through collective instructions and the CTA's barrier, as the roles of a kernel
// do.  answers[block] gets the ballot of the lanes' answers.  C ABI only; built by the
// test that uses it.
#include <cstdint>
#include <cuda_runtime.h>

#include "../w4_gemm_keyed_gb300/csrc/tf_ptx.cuh"

namespace {

// Bounded busy time of about n steps.
__device__ unsigned spend(unsigned n, unsigned x) {
    for (unsigned i = 0; i < n; ++i) x = x * 1664525u + 1013904223u;
    return x;
}

// what: 0 the flag alone, 1 the phase, then the flag, 2 the flag, then the phase, 3 the phase alone
__global__ void warp_wait_kernel(unsigned what, unsigned gap, unsigned *answers, unsigned *sink) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        tfk::mbar_init(&bar, 1);
        abort_flag = 0;
        tfk::fence_mbar_init();
    }
    __syncthreads();
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned x = lane;
    if (warp == 0) {
        x = spend((lane * 37 + blockIdx.x) % 64, x);
        __syncwarp();
        const bool ok = tfk::mbar_warp_wait_or_abort(&abort_flag, &bar, 0);
        const unsigned all = __ballot_sync(0xFFFFFFFFu, ok);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
        if (lane == 0) answers[blockIdx.x] = all;
    } else if (lane == 0) {
        x = spend(200 + blockIdx.x % 512, x);
        if (what == 1 || what == 3) tfk::mbar_arrive(&bar);
        if (what == 1 || what == 2) x = spend(gap, x);
        if (what != 3) *reinterpret_cast<volatile int *>(&abort_flag) = 1;
        if (what == 2) tfk::mbar_arrive(&bar);
    }
    __syncthreads();
    if (x == 0x12345678u) *sink = x;      // keeps the busy time
}

}  // namespace

extern "C" int warp_wait_check(unsigned what, unsigned gap, unsigned blocks, unsigned *answers, unsigned *sink) {
    if (what > 3 || gap > 4096 || blocks < 1 || blocks > 65536 || !answers || !sink) return 1;
    warp_wait_kernel<<<blocks, 64>>>(what, gap, answers, sink);
    if (cudaGetLastError() != cudaSuccess) return 2;
    return cudaDeviceSynchronize() == cudaSuccess ? 0 : 3;
}
