// glq_selftest.cu -- a check of the library's bounded device waits, for
// testing failure detection without faulting or hanging the GPU.
//
// Every wait in the layer's kernels (the tensor-core pipeline's mbarriers,
// its cluster-scope ones, the codebook-table loads of the GEMV and the W
// reconstruction) gives up after a limit and reports GLQ_DEVERR_TIMEOUT
// through the layer's device error word.  This kernel runs the same wait
// helpers on an mbarrier that only some of its expected arrivals reach, so
// that the wait runs out for certain (a flag that nothing sets), with a
// short limit chosen by the caller; no copy or other memory operation is
// pending on the barrier.
#include "glq_fp8.cuh"
#include "glq_kernels.cuh"
#include "glq_sm100.cuh"

namespace glq {

namespace {

__global__ void wait_selftest_kernel(unsigned *err, int kind, int arrivals, unsigned long long limit) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) mbar_init(&bar, 2);  // phase 0 completes after two arrivals
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 0; i < arrivals; ++i) sm100::mbar_arrive(&bar);
    bool ok;
    if (kind == 0) ok = sm100::mbar_wait(&bar, 0, limit);
    else if (kind == 1) ok = sm100::mbar_wait_cluster(&bar, 0, limit);
    else ok = mbar_wait_bounded(&bar, 0, (uint32_t)limit);
    if (!ok) atomicOr(err, GLQ_DEVERR_TIMEOUT);
}

// The same for the waits of the 8-bit float kernels, at CTA scope (warp 0)
// and at cluster scope (warp 1) at once; should only one of them run out,
// the word says so with GLQ_DEVERR_BOUNDS.
__global__ void fp8_wait_selftest_kernel(unsigned *err, int arrivals, unsigned long long limit) {
    __shared__ uint64_t bar[2];
    __shared__ volatile int abort[2];
    __shared__ unsigned ran_out[2];
    const int t = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
        mbar_init(&bar[t], 2);
        abort[t] = 0;
        ran_out[t] = 0;
        for (int i = 0; i < arrivals; ++i) sm100::mbar_arrive(&bar[t]);
        if (t == 0) fp8::wait_bounded<false>(&bar[t], 0, &abort[t], &ran_out[t], limit);
        else fp8::wait_bounded<true>(&bar[t], 0, &abort[t], &ran_out[t], limit);
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    if (ran_out[0] != ran_out[1]) atomicOr(err, GLQ_DEVERR_BOUNDS);
    else if (ran_out[0]) atomicOr(err, ran_out[0]);
}

// The experts' grid barrier over G CTAs, of which the launch has G or one less.
__global__ void moe_wait_selftest_kernel(uint64_t *bar, unsigned *err, uint32_t G, unsigned long long limit) {
    __shared__ volatile int abort;
    if (threadIdx.x != 0) return;
    abort = 0;
    fp8::grid_barrier(bar, G, &abort, err, limit);
}

}  // namespace

cudaError_t launch_moe_wait_selftest(uint64_t *bar, unsigned *err, int grid, bool all, unsigned long long limit,
                                     cudaStream_t s) {
    uint32_t G = grid;
    void *args[] = {&bar, &err, &G, &limit};
    return cudaLaunchCooperativeKernel((const void *)moe_wait_selftest_kernel, dim3(all ? grid : grid - 1), dim3(32), args,
                                       0, s);
}

cudaError_t launch_fp8_wait_selftest(unsigned *err, int arrivals, unsigned long long limit, cudaStream_t s) {
    fp8_wait_selftest_kernel<<<1, 64, 0, s>>>(err, arrivals, limit);
    return cudaGetLastError();
}

cudaError_t launch_wait_selftest(unsigned *err, int kind, int arrivals, unsigned long long limit, cudaStream_t s) {
    wait_selftest_kernel<<<1, 32, 0, s>>>(err, kind, arrivals, limit);
    return cudaGetLastError();
}

}  // namespace glq
