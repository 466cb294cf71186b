// A barrier that nothing completes, waited for with the attention kernels' own bounded wait.
#include "../e8_lattice_vector_gb300/csrc_paged/nq_paged_device.cuh"

namespace {
// Waits `times` times; result: the waits that passed, the flag afterwards, nanoseconds.
__global__ void wait_for_nothing(int gave_up, int times, long long* result) {
    __shared__ uint64_t bar;
    __shared__ int flag;
    flag = gave_up;
    nq::mbar_init(nq::smem_ptr(&bar), 1);
    nq::mbar_init_fence();
    const uint64_t from = nq::global_ns();
    long long passed = 0;
    for (int i = 0; i < times; ++i) passed += nq::mbar_wait(nq::smem_ptr(&bar), 0, &flag);
    result[0] = passed;
    result[1] = flag;
    result[2] = (long long)(nq::global_ns() - from);
}
}  // namespace

extern "C" int wait_for_nothing_once(int gave_up, int times, long long* result) {
    wait_for_nothing<<<1, 1>>>(gave_up, times, result);
    return int(cudaGetLastError() != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess);
}
