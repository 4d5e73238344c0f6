// selftest.cu -- exercise of the bounded-wait failure path on the device.
//
// One CTA of two warps initialises mbarriers that nothing ever arrives on and
// waits for them with the library's two bounded waits.  A wait gives up after
// IC_WAIT_LIMIT_NS, sets IC_DEV_TIMEOUT in the status word and the kernel
// returns normally, so the context stays usable.  These are the waits that
// every pipeline of the library uses; the entry point lets a test check,
// without faulting or hanging anything, that a stalled pipeline ends with a
// status the host can read.
#include "sm100.cuh"

namespace ic {
namespace {

__global__ void __launch_bounds__(64) wait_timeout_kernel(uint32_t* status) {
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag[2];
    if (threadIdx.x < 2) {
        sm100::mbar_init(&bar[threadIdx.x], 1);
        abort_flag[threadIdx.x] = 0;
        sm100::fence_mbar_init();
    }
    __syncthreads();
    // phase 0 never completes: no thread arrives
    if (threadIdx.x < 32) sm100::warp_wait(&bar[0], 0, status, &abort_flag[0]);
    else sm100::wait_for(&bar[1], 0, status, &abort_flag[1], 0);
    __syncthreads();
    // a wait that ended without its own time running out would hide here
    if (threadIdx.x == 0 && !(abort_flag[0] && abort_flag[1])) atomicAnd(status, ~(uint32_t)IC_DEV_TIMEOUT);
}

}  // namespace
}  // namespace ic

extern "C" ic_status ic_selftest_wait_timeout(void* ws, size_t ws_bytes, void* stream) {
    if (ws == nullptr || ws_bytes < IC_STATUS_BYTES || ((uintptr_t)ws & 255)) return IC_ERR_INVALID_ARG;
    ic::wait_timeout_kernel<<<1, 64, 0, (cudaStream_t)stream>>>(static_cast<uint32_t*>(ws));
    return ic::last_launch_status();
}
