// Self-test of the bounded waits of the library's kernels: that of most of them (rx_device.cuh:
// mbar_wait) and that of prompt_attention's bf16 kernel (prompt_wait.cuh: pt_wait).
//
// One warp waits on mbarriers that no thread ever arrives at.  Each wait gives up after its
// time limit; the first records RX_DEV_TIMEOUT as it does, the second sets the flag that ends the
// other waits (a third, of the full limit, returns at once) and the kernel records it at its end.
// Only if all of them did so is RX_DEV_TIMEOUT in the status word: the path a real kernel takes
// when a copy or a partner never completes, exercised on purpose without faulting or hanging the
// device (the context stays usable afterwards).
#include <cuda_runtime.h>

#include "prompt_wait.cuh"
#include "radix_attn.h"
#include "rx_common.h"
#include "rx_device.cuh"

namespace rx {

__global__ void __launch_bounds__(32) wait_selftest_kernel(int32_t* status, uint32_t limit_ns) {
    __shared__ __align__(8) uint64_t bar[3];
    __shared__ int abort_flag[2];
    __shared__ int32_t code[2];          // what each of the two kinds records
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&bar[i]), 1);   // one arrival expected, none will come
        abort_flag[0] = abort_flag[1] = code[0] = code[1] = 0;
        fence_mbar_init();
    }
    __syncthreads();
    bool ok = false;
    if (threadIdx.x == 0) ok = mbar_wait(smem_u32(&bar[0]), 0, &abort_flag[0], &code[0], limit_ns);
    __syncwarp();
    ok |= pt_wait(smem_u32(&bar[1]), 0, &abort_flag[1], limit_ns);
    __syncwarp();
    const uint64_t t0 = global_ns();
    ok |= pt_wait(smem_u32(&bar[2]), 0, &abort_flag[1]);
    ok |= global_ns() - t0 > 1000000000ull;          // it was ended by the flag, not by its limit of 2 s
    if (threadIdx.x == 0 && abort_flag[1]) report(&code[1], RX_DEV_TIMEOUT);
    __syncthreads();
    if (!__any_sync(0xffffffffu, ok) && threadIdx.x == 0 && code[0] == RX_DEV_TIMEOUT && code[1] == RX_DEV_TIMEOUT)
        report(status, RX_DEV_TIMEOUT);
}

}  // namespace rx

extern "C" int rx_wait_selftest(int32_t* d_status, uint64_t limit_ns, void* stream) {
    RX_REQUIRE(d_status != nullptr, "rx_wait_selftest: d_status is NULL");
    const uint64_t lim = limit_ns < 1000ull ? 1000ull : (limit_ns > 100000000ull ? 100000000ull : limit_ns);
    rx::wait_selftest_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(d_status, (uint32_t)lim);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        rx::set_error("rx_wait_selftest: launch failed: %s", cudaGetErrorString(e));
        return RX_ECUDA;
    }
    return RX_OK;
}
