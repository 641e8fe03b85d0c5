// Check of the kernels' failure detection: a bounded wait that runs out.
//
// Every decode kernel waits on mbarriers that asynchronous copies complete.
// Such a wait is bounded: past its limit the kernel records PA_ERR_TIMEOUT in
// the device status word, stops its loop, drains what it issued and returns,
// so the context stays usable and the host learns of it through
// pa_device_status. Nothing in a correct run lets a wait run out, so this
// file gives that path a run of its own. One CTA is laid out as the decode
// kernels are (a producer warp that arms a ring stage, a consumer warp that
// waits for it), except that the producer arms the stage for a copy it never
// issues: the phase cannot complete, the consumer's wait gives up after the
// caller's limit, records the timeout and raises the abort flag; the producer,
// seeing it, stops; the drain's own bounded wait gives up too (it records
// the same code), and the CTA returns. No copy is in flight at any point,
// so nothing lands in shared memory after the CTA has gone.
//
// The consumer is a whole warp, whose lanes have to agree on the outcome. Half
// of them are given four times the limit, and the producer completes the phase
// once the others have given up: had each lane its own answer, the patient ones
// would go on alone. A warp that does not agree is recorded as PA_ERR_CUDA.
#include "../../include/pa.h"
#include "device_common.cuh"
#include "internal.h"

namespace pa {

namespace {

__global__ void __launch_bounds__(64, 1) wait_timeout_check_kernel(int *status, unsigned long long limit_ns) {
    __shared__ __align__(8) uint64_t bars[3];   // a stage's full and empty barriers; one the warp has to agree on
    __shared__ int s_abort, s_gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t full = smem_addr(&bars[0]), empty = smem_addr(&bars[1]), late = smem_addr(&bars[2]);
    if (threadIdx.x == 0) {
        mbar_init(full, 1);
        mbar_init(empty, 1);
        mbar_init(late, 1);
        s_abort = s_gave_up = 0;
        mbar_fence_init();
    }
    __syncthreads();
    if (warp == 1) {
        // producer: arm stage 0 for 1 KiB of copies, then (as for a second
        // round of the ring) wait for the consumer to release it
        if (lane == 0) {
            mbar_arrive_expect_tx(full, 1024u);   // no copy is ever issued
            while (!*reinterpret_cast<volatile int *>(&s_abort)) {
                if (mbar_wait_for(empty, 0, limit_ns)) break;   // (never: the consumer does not release)
                record_status(status, kStatusTimeout);
                s_abort = 1;
            }
        }
    } else {
        // consumer: the kernels' wait for a stage to fill
        if (mbar_wait_warp(full, 0, status, &s_abort, limit_ns) && lane == 0) mbar_arrive(empty);
    }
    __syncthreads();
    if (warp == 1) {
        if (lane == 0) {
            const uint64_t t0 = global_timer_ns();
            while (!*reinterpret_cast<volatile int *>(&s_gave_up) && global_timer_ns() - t0 < 2 * limit_ns) {
            }
            mbar_arrive(late);   // the phase completes after half of the lanes have given up
        }
    } else {
        const bool ok = mbar_wait_warp(late, 0, status, &s_gave_up, lane < 16 ? limit_ns : 4 * limit_ns);
        const unsigned went_on = __ballot_sync(0xffffffffu, ok);
        if (lane == 0 && status && went_on != 0u && went_on != 0xffffffffu) atomicExch(status, kStatusCuda);
    }
    __syncthreads();
    // drain: the last phase the producer armed (bounded as well)
    if (threadIdx.x == 0 && !mbar_wait_for(full, 0, limit_ns)) record_status(status, kStatusTimeout);
}

}  // namespace

cudaError_t launch_wait_timeout_check(int *status, unsigned long long limit_ns, cudaStream_t stream) {
    wait_timeout_check_kernel<<<1, 64, 0, stream>>>(status, limit_ns);
    return cudaGetLastError();
}

}  // namespace pa

extern "C" PA_API pa_status pa_check_wait_timeout(unsigned timeout_us, void *stream) {
    if (timeout_us == 0 || timeout_us > 2000000u) return PA_ERR_INVALID_ARG;
    int *status = pa::device_status_word();
    if (!status) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_wait_timeout_check(status, 1000ull * timeout_us,
                                                        reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
