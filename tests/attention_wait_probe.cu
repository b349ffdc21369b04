// Test probe, not part of the library: waits of the attention kernels' own kind on a
// barrier that nothing completes, beside one that is.  Built and run by
// tests/test_gpu_attention_wait.py.
#include "../block_draft_proposal_gb300/csrc/attention_tc.cuh"

using namespace dflash2;

__global__ void attention_wait_probe_kernel(int32_t *err, unsigned long long *elapsed_ns, int *result) {
    __shared__ uint64_t never, done;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&never, 1);
        mbar_init(&done, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        mbar_arrive(&done);
        result[0] = attn::bar_wait(&done, 0, &abort_flag, err) ? 1 : 0;
        uint64_t t0 = global_timer_ns();
        // phase 0 of a barrier with one expected arrival: nobody arrives
        result[1] = attn::bar_wait(&never, 0, &abort_flag, err) ? 1 : 0;
        elapsed_ns[0] = global_timer_ns() - t0;
        result[2] = abort_flag;
        t0 = global_timer_ns();
        result[3] = attn::bar_wait(&never, 0, &abort_flag, nullptr) ? 1 : 0;  // sees the flag
        elapsed_ns[1] = global_timer_ns() - t0;
        result[4] = attn::bar_wait(&done, 0, &abort_flag, nullptr) ? 1 : 0;   // is complete all the same
    }
}

extern "C" int attention_wait_probe(int32_t *err, unsigned long long *elapsed_ns, int *result) {
    attention_wait_probe_kernel<<<1, 32>>>(err, elapsed_ns, result);
    return (int)cudaDeviceSynchronize();
}
