// Test helper: the gated scan's kernels with a wait for tokens that is told to
// have run out.  Every wait is made as the library makes it, and the tokens are
// there; the chosen CTA's workers only get the answer "not in time" at one step,
// so nothing here can hang or read what is not there.
#include <cstdint>

#include "lq_common.cuh"

namespace lq {

constexpr int kProbeBlocks = 4096, kProbeThreads = 320;
__device__ int probe_calls[kProbeBlocks * kProbeThreads];     // waits that a thread has made
__device__ int probe_block, probe_step;

// In step order: a worker waits once a step before the step in question.  The
// last warp is the loader, whose waits are left alone.
__device__ __forceinline__ bool probe_wait(uint64_t *bar, uint32_t parity, long long budget) {
    const bool ok = mbar_wait(bar, parity, budget);
    const int block = blockIdx.x, thread = threadIdx.x;
    if (block != probe_block || block >= kProbeBlocks || thread >= kProbeThreads || thread >= (int)blockDim.x - 32) return ok;
    return ok && probe_calls[block * kProbeThreads + thread]++ != probe_step;
}

}  // namespace lq

#define mbar_wait probe_wait
#include "lq_scan.cu"
#undef mbar_wait

namespace lq {

cudaError_t tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000 *out) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q);
    if (e != cudaSuccess) return e;
    *out = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return q == cudaDriverEntryPointSuccess && fn != nullptr ? cudaSuccess : cudaErrorNotSupported;
}

}  // namespace lq

// One call of the forward (grads NULL) or backward pass whose CTA `block` is
// late at its step `step` (-1: none), to its end.  Returns the CUDA error code.
extern "C" int lq_test_scan_late(const lq_scan_config *c, const lq_scan_args *a, const lq_scan_grads *g, int block, int step) {
    void *calls = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&calls, lq::probe_calls);
    if (e == cudaSuccess) e = cudaMemset(calls, 0, sizeof(int) * lq::kProbeBlocks * lq::kProbeThreads);
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(lq::probe_block, &block, sizeof(int));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(lq::probe_step, &step, sizeof(int));
    if (e == cudaSuccess)
        e = g == nullptr ? lq::launch_scan_forward(*c, *a, true, nullptr) : lq::launch_scan_backward(*c, *a, *g, true, nullptr);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    return (int)e;
}
