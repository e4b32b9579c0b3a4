// ua_launch.h -- launching a kernel that may be scheduled while the kernel before
// it in the stream still drains (internal).
#pragma once

#include <cuda_runtime.h>

namespace ua {

// For the second and later kernels of one call: the first is launched the usual way
// or begins with griddep_wait(), so everything that came before the call is complete
// when they start.  Each calls griddep_wait() in every thread, at the latest before it
// ends, and before it touches what the kernel in front of it writes (by plain loads: a
// read-only load may be moved in front of the wait).  A first kernel that is launched
// like this calls it before its first access to global memory, and has no read-only
// loads at all (any input may be what the kernel in front writes): only its launch
// and what it sets up on chip run under the end of whatever came before.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace ua
