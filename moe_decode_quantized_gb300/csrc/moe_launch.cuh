// moe_launch.cuh -- what the library's translation units share on the host side of
// a launch: the check of a CUDA call, a launch behind the stream's last kernel.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_host.cuh"

namespace moe {

#define MOE_CUDA_OK(expr)                                                                               \
    do {                                                                                                \
        cudaError_t e_ = (expr);                                                                        \
        if (e_ != cudaSuccess)                                                                          \
            return host_fail(MOE_ECUDA, "%s: %s (%s)", #expr, cudaGetErrorString(e_), cudaGetErrorName(e_)); \
    } while (0)

// Launches behind the stream's last kernel while that still runs (the kernels wait for its end before they touch
// memory): one token over 511, call after call, 12.0 us a call, launched the plain way 16.4.
template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t shared, moe_stream_t stream, A... args)
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = shared;
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace moe
