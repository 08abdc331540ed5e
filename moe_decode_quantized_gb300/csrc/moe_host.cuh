// moe_host.cuh -- host helpers that the library's translation units share:
// the calling thread's error message, the bound on waits inside kernels, tensor maps.
// Host code only; defined in moe_abi.cu.
#pragma once
#include <cuda.h>

#include "../../include/moe.h"

namespace moe {

// records the message of the calling thread (moe_last_error) and returns `code`
__attribute__((format(printf, 2, 3), visibility("hidden"))) int host_fail(int code, const char *fmt, ...);

// moe_set_wait_limit_ns's value
__attribute__((visibility("hidden"))) unsigned long long host_wait_ns();

// a tensor map of bf16 elements in the 128-byte swizzle: rank 2 or 3, dims and box innermost first, strides
// (bytes) of the dimensions after the first; what lies outside reads as zeros
__attribute__((visibility("hidden"))) int host_map_bf16(CUtensorMap *m, const void *base, int rank, const uint64_t *dims,
                                                        const uint64_t *strides, const uint32_t *box);

}  // namespace moe
