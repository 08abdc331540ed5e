// moe_host.cuh -- host helpers that the library's translation units share:
// the calling thread's error message and the bound on waits inside kernels.
// Host code only; defined in moe_abi.cu.
#pragma once
#include "../../include/moe.h"

namespace moe {

// records the message of the calling thread (moe_last_error) and returns `code`
__attribute__((format(printf, 2, 3), visibility("hidden"))) int host_fail(int code, const char *fmt, ...);

// moe_set_wait_limit_ns's value
__attribute__((visibility("hidden"))) unsigned long long host_wait_ns();

}  // namespace moe
