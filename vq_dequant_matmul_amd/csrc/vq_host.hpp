// vq_host.hpp -- what the C ABI's translation units share on the host: the
// thread's error message and the pointer checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/vq.h"

#define VQ_EXPORT extern "C" __attribute__((visibility("default")))

namespace vq {

// Set the thread's message and return st / clear it and return VQ_OK.
vq_status fail(vq_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
vq_status ok();
vq_status hip_fail(hipError_t e, const char *what);

// vq_moe_ffn's checks of tensors and sizes: what passes fails later only by a
// pointer, a workspace or a launch.
vq_status check_moe_ffn(const vq_tensor *gate, const vq_tensor *up, const vq_tensor *down,
                        int32_t n_tokens, int32_t top_k);

inline bool aligned(const void *p, size_t a)
{
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

}  // namespace vq
