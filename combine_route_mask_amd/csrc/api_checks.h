// Host-side checks shared by the entry points of the expert layer.  No
// exception leaves an entry point.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "moe_ep.h"

namespace moe_ep {

// Message and code of the calling thread's last call (api.cpp).
int fail(int code, const std::string &msg);
int ok();

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int bad(const char *msg) { return fail(MOE_EP_ERR_INVALID_ARG, msg); }

// A required device pointer: present and aligned.
inline bool good(const void *p, uintptr_t a) { return p && aligned(p, a); }

template <typename F>
int guarded(F f)
{
    try {
        return f();
    } catch (...) {
        return MOE_EP_ERR_HIP; // no memory for a message
    }
}

// Launches; an error that an earlier call of the thread left behind is not
// this call's.
template <typename F>
int launched(const char *what, F launch)
{
    (void)hipGetLastError();
    const hipError_t e = launch();
    if (e == hipErrorInvalidConfiguration) // the launchers' own limit
        return fail(MOE_EP_ERR_CAPACITY, std::string(what) + " needs more workgroups than a launch holds");
    if (e != hipSuccess)
        return fail(MOE_EP_ERR_HIP, std::string(what) + " launch failed: " + hipGetErrorString(e));
    return ok();
}

// Bytes of one element, 0 for an unknown type.
inline int64_t item_bytes(int32_t row_type)
{
    return row_type == MOE_EP_BF16_ROWS ? 2 : row_type == MOE_EP_FP32_ROWS ? 4 : 0;
}

} // namespace moe_ep
