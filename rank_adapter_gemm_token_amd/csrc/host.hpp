// host.hpp -- host-side pieces shared by the C entry points' source files.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

namespace lora {

// Keeps the HIP error's text for lora_last_hip_error and returns LORA_EHIP
// (defined in api.cpp).  The runtime remembers a failed call until it is asked
// for its last error: it is asked here, or the check after the next launch
// would report this call's failure as the launch's.
int hip_fail(hipError_t e);

// The status of a failed call that allocates: LORA_ENOMEM where that was the
// reason.
int alloc_status(hipError_t e);

#define HIP_TRY(expr)                                    \
    do {                                                 \
        hipError_t e_ = (expr);                          \
        if (e_ != hipSuccess) return lora::hip_fail(e_); \
    } while (0)

// Make a handle's device current for the duration of a call.
class DeviceGuard {
public:
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev_) != hipSuccess) {
            prev_ = -1;
            return;
        }
        if (prev_ != dev) err_ = hipSetDevice(dev);
        switched_ = prev_ != dev;
    }
    ~DeviceGuard() {
        if (prev_ >= 0 && switched_) (void)hipSetDevice(prev_);
    }
    hipError_t error() const { return err_; }

private:
    int prev_ = -1;
    bool switched_ = false;
    hipError_t err_ = hipSuccess;
};

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }

}  // namespace lora
