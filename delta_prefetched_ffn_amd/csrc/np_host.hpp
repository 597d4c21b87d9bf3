// What the host files of the library share: error reporting, the device guard, pointer checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "np.h"

namespace np {

// Records the calling thread's error text (np_last_error) and returns st.
__attribute__((format(printf, 2, 3))) np_status fail(np_status st, const char* fmt, ...);

// p must be memory device `dev` can read and write: its own device memory or pinned host memory
// mapped for it. A pageable host pointer (or another device's memory) would fault the GPU instead
// of failing here. `owner` names what lives on `dev` in the error text.
np_status check_io_ptr(const void* p, int dev, const char* what, const char* owner = "layer");

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

#define NP_HIP(call)                                                                          \
    do {                                                                                      \
        hipError_t e_ = (call);                                                               \
        if (e_ != hipSuccess) return fail(NP_EHIP, "%s failed: %s", #call, hipGetErrorString(e_)); \
    } while (0)

// Makes `dev` current for the scope and restores the previous device.
struct DeviceGuard {
    int prev = -1;
    bool ok = true;
    explicit DeviceGuard(int dev) {
        if (hipGetDevice(&prev) != hipSuccess) prev = -1;
        if (prev != dev) ok = hipSetDevice(dev) == hipSuccess;
    }
    ~DeviceGuard() {
        int cur = -1;
        if (prev >= 0 && hipGetDevice(&cur) == hipSuccess && cur != prev) (void)hipSetDevice(prev);
    }
};

// What a handle's destruction does within this scope leaves streams alone that are being captured: Python's collector may
// drop a handle at any time. hipDeviceSynchronize would end the capture nevertheless; hipFree waits for the device as well, and does
// not. (The runtime has the call; a host build over a stand-in for it may lack it.)
extern "C" hipError_t hipThreadExchangeStreamCaptureMode(hipStreamCaptureMode*) __attribute__((weak));
struct CaptureGuard {
    hipStreamCaptureMode mode = hipStreamCaptureModeRelaxed;
    static void exchange(hipStreamCaptureMode* m) {
        if (hipThreadExchangeStreamCaptureMode) (void)hipThreadExchangeStreamCaptureMode(m);
    }
    CaptureGuard() { exchange(&mode); }
    ~CaptureGuard() { exchange(&mode); }
};

}  // namespace np
