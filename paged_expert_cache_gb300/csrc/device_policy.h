// device_policy.h -- what the attention entry points keep of a device, free of
// CUDA so that it compiles and runs on its own (the CPU tests do).
#pragma once

#include <atomic>

namespace moe {

constexpr int kMaxDevices = 64;

// A setting that belongs to a device (a kernel's shared-memory limit): made on
// each device's first call. A failure is not kept, so that a later call tries
// again. Threads that come at once may both make it, which does no harm.
struct DeviceOnce {
    std::atomic<bool> done[kMaxDevices] = {};
    // set() returns a status whose zero is success.
    template <class F>
    auto run(int device, F set) -> decltype(set()) {
        const bool kept = device >= 0 && device < kMaxDevices;
        if (kept && done[device].load(std::memory_order_acquire)) return {};
        const auto status = set();
        if (kept && status == decltype(set()){}) done[device].store(true, std::memory_order_release);
        return status;
    }
};

}  // namespace moe
