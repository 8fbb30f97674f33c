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

// Makes a device current while it lives, and then the caller's again. Runtime
// has get(int*) and set(int), with statuses whose zero is success.
template <class Runtime>
struct DeviceScope {
    using Status = decltype(Runtime::set(0));
    int before = -1;
    Status status;
    explicit DeviceScope(int device) {
        status = Runtime::get(&before);
        if (status != Status{}) before = -1;
        else if (before != device) status = Runtime::set(device);
    }
    ~DeviceScope() {
        int now = -1;
        if (before >= 0 && Runtime::get(&now) == Status{} && now != before) Runtime::set(before);
    }
    DeviceScope(const DeviceScope&) = delete;
    DeviceScope& operator=(const DeviceScope&) = delete;
};

}  // namespace moe
