// Drives device_policy.h: each input line is "once <device> <status>", a call
// on that device whose setting would return the status; prints how often the
// setting has been made so far, and the call's status.
#include <cstdio>

#include "device_policy.h"

int main() {
    static moe::DeviceOnce once;
    int device, status, made = 0;
    while (std::scanf(" once %d %d", &device, &status) == 2) {
        const int got = once.run(device, [&] {
            ++made;
            return status;
        });
        std::printf("%d %d\n", made, got);
    }
    return 0;
}
