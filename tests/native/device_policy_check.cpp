// Drives device_policy.h. Input lines:
//   once <device> <status>            a call on that device whose setting would
//     return the status; prints how often the setting has been made so far, and
//     the call's status
//   scope <current> <device> <fails>  a scope of the device while another is
//     current, with a runtime that refuses to set device <fails>; prints the
//     scope's status, the device current inside, and the one after it
#include <cstdio>
#include <cstring>

#include "device_policy.h"

static int current, refused;
struct Fake {
    static int get(int* device) {
        *device = current;
        return current < 0 ? 3 : 0;
    }
    static int set(int device) {
        if (device == refused) return 101;
        current = device;
        return 0;
    }
};

int main() {
    static moe::DeviceOnce once;
    char what[16];
    int device, status, made = 0;
    while (std::scanf(" %15s", what) == 1) {
        if (std::strcmp(what, "once") == 0 && std::scanf("%d %d", &device, &status) == 2) {
            const int got = once.run(device, [&] {
                ++made;
                return status;
            });
            std::printf("%d %d\n", made, got);
        } else if (std::strcmp(what, "scope") == 0 && std::scanf("%d %d %d", &current, &device, &refused) == 3) {
            int inside;
            {
                const moe::DeviceScope<Fake> scope(device);
                status = scope.status;
                inside = current;
            }
            std::printf("%d %d %d\n", status, inside, current);
        } else {
            return 1;
        }
    }
    return 0;
}
