// Drives device_policy.h. Input lines:
//   once <device> <status>            a call on that device whose setting would
//     return the status; prints how often the setting has been made so far, and
//     the call's status
//   scope <current> <device> <fails>  a scope of the device while another is
//     current, with a runtime that refuses to set device <fails>; prints the
//     scope's status, the device current inside, and the one after it
//   heads <tasks> <sms>               whether append takes 32 heads a warp
//   halves <pairs> <head_dim> <keys per sequence> <sms>   whether a prompt's
//     items are one tile with its keys in halves
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
    long long n, keys;
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
        } else if (std::strcmp(what, "heads") == 0 && std::scanf("%lld %d", &n, &device) == 2) {
            std::printf("%d\n", moe::append_takes_32_heads(n, device));
        } else if (std::strcmp(what, "halves") == 0 && std::scanf("%lld %d %lld %d", &n, &status, &keys, &device) == 4) {
            std::printf("%d\n", moe::prompt_in_halves(n, status, keys, device));
        } else {
            return 1;
        }
    }
    return 0;
}
