// Drives the rules of device_policy.h for attention over common positions. Input lines:
//   pays <rows> <sequences> <positions> <kv_heads> <head_dim>   whether it is worth its own kernels
//   single <rows> <groups> <tile>                               whether rows are taken a tile at a time
#include <cstdio>
#include <cstring>

#include "device_policy.h"

int main() {
    char what[16];
    long long rows, sequences, positions;
    int a, b;
    while (std::scanf(" %15s", what) == 1) {
        if (std::strcmp(what, "pays") == 0 && std::scanf("%lld %lld %lld %d %d", &rows, &sequences, &positions, &a, &b) == 5) {
            std::printf("%d\n", moe::sharing_pays(rows, sequences, positions, a, b));
        } else if (std::strcmp(what, "single") == 0 && std::scanf("%lld %d %d", &rows, &a, &b) == 3) {
            std::printf("%d\n", moe::shared_in_single_tiles(rows, a, b));
        } else {
            return 1;
        }
    }
    return 0;
}
