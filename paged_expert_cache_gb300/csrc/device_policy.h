// device_policy.h -- what the attention entry points keep of a device and how
// they choose by its SMs, free of CUDA so that it compiles and runs on its own
// (the CPU tests do).
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

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

// Whether a warp of the append kernel takes 32 query heads of a token, so that
// the rotation is read once for them; 8 where there are too few tokens to fill
// the GPU that way. tasks: warps of the former kind.
inline bool append_takes_32_heads(int64_t tasks, int sms) { return tasks >= (int64_t)sms * 16; }

// Whether prompt attention takes items of one tile, its keys in two halves, in
// place of pairs of tiles. The former are twice as many and half as long, but
// each loads its keys for itself: taken where pairs would leave half of the SMs
// idle (152 SMs, 600 tokens, 32 heads over 4: 11.6 us, in pairs 16.0), and at
// head_dim 128 up to two and a half pairs per SM for long sequences, whose pairs
// differ most (2451 tokens 53.0 and 61.1 us; 3000, 376 pairs, 71.5 and 75.3; 3400,
// 428 pairs, 88.1 and 82.6). Not at 64 (1500 tokens 23.3 and 22.2 us, 2451 44.6 and
// 40.0), nor for shorter ones (4 of 600 tokens at 64: 23.3 and 19.7). The lengths
// are on the device, so the call's rows stand for them: `pairs` is the most that
// there can be, and a long sequence among many short ones counts as short.
inline bool prompt_in_halves(int64_t pairs, int head_dim, int64_t keys_per_sequence, int sms) {
    const bool long_ones = head_dim == 128 && keys_per_sequence >= 1000;
    return 2 * pairs <= (long_ones ? 5 : 1) * (int64_t)sms;
}

// Whether reading what groups have in common once pays for its own kernels, against
// attention over each sequence by itself: by the most work that the call can hold, in
// cells of 16 positions and 64 dims for 8 rows (rows: of queries a key/value head;
// positions: what a row of the block table has room for). The common positions cost as
// much as 3 such row tiles whatever their rows are, and 8 us (32 query heads over 4,
// head_dim 128: 16 sequences behind 2451 positions 23.4 us, each by itself 15.2; behind
// 10000 27.1 and 27.0, 20000 30.8 and 42.2; 8 behind 10000 23.1 and 19.5; 48 behind
// 2451 30.7 and 25.9, 5000 32.9 and 37.2. 16 heads of their own, head_dim 64: 4 behind
// 20000 33.6 and 26.5, 8 behind 10000 25.9 and 27.5, 16 behind 5000 21.9 and 29.0.)
// Lengths and groups are on the device, so the room stands for them: in a table with
// much more of it than is held, short prefixes are read once for their group as well.
constexpr int64_t kSharedWork = 1 << 16;
inline bool sharing_pays(int64_t rows, int64_t sequences, int64_t positions, int kv_heads, int head_dim) {
    const int64_t tiles = std::max((rows + 7) / 8, std::min(sequences, rows));
    return tiles * (positions / 16) * kv_heads * (head_dim / 64) >= kSharedWork + 3 * kSharedWork / std::max<int64_t>(tiles, 1);
}

// Whether attention over common positions takes rows a tile at a time, its key tiles
// in turn between the two halves of a CTA, in place of pairs of tiles. A single tile
// costs two thirds of a pair, so it is taken where groups fill one tile or three (32
// rows, head_dim 64: 25.4 us, in pairs 27.1; 320 rows behind 2451 positions 29.3 and
// 33.3, behind 20000 45.2 and 46.8), not for two, four or more (160 rows 26.5 and 24.9;
// 512 rows behind 32768 139 and 114). The groups are on the device: their average
// stands for them.
inline bool shared_in_single_tiles(int64_t rows, int groups, int tile) {
    const int64_t tiles = (rows + (int64_t)groups * tile - 1) / ((int64_t)groups * tile);
    return tiles <= 1 || tiles == 3;
}

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
