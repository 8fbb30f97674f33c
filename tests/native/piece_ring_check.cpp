// Drives piece_ring.h with a thread for each warp: one that puts pieces, 15 that take
// them, four of which vote on every step of a piece. Barriers are the GPU's: an arrival
// count, phases told apart by parity, waits that give up.
//
// Input lines: <pieces> <who> <piece> <ms>   warp <who> (0 the putter, 1 .. 15 the
//   takers, 12 .. 15 the voters) sleeps for so long before it puts, or inside, that
//   piece; <who> < 0: nobody does. Waits give up after 40 ms.
// Prints: pieces taken by all, whether a wait gave up, and the faults seen: pieces
//   read that were not put, pieces written over while a taker was at work on the
//   place's last one, votes that came out unlike among warps none of which gave up.
#include <atomic>
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>
#include <vector>

#include "piece_ring.h"

constexpr int kTakers = 15, kSteps = 5;

struct Barrier {
    std::mutex m;
    std::condition_variable cv;
    int count, pending;
    unsigned phase = 0;
    explicit Barrier(int n) : count(n), pending(n) {}
    void arrive() {
        const std::lock_guard<std::mutex> lock(m);
        if (--pending == 0) pending = count, ++phase, cv.notify_all();
    }
    bool wait(uint32_t parity, int ms) {  // true once the phase of that parity has completed
        std::unique_lock<std::mutex> lock(m);
        return cv.wait_for(lock, std::chrono::milliseconds(ms), [&] { return (phase & 1) != parity; });
    }
};

struct Place {
    std::atomic<int> piece{-12345}, end{-12345}, at_work{0};  // nothing has been put yet
};

int main() {
    int pieces, who, stall, ms;
    while (std::scanf("%d %d %d %d", &pieces, &who, &stall, &ms) == 4) {
        Place places[2];
        Barrier full[2] = {Barrier(1), Barrier(1)}, empty[2] = {Barrier(kTakers), Barrier(kTakers)}, voted(4);
        moe::Votes votes = {};
        std::atomic<int> gave_up{0}, faults{0}, least{1 << 30};
        std::vector<std::vector<int>> answers(4);
        auto sleep = [&](int warp, int piece) {
            if (warp == who && piece == stall) std::this_thread::sleep_for(std::chrono::milliseconds(ms));
        };
        auto wait = [&](Barrier& b, uint32_t parity) {
            const bool there = b.wait(parity, 40);
            if (!there) gave_up = 1;
            return there;
        };
        std::vector<std::thread> warps;
        warps.emplace_back([&] {
            for (int n = 0; n <= pieces; ++n) {
                sleep(0, n);
                if (!moe::put_piece(n, [&](int place, uint32_t parity) { return wait(empty[place], parity); },
                                    [&](int place) {
                                        if (places[place].at_work) ++faults;
                                        places[place].piece = n;
                                        places[place].end = n == pieces;
                                        full[place].arrive();
                                    }))
                    break;
            }
        });
        for (int w = 1; w <= kTakers; ++w)
            warps.emplace_back([&, w] {
                int n = 0, question = 0;
                for (;; ++n) {
                    if (!moe::take_piece(n, [&](int place, uint32_t parity) { return wait(full[place], parity); },
                                         [&](int place) {
                                             if (places[place].piece != n) ++faults;
                                             return places[place].end != 0;
                                         }))
                        break;
                    Place& p = places[n & 1];
                    ++p.at_work;
                    if (p.piece != n) ++faults;
                    sleep(w, n);
                    if (w >= 12)
                        for (int step = 0; step < kSteps; ++step, ++question)
                            answers[w - 12].push_back(moe::any_of_four(
                                votes, question, w - 12, question % 7 == w - 12,
                                [&](auto vote) {
                                    vote();
                                    voted.arrive();
                                },
                                [&](uint32_t parity) { wait(voted, parity); }));
                    if (p.piece != n) ++faults;
                    --p.at_work;
                    empty[n & 1].arrive();
                }
                int seen = least;
                while (n < seen && !least.compare_exchange_weak(seen, n)) {
                }
            });
        for (std::thread& t : warps) t.join();
        if (!gave_up)
            for (int w = 0; w < 4; ++w)
                for (int q = 0; q < pieces * kSteps; ++q) faults += answers[w][q] != (q % 7 < 4);
        std::printf("%d %d %d\n", least.load(), gave_up.load(), faults.load());
        std::fflush(stdout);
    }
    return 0;
}
